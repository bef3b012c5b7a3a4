// Forward products of a few rows (nvfp4_ffn.h): bound by reading the weights once.
//
// A workgroup has 16 columns of an expert (gated: 8 of each projection) and its rows, 16 at a time; its sixteen waves
// share k. Weights go from memory straight to the registers of v_mfma_f32_16x16x32, where a load takes 64 bytes of each
// of 16 rows: nothing is staged, the other three waves of a SIMD have their loads under way while one multiplies, and
// no wave waits for another before the end, where the waves' sums meet in LDS in the order of k.
#include "ffn_gemm.h"

namespace ffn {

template <class T> __device__ __forceinline__ f32x4 mfma16(s16x8 a, s16x8 b, f32x4 c) {
  if constexpr (T::kId == NVFP4_MOE_F16) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  } else {
    typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  }
}

// 16 bytes at an offset from a buffer's base, 0 outside of it: no branch, so that the compiler counts the loads in flight.
typedef __amdgpu_buffer_rsrc_t Buffer;
template <int AUX> __device__ __forceinline__ s16x8 load16(Buffer b, int offset) {
  return __builtin_bit_cast(s16x8, __builtin_amdgcn_raw_buffer_load_b128(b, offset, 0, AUX));
}

template <class T, bool GATED> __global__ __launch_bounds__(1024, 4) void few_kernel(const Product p) {
  constexpr int NW = 16, ROWS = 16, U = 8;  // steps of 32 k in a chunk
  constexpr int kStream = 2;                // read once: not kept in the caches
  __shared__ __attribute__((aligned(16))) float room[NW][ROWS][20];  // rows padded: 16 lanes' writes take all banks
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int e = blockIdx.y, i = lane & 15, q = lane >> 4;
  const bool live = !p.rows.offsets || e < p.rows.experts;
  const int64_t lo = first_row(p.rows, e), hi = p.rows.offsets && !live ? p.rows.rows : first_row(p.rows, e + 1);
  const int n0 = blockIdx.x * (GATED ? 8 : 16);
  const int w_row = GATED ? (i < 8 ? n0 + i : p.ep.inner + n0 + i - 8) : n0 + i;
  const Buffer weights = __builtin_amdgcn_make_buffer_rsrc((void*)((const uint16_t*)p.b + (live ? e : 0) * p.b_step), 0, kMostBytes, 0x00020000);
  const int w_at = GATED || w_row < p.n ? (int)((int64_t)w_row * p.ldb * 2) + q * 16 : kOutside;
  // this wave's steps, by twos: whole lines of 128 bytes
  const int twos = ceil_div(p.k, 64);
  const int begin = 2 * (twos * wave / NW), end = 2 * (twos * (wave + 1) / NW);
  const int last = min(p.k, end * 32) - q * 8;  // the lane's k are below

  for (int64_t row0 = lo; row0 < hi; row0 += ROWS) {
    // what the finishing threads need, before the weights
    constexpr int EIGHTS = GATED ? 1 : 2;
    const int my_row = threadIdx.x / EIGHTS, my_col = n0 + threadIdx.x % EIGHTS * 8;
    const bool mine = my_row < ROWS && row0 + my_row < hi && my_col < (GATED ? p.ep.inner : p.n);
    float bias[8] = {}, residual[8] = {};
    if (!GATED && mine && live) {
      if (p.ep.bias) param8<T>(p.ep.bias, (int64_t)e * p.n + my_col, p.ep.bias_f32, true, bias);
      if (p.ep.residual) load8<T>(p.ep.residual, (row0 + my_row) * p.ep.ldr + my_col, true, residual);
    }
    f32x4 acc = {0, 0, 0, 0};
    if (live) {
      const Buffer rows = __builtin_amdgcn_make_buffer_rsrc((void*)((const uint16_t*)p.a + (p.rows.row_slots ? 0 : row0 * p.lda)), 0, kMostBytes, 0x00020000);
      const int64_t r = row0 + i, from = r >= hi ? -1 : p.rows.row_slots ? source_row(p.rows, r) : i;
      const int x_at = from < 0 ? kOutside : (int)(from * p.lda * 2) + q * 16;
      for (int s = begin; s < end; s += U) {
        s16x8 w[U], x[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int k = (s + u) * 32;
          w[u] = load16<kStream>(weights, k < last ? w_at + k * 2 : kOutside);
          x[u] = load16<0>(rows, k < last ? x_at + k * 2 : kOutside);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) acc = mfma16<T>(w[u], x[u], acc);
      }
    }
    *(f32x4*)&room[wave][i][4 * q] = acc;
    __syncthreads();
    if (mine) {
      float v[8] = {}, u[8] = {};
#pragma unroll
      for (int s = 0; s < NW; ++s) {
        const float* from = &room[s][my_row][GATED ? 0 : my_col - n0];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          v[j] += from[j];
          if (GATED) u[j] += from[8 + j];
        }
      }
      if constexpr (GATED) finish_gated<T>(p.ep, row0 + my_row, my_col, v, u);
      else finish_linear<T>(p.ep, p.n, row0 + my_row, my_col, v, bias, residual);
    }
    __syncthreads();
  }
}

int run_few(const Product& p, int dtype, bool gated, hipStream_t stream) {
  const dim3 grid(ceil_div(gated ? p.ep.inner : p.n, gated ? 8 : 16), p.rows.offsets ? p.rows.experts + (p.rows.clear ? 1 : 0) : 1);
  with_type16(dtype, [&](auto type) {
    using T = decltype(type);
    if (gated) few_kernel<T, true><<<grid, 1024, 0, stream>>>(p);
    else few_kernel<T, false><<<grid, 1024, 0, stream>>>(p);
    return 0;
  });
  return launched();
}

}  // namespace ffn
