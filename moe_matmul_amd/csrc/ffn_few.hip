// Forward products of a few rows (nvfp4_ffn.h): bound by reading the weights once.
//
// A workgroup has 16 columns of an expert (gated: 8 of each projection) and its rows, R at a time; its sixteen waves share
// k, in chunks of up to 8192. Weights go from memory straight to the registers of v_mfma_f32_16x16x32, where a load
// takes 64 bytes of each of 16 rows, and all of a wave's loads of a chunk are under way at once (U of them: 4 where k is
// at most 2048, so that two workgroups share a compute unit). The rows lie in LDS: their loads are issued first, so
// that they are there while the weights are on the way. The waves' sums meet in LDS in the order of k.
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
__device__ __forceinline__ s16x8 load16(Buffer b, int offset) {
  return __builtin_bit_cast(s16x8, __builtin_amdgcn_raw_buffer_load_b128(b, offset, 0, 0));
}

constexpr int kFewWaves = 16;

// Bytes between rows in LDS: 64 more than their elements', so that eight rows' chunks lie in different banks.
__host__ __device__ inline int few_stride(int k) { return (k < 32 * 16 * kFewWaves ? k + 31 : 32 * 16 * kFewWaves) / 32 * 64 + 64; }

template <class T, int U, int R, bool GATED> __global__ __launch_bounds__(1024, U <= 4 ? 8 : 4) void few_kernel(const Product p) {
  constexpr int NW = kFewWaves, CHUNK = 32 * U * NW;  // k of a chunk
  extern __shared__ __attribute__((aligned(16))) uint8_t few_lds[];
  float(*room)[16][20] = (float(*)[16][20])few_lds;  // the waves' sums; rows padded: 16 lanes' writes take all banks
  uint8_t* xs = few_lds + NW * 16 * 20 * 4;          // R rows of a chunk
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int e = blockIdx.y, i = lane & 15, q = lane >> 4;
  const bool live = !p.rows.offsets || e < p.rows.experts;
  const int64_t lo = first_row(p.rows, e), hi = p.rows.offsets && !live ? p.rows.rows : first_row(p.rows, e + 1);
  const int n0 = blockIdx.x * (GATED ? 8 : 16);
  const int w_row = GATED ? (i < 8 ? n0 + i : p.ep.inner + n0 + i - 8) : n0 + i;
  const Buffer weights = __builtin_amdgcn_make_buffer_rsrc((void*)((const uint16_t*)p.b + (live ? e : 0) * p.b_step), 0, kMostBytes, 0x00020000);
  const int w_at = GATED || w_row < p.n ? (int)((int64_t)w_row * p.ldb * 2) + q * 16 : kOutside;
  const int stride = few_stride(p.k);
  const uint8_t* x_at = xs + i % R * stride + q * 16;  // (rows from R on are never stored: any of them will do)

  for (int64_t row0 = lo; row0 < hi; row0 += R) {
    // the residual (or dh) of the finishing threads, before the weights
    constexpr int EIGHTS = GATED ? 1 : 2;
    const int my_row = threadIdx.x / EIGHTS, my_col = n0 + threadIdx.x % EIGHTS * 8;
    const bool mine = my_row < R && row0 + my_row < hi && my_col < (GATED ? p.ep.inner : p.n);
    u32x4 residual = {0, 0, 0, 0};
    if (mine && live && p.ep.residual)
      residual = *(const u32x4*)((const uint16_t*)p.ep.residual + (row0 + my_row) * p.ep.ldr + my_col);
    f32x4 acc = {0, 0, 0, 0};
    if (live) {
      const Buffer rows = __builtin_amdgcn_make_buffer_rsrc((void*)((const uint16_t*)p.a + (p.rows.row_slots ? 0 : row0 * p.lda)), 0, kMostBytes, 0x00020000);
      for (int k0 = 0; k0 < p.k; k0 += CHUNK) {
        const int size = min(CHUNK, p.k - k0), wide = (size + 31) / 32 * 4;  // 16-byte pieces of a row, whole steps
        // the first pieces of the rows' chunk, then the wave's weights, then the other pieces
        auto piece = [&](int at) __attribute__((always_inline)) {
          const int r = at / wide, c = at - r * wide;
          const int64_t from = row0 + r >= hi || at >= R * wide ? -1 : p.rows.row_slots ? source_row(p.rows, row0 + r) : r;
          return load16(rows, from >= 0 && c * 8 < size ? (int)((from * p.lda + k0 + c * 8) * 2) : kOutside);
        };
        auto put = [&](int at, s16x8 v) __attribute__((always_inline)) {
          const int r = at / wide, c = at - r * wide;
          if (at < R * wide) *(s16x8*)(xs + r * stride + c * 16) = v;
        };
        const s16x8 x0 = piece(threadIdx.x);
        const int twos = (size + 63) / 64, begin = 2 * (twos * wave / NW), end = 2 * (twos * (wave + 1) / NW);
        const int last = min(p.k, k0 + end * 32) - q * 8;  // the lane's k are below
        s16x8 w[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int k = k0 + (begin + u) * 32;
          w[u] = load16(weights, k < last ? w_at + k * 2 : kOutside);
        }
        put(threadIdx.x, x0);
        for (int at = threadIdx.x + 1024; at < R * wide; at += 1024) put(at, piece(at));
        __syncthreads();
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (begin + u < end && (begin + u) * 32 < size) acc = mfma16<T>(w[u], *(const s16x8*)(x_at + (begin + u) * 64), acc);
        __syncthreads();
      }
    }
    *(f32x4*)&room[wave][i][4 * q] = acc;
    __syncthreads();
    if (threadIdx.x < R * 16) {
      float* sum = &room[0][threadIdx.x / 16][threadIdx.x % 16];
      float v = 0.f;
#pragma unroll
      for (int s = 0; s < NW; ++s) v += sum[s * 16 * 20];
      *sum = v;
    }
    __syncthreads();
    if (mine) {
      float v[8], u[8];
      load8<F32>(&room[0][my_row][GATED ? 0 : my_col - n0], 0, true, v);
      if (GATED) load8<F32>(&room[0][my_row][8], 0, true, u);
      if constexpr (GATED) {
        if (p.ep.residual) finish_gated_dz<T>(p.ep, row0 + my_row, my_col, v, u, residual);
        else finish_gated<T>(p.ep, row0 + my_row, my_col, v, u);
      } else {
        float bias[8] = {}, r[8];
        if (p.ep.bias && live) param8<T>(p.ep.bias, (int64_t)e * p.n + my_col, p.ep.bias_f32, true, bias);
        unpack16x8<T>(residual, r);
        finish_linear<T>(p.ep, p.n, row0 + my_row, my_col, v, bias, r);
      }
    }
    __syncthreads();
  }
}

int run_few(const Product& p, int dtype, bool gated, hipStream_t stream) {
  const dim3 grid(ceil_div(gated ? p.ep.inner : p.n, gated ? 8 : 16), p.rows.offsets ? p.rows.experts + (p.rows.clear ? 1 : 0) : 1);
  with_type16(dtype, [&](auto type) {
    using T = decltype(type);
    auto go = [&](auto steps, auto rows) {
      constexpr int U = decltype(steps)::value, R = decltype(rows)::value;
      const size_t lds = kFewWaves * 16 * 20 * 4 + R * few_stride(p.k);
      auto kernel = gated ? few_kernel<T, U, R, true> : few_kernel<T, U, R, false>;
      static thread_local size_t allowed[2][16];  // by device
      int device = 0;
      if (lds > 65536 && hipGetDevice(&device) == hipSuccess && (device >= 16 || allowed[gated][device] < lds)) {
        if (hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds) == hipSuccess && device < 16)
          allowed[gated][device] = lds;
      }
      kernel<<<grid, 1024, lds, stream>>>(p);
    };
    auto by_rows = [&](auto steps) {
      if (p.m == 1) go(steps, std::integral_constant<int, 1>{});
      else go(steps, std::integral_constant<int, 8>{});
    };
    if (p.k <= 32 * 4 * kFewWaves) by_rows(std::integral_constant<int, 4>{});
    else by_rows(std::integral_constant<int, 16>{});
    return 0;
  });
  return launched();
}

}  // namespace ffn
