// Forward products of a few rows (nvfp4_ffn.h): bound by reading the weights once.
//
// A workgroup of sixteen waves has some of an expert's columns and its rows, R at a time. A wave has 16 columns (gated: 8
// of each projection) and a part of k: weights go from memory straight to the registers of v_mfma_f32_16x16x32, where a
// load takes 64 bytes of each of 16 rows, and all of a wave's loads of a chunk (U of them) are under way at once. The
// rows lie in LDS: their loads are issued first, so that they are there while the weights are on the way. The sums of
// the waves that share a column meet in LDS, in the order of k.
//
// Where workgroups are few, what counts is how soon all weights are asked for: U = 16, one workgroup to a compute unit
// (1 row, 4096 x 7168: 15.4 us; U = 4 16.9). Where there are several rounds of them, two share a unit, so that one's
// weights are under way while the other adds up: U = 4, the registers allow no more (1 row, 28672 x 4096: 44 us, 5.3
// TB/s; U = 16 54. 32 experts of 4096 x 7168: 208 and 311). Where k is short, all sixteen waves would have little to do
// for a few columns: fewer share k, and the workgroup has more columns (256 experts of 2048 x 512, 64 rows: 35 us, 90
// with 16 columns to a workgroup). Under a kernel trace: 1 x 7168 x 2048 8.5 us, gated 1 x 2 x 2048 x 7168 12.5 (58.7 MB:
// 4.7 TB/s; a launch that does nothing takes 3).
#include <atomic>

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
__host__ __device__ constexpr int few_stride(int k, int chunk) { return ((k < chunk ? k : chunk) + 31) / 32 * 64 + 64; }

// The expert of a workgroup and its rows: the blockIdx.y-th, or of those that have any, if there are fewer workgroups
// than experts; with `clear` the last has the rows of none. False: no such expert, or no rows.
__device__ __forceinline__ bool few_expert(const Rows& p, int lane, int& expert, int64_t& lo, int64_t& hi) {
  if (!p.offsets) {
    hi = p.rows;
    return true;
  }
  const int high = (int)gridDim.y - (p.clear ? 1 : 0);
  if ((int)blockIdx.y == high || high == p.experts) {
    expert = (int)blockIdx.y == high ? p.experts : (int)blockIdx.y;
    lo = (int64_t)uniform((uint64_t)first_row(p, expert));
    hi = expert == p.experts ? p.rows : (int64_t)uniform((uint64_t)first_row(p, expert + 1));
    return lo < hi;
  }
  int before = 0;
  for (int c = 0; c < p.experts; c += 64) {
    const int mine = c + lane;
    const int64_t first = mine < p.experts ? first_row(p, mine) : 0, after = mine < p.experts ? first_row(p, mine + 1) : 0;
    const uint64_t some = __ballot(after > first);
    const int rank = before + __builtin_popcountll(some & (((uint64_t)1 << lane) - 1));
    const uint64_t found = __ballot(after > first && rank == (int)blockIdx.y);
    if (found) {
      const int src = __builtin_ctzll(found);
      expert = c + src;
      lo = __builtin_amdgcn_readlane((int)first, src);
      hi = __builtin_amdgcn_readlane((int)after, src);
      return true;
    }
    before += __builtin_popcountll(some);
  }
  return false;
}

// share_log: 2^share_log waves share k.
template <class T, int U, int R, bool GATED> __global__ __launch_bounds__(1024, U <= 4 ? 8 : 4) void few_kernel(const Product p, int share_log) {
  constexpr int CHUNK = 32 * U * kFewWaves;  // k of a chunk (one that fewer waves share is the only one)
  constexpr int COLS = GATED ? 8 : 16, EIGHTS = COLS / 8;
  extern __shared__ __attribute__((aligned(16))) uint8_t few_lds[];
  uint8_t* xs = few_lds;                             // R rows of a chunk
  float(*room)[16][20] = (float(*)[16][20])few_lds;  // then the waves' sums; rows padded: 16 lanes' writes take all banks
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int sharing = 1 << share_log, part = wave & (sharing - 1), groups = kFewWaves >> share_log, group = wave >> share_log;
  const int i = lane & 15, q = lane >> 4;
  int e = 0;
  int64_t lo = 0, hi = 0;
  if (!few_expert(p.rows, lane, e, lo, hi)) return;
  const bool live = !p.rows.offsets || e < p.rows.experts;
  const int cols = GATED ? p.ep.inner : p.n, n_block = blockIdx.x * groups * COLS, n0 = n_block + group * COLS;
  const int w_row = GATED ? (i < 8 ? n0 + i : p.ep.inner + n0 + i - 8) : n0 + i;
  const Buffer weights = __builtin_amdgcn_make_buffer_rsrc((void*)((const uint16_t*)p.b + (live ? e : 0) * p.b_step), 0, kMostBytes, 0x00020000);
  const int w_at = (GATED ? n0 : w_row) < cols ? (int)((int64_t)w_row * p.ldb * 2) + q * 16 : kOutside;
  const int stride = few_stride(p.k, CHUNK);
  const uint8_t* x_at = xs + i % R * stride + q * 16;  // (rows from R on are never stored: any of them will do)

  for (int64_t row0 = lo; row0 < hi; row0 += R) {
    const int here = (int)min((int64_t)R, hi - row0);
    // where this thread finishes: eight columns of a row
    struct Mine { int row, eight, col; bool in, residual; };
    auto mine_at = [&](int thread) __attribute__((always_inline)) {
      const int row_log = 4 - share_log + (EIGHTS == 2);  // groups * EIGHTS threads a row
      Mine m;
      m.row = thread >> row_log;
      m.eight = thread & ((1 << row_log) - 1);
      m.col = n_block + m.eight * 8;
      m.in = m.row < here && m.col < cols;
      m.residual = m.in && live && p.ep.residual;
      return m;
    };
    auto residual_at = [&](const Mine& m) __attribute__((always_inline)) {
      return *(const u32x4*)((const uint16_t*)p.ep.residual + (row0 + m.row) * p.ep.ldr + m.col);
    };
    u32x4 residual = {0, 0, 0, 0};
    // (before the weights, so that it is there; two workgroups of a compute unit have no registers for it)
    constexpr bool EARLY = U > 4;
    if constexpr (EARLY) {
      const Mine m = mine_at(threadIdx.x);
      if (m.residual) residual = residual_at(m);
    }
    f32x4 acc = {0, 0, 0, 0};
    if (live) {
      const Buffer rows = __builtin_amdgcn_make_buffer_rsrc((void*)((const uint16_t*)p.a + (p.rows.row_slots ? 0 : row0 * p.lda)), 0, kMostBytes, 0x00020000);
      for (int k0 = 0; k0 < p.k; k0 += CHUNK) {
        const int size = min(CHUNK, p.k - k0), wide = (size + 31) / 32 * 4;  // 16-byte pieces of a row, whole steps
        // the first pieces of the rows' chunk, then the wave's weights, then the other pieces
        auto row_of = [&](int at) __attribute__((always_inline)) {  // at / wide
          int r = 0;
#pragma unroll
          for (int j = 1; j < R; ++j) r += at >= j * wide;
          return r;
        };
        auto piece = [&](int at) __attribute__((always_inline)) {
          const int r = row_of(at), c = at - r * wide;
          const int64_t from = at >= here * wide ? -1 : p.rows.row_slots ? source_row(p.rows, row0 + r) : r;
          return load16(rows, from >= 0 && c * 8 < size ? (int)((from * p.lda + k0 + c * 8) * 2) : kOutside);
        };
        auto put = [&](int at, s16x8 v) __attribute__((always_inline)) {
          const int r = row_of(at), c = at - r * wide;
          if (at < here * wide) *(s16x8*)(xs + r * stride + c * 16) = v;
        };
        const s16x8 x0 = piece(threadIdx.x);
        const int twos = (size + 63) / 64, begin = 2 * (twos * part >> share_log), end = 2 * (twos * (part + 1) >> share_log);
        const int last = min(p.k, k0 + end * 32) - q * 8;  // the lane's k are below
        s16x8 w[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int k = k0 + (begin + u) * 32;
          w[u] = load16(weights, k < last ? w_at + k * 2 : kOutside);
        }
        put(threadIdx.x, x0);
        for (int at = threadIdx.x + 1024; at < here * wide; at += 1024) put(at, piece(at));
        __syncthreads();
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (begin + u < end && (begin + u) * 32 < size) acc = mfma16<T>(w[u], *(const s16x8*)(x_at + (begin + u) * 64), acc);
        __syncthreads();
      }
    }
    *(f32x4*)&room[wave][i][4 * q] = acc;
    __syncthreads();
    int thread = threadIdx.x;
    asm volatile("" : "+v"(thread));  // nothing of what follows is kept in registers over the weights
    if (thread < R * 16 * groups) {
      float* sum = &room[thread / (R * 16) << share_log][thread / 16 % R][thread % 16];
      float v = 0.f;
#pragma unroll 4
      for (int s = 0; s < sharing; ++s) v += sum[s * 16 * 20];
      *sum = v;
    }
    __syncthreads();
    const Mine m = mine_at(thread);
    if (m.in) {
      if (!EARLY && m.residual) residual = residual_at(m);
      const int64_t row = row0 + m.row;
      const float* sums = room[m.eight / EIGHTS << share_log][m.row];
      float v[8], u[8];
      load8<F32>(sums, GATED ? 0 : m.eight % EIGHTS * 8, true, v);
      if constexpr (GATED) {
        load8<F32>(sums, 8, true, u);
        if (p.ep.residual) finish_gated_dz<T>(p.ep, row, m.col, v, u, residual);
        else finish_gated<T>(p.ep, row, m.col, v, u);
      } else {
        float bias[8] = {}, r[8];
        if (p.ep.bias && live) param8<T>(p.ep.bias, (int64_t)e * p.n + m.col, p.ep.bias_f32, true, bias);
        unpack16x8<T>(residual, r);
        finish_linear<T>(p.ep, p.n, row, m.col, v, bias, r);
      }
    }
    __syncthreads();
  }
}

int run_few(const Product& p, int dtype, bool gated, hipStream_t stream) {
  constexpr int kDeep = 16, kShallow = 4;  // loads of a wave under way
  const int experts = p.rows.offsets ? p.rows.experts : 1, units = compute_units();
  const int blocks = ceil_div(gated ? p.ep.inner : p.n, gated ? 8 : 16);  // of sixteen waves' columns
  const int busy = (int)(experts < p.m ? experts : p.m);                  // experts that can have rows
  const bool deep = p.k > 32 * kShallow * kFewWaves && (int64_t)blocks * busy <= units;
  // fewer waves share k as long as they cover it at once and there are two rounds of two workgroups to a unit
  int share_log = 4;
  while (!deep && share_log > 1 && p.k <= 32 * kShallow << (share_log - 1) && (int64_t)blocks * busy >> (4 - share_log) >= 4 * units) --share_log;
  // To look for the experts that have rows costs every workgroup its time, idle workgroups cost a launch of theirs: 8 of 64
  // experts (1 token, 2 x 1024 x 2048) 19 us and 25, 32 rows of 64 56 and 54; up to a quarter of the experts the search pays.
  const int high = p.m * 4 <= experts ? busy : experts;
  const dim3 grid(ceil_div(blocks, kFewWaves >> share_log), p.rows.offsets ? high + (p.rows.clear ? 1 : 0) : 1);
  with_type16(dtype, [&](auto type) {
    using T = decltype(type);
    auto go = [&](auto steps, auto rows) {
      constexpr int U = decltype(steps)::value, R = decltype(rows)::value;
      const int rows_bytes = R * few_stride(p.k, 32 * U * kFewWaves), sums_bytes = kFewWaves * 16 * 20 * 4;
      const size_t lds = rows_bytes > sums_bytes ? rows_bytes : sums_bytes;
      auto kernel = gated ? few_kernel<T, U, R, true> : few_kernel<T, U, R, false>;
      // what a kernel is allowed belongs to the process, so it is always the most that the kernel ever asks for
      constexpr int most = R * few_stride(1 << 20, 32 * U * kFewWaves);
      if constexpr (most > 65536) {
        static std::atomic<bool> allowed[2][16];  // by device
        int device = 0;
        if (hipGetDevice(&device) != hipSuccess || device >= 16) device = -1;
        if (device < 0 || !allowed[gated][device]) {
          const bool done = hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, most) == hipSuccess;
          if (done && device >= 0) allowed[gated][device] = true;
        }
      }
      kernel<<<grid, 1024, lds, stream>>>(p, share_log);
    };
    auto by_rows = [&](auto steps) {
      if (p.m == 1) go(steps, std::integral_constant<int, 1>{});
      else go(steps, std::integral_constant<int, 8>{});
    };
    if (deep) by_rows(std::integral_constant<int, kDeep>{});
    else by_rows(std::integral_constant<int, kShallow>{});
    return 0;
  });
  return launched();
}

}  // namespace ffn
