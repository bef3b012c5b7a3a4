// Matrix products in 16 bits with fp32 accumulation, for the entry points of
// nvfp4_ffn.h: C[m][n] = sum over k of A(m, k) B(n, k), each operand with adjacent k
// ("k inside": rows and weights of a forward product) or with adjacent m or n ("k
// outside": weights of a gradient of rows, both operands of a gradient of weights).
//
// A workgroup of four waves computes a tile of BM x BN, each wave a quarter (2 x 2)
// by v_mfma_f32_32x32x16. Operands go from memory to LDS by direct buffer loads in
// stages of BK, NS stages deep; an operand with k outside keeps its layout in LDS and
// is transposed by ds_read_b64_tr_b16 on the way to registers. One barrier a stage,
// before its last step of 16 k: the fragments of a step are read during the MFMAs of
// the one before, the loads of a stage are issued half in the last step of the stage
// whose buffer they take, half in the step after.
#pragma once

#include <type_traits>

#include "ffn_common.h"

namespace ffn {

// ---- direct loads ---------------------------------------------------------------
constexpr int kOutside = (int)0x80000000;  // an offset that no resource holds: the load gives 0
constexpr int kMostBytes = 0x7FFFFFFF;

__device__ __forceinline__ uint64_t uniform(uint64_t v) {
  return (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(v >> 32)) << 32 | (uint32_t)__builtin_amdgcn_readfirstlane((int)v);
}
// A raw buffer of num_bytes from a wave-uniform address on. A scalar register that a vector instruction wrote
// (readfirstlane) may be read by a buffer load five wait states later; the compiler keeps to that for its own loads,
// but does not see those in asm, so the resource's words pass through that wait here.
__device__ __forceinline__ i32x4 buffer_at(uint64_t base, int num_bytes) {
  i32x4 r = {__builtin_amdgcn_readfirstlane((int)base), __builtin_amdgcn_readfirstlane((int)((base >> 32) & 0xFFFFu)),
             __builtin_amdgcn_readfirstlane(num_bytes), 0x00020000};
  asm volatile("s_nop 4" : "+s"(r));
  return r;
}
// 16 bytes of each lane to LDS at `lds` + 16 * lane; counted by vmcnt, which the kernel waits for itself. (A load to
// LDS reads M0 one wait state after it was written, again unseen by the compiler.)
__device__ __forceinline__ void load_lds16(i32x4 rsrc, uint32_t lds, int offset) {
  const uint32_t at = __builtin_amdgcn_readfirstlane(lds);
  asm volatile("s_nop 0\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds" ::"v"(offset), "s"(rsrc), "{m0}"(at) : "memory");
}
// LDS reads of this wave are done, then the workgroup's barrier; loads in flight stay so.
__device__ __forceinline__ void block_sync() {
  __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
  asm volatile("s_barrier" ::: "memory");
}
template <int N> __device__ __forceinline__ void wait_loads() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 0xF) | ((N >> 4) << 14) | (0x7 << 4) | (0xF << 8));
  asm volatile("" ::: "memory");
}

template <class T> __device__ __forceinline__ f32x16 mfma32(s16x8 a, s16x8 b, f32x16 c) {
  if constexpr (T::kId == NVFP4_MOE_F16) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  } else {
    typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  }
}

// ---- epilogues ------------------------------------------------------------------
// What becomes of a product's sums. Columns come in eights at multiples of 8; every address is 16-byte aligned.
struct Epilogue {
  void* y;                 // [m][n], rows ldy apart
  int64_t ldy;
  int y_f32;               // fp32 in place of the rows' type
  const void* bias;        // [n] of each expert
  int bias_f32, act;
  const void* residual;    // rows ldr apart
  int64_t ldr;
  void* z;                 // [m][n]
  // gated: n = 2 * inner columns, y [m][inner]
  int inner;
  void* kept;              // [m][2 * inner]
  uint8_t *codes, *scales;
};

// `live`: a row of an expert; the others become 0.
template <class T>
__device__ __forceinline__ void finish_linear(const Epilogue& p, int n, int e, bool live, int64_t row, int col, float* v) {
  if (p.bias && live) {
    float b[8];
    param8<T>(p.bias, (int64_t)e * n + col, p.bias_f32, true, b);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] += b[j];
  }
  if (p.z) store8<T>(p.z, row * n + col, true, v);
  if (p.act != NVFP4_FFN_NONE) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = activation(v[j], p.act);
  }
  if (p.residual && live) {
    float r[8];
    load8<T>(p.residual, row * p.ldr + col, true, r);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] += r[j];
  }
  if (p.y_f32) store8<F32>(p.y, row * p.ldy + col, true, v);
  else store8<T>(p.y, row * p.ldy + col, true, v);
}
// h, and g and u where they are kept in 16 bits, of eight columns.
template <class T>
__device__ __forceinline__ void finish_gated(const Epilogue& p, int64_t row, int col, const float* g, const float* u) {
  if (p.kept) {
    store8<T>(p.kept, row * 2 * p.inner + col, true, g);
    store8<T>(p.kept, row * 2 * p.inner + p.inner + col, true, u);
  }
  float h[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) h[j] = activation(g[j], p.act) * u[j];
  store8<T>(p.y, row * p.ldy + col, true, h);
}
__device__ __forceinline__ uint32_t top8(const float* v) {
  uint32_t top = abs_bits(v[0]);
#pragma unroll
  for (int j = 1; j < 8; ++j) top = umax(top, abs_bits(v[j]));
  return top;
}
__device__ __forceinline__ void store_codes8(uint8_t* at, const float* v, float inverse) {
  u32x2 w;
  w.x = encode4(v[0], v[1], v[2], v[3], inverse);
  w.y = encode4(v[4], v[5], v[6], v[7], inverse);
  *(u32x2*)at = w;
}

// ---- the product ------------------------------------------------------------------
struct Product {
  const void *a, *b;
  int64_t lda, ldb;        // elements from a row to the next: of m and n with k inside, of k with k outside
  int64_t m;               // output rows (with a plan: the most there can be); with the plan over k, all experts' k rows are rows.rows
  int n, k;
  int64_t b_step;          // elements from an expert's B to the next's
  Rows rows;               // over the output's rows, or over k
  int tiles_m, tiles_n;    // dense, or of each expert where the plan is over k
  int splits;              // parts of k; more than one: fp32 sums to `partial` [splits][m][n]
  float* partial;
  int64_t partial_step;    // floats of one part
  Epilogue ep;
};

constexpr int kInside = 0, kOutsideK = 1;

constexpr int kXcds = 8;         // workgroups go round-robin over them; each has an L2
constexpr int kRasterWidth = 8;  // columns of tiles walked down together: 32 workgroups of an XCD share 4 + 8 panels

// Workgroup b of `total` in the order in which neighbours share an XCD.
__device__ __forceinline__ int64_t xcd_order(int64_t b, int64_t total) {
  const int64_t x = b % kXcds, i = b / kXcds, whole = total / kXcds, more = total % kXcds;
  return x * whole + (x < more ? x : more) + i;
}

// BX rows or columns of an operand in stages of BK.
template <class T, int LAYOUT, int BX, int BK, int NW> struct Operand {
  static constexpr int kLineChunks = LAYOUT == kInside ? BK / 8 : BX / 8;  // 16-byte chunks of a line in LDS
  static constexpr int kLines = 64 / kLineChunks;                        // lines of a load of one wave
  static constexpr int kLoads = BX * BK / 8 / (64 * NW);
  static constexpr int kBytes = BX * BK * 2;
  static_assert(LAYOUT == kInside || (kLines * NW) % 4 == 0, "the swizzle of a lane is that of its every load");
  static_assert(LAYOUT == kOutsideK || (BK == 32 || (BK == 64 && NW % 2 == 0)), "the swizzle of a lane is that of its every load");

  int voff[kLoads];
  int chunk_k;           // k inside: the lane's first k of a stage
  uint64_t base;         // of the tile
  int64_t ld_bytes;

  // k inside: chunk c of line r lies at c ^ swizzle(r), so that 8 and 16 consecutive
  // lines hold one chunk in different banks (windows of 128 and 256 bytes).
  __device__ static __forceinline__ int swizzle(int r) {
    return BK == 32 ? ((r >> 1) & 3) ^ ((r >> 3) & 1) : ((r >> 1) & 7) ^ ((r & 1) << 2);
  }

  // `row_of(line)`: the operand's row for a line of the tile, -1 for none.
  template <class Fn> __device__ __forceinline__ void set_inside(const void* at, int64_t ld, int wave, int lane, Fn row_of) {
    base = uniform((uint64_t)at);
    ld_bytes = ld * 2;
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      const int line = (u * NW + wave) * kLines + lane / kLineChunks;
      const int chunk = (lane % kLineChunks) ^ swizzle(line);
      const int64_t row = row_of(line);
      chunk_k = chunk * 8;
      voff[u] = row < 0 ? kOutside : (int)(row * ld_bytes) + chunk * 16;
    }
  }
  // k outside: lines of BX elements, one for each k; 32-byte units swizzled by the line's
  // last two bits, so that the four lines that a transposing read takes lie in different banks.
  __device__ __forceinline__ void set_outside(const void* at, int64_t ld, int width, int wave, int lane) {
    base = uniform((uint64_t)at);
    ld_bytes = ld * 2;
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      const int line = (u * NW + wave) * kLines + lane / kLineChunks;
      const int col = ((lane % kLineChunks) ^ (4 * (line & 3))) * 8;
      voff[u] = col < width ? (int)(line * ld_bytes) + col * 2 : kOutside;
    }
  }

  // Loads U0 .. U1-1 of the stage that begins at k, of which `left` elements are there (0 or less: none).
  template <int U0, int U1> __device__ __forceinline__ void issue(uint32_t lds, int wave, int64_t k, int64_t left) const {
    if constexpr (LAYOUT == kInside) {
      const i32x4 r = buffer_at(base + k * 2, kMostBytes);
      if (left >= BK) {
#pragma unroll
        for (int u = U0; u < U1; ++u) load_lds16(r, lds + (u * NW + wave) * 1024, voff[u]);
      } else {
        const bool there = chunk_k < left;
#pragma unroll
        for (int u = U0; u < U1; ++u) load_lds16(r, lds + (u * NW + wave) * 1024, there ? voff[u] : kOutside);
      }
    } else {
      const int64_t lines = left < 0 ? 0 : left < BK ? left : BK;
      const i32x4 r = buffer_at(base + k * ld_bytes, (int)(lines * ld_bytes));
#pragma unroll
      for (int u = U0; u < U1; ++u) load_lds16(r, lds + (u * NW + wave) * 1024, voff[u]);
    }
  }
};

// The lane's places in a stage of an operand, for a wave's BLOCKS blocks of 32 from `first` on.
template <int LAYOUT, int BX, int BK, int BLOCKS> struct Reader {
  static constexpr int kPlaces = LAYOUT == kInside ? BK / 16 : BLOCKS;
  uint32_t at[kPlaces];

  __device__ __forceinline__ void set(int first, int lane) {
    if constexpr (LAYOUT == kInside) {
      const int r = lane & 31;
      const int sw = BK == 32 ? ((r >> 1) & 3) ^ ((r >> 3) & 1) : ((r >> 1) & 7) ^ ((r & 1) << 2);
#pragma unroll
      for (int s = 0; s < kPlaces; ++s) at[s] = (first + r) * BK * 2 + (((2 * s + (lane >> 5)) ^ sw) << 4);
    } else {
      // of 16 lanes, four give the four lines' 32 bytes each; a lane gets one column's four k
      const int kk = (lane >> 2) & 3, unit = first / 16 + ((lane >> 4) & 1);
#pragma unroll
      for (int j = 0; j < kPlaces; ++j)
        at[j] = ((lane >> 5) * 8 + kk) * BX * 2 + (((unit + 2 * j) ^ (2 * kk)) << 5) + (lane & 3) * 8;
    }
  }
  // Block j of step s (16 k) of the stage at `lds`.
  __device__ __forceinline__ s16x8 read(const uint8_t* lds, int j, int s) const {
    if constexpr (LAYOUT == kInside) {
      return *(const s16x8*)(lds + at[s] + j * 32 * BK * 2);
    } else {
      typedef s16x4 __attribute__((address_space(3))) * lds4;
      const uint8_t* p = lds + at[j] + s * 16 * BX * 2;
      const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)p);
      const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(p + 4 * BX * 2));
      return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
    }
  }
};

// Which tile of which expert a workgroup has, and what it reads.
struct Place {
  int expert, live;   // live 0: rows of no expert
  int64_t row, rows;  // first output row, and the row after the expert's last
  int col;
  int64_t k_row, k;   // first row of the reduction (plan over k), its length
  int split;
};

// The plan is over the output's rows: the expert and rows of the tile `mt`, counted over all experts. False: no such tile.
template <int BM> __device__ __forceinline__ bool find_rows(const Rows& p, int64_t mt, int lane, Place& at) {
  int64_t before = 0;
  for (int c = 0; c <= p.experts; c += 64) {
    const int e = c + lane;
    const int64_t lo = e <= p.experts ? first_row(p, e) : 0;
    const int64_t hi = e < p.experts ? first_row(p, e + 1) : e == p.experts && p.clear ? p.rows : 0;
    const int tiles = hi > lo ? (int)((hi - lo + BM - 1) / BM) : 0;
    int upto = tiles;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int v = __shfl_up(upto, d, 64);
      if (lane >= d) upto += v;
    }
    const uint64_t found = __ballot(before + upto > mt);
    if (found) {
      const int src = __builtin_ctzll(found);
      const int64_t first = before + __shfl(upto - tiles, src, 64);
      at.expert = __builtin_amdgcn_readfirstlane(c + src);
      at.live = at.expert < p.experts;
      at.row = (int64_t)uniform((uint64_t)((int64_t)__shfl((int)lo, src, 64) + (mt - first) * BM));
      at.rows = __builtin_amdgcn_readfirstlane(__shfl((int)hi, src, 64));
      return true;
    }
    before += __shfl(upto, 63, 64);
  }
  return false;
}

template <class T, int AL, int BL, bool GATED, int BM, int BN, int BK, int NS, int PER_CU>
__global__ __launch_bounds__(256, PER_CU) void product_kernel(const Product p) {
  constexpr int NW = 4, MI = BM / 64, NI = BN / 64, STEPS = BK / 16;
  using A = Operand<T, AL, BM, BK, NW>;
  using B = Operand<T, BL, BN, BK, NW>;
  constexpr int STAGE = A::kBytes + B::kBytes, L = A::kLoads + B::kLoads;
  static_assert(STEPS % 2 == 0 && NS >= 2 && (NS - 1) * L < 64, "fragments alternate, loads are counted");
  static_assert(!GATED || (AL == kInside && BL == kInside && NI % 2 == 0 && BK == 32), "gate and up blocks of a wave");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[NS * STAGE];
  const uint32_t lds_at = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds;

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave >> 1, wn = wave & 1;

  // ---- the tile
  Place at;
  const int tile_cols = GATED ? BN / 2 : BN;
  constexpr bool OVER_K = AL == kOutsideK;  // the plan is over k
  at.expert = 0;
  at.live = 1;
  at.k_row = 0;
  at.k = p.k;
  if (OVER_K || !p.rows.offsets) {
    const int64_t tiles = (int64_t)p.tiles_m * p.tiles_n;
    int64_t v = xcd_order(blockIdx.x, gridDim.x);
    at.split = (int)(v % p.splits);
    v /= p.splits;
    at.expert = (int)(v / tiles);
    v -= at.expert * tiles;
    // down columns of kRasterWidth tiles
    const int64_t wide = (int64_t)p.tiles_m * kRasterWidth;
    const int super = (int)(v / wide), width = min(kRasterWidth, p.tiles_n - super * kRasterWidth);
    v -= super * wide;
    at.row = (v / width) * BM;
    at.col = (int)(super * kRasterWidth + v % width) * tile_cols;
    at.rows = p.m;
    if (OVER_K) {
      at.k_row = first_row(p.rows, at.expert);
      at.k = first_row(p.rows, at.expert + 1) - at.k_row;
      if (at.k < 0) at.k = 0;
    }
  } else {
    // the number of tiles is only known on the device: runs of eight to an XCD
    const int64_t b = blockIdx.x, x = b % kXcds, i = b / kXcds;
    int64_t v = i / 8 * (8 * kXcds) + x * 8 + i % 8;
    at.split = (int)(v % p.splits);
    v /= p.splits;
    at.col = (int)(v % p.tiles_n) * tile_cols;
    if (!find_rows<BM>(p.rows, v / p.tiles_n, lane, at)) return;
    if (!at.live) at.k = 0;
  }
  const int stages_all = (int)((at.k + BK - 1) / BK);
  const int first = (int)((int64_t)stages_all * at.split / p.splits);
  const int stages = (int)((int64_t)stages_all * (at.split + 1) / p.splits) - first;

  // ---- operands
  A a;
  B b;
  if constexpr (AL == kInside) {
    if (p.rows.row_slots) {
      a.set_inside(p.a, p.lda, wave, lane, [&](int line) {
        const int64_t r = at.row + line;
        return r < at.rows && at.live ? source_row(p.rows, r) : (int64_t)-1;
      });
    } else {
      a.set_inside((const uint16_t*)p.a + at.row * p.lda, p.lda, wave, lane,
                   [&](int line) { return at.row + line < at.rows ? (int64_t)line : (int64_t)-1; });
    }
  } else {
    a.set_outside((const uint16_t*)p.a + at.k_row * p.lda + at.row, p.lda, (int)min((int64_t)BM, p.m - at.row), wave, lane);
  }
  const uint16_t* be = (const uint16_t*)p.b + (OVER_K ? 0 : (at.live ? at.expert : 0) * p.b_step);
  if constexpr (GATED) {
    // blocks of a wave's columns: gate rows in the first half, the same columns' up rows in the second
    b.set_inside(be + at.col * p.ldb, p.ldb, wave, lane, [&](int line) {
      const int j = line % (BN / 2) / 32, col = line / (BN / 2) * (BN / 4) + j % (NI / 2) * 32 + line % 32;
      return at.col + col < p.ep.inner ? (int64_t)col + (j < NI / 2 ? 0 : p.ep.inner) : (int64_t)-1;
    });
  } else if constexpr (BL == kInside) {
    b.set_inside(be + at.col * p.ldb, p.ldb, wave, lane,
                 [&](int line) { return at.col + line < p.n ? (int64_t)line : (int64_t)-1; });
  } else {
    b.set_outside(be + at.k_row * p.ldb + at.col, p.ldb, min(BN, p.n - at.col), wave, lane);
  }
  Reader<AL, BM, BK, MI> ra;
  Reader<BL, BN, BK, NI> rb;
  ra.set(wm * (BM / 2), lane);
  rb.set(wn * (BN / 2), lane);

  f32x16 acc[MI][NI];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NI; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;

  if (stages > 0) {
    const int64_t k_end = min(at.k, (int64_t)(first + stages) * BK);
    // Half H of the loads of stage s (of the tile's) to its buffer: A's or B's.
    auto issue = [&](auto half, int s) __attribute__((always_inline)) {
      const uint32_t to = lds_at + (uint32_t)(s % NS) * STAGE;
      const int64_t k = (int64_t)(first + s) * BK;
      if constexpr (decltype(half)::value == 0) a.template issue<0, A::kLoads>(to, wave, k, k_end - k);
      else b.template issue<0, B::kLoads>(to + A::kBytes, wave, k, k_end - k);
    };
    std::integral_constant<int, 0> kA;
    std::integral_constant<int, 1> kB;
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      issue(kA, s);
      if (s < NS - 1) issue(kB, s);
    }
    s16x8 fa[2][MI], fb[2][NI];
    auto read = [&](int buf, const uint8_t* stage, int step) __attribute__((always_inline)) {
#pragma unroll
      for (int j = 0; j < NI; ++j) fb[buf][j] = rb.read(stage + A::kBytes, j, step);
#pragma unroll
      for (int i = 0; i < MI; ++i) fa[buf][i] = ra.read(stage, i, step);
    };
    wait_loads<(NS - 2) * L + A::kLoads>();
    block_sync();
    read(0, lds, 0);
    uint32_t now = 0;  // LDS offset of the stage under way
    for (int s = 0; s < stages; ++s) {
      const uint32_t next = now == (NS - 1) * STAGE ? 0 : now + STAGE;
#pragma unroll
      for (int t = 0; t < STEPS; ++t) {
        if (t == STEPS - 1) {
          wait_loads<(NS - 2) * L>();
          block_sync();
          issue(kA, s + NS);
        }
        if (t == 0) issue(kB, s + NS - 1);
        __builtin_amdgcn_sched_barrier(0);
        read((t + 1) & 1, lds + (t == STEPS - 1 ? next : now), (t + 1) % STEPS);
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
          for (int j = 0; j < NI; ++j) acc[i][j] = mfma32<T>(fb[t & 1][j], fa[t & 1][i], acc[i][j]);
        // the reads of the next step among the MFMAs of this one
        constexpr int READS = (AL == kInside ? MI : 2 * MI) + (BL == kInside ? NI : 2 * NI), PER = (READS + MI * NI - 1) / (MI * NI);
#pragma unroll
        for (int q = 0; q < READS / PER; ++q) {
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
          __builtin_amdgcn_sched_group_barrier(0x100, PER, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      now = next;
    }
    wait_loads<0>();  // nothing is written to LDS after the workgroup's end
  }

  // ---- the epilogue. A lane holds row lane % 32 of a block, and of its columns four of
  // every eight; one exchange with the lane 32 away gives it eight columns side by side.
  const int half = lane >> 5;
  auto columns8 = [&](const f32x16& c, int part, float* v) __attribute__((always_inline)) {
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      // copies: bit_cast of a vector's element itself takes the first one
      const float low = c[part * 8 + r], high = c[part * 8 + 4 + r];
      const auto x = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, low), __builtin_bit_cast(uint32_t, high), false, false);
      const uint32_t first = x[0], second = x[1];
      v[r] = __builtin_bit_cast(float, first);
      v[r + 4] = __builtin_bit_cast(float, second);
    }
  };
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    const int64_t row = at.row + wm * (BM / 2) + i * 32 + (lane & 31);
    const bool in = row < at.rows;
    if constexpr (GATED) {
#pragma unroll
      for (int j = 0; j < NI / 2; ++j) {
        const int col0 = at.col + wn * (BN / 4) + j * 32;
        float g[2][8], u[2][8];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          columns8(acc[i][j], q, g[q]);
          columns8(acc[i][j + NI / 2], q, u[q]);
        }
        if (p.splits > 1) {
          float* to = p.partial + at.split * p.partial_step + row * p.n;
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const int col = col0 + 16 * q + 8 * half;
            if (in && col < p.ep.inner) {
              store8<F32>(to, col, true, g[q]);
              store8<F32>(to, p.ep.inner + col, true, u[q]);
            }
          }
          continue;
        }
        if (p.ep.codes) {
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            const float(&v)[2][8] = w ? u : g;
            uint32_t top = umax(top8(v[0]), top8(v[1]));
            top = umax(top, from_lane_xor(top, 32));
            const uint32_t byte = scale8(top);
            if (in && col0 < p.ep.inner) {
              const int64_t k = row * 2 * p.ep.inner + w * p.ep.inner + col0;
#pragma unroll
              for (int q = 0; q < 2; ++q) store_codes8(p.ep.codes + k + 16 * q + 8 * half, v[q], scale8_inverse(byte));
              if (half == 0) p.ep.scales[k / 32] = (uint8_t)byte;
            }
          }
        }
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int col = col0 + 16 * q + 8 * half;
          if (in && col < p.ep.inner) finish_gated<T>(p.ep, row, col, g[q], u[q]);
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < NI; ++j)
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int col = at.col + wn * (BN / 2) + j * 32 + 16 * q + 8 * half;
          float v[8];
          columns8(acc[i][j], q, v);
          if (in && col < p.n) {
            if (p.splits > 1) {
              store8<F32>(p.partial + at.split * p.partial_step + ((OVER_K ? at.expert * p.m : 0) + row) * p.n, col, true, v);
            } else if constexpr (OVER_K) {
              Epilogue ep = p.ep;
              finish_linear<T>(ep, p.n, 0, true, at.expert * p.m + row, col, v);
            } else {
              finish_linear<T>(p.ep, p.n, at.expert, at.live, row, col, v);
            }
          }
        }
    }
  }
}

// ---- host: sizes of tiles, parts of k ----------------------------------------------
struct Tiling {
  int big;     // 256 x 256 tiles, else 128 x 128
  int splits;
};
// For tiles of rows (at most `rows` of them, by experts) and cols, k long; over_k: rows x cols of each expert.
Tiling choose_tiling(int64_t rows, int cols, int64_t k, int experts, bool over_k, int units);
// Adds the parts of k and applies the epilogue.
int finish_splits(const Product& p, int dtype, bool gated, bool over_k, void* stream);

template <class T, int AL, int BL, bool GATED> inline int launch_product(Product& p, const Tiling& t, hipStream_t stream) {
  constexpr bool OVER_K = AL == kOutsideK;
  const int bm = t.big ? 256 : 128, cols = (t.big ? 256 : 128) / (GATED ? 2 : 1);
  p.splits = t.splits;
  p.tiles_m = (int)ceil_div64(p.m, bm);
  p.tiles_n = ceil_div(GATED ? p.ep.inner : p.n, cols);
  int64_t tiles;
  if (OVER_K) {
    tiles = (int64_t)p.tiles_m * p.tiles_n * (p.rows.offsets ? p.rows.experts : 1);
  } else if (p.rows.offsets) {
    const int64_t most = p.m / bm + (p.rows.experts < p.m ? p.rows.experts : p.m) + 1;  // whole tiles, and a part of one for each
    tiles = ceil_div64(most * p.tiles_n * p.splits, 8 * kXcds) * (8 * kXcds);
  } else {
    tiles = (int64_t)p.tiles_m * p.tiles_n;
  }
  if (OVER_K || !p.rows.offsets) tiles *= p.splits;
  if (tiles > 0x7FFFFF) return NVFP4_ERR_INVALID;
  if (t.big) product_kernel<T, AL, BL, GATED, 256, 256, 32, 4, 1><<<(int)tiles, 256, 0, stream>>>(p);
  else product_kernel<T, AL, BL, GATED, 128, 128, 32, 4, 2><<<(int)tiles, 256, 0, stream>>>(p);
  return launched();
}

}  // namespace ffn
