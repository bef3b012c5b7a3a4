// Matrix products in 16 bits with fp32 accumulation, for the entry points of
// nvfp4_ffn.h: C[m][n] = sum over k of A(m, k) B(n, k), each operand with adjacent k
// ("k inside": rows and weights of a forward product) or with adjacent m or n ("k
// outside": weights of a gradient of rows, both operands of a gradient of weights).
//
// A workgroup computes a tile of BM x BN by v_mfma_f32_32x32x16, its waves WM x WN parts of it. Operands go from memory to
// LDS by direct buffer loads in stages of BK, SA and SB stages deep; an operand with k outside keeps its layout in LDS and
// is transposed by ds_read_b64_tr_b16 on the way to registers. One barrier a stage, before its last step of 16 k: the
// fragments of a step are read during the MFMAs of the one before; B's next loads are issued in the last step of the stage
// whose buffer they take, A's in the step after, so that neither waits in one queue behind the other.
//
// What bounds it: the card's power in large products (8192 x 4096 x 7168: 1.28 to 1.37 PFLOP/s at 1.5 to 1.6 GHz, matrix
// units busy 78% of the cycles; a large library product 1.42). LDS is next: 256 x 256 with waves of 128 x 64 reads 384
// cycles and writes 128 of the 512 that the MFMAs of a step take. Hence that tile, A's stages one deeper than B's (3 and 2
// fill the 160 KB). In products of few tiles the rounds of tiles bound, hence the other shapes: see launch_product.
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

// f(0), f(1), .., f(N - 1), each a constant.
template <int N, class Fn> __device__ __forceinline__ void each(Fn f) {
  if constexpr (N > 0) {
    each<N - 1>(f);
    f(std::integral_constant<int, N - 1>{});
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
  const void* residual;    // rows ldr apart; gated: dh, and y is dz [m][2 * inner] instead of h
  int64_t ldr;
  void* z;                 // [m][n]
  // gated: n = 2 * inner columns, y [m][inner]
  int inner;
  void* kept;              // [m][2 * inner]
  uint8_t *codes, *scales;
};

// Eight sums v of a row, the bias (b) and the residual (r) of their columns, 0 for none: z, its activation and y.
// `live`: a row of an expert; the others become 0.
template <class T>
__device__ __forceinline__ void finish_linear(const Epilogue& p, int n, int64_t row, int col, float* v, const float* b, const float* r) {
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] += b[j];
  if (p.z) *(u32x4*)((uint16_t*)p.z + row * n + col) = pack16x8<T>(v);
  activation8(v, p.act);
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] += r[j];
  if (p.y_f32) store8<F32>(p.y, row * p.ldy + col, true, v);
  else *(u32x4*)((uint16_t*)p.y + row * p.ldy + col) = pack16x8<T>(v);
}
// dz of eight columns from g, u and dh.
template <class T>
__device__ __forceinline__ void finish_gated_dz(const Epilogue& p, int64_t row, int col, float* g, float* u, u32x4 dh) {
  float d[8], a[8];
  unpack16x8<T>(dh, d);
  values_slopes8(g, a, p.act);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    g[j] *= d[j] * u[j];
    u[j] = d[j] * a[j];
  }
  uint16_t* at = (uint16_t*)p.y + row * p.ldy + col;
  *(u32x4*)at = pack16x8<T>(g);
  *(u32x4*)(at + p.inner) = pack16x8<T>(u);
}
// h, and g and u where they are kept in 16 bits, of eight columns.
template <class T>
__device__ __forceinline__ void finish_gated(const Epilogue& p, int64_t row, int col, const float* g, const float* u) {
  if (p.kept) {
    uint16_t* at = (uint16_t*)p.kept + row * 2 * p.inner + col;
    *(u32x4*)at = pack16x8<T>(g);
    *(u32x4*)(at + p.inner) = pack16x8<T>(u);
  }
  float h[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) h[j] = g[j];
  activation8(h, p.act);
#pragma unroll
  for (int j = 0; j < 8; ++j) h[j] *= u[j];
  *(u32x4*)((uint16_t*)p.y + row * p.ldy + col) = pack16x8<T>(h);
}
__device__ __forceinline__ uint32_t top8(const float* v) {
  uint32_t top = abs_bits(v[0]);
#pragma unroll
  for (int j = 1; j < 8; ++j) top = umax(top, abs_bits(v[j]));
  return top;
}
// g and u in 8 bits: four lanes side by side hold a block of 32 columns (`in` alike in all four).
__device__ __forceinline__ void finish_codes(const Epilogue& p, int64_t row, int col, bool in, const float* g, const float* u) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = h ? u[j] : g[j];
    uint32_t top = top8(v);
    top = umax(top, from_lane_xor(top, 1));
    top = umax(top, from_lane_xor(top, 2));
    if (!in) continue;
    const uint32_t byte = scale8(top);
    const float inverse = scale8_inverse(byte);
    const int64_t k = row * 2 * p.inner + h * p.inner + col;
    u32x2 w;
    w.x = encode4(v[0], v[1], v[2], v[3], inverse);
    w.y = encode4(v[4], v[5], v[6], v[7], inverse);
    *(u32x2*)(p.codes + k) = w;
    if (col % 32 == 0) p.scales[k / 32] = (uint8_t)byte;
  }
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
  int tile_rows;           // dense rows of a tile
  int splits;              // parts of k; more than one: fp32 sums to `partial` [splits][m][n]
  float* partial;
  int64_t partial_step;    // floats of one part
  Epilogue ep;
};

constexpr int kInside = 0, kOutsideK = 1;

constexpr int64_t kMostTiles = 0x7FFFFF;  // workgroups of 512 threads in a launch: below 2^32 threads
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

  // The buffer of the stage that begins at k, of which `left` elements are there (0 or less: none).
  __device__ __forceinline__ i32x4 stage(int64_t k, int64_t left) const {
    if constexpr (LAYOUT == kInside) {
      return buffer_at(base + k * 2, kMostBytes);
    } else {
      const int64_t lines = left < 0 ? 0 : left < BK ? left : BK;
      return buffer_at(base + k * ld_bytes, (int)(lines * ld_bytes));
    }
  }
  // Load u of that stage.
  template <int U> __device__ __forceinline__ void load(i32x4 buffer, uint32_t lds, int wave, int64_t left) const {
    const bool there = LAYOUT == kOutsideK || chunk_k < left;
    load_lds16(buffer, lds + (U * NW + wave) * 1024, there ? voff[U] : kOutside);
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
  int64_t row, rows;  // first output row, and the row after the tile's last
  int col;
  int64_t k_row, k;   // first row of the reduction (plan over k), its length
  int split;
};

// Rows of a tile where so many are covered by as few tiles of up to BM as can be: the same in all but the last, in blocks of 32.
__device__ __host__ __forceinline__ uint32_t even_rows(uint32_t rows, uint32_t bm) {
  const uint32_t tiles = (rows + bm - 1) / bm;
  return ((rows + tiles - 1) / tiles + 31) / 32 * 32;
}

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
      const int64_t first = before + __builtin_amdgcn_readlane(upto - tiles, src);
      at.expert = c + src;
      at.live = at.expert < p.experts;
      const int64_t from = __builtin_amdgcn_readlane((int)lo, src), end = __builtin_amdgcn_readlane((int)hi, src), rows = even_rows((uint32_t)(end - from), BM);
      at.row = from + (mt - first) * rows;
      at.rows = min(end, at.row + rows);
      return true;
    }
    before += __builtin_amdgcn_readlane(upto, 63);
  }
  return false;
}

template <class T, int AL, int BL, bool GATED, int BM, int BN, int WM, int WN, int BK, int SA, int SB, int PER_SIMD>
__global__ __launch_bounds__(64 * WM * WN, PER_SIMD) void product_kernel(const Product p) {
  constexpr int NW = WM * WN, TM = BM / WM, TN = BN / WN;  // a wave's part of the tile
  constexpr int MI = TM / 32, NI = TN / 32, STEPS = BK / 16;
  using A = Operand<T, AL, BM, BK, NW>;
  using B = Operand<T, BL, BN, BK, NW>;
  constexpr int B_AT = SA * A::kBytes, LDS = B_AT + SB * B::kBytes;  // A's stages, then B's
  static_assert(STEPS % 2 == 0 && SB >= 2 && (SA == SB || SA == SB + 1) && SA * A::kLoads + SB * B::kLoads < 64, "fragments alternate, loads are counted");
  static_assert(!GATED || (AL == kInside && BL == kInside && NI % 2 == 0), "gate and up blocks of a wave");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[LDS];
  const uint32_t lds_at = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds;

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WN, wn = wave % WN;

  // ---- the tile
  Place at;
  const int tile_cols = GATED ? BN / 2 : BN;
  constexpr bool OVER_K = AL == kOutsideK;  // the plan is over k
  at.expert = 0;
  at.live = 1;
  at.k_row = 0;
  at.k = p.k;
  if (OVER_K || !p.rows.offsets) {
    int64_t v;
    if (OVER_K && p.rows.offsets) {
      // experts have more and fewer rows: every XCD has its share of each one's tiles
      const int64_t tiles = (int64_t)p.tiles_m * p.tiles_n * p.splits, share = (tiles + kXcds - 1) / kXcds;
      const int64_t i = blockIdx.x / kXcds;
      at.expert = (int)(i / share);
      v = blockIdx.x % kXcds * share + i % share;
      if (v >= tiles) return;
    } else {
      v = xcd_order(blockIdx.x, gridDim.x);
    }
    at.split = (int)(v % p.splits);
    v /= p.splits;
    // down columns of kRasterWidth tiles
    const int64_t wide = (int64_t)p.tiles_m * kRasterWidth;
    const int super = (int)(v / wide), width = min(kRasterWidth, p.tiles_n - super * kRasterWidth);
    v -= super * wide;
    at.col = (int)(super * kRasterWidth + v % width) * tile_cols;
    const int64_t rows = p.tile_rows;
    at.row = (v / width) * rows;
    at.rows = min(p.m, at.row + rows);
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
    if (!find_rows<BM>(p.rows, (int64_t)uniform((uint64_t)(v / p.tiles_n)), lane, at)) return;
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
      const int j = line % TN / 32, col = line / TN * (TN / 2) + j % (NI / 2) * 32 + line % 32;
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
  // the tile's blocks of 32 rows are shared evenly by the rows of waves
  const int tile_blocks = (int)((at.rows - at.row + 31) / 32), blocks = (tile_blocks + WM - 1) / WM;
  const int wave_row = wm * blocks * 32;
  const int64_t wave_end = min(at.rows, at.row + wave_row + blocks * 32);
  ra.set(wave_row, lane);
  rb.set(wn * TN, lane);

  f32x16 acc[MI][NI];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NI; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;

  if (stages > 0) {
    const int64_t k_end = min(at.k, (int64_t)(first + stages) * BK);
    // Load u of A's or B's part of stage s (of the tile's) to its buffer.
    struct Stage { i32x4 buffer; uint32_t lds; int64_t left; };
    auto stage_a = [&](int s) __attribute__((always_inline)) {
      const int64_t k = (int64_t)(first + s) * BK;
      return Stage{a.stage(k, k_end - k), lds_at + (uint32_t)(s % SA) * A::kBytes, k_end - k};
    };
    auto stage_b = [&](int s) __attribute__((always_inline)) {
      const int64_t k = (int64_t)(first + s) * BK;
      return Stage{b.stage(k, k_end - k), lds_at + B_AT + (uint32_t)(s % SB) * B::kBytes, k_end - k};
    };
    auto load_a = [&](auto u, const Stage& s) __attribute__((always_inline)) { a.template load<decltype(u)::value>(s.buffer, s.lds, wave, s.left); };
    auto load_b = [&](auto u, const Stage& s) __attribute__((always_inline)) { b.template load<decltype(u)::value>(s.buffer, s.lds, wave, s.left); };
#pragma unroll
    for (int s = 0; s < SB; ++s) {
      if (s < SA - 1) {
        const Stage sa = stage_a(s);
        each<A::kLoads>([&](auto u) __attribute__((always_inline)) { load_a(u, sa); });
      }
      const Stage sb = stage_b(s);
      each<B::kLoads>([&](auto u) __attribute__((always_inline)) { load_b(u, sb); });
    }
    s16x8 fa[2][MI], fb[2][NI];
    // Fragment f of a step: B's, then A's, as the MFMAs want them.
    auto read = [&](int buf, uint32_t in_a, uint32_t in_b, int step, int f) __attribute__((always_inline)) {
      if (f < NI) fb[buf][f] = rb.read(lds + in_b, f, step);
      else fa[buf][f - NI] = ra.read(lds + in_a, f - NI, step);
    };
    wait_loads<(SA - 2) * A::kLoads + (SB - 1) * B::kLoads>();
    block_sync();
#pragma unroll
    for (int f = 0; f < NI + MI; ++f) read(0, 0, B_AT, 0, f);
    // The wave's blocks of 32 rows that the output has: a loop for each number of them, so that nothing in it depends on
    // it (all in one with the others skipped takes registers that the largest tile does not have: 203 us where whole
    // tiles take 141). A wave without rows loads its share and keeps the barriers.
    auto run = [&](auto of) __attribute__((always_inline)) {
      constexpr int ACTIVE = decltype(of)::value;
      uint32_t now_a = 0, now_b = B_AT;  // LDS offsets of the stage under way
      for (int s = 0; s < stages; ++s) {
        const uint32_t next_a = now_a == (SA - 1) * A::kBytes ? 0 : now_a + A::kBytes;
        const uint32_t next_b = now_b == B_AT + (SB - 1) * B::kBytes ? B_AT : now_b + B::kBytes;
        Stage sa = stage_a(s + SA - 1), sb;
        // a step: for every row block its share of the next step's reads, a load, its MFMAs
        each<STEPS>([&](auto step) __attribute__((always_inline)) {
          constexpr int t = decltype(step)::value;
          if constexpr (t == STEPS - 1) {
            sb = stage_b(s + SB);
            wait_loads<(SA - 2) * A::kLoads + (SB - 2) * B::kLoads>();
            block_sync();
          }
          each<MI>([&](auto block) __attribute__((always_inline)) {
            constexpr int i = decltype(block)::value;
            if constexpr (t == STEPS - 1) each<B::kLoads>([&](auto u) __attribute__((always_inline)) {
              if constexpr (decltype(u)::value * MI / B::kLoads == i) load_b(u, sb);
            });
            if constexpr (t == 0) each<A::kLoads>([&](auto u) __attribute__((always_inline)) {
              if constexpr (decltype(u)::value * MI / A::kLoads == i) load_a(u, sa);
            });
#pragma unroll
            for (int f = i * (NI + MI) / MI; f < (i + 1) * (NI + MI) / MI; ++f)
              if ((f < NI ? 0 : f - NI) < ACTIVE)
                read((t + 1) & 1, t == STEPS - 1 ? next_a : now_a, t == STEPS - 1 ? next_b : now_b, (t + 1) % STEPS, f);
            if (i < ACTIVE)
#pragma unroll
              for (int j = 0; j < NI; ++j) acc[i][j] = mfma32<T>(fb[t & 1][j], fa[t & 1][i], acc[i][j]);
            __builtin_amdgcn_sched_barrier(0);
          });
        });
        now_a = next_a;
        now_b = next_b;
      }
    };
    const int active = at.row + wave_row < wave_end ? blocks : 0;
    each<MI + 1>([&](auto of) __attribute__((always_inline)) {
      if (active == decltype(of)::value) run(of);
    });
    // nothing more is written to the stages, nor read from them
    wait_loads<0>();
    block_sync();
  }

  // ---- the epilogue. A lane holds row lane % 32 of a block and four of every eight columns: 32 rows at a time go
  // through LDS (of the wave's own), so that a row's lanes then have eight columns each side by side, and global
  // loads and stores take whole lines. Rows are padded by 16 bytes: 16 lanes' writes take all banks once.
  constexpr int C = TN, ROOM = C + 4;                 // columns of a wave
  constexpr int LANES = (GATED ? C / 2 : C) / 8;      // of a row
  constexpr int PASS = 64 / LANES, PASSES = 32 / PASS;
  static_assert(NW * 32 * ROOM * 4 <= LDS, "the stages hold the waves' rooms");
  float* room = (float*)lds + wave * 32 * ROOM;
  const int my_row = lane / LANES, my_col = lane % LANES * 8;
  const int col = at.col + wn * (GATED ? C / 2 : C) + my_col;
  const int64_t row0 = at.row + wave_row + my_row;
  const bool in_cols = col < (GATED ? p.ep.inner : p.n), parts = p.splits > 1;
  const int64_t out0 = OVER_K ? at.expert * p.m : 0;  // output row of the tile's row 0
  float* partial = parts ? p.partial + at.split * p.partial_step + out0 * p.n : nullptr;
  const bool has_bias = !GATED && BL == kInside && p.ep.bias && at.live && !parts;
  const bool has_residual = BL == kInside && p.ep.residual && at.live && !parts;
  float bias[8] = {};
  if (has_bias && in_cols) param8<T>(p.ep.bias, (int64_t)at.expert * p.n + col, p.ep.bias_f32, true, bias);
  // the residual of a pass; out of range: 0
  auto residual_at = [&](int64_t row) __attribute__((always_inline)) {
    return row < wave_end && in_cols ? *(const u32x4*)((const uint16_t*)p.ep.residual + row * p.ep.ldr + col) : u32x4{0, 0, 0, 0};
  };
  constexpr bool GRADIENT = BL == kOutsideK;  // no bias, activation or residual
  const bool plain = !GATED && !parts && !p.ep.y_f32 && (GRADIENT || (p.ep.act == NVFP4_FFN_NONE && !p.ep.z));
  u32x4 residual[PASSES];
  if (has_residual && plain) {
#pragma unroll
    for (int q = 0; q < PASSES; ++q) residual[q] = residual_at(row0 + q * PASS);
  }
  each<MI>([&](auto block) __attribute__((always_inline)) {
    constexpr int i = decltype(block)::value;
    if (at.row + wave_row + i * 32 >= wave_end) return;
    // a wave's LDS operations keep their order; the fence keeps the compiler to it
    wave_sync();
#pragma unroll
    for (int j = 0; j < NI; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const f32x4 v = {acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
        *(f32x4*)(room + (lane & 31) * ROOM + j * 32 + 8 * q + 4 * (lane >> 5)) = v;
      }
    wave_sync();
    const float* from = room + my_row * ROOM + my_col;
    const int64_t first_of = row0 + i * 32;
    if constexpr (!GATED) {
      if (plain) {
        // (the next block's residual is under way before this one's stores, which its wait would else include)
        u32x4 mine[PASSES];
        if (has_residual) {
#pragma unroll
          for (int q = 0; q < PASSES; ++q) {
            mine[q] = residual[q];
            if (i + 1 < MI) residual[q] = residual_at(first_of + 32 + q * PASS);
          }
        }
#pragma unroll
        for (int q = 0; q < PASSES; ++q) {
          const int64_t row = first_of + q * PASS;
          float v[8];
          load8<F32>(from, q * PASS * ROOM, true, v);
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] += bias[j];
          if (has_residual) {
            float r[8];
            unpack16x8<T>(mine[q], r);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] += r[j];
          }
          if (row < wave_end && in_cols) *(u32x4*)((uint16_t*)p.ep.y + (out0 + row) * p.ep.ldy + col) = pack16x8<T>(v);
        }
        return;
      }
      u32x4 next = has_residual ? residual_at(first_of) : u32x4{0, 0, 0, 0};
#pragma unroll 1
      for (int q = 0; q < PASSES; ++q) {
        const int64_t row = first_of + q * PASS;
        const u32x4 mine = next;
        if (has_residual && q + 1 < PASSES) next = residual_at(row + PASS);
        float v[8], r[8];
        load8<F32>(from, q * PASS * ROOM, true, v);
        if (row >= wave_end || !in_cols) continue;
        if (parts) {
          store8<F32>(partial, row * p.n + col, true, v);
          continue;
        }
        if constexpr (GRADIENT) {  // fp32
          store8<F32>(p.ep.y, (out0 + row) * p.ep.ldy + col, true, v);
          continue;
        }
        unpack16x8<T>(mine, r);
        finish_linear<T>(p.ep, p.n, out0 + row, col, v, bias, r);
      }
    } else {
      u32x4 next = has_residual ? residual_at(first_of) : u32x4{0, 0, 0, 0};
#pragma unroll 1
      for (int q = 0; q < PASSES; ++q) {
        const int64_t row = first_of + q * PASS;
        const bool in = row < wave_end && in_cols;
        const u32x4 dh = next;
        if (has_residual && q + 1 < PASSES) next = residual_at(row + PASS);
        float g[8], u[8];
        load8<F32>(from, q * PASS * ROOM, true, g);
        load8<F32>(from, q * PASS * ROOM + C / 2, true, u);
        if (parts) {
          if (in) {
            store8<F32>(partial, row * p.n + col, true, g);
            store8<F32>(partial, row * p.n + p.ep.inner + col, true, u);
          }
          continue;
        }
        if (has_residual) {
          if (in) finish_gated_dz<T>(p.ep, row, col, g, u, dh);
          continue;
        }
        if (p.ep.codes) finish_codes(p.ep, row, col, in, g, u);
        if (in) finish_gated<T>(p.ep, row, col, g, u);
      }
    }
  });
}

// ---- host: sizes of tiles, parts of k ----------------------------------------------
struct Tiling {
  int shape;   // 0: 128 x 128, 1: 256 x 128, 2: 256 x 256; of rows with k inside also 3: 64 x 128, 4: 320 x 128, 5: 320 x 256
  int splits;
};
constexpr int kShapes = 6, kShapesOverK = 3;
constexpr int tile_rows(int shape) { return shape >= 4 ? 320 : shape == 3 ? 64 : shape ? 256 : 128; }
constexpr int tile_cols(int shape) { return shape == 2 || shape == 5 ? 256 : 128; }

// Tile, waves, stages: time in us of a product that it fits, bf16, forward.
//   256 x 256, 8, 3 + 2: 4096 x 4096 x 4096 106 (1.29 PFLOP/s)
//   320 x 256, 8, 2 + 2: 5120 x 4096 x 2048 73 (1.18; 256 x 256 takes two rounds, 98)
//   320 x 128, 4, 3 + 2: 5120 x 2048 x 2048 43 (1.01; 256 x 256 44, 128 x 128 57), 2051 x 4104 x 2048 41 (46, 58)
//   256 x 128, 8, 3 + 3: 1500 x 1536 x 6144, in parts, 42 (128 x 128 43)
//   128 x 128, 4, 2 + 2, two to a unit: 1000 x 4096 x 2048 27 (256 x 128 29)
//    64 x 128, 4, 3 + 3, two to a unit: 128 x 4096 x 4096, in parts, 19 (128 x 128 21); experts of few rows
// Four waves of 128 x 128 in place of eight of 128 x 64 take the same time in 256 x 256.
template <class T, int AL, int BL, bool GATED> inline int launch_product(Product& p, const Tiling& t, hipStream_t stream) {
  constexpr bool OVER_K = AL == kOutsideK;
  const int bm = tile_rows(t.shape), cols = tile_cols(t.shape) / (GATED ? 2 : 1);
  p.splits = t.splits;
  p.tiles_m = (int)ceil_div64(p.m, bm);
  p.tile_rows = (int)even_rows((uint32_t)p.m, bm);
  p.tiles_n = ceil_div(GATED ? p.ep.inner : p.n, cols);
  int64_t tiles;
  if (OVER_K) {
    tiles = (int64_t)p.tiles_m * p.tiles_n * p.splits;
    if (p.rows.offsets) tiles = ceil_div64(tiles, kXcds) * kXcds * p.rows.experts;
  } else if (p.rows.offsets) {
    const int64_t most = p.m / bm + (p.rows.experts < p.m ? p.rows.experts : p.m) + 1;  // whole tiles, and a part of one for each
    tiles = ceil_div64(most * p.tiles_n * p.splits, 8 * kXcds) * (8 * kXcds);
  } else {
    tiles = (int64_t)p.tiles_m * p.tiles_n * p.splits;
  }
  if (tiles > kMostTiles) return NVFP4_ERR_INVALID;
  const dim3 grid((unsigned)tiles);
  if (t.shape == 2) product_kernel<T, AL, BL, GATED, 256, 256, 2, 4, 64, 3, 2, 2><<<grid, 512, 0, stream>>>(p);
  else if (t.shape == 1) product_kernel<T, AL, BL, GATED, 256, 128, 4, 2, 64, 3, 3, 2><<<grid, 512, 0, stream>>>(p);
  else if (t.shape == 0) product_kernel<T, AL, BL, GATED, 128, 128, 2, 2, 64, 2, 2, 2><<<grid, 256, 0, stream>>>(p);
  else if constexpr (AL == kInside) {
    if (t.shape == 3) product_kernel<T, AL, BL, GATED, 64, 128, 2, 2, 64, 3, 3, 2><<<grid, 256, 0, stream>>>(p);
    else if (t.shape == 4) product_kernel<T, AL, BL, GATED, 320, 128, 2, 2, 64, 3, 2, 1><<<grid, 256, 0, stream>>>(p);
    else product_kernel<T, AL, BL, GATED, 320, 256, 2, 4, 64, 2, 2, 2><<<grid, 512, 0, stream>>>(p);
  }
  return launched();
}

}  // namespace ffn
