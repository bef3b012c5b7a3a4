// Quantisation to NVFP4 operands (codes and tiled scales), of plain rows, of
// rows sent to their experts, and of the experts' gated activations; and back.
#include "moe_common.h"

namespace moe {
namespace {

constexpr int kTileThreads = 512;
constexpr int kTileAtoms = 4;                        // atoms along K of a tile: 256 K-elements
constexpr int kTileBlocks = kTileAtoms * 4;          // 16-element blocks of a tile's row
constexpr int kRowThreads = 256;
constexpr int64_t kMaxGrid = (1 << 23) - 1;          // workgroups: fewer than 2^32 threads, and 2^31 of a row kernel

// ---- one block of 16 ---------------------------------------------------------
// The rounding of a quotient to few bits is exact where the quotient is rounded
// to odd before: the nearest fp32 q to a / s, moved towards zero if it is above
// a / s, with the last bit set if it is not a / s itself. `inverse` is the
// nearest fp32 to 1 / s. a * inverse can be an ulp off; a fused multiply-add with
// what it leaves gives the nearest quotient (Markstein's correction), and the
// sign of a - q s, without error from another one, its side. On magnitudes.
__device__ inline uint32_t quotient_to_odd(float a, float s, float inverse) {
  const float near = a * inverse, q = fmaf(fmaf(-near, s, a), inverse, near), rest = fmaf(-q, s, a);
  uint32_t u = __builtin_bit_cast(uint32_t, q);
  u -= rest < 0.f;
  return u | (rest != 0.f);
}
// An fp64 value >= 0 to fp32, to odd.
__device__ inline float to_odd(double d) {
  const float f = (float)d;
  uint32_t u = __builtin_bit_cast(uint32_t, f);
  u -= (double)f > d;
  u |= (double)f != d;
  return __builtin_bit_cast(float, u);
}

__device__ inline uint32_t e4m3_of(float v) {  // v >= 0
  return __builtin_amdgcn_cvt_pk_fp8_f32(fminf(v, 448.f), 0.f, 0, false) & 0xFF;
}
__device__ inline float e4m3_value(uint32_t byte) { return __builtin_amdgcn_cvt_f32_fp8((int)byte, 0); }

// Two E2M1 codes into byte kByte of `into`; values beyond 6 give 6.
template <int kByte> __device__ inline uint32_t e2m1_pair(uint32_t into, float a, float b) {
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(into, a, b, 1.f, kByte);
}
__device__ inline uint32_t e2m1_word(const float* q) {
  uint32_t w = 0;
  w = e2m1_pair<0>(w, q[0], q[1]);
  w = e2m1_pair<1>(w, q[2], q[3]);
  w = e2m1_pair<2>(w, q[4], q[5]);
  return e2m1_pair<3>(w, q[6], q[7]);
}

struct Block {
  u32x2 codes;
  uint32_t scale;  // E4M3 byte
};

constexpr uint32_t kInfBits = 0x7F800000u, kScaleNan = 0x7Fu;

__device__ inline Block encode(const float (&v)[16]) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) top = max(top, __builtin_bit_cast(uint32_t, v[i]) & 0x7FFFFFFFu);
  Block b;
  const float sixth = __builtin_bit_cast(float, quotient_to_odd(__builtin_bit_cast(float, top), 6.f, 1.f / 6.f));
  b.scale = e4m3_of(sixth);
  const float s = e4m3_value(b.scale), inverse = s == 0.f ? 0.f : 1.f / s;
  float q[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const uint32_t u = quotient_to_odd(fabsf(v[i]), s, inverse);
    q[i] = __builtin_bit_cast(float, u | (__builtin_bit_cast(uint32_t, v[i]) & 0x80000000u));
  }
  b.codes.x = e2m1_word(q);
  b.codes.y = e2m1_word(q + 8);
  if (top >= kInfBits) {  // an infinity or NaN in the block
    b.scale = kScaleNan;
    b.codes = u32x2{0u, 0u};
  } else if (b.scale == 0) {
    b.codes = u32x2{0u, 0u};
  }
  return b;
}

// ---- where blocks come from ----------------------------------------------------
template <class T> struct RowSource {
  const void* x;
  int64_t row_stride, batch_stride;
  int64_t m;  // rows of a batch
  float scale;
  int vec;

  __device__ inline Block block(int64_t row, int, int kb) const {
    const int64_t at = (m > 0 ? row / m * batch_stride + row % m * row_stride : row * row_stride) + kb * 16;
    Raw8<T> raw[2];
    raw[0].load(x, at, vec);
    raw[1].load(x, at + 8, vec);
    float v[16];
    raw[0].values(v);
    raw[1].values(v + 8);
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] *= scale;
    return encode(v);
  }
};

// silu(g alpha) (u alpha) scale. In fp32 first, with a bound on its error: the
// products, 1 + e^-g, its reciprocal and e^-g itself (|g| 2^-24 through its
// argument, |g| < 100 where it counts) stay within kUnsure of the exact value.
// Where a code or the scale would be another one within that bound, the block
// is done again in fp64. So the results are those of the exact activation, and
// do not depend on how exp is computed.
constexpr float kUnsure = 1.f / 65536;

__device__ inline double silu_f64(double g) { return g / (1.0 + exp(-g)); }

__device__ inline Block encode_f64(const double (&v)[16]) {
  double top = 0.0;
#pragma unroll
  for (int i = 0; i < 16; ++i) top = fmax(top, fabs(v[i]));
  Block b;
  b.scale = e4m3_of(to_odd(top / 6.0));
  const double s = e4m3_value(b.scale), inverse = s == 0.0 ? 0.0 : 1.0 / s;
  float q[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) q[i] = copysignf(to_odd(fmin(fabs(v[i]) * inverse, 16.0)), (float)v[i]);
  b.codes.x = e2m1_word(q);
  b.codes.y = e2m1_word(q + 8);
  if (b.scale == 0) b.codes = u32x2{0u, 0u};
  return b;
}

template <class T> struct SwigluSource {
  const void* c;
  int64_t row_stride;
  const float* alpha;
  int k, vec;
  float scale;

  __device__ inline Block block(int64_t row, int expert, int kb) const {
    const int64_t at = row * row_stride + kb * 16;
    Raw8<T> raw[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) raw[i].load(c, at + i / 2 * k + i % 2 * 8, vec);
    float g[16], u[16], v[16];
    raw[0].values(g);
    raw[1].values(g + 8);
    raw[2].values(u);
    raw[3].values(u + 8);
    const float al = alpha == nullptr ? 1.f : alpha[expert];
    uint32_t top = 0;
    float factor = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float ga = g[i] * al, ua = u[i] * al * scale;
      const float sigmoid = __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(ga * -1.44269502f));
      v[i] = ga * sigmoid * ua;
      factor = fmaxf(factor, fabsf(ua));
      top = max(top, __builtin_bit_cast(uint32_t, v[i]) & 0x7FFFFFFFu);
    }
    Block b;
    const float sixth = __builtin_bit_cast(float, top) * (1.f / 6.f);
    b.scale = e4m3_of(sixth * (1.f - kUnsure));
    // a sigmoid below 2^-126 is 0 here: g times it would count with a factor this large only
    bool unsure = factor > 0x1p+90f || b.scale != e4m3_of(sixth * (1.f + kUnsure));
    const float s = e4m3_value(b.scale), inverse = s == 0.f ? 0.f : __builtin_amdgcn_rcpf(s);
    const float low = inverse * (1.f - kUnsure), high = inverse * (1.f + kUnsure);
    float q[16], r[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      q[i] = v[i] * low;
      r[i] = v[i] * high;
    }
    b.codes.x = e2m1_word(q);
    b.codes.y = e2m1_word(q + 8);
    unsure |= b.codes.x != e2m1_word(r) || b.codes.y != e2m1_word(r + 8);
    if (top >= kInfBits) {
      // an infinity or NaN in an operand, or a product beyond fp32
      b.scale = kScaleNan;
      b.codes = u32x2{0u, 0u};
    } else if (unsure) {
      double w[16];
#pragma unroll
      for (int i = 0; i < 16; ++i)
        w[i] = silu_f64((double)g[i] * al) * ((double)u[i] * al) * scale;
      b = encode_f64(w);
    } else if (b.scale == 0) {
      b.codes = u32x2{0u, 0u};
    }
    return b;
  }
};

// ---- where rows lie ------------------------------------------------------------
// Rows in batches of m (offsets null), or sorted by expert.
struct Rows {
  const int32_t *offsets, *atoms;
  int experts;
  int64_t rows, m;  // all of them, of a batch

  __device__ inline int last_at_most(const int32_t* starts, int v) const {
    int low = 0, high = experts;  // starts[low] <= v < starts[high]
    while (high - low > 1) {
      const int mid = (low + high) / 2;
      if (starts[mid] <= v) low = mid;
      else high = mid;
    }
    return low;
  }
  // Expert (or batch) of a row, its atom row and its row in that.
  __device__ inline void find(int64_t row, int& expert, int64_t& atom, int& r) const {
    if (offsets == nullptr) {
      const int64_t batch = row / m, at = row % m;
      expert = 0;
      atom = batch * ceil_div64(m, kAtomRows) + at / kAtomRows;
      r = (int)(at % kAtomRows);
    } else {
      expert = last_at_most(offsets, (int)row);
      const int at = (int)row - offsets[expert];
      atom = atoms[expert] + at / kAtomRows;
      r = at % kAtomRows;
    }
  }
  // First row of an atom row, how many rows it holds (0: there is no such atom row), its expert.
  __device__ inline int64_t first_row(int64_t atom, int& count, int& expert) const {
    if (offsets == nullptr) {
      const int64_t per = ceil_div64(m, kAtomRows), batch = atom / per, at = atom % per * kAtomRows;
      expert = 0;
      count = (int)min((int64_t)kAtomRows, m - at);
      return batch * m + at;
    }
    if (atom >= atoms[experts]) {
      count = expert = 0;
      return 0;
    }
    expert = last_at_most(atoms, (int)atom);
    const int at = ((int)atom - atoms[expert]) * kAtomRows, first = offsets[expert] + at;
    count = min(kAtomRows, offsets[expert + 1] - first);
    return first;
  }
};

__device__ inline uint32_t or_quad(uint32_t v) {
  v |= __builtin_amdgcn_mov_dpp(v, 0xB1, 0xF, 0xF, false);
  return v | __builtin_amdgcn_mov_dpp(v, 0x4E, 0xF, 0xF, false);
}

// A row of blocks, padded to whole atoms: block kb of row `row`, from the index
// of a thread.
struct Place {
  int64_t row;
  int kb;
};
__device__ inline Place place_of(uint32_t index, uint32_t padded) {
  return {(int64_t)(index / padded), (int)(index % padded)};
}

// Few rows per expert: a thread per block; four lanes join their scales to the
// word of an atom's row.
template <class Source>
__global__ void __launch_bounds__(kRowThreads)
    nvfp4_quantize_rows_kernel(Source src, Rows rows, int blocks, uint8_t* a, uint8_t* sfa) {
  const int padded = ceil_div(blocks, 4) * 4;
  const Place p = place_of(blockIdx.x * kRowThreads + threadIdx.x, padded);
  const int64_t end = rows.offsets == nullptr ? rows.rows : rows.offsets[rows.experts];
  if (p.row >= end) return;  // for four lanes at a time
  int expert, r;
  int64_t atom;
  rows.find(p.row, expert, atom, r);
  uint32_t scale = 0;
  if (p.kb < blocks) {
    const Block b = src.block(p.row, expert, p.kb);
    *(u32x2*)(a + (p.row * blocks + p.kb) * 8) = b.codes;
    scale = b.scale << (p.kb % 4 * 8);
  }
  scale = or_quad(scale);
  if (p.kb % 4 == 0) *(uint32_t*)(sfa + (atom * (padded / 4) + p.kb / 4) * kAtomBytes + atom_row(r)) = scale;
}

// Many rows: a workgroup per tile of 128 rows x 256 K-elements. Codes are
// stored 128 bytes of a row at a time; the tile's scales are collected in
// shared memory and stored as the 2 KB that they are.
template <class Source>
__global__ void __launch_bounds__(kTileThreads)
    nvfp4_quantize_tiles_kernel(Source src, Rows rows, int blocks, uint8_t* a, uint8_t* sfa) {
  __shared__ uint32_t s_sf[kTileAtoms * kAtomBytes / 4];
  const int along = ceil_div(blocks, 4), chunks = ceil_div(along, kTileAtoms);
  const int64_t atom = blockIdx.x / chunks;
  const int first_atom = blockIdx.x % chunks * kTileAtoms;
  int count, expert;
  const int64_t first = rows.first_row(atom, count, expert);
  if (count == 0) return;
  const int kt = threadIdx.x % kTileBlocks, kb = first_atom * 4 + kt;
#pragma unroll
  for (int pass = 0; pass < kAtomRows / (kTileThreads / kTileBlocks); ++pass) {
    const int r = pass * (kTileThreads / kTileBlocks) + threadIdx.x / kTileBlocks;
    uint32_t scale = 0;
    if (r < count && kb < blocks) {
      const Block b = src.block(first + r, expert, kb);
      *(u32x2*)(a + ((first + r) * blocks + kb) * 8) = b.codes;
      scale = b.scale;
    }
    ((uint8_t*)s_sf)[kt / 4 * kAtomBytes + atom_row(r) + kt % 4] = (uint8_t)scale;
  }
  __syncthreads();
  const int words = min(kTileAtoms, along - first_atom) * (kAtomBytes / 4);
  uint32_t* to = (uint32_t*)(sfa + (atom * along + first_atom) * kAtomBytes);
  for (int i = threadIdx.x; i < words; i += kTileThreads) to[i] = s_sf[i];
}

// Dispatch: a token's row is quantised once and its codes stored to the rows of
// all its slots. kDirect: so are its scales, a word at a time; else they go to
// token_scales [tokens][atoms along k, padded to fours] and nvfp4_dispatch_scales_kernel lays them out.
struct Slots {
  const int32_t *ids, *slot_rows, *offsets, *atoms;
  int topk, experts;
};
template <class T, bool kDirect>
__global__ void __launch_bounds__(kRowThreads)
    nvfp4_dispatch_kernel(RowSource<T> src, Slots slots, int64_t tokens, int blocks, uint8_t* a, uint8_t* sfa,
                          uint32_t* token_scales) {
  const int padded = ceil_div(blocks, 4) * 4;
  const Place p = place_of(blockIdx.x * kRowThreads + threadIdx.x, padded);
  if (p.row >= tokens) return;
  Block b = {u32x2{0u, 0u}, 0u};
  if (p.kb < blocks) b = src.block(p.row, 0, p.kb);
  const uint32_t word = or_quad(b.scale << (p.kb % 4 * 8));
  for (int j = 0; j < slots.topk; ++j) {
    const int64_t slot = p.row * slots.topk + j;
    const int row = slots.slot_rows[slot];
    if (row < 0) continue;
    if (p.kb < blocks) *(u32x2*)(a + ((int64_t)row * blocks + p.kb) * 8) = b.codes;
    if (kDirect && p.kb % 4 == 0) {
      const int e = slots.ids[slot], at = row - slots.offsets[e];
      const int64_t atom = slots.atoms[e] + at / kAtomRows;
      *(uint32_t*)(sfa + (atom * (padded / 4) + p.kb / 4) * kAtomBytes + atom_row(at % kAtomRows)) = word;
    }
  }
  if (!kDirect && p.kb % 4 == 0) token_scales[p.row * (ceil_div(padded, 16) * 4) + p.kb / 4] = word;
}

// Scales of the rows sorted by expert, whole atoms at a time: thread = row of
// the atom row, in the order in which its words lie. A token's words are padded
// to a multiple of four, so that they are read four atoms at a time.
constexpr int kScaleThreads = 128;
constexpr int kScaleAtoms = 16;  // along K, of a workgroup
__global__ void __launch_bounds__(kScaleThreads)
    nvfp4_dispatch_scales_kernel(const uint32_t* token_scales, const int32_t* row_slots, int topk, Rows rows,
                                 int along, uint8_t* sfa) {
  const int chunks = ceil_div(along, kScaleAtoms), stride = ceil_div(along, 4) * 4;
  const int64_t atom = blockIdx.x / chunks;
  const int from = blockIdx.x % chunks * kScaleAtoms;
  int count, expert;
  const int64_t first = rows.first_row(atom, count, expert);
  if (count == 0) return;
  const int r = threadIdx.x / 4 + threadIdx.x % 4 * 32;
  const int64_t token = r < count ? row_slots[first + r] / topk : -1;
  const uint32_t* in = token_scales + token * stride;
  uint32_t* out = (uint32_t*)(sfa + atom * along * kAtomBytes) + threadIdx.x;
  u32x4 word[kScaleAtoms / 4];
#pragma unroll
  for (int i = 0; i < kScaleAtoms / 4; ++i)
    word[i] = token >= 0 && from + i * 4 < along ? *(const u32x4*)(in + from + i * 4) : u32x4{0u, 0u, 0u, 0u};
#pragma unroll
  for (int i = 0; i < kScaleAtoms; ++i)
    if (from + i < along) out[(from + i) * (kAtomBytes / 4)] = word[i / 4][i % 4];
}

// ---- back to values ---------------------------------------------------------------
// Eight values to a thread: a wave's stores then fill whole lines at once.
__device__ inline void decode(uint32_t codes, uint32_t scale, float (&v)[8]) {
  const float s = e4m3_value(scale);
  const f32x2 p0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.f, 0);
  const f32x2 p1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.f, 1);
  const f32x2 p2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.f, 2);
  const f32x2 p3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.f, 3);
  v[0] = p0.x * s;
  v[1] = p0.y * s;
  v[2] = p1.x * s;
  v[3] = p1.y * s;
  v[4] = p2.x * s;
  v[5] = p2.y * s;
  v[6] = p3.x * s;
  v[7] = p3.y * s;
}

template <class T>
__global__ void __launch_bounds__(kRowThreads)
    nvfp4_dequantize_rows_kernel(const uint32_t* a, const uint8_t* sfa, Rows rows, int blocks, void* out,
                                 int64_t row_stride, int vec) {
  const Place p = place_of(blockIdx.x * kRowThreads + threadIdx.x, 2 * blocks);  // halves of blocks
  const int64_t end = rows.offsets == nullptr ? rows.rows : rows.offsets[rows.experts];
  if (p.row >= end) return;
  int expert, r;
  int64_t atom;
  rows.find(p.row, expert, atom, r);
  const int kb = p.kb / 2;
  float v[8];
  decode(a[p.row * 2 * blocks + p.kb], sfa[(atom * ceil_div(blocks, 4) + kb / 4) * kAtomBytes + atom_row(r) + kb % 4], v);
  store8<T>(out, p.row * row_stride + p.kb * 8, vec, v);
}

template <class T>
__global__ void __launch_bounds__(kTileThreads)
    nvfp4_dequantize_tiles_kernel(const uint32_t* a, const uint8_t* sfa, Rows rows, int blocks, void* out,
                                  int64_t row_stride, int vec) {
  __shared__ uint32_t s_sf[kTileAtoms * kAtomBytes / 4];
  constexpr int kHalves = 2 * kTileBlocks, kPassRows = kTileThreads / kHalves;
  const int along = ceil_div(blocks, 4), chunks = ceil_div(along, kTileAtoms);
  const int64_t atom = blockIdx.x / chunks;
  const int first_atom = blockIdx.x % chunks * kTileAtoms;
  int count, expert;
  const int64_t first = rows.first_row(atom, count, expert);
  if (count == 0) return;
  const int half = threadIdx.x % kHalves, kh = first_atom * 8 + half;
  uint32_t codes[kAtomRows / kPassRows];
#pragma unroll
  for (int pass = 0; pass < kAtomRows / kPassRows; ++pass) {
    const int r = pass * kPassRows + threadIdx.x / kHalves;
    codes[pass] = r < count && kh < 2 * blocks ? __builtin_nontemporal_load(a + (first + r) * 2 * blocks + kh) : 0u;
  }
  const int words = min(kTileAtoms, along - first_atom) * (kAtomBytes / 4);
  const uint32_t* from = (const uint32_t*)(sfa + (atom * along + first_atom) * kAtomBytes);
  for (int i = threadIdx.x; i < words; i += kTileThreads) s_sf[i] = from[i];
  __syncthreads();
  if (kh >= 2 * blocks) return;
#pragma unroll
  for (int pass = 0; pass < kAtomRows / kPassRows; ++pass) {
    const int r = pass * kPassRows + threadIdx.x / kHalves;
    if (r >= count) break;
    float v[8];
    decode(codes[pass], ((const uint8_t*)s_sf)[half / 8 * kAtomBytes + atom_row(r) + half / 2 % 4], v);
    store8<T>(out, (first + r) * row_stride + kh * 8, vec, v);
  }
}

// ---- host ---------------------------------------------------------------------------
// Atom rows that `rows` rows can have.
int64_t atom_rows(const Rows& r, int64_t batches) {
  if (r.offsets == nullptr) return batches * ceil_div64(r.m, kAtomRows);
  const int64_t used = r.rows < r.experts ? r.rows : r.experts;
  return (r.rows - used) / kAtomRows + used;
}

// Tiles pay from 16 rows of an atom on (of 128: below, most threads of a tile have no row).
bool tiles_pay(const Rows& r) { return r.offsets == nullptr ? r.m >= 16 : r.rows >= (int64_t)16 * r.experts; }

template <class Source>
int launch_quantize(const Source& src, const Rows& rows, int64_t batches, int blocks, void* a, void* sfa, hipStream_t st) {
  if (tiles_pay(rows)) {
    const int64_t grid = atom_rows(rows, batches) * ceil_div(ceil_div(blocks, 4), kTileAtoms);
    if (grid > kMaxGrid) return NVFP4_ERR_INVALID;
    nvfp4_quantize_tiles_kernel<<<(unsigned)grid, kTileThreads, 0, st>>>(src, rows, blocks, (uint8_t*)a, (uint8_t*)sfa);
  } else {
    const int64_t grid = ceil_div64(rows.rows * (ceil_div(blocks, 4) * 4), kRowThreads);
    if (grid > kMaxGrid) return NVFP4_ERR_INVALID;
    nvfp4_quantize_rows_kernel<<<(unsigned)grid, kRowThreads, 0, st>>>(src, rows, blocks, (uint8_t*)a, (uint8_t*)sfa);
  }
  return launched();
}

constexpr int64_t kMaxRows = (int64_t)1 << 31, kMaxStride = (int64_t)1 << 40;

int check_operand(int64_t rows, int k, const void* a, const void* sfa) {
  if (rows < 0 || rows >= kMaxRows || k < 0 || k % 32 || k > 1 << 22) return NVFP4_ERR_INVALID;
  if (rows > 0 && k > 0 && (a == nullptr || sfa == nullptr)) return NVFP4_ERR_INVALID;
  return aligned(a, 16) && aligned(sfa, 16) ? NVFP4_OK : NVFP4_ERR_MISALIGNED;
}
int check_source(const void* x, int dtype, int64_t rows, int width, int64_t stride) {
  if (!known_type(dtype) || stride < width || stride > kMaxStride) return NVFP4_ERR_INVALID;
  if (rows > 0 && width > 0 && x == nullptr) return NVFP4_ERR_INVALID;
  return aligned(x, element_bytes(dtype)) ? NVFP4_OK : NVFP4_ERR_MISALIGNED;
}
int check_sorted(const int32_t* offsets, const int32_t* atoms, int experts) {
  if (experts < 1 || experts > NVFP4_MOE_MAX_EXPERTS) return NVFP4_ERR_INVALID;
  if ((offsets == nullptr) != (atoms == nullptr) || (offsets == nullptr && experts != 1)) return NVFP4_ERR_INVALID;
  return aligned(offsets, 4) && aligned(atoms, 4) ? NVFP4_OK : NVFP4_ERR_MISALIGNED;
}

// Scales go straight to their atoms where an expert has few rows: its atoms'
// lines would not fill up in any order, and one launch is saved.
bool direct_scales(int64_t tokens, int topk, int experts) { return tokens * topk < (int64_t)16 * experts; }

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int nvfp4_moe_quantize(const void* x, int dtype, int l, int64_t m, int k, int64_t batch_stride, int64_t row_stride,
                       float scale, void* a, void* sfa, void* stream) {
  if (l < 1 || m < 0 || m >= kMaxRows || l * m >= kMaxRows) return NVFP4_ERR_INVALID;
  if (int rc = check_source(x, dtype, m, k, row_stride)) return rc;
  if (int rc = check_operand(l * m, k, a, sfa)) return rc;
  if (batch_stride < 0 || batch_stride > kMaxStride) return NVFP4_ERR_INVALID;
  if (m == 0 || k == 0) return NVFP4_OK;
  const bool vec = wide_rows(x, dtype, row_stride) && (l == 1 || batch_stride * element_bytes(dtype) % 16 == 0);
  const Rows rows = {nullptr, nullptr, 1, l * m, m};
  return with_type(dtype, [&](auto t) {
    const RowSource<decltype(t)> src = {x, row_stride, batch_stride, l > 1 ? m : 0, scale, vec};
    return launch_quantize(src, rows, l, k / 16, a, sfa, (hipStream_t)stream);
  });
}

size_t nvfp4_moe_dispatch_workspace_bytes(int64_t tokens, int topk, int k, int experts) {
  if (tokens <= 0 || topk < 1 || k <= 0 || direct_scales(tokens, topk, experts)) return 0;
  return (size_t)tokens * ceil_div(k, 4 * kAtomK) * 16;
}

int nvfp4_moe_dispatch(const void* x, int dtype, int64_t tokens, int topk, int k, int64_t row_stride, float scale,
                       const int32_t* ids, const int32_t* slot_rows, const int32_t* row_slots,
                       const int32_t* offsets, const int32_t* atoms, int experts, void* a, void* sfa,
                       void* workspace, size_t workspace_bytes, void* stream) {
  if (topk < 1 || topk > NVFP4_MOE_MAX_TOPK || tokens < 0 || tokens * topk > (int64_t)1 << 30) return NVFP4_ERR_INVALID;
  if (int rc = check_source(x, dtype, tokens, k, row_stride)) return rc;
  if (int rc = check_operand(tokens * topk, k, a, sfa)) return rc;
  if (offsets == nullptr) return NVFP4_ERR_INVALID;
  if (int rc = check_sorted(offsets, atoms, experts)) return rc;
  if (tokens > 0 && (ids == nullptr || slot_rows == nullptr || row_slots == nullptr)) return NVFP4_ERR_INVALID;
  if (!aligned(ids, 4) || !aligned(slot_rows, 4) || !aligned(row_slots, 4)) return NVFP4_ERR_MISALIGNED;
  if (tokens == 0 || k == 0) return NVFP4_OK;
  const size_t need = nvfp4_moe_dispatch_workspace_bytes(tokens, topk, k, experts);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return NVFP4_ERR_WORKSPACE;
  if (need > 0 && !aligned(workspace, 256)) return NVFP4_ERR_MISALIGNED;
  const int blocks = k / 16, along = ceil_div(blocks, 4);
  const int64_t grid = ceil_div64(tokens * along * 4, kRowThreads);
  const Rows rows = {offsets, atoms, experts, tokens * topk, 0};
  const int64_t scale_grid = atom_rows(rows, 1) * ceil_div(along, kScaleAtoms);
  if (grid > kMaxGrid || scale_grid > kMaxGrid) return NVFP4_ERR_INVALID;
  const Slots slots = {ids, slot_rows, offsets, atoms, topk, experts};
  const hipStream_t st = (hipStream_t)stream;
  int rc = with_type(dtype, [&](auto t) {
    using T = decltype(t);
    const RowSource<T> src = {x, row_stride, 0, 0, scale, wide_rows(x, dtype, row_stride)};
    if (need == 0)
      nvfp4_dispatch_kernel<T, true><<<(unsigned)grid, kRowThreads, 0, st>>>(src, slots, tokens, blocks, (uint8_t*)a,
                                                                            (uint8_t*)sfa, nullptr);
    else
      nvfp4_dispatch_kernel<T, false><<<(unsigned)grid, kRowThreads, 0, st>>>(src, slots, tokens, blocks, (uint8_t*)a,
                                                                             (uint8_t*)sfa, (uint32_t*)workspace);
    return launched();
  });
  if (rc != NVFP4_OK || need == 0) return rc;
  nvfp4_dispatch_scales_kernel<<<(unsigned)scale_grid, kScaleThreads, 0, st>>>((const uint32_t*)workspace, row_slots, topk,
                                                                            rows, along, (uint8_t*)sfa);
  return launched();
}

int nvfp4_moe_swiglu(const void* c, int dtype, int64_t rows, int k, int64_t row_stride, const float* alpha,
                     float scale, const int32_t* offsets, const int32_t* atoms, int experts, void* a, void* sfa,
                     void* stream) {
  if (int rc = check_operand(rows, k, a, sfa)) return rc;
  if (int rc = check_source(c, dtype, rows, 2 * k, row_stride)) return rc;
  if (int rc = check_sorted(offsets, atoms, experts)) return rc;
  if (!aligned(alpha, 4)) return NVFP4_ERR_MISALIGNED;
  if (rows == 0 || k == 0) return NVFP4_OK;
  const Rows where = {offsets, atoms, experts, rows, rows};
  return with_type(dtype, [&](auto t) {
    const SwigluSource<decltype(t)> src = {c, row_stride, alpha, k, wide_rows(c, dtype, row_stride), scale};
    return launch_quantize(src, where, 1, k / 16, a, sfa, (hipStream_t)stream);
  });
}

int nvfp4_moe_dequantize(const void* a, const void* sfa, int l, int64_t m, int k, const int32_t* offsets,
                         const int32_t* atoms, int experts, void* out, int dtype, int64_t row_stride, void* stream) {
  if (l < 1 || m < 0 || m >= kMaxRows || l * m >= kMaxRows || (offsets != nullptr && l != 1)) return NVFP4_ERR_INVALID;
  if (int rc = check_operand(l * m, k, a, sfa)) return rc;
  if (int rc = check_source(out, dtype, m, k, row_stride)) return rc;
  if (int rc = check_sorted(offsets, atoms, experts)) return rc;
  if (m == 0 || k == 0) return NVFP4_OK;
  const Rows rows = {offsets, atoms, experts, l * m, m};
  const int blocks = k / 16;
  const bool tiles = tiles_pay(rows);
  const int64_t grid = tiles ? atom_rows(rows, l) * ceil_div(ceil_div(blocks, 4), kTileAtoms)
                             : ceil_div64(rows.rows * 2 * blocks, kRowThreads);
  if (grid > kMaxGrid) return NVFP4_ERR_INVALID;
  const hipStream_t st = (hipStream_t)stream;
  return with_type(dtype, [&](auto t) {
    using T = decltype(t);
    const int vec = wide_rows(out, dtype, row_stride);
    if (tiles)
      nvfp4_dequantize_tiles_kernel<T><<<(unsigned)grid, kTileThreads, 0, st>>>((const uint32_t*)a, (const uint8_t*)sfa, rows,
                                                                                blocks, out, row_stride, vec);
    else
      nvfp4_dequantize_rows_kernel<T><<<(unsigned)grid, kRowThreads, 0, st>>>((const uint32_t*)a, (const uint8_t*)sfa, rows,
                                                                              blocks, out, row_stride, vec);
    return launched();
  });
}

}  // extern "C"
