// Quantisation to NVFP4 operands (codes and tiled scales), of plain rows, of
// rows sent to their experts, and of the experts' gated activations; and back.
#include "moe_common.h"

namespace moe {
namespace {

constexpr int kTileThreads = 1024;
constexpr int kTileAtoms = 4;                        // atoms along K of a tile: 256 K-elements
constexpr int kTileHalves = kTileAtoms * 8;          // halves of 16-element blocks of a tile's row
constexpr int kRowThreads = 256;
constexpr int64_t kMaxGrid = (1 << 23) - 1;          // workgroups of a row kernel: fewer than 2^31 threads
constexpr int64_t kMaxTiles = (1 << 22) - 1;         // of a tile kernel: fewer than 2^32 threads, which a launch can have

// ---- half a block of 16 to a lane: a wave's loads and stores take whole lines ---------------------------------------------------------
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

// The other lane of a block's two.
__device__ inline uint32_t pair(uint32_t v) { return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, false); }
__device__ inline double pair(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  return __builtin_bit_cast(double, (uint64_t)pair((uint32_t)(u >> 32)) << 32 | pair((uint32_t)u));
}

struct Half {
  uint32_t codes;  // of eight elements
  uint32_t scale;  // E4M3 byte of their block
};

constexpr uint32_t kInfBits = 0x7F800000u, kScaleNan = 0x7Fu;

__device__ inline Half encode(const float (&v)[8]) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, __builtin_bit_cast(uint32_t, v[i]) & 0x7FFFFFFFu);
  top = max(top, pair(top));
  Half b;
  const float sixth = __builtin_bit_cast(float, quotient_to_odd(__builtin_bit_cast(float, top), 6.f, 1.f / 6.f));
  b.scale = e4m3_of(sixth);
  const float s = e4m3_value(b.scale), inverse = s == 0.f ? 0.f : 1.f / s;
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t u = quotient_to_odd(fabsf(v[i]), s, inverse);
    q[i] = __builtin_bit_cast(float, u | (__builtin_bit_cast(uint32_t, v[i]) & 0x80000000u));
  }
  b.codes = b.scale == 0 ? 0u : e2m1_word(q);
  if (top >= kInfBits) b = {0u, kScaleNan};  // an infinity or NaN in the block
  return b;
}

// The same for 16-bit values as they are. They and the borders of the rounding
// (s times 3-bit numbers) have so few bits that a quotient either is a border or
// is off it by 2^-8 (bf16) or 2^-11 (fp16) of its value: bf16 quotients may lose
// all but 11 bits before, which restores those that are borders from an error of
// an ulp or two; fp16 ones are made the nearest fp32 as above.
template <class T> __device__ inline Half encode_16bit(const Raw8<T>& x) {
  typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
  constexpr uint32_t kInf16 = T::kId == NVFP4_MOE_F16 ? 0x7C00u : 0x7F80u;
  u16x2 tops = {0, 0};  // magnitudes order as whole numbers
#pragma unroll
  for (int i = 0; i < 4; ++i) tops = __builtin_elementwise_max(tops, __builtin_bit_cast(u16x2, x.w[0][i] & 0x7FFF7FFFu));
  uint32_t top = max((uint32_t)tops.x, (uint32_t)tops.y);
  top = max(top, pair(top));
  float largest, unused, v[8];
  unpack2<T>(top, largest, unused);
  Half b;
  b.scale = e4m3_of(__builtin_bit_cast(float, quotient_to_odd(largest, 6.f, 1.f / 6.f)));
  const float s = e4m3_value(b.scale), inverse = s == 0.f ? 0.f : 1.f / s;
  x.values(v);
  if constexpr (T::kId == NVFP4_MOE_BF16) {
    f16x2 q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // a saturated scale leaves quotients beyond f16's range
      q[i].x = (_Float16)__builtin_amdgcn_fmed3f(v[2 * i] * inverse, -16.f, 16.f);
      q[i].y = (_Float16)__builtin_amdgcn_fmed3f(v[2 * i + 1] * inverse, -16.f, 16.f);
    }
    b.codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(0u, q[0], 1.f, 0);
    b.codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(b.codes, q[1], 1.f, 1);
    b.codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(b.codes, q[2], 1.f, 2);
    b.codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(b.codes, q[3], 1.f, 3);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float near = v[i] * inverse;
      v[i] = fmaf(fmaf(-near, s, v[i]), inverse, near);
    }
    b.codes = e2m1_word(v);
  }
  if (b.scale == 0) b.codes = 0u;
  if (top >= kInf16) b = {0u, kScaleNan};
  return b;
}

// ---- where halves come from ----------------------------------------------------
// kAsIs: 16-bit rows whose factor is 1.
template <class T, bool kAsIs> struct RowSource {
  const void* x;
  int64_t row_stride, batch_stride;
  int64_t m;  // rows of a batch
  float scale;
  int vec;

  // Half kh of a row.
  __device__ inline Half half(int64_t row, int, int kh) const {
    Raw8<T> raw;
    raw.load(x, (m > 0 ? row / m * batch_stride + row % m * row_stride : row * row_stride) + kh * 8, vec);
    if constexpr (kAsIs) {
      return encode_16bit<T>(raw);
    } else {
      float v[8];
      raw.values(v);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] *= scale;
      return encode(v);
    }
  }
};

// silu(g alpha) (u alpha) scale. In fp32 first, with a bound on its error: the
// products, 1 + e^-g, its reciprocal and e^-g itself (|g| 2^-24 through its
// argument, |g| < 100 where it counts) stay within kUnsure of the exact value.
// Where a code or the scale would be another one within that bound, the block
// is done again in fp64; so are blocks whose factors leave the range where the
// bound holds, and those that come out infinite or NaN. So the results are those
// of the exact activation, and do not depend on how exp is computed.
constexpr float kUnsure = 1.f / 65536;

__device__ inline double silu_f64(double g) { return g / (1.0 + exp(-g)); }

__device__ inline Half encode_f64(const double (&v)[8]) {
  double top = 0.0;
  uint32_t bad = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    top = fmax(top, fabs(v[i]));
    bad |= !(fabsf((float)v[i]) < INFINITY);  // beyond fp32, or NaN
  }
  top = fmax(top, pair(top));
  if (bad | pair(bad)) return {0u, kScaleNan};
  Half b;
  b.scale = e4m3_of(to_odd(top / 6.0));
  const double s = e4m3_value(b.scale), inverse = s == 0.0 ? 0.0 : 1.0 / s;
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = copysignf(to_odd(fmin(fabs(v[i]) * inverse, 16.0)), (float)v[i]);
  b.codes = b.scale == 0 ? 0u : e2m1_word(q);
  return b;
}

template <class T> struct SwigluSource {
  const void* c;
  int64_t row_stride;
  const float* alpha;
  int k, vec;
  float scale;

  __device__ inline Half half(int64_t row, int expert, int kh) const {
    const int64_t at = row * row_stride + kh * 8;
    Raw8<T> raw[2];
    raw[0].load(c, at, vec);
    raw[1].load(c, at + k, vec);
    float g[8], u[8], v[8];
    raw[0].values(g);
    raw[1].values(u);
    const float al = alpha == nullptr ? 1.f : alpha[expert], al_scale = al * scale;
    // (an infinite one makes `factor` infinite, or `top` NaN)
    const bool in_range = fabsf(al_scale) >= 0x1p-126f || al == 0.f || scale == 0.f;
    uint32_t top = 0;
    float factor = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float ga = g[i] * al, ua = u[i] * al_scale;
      const float sigmoid = __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(ga * -1.44269502f));
      v[i] = ga * sigmoid * ua;
      factor = fmaxf(fmaxf(factor, fabsf(ua)), fabsf(ga));
      top = max(top, __builtin_bit_cast(uint32_t, v[i]) & 0x7FFFFFFFu);
    }
    top = max(top, pair(top));
    Half b;
    const float sixth = __builtin_bit_cast(float, top) * (1.f / 6.f);
    b.scale = e4m3_of(sixth * (1.f - kUnsure));
    // a factor or a sigmoid below 2^-126 has lost bits or is 0: it would count beside one this large only, but
    // alpha times scale counts beside any u
    uint32_t unsure = top >= kInfBits || factor > 0x1p+90f || !in_range ||
                      b.scale != e4m3_of(sixth * (1.f + kUnsure));
    const float s = e4m3_value(b.scale), inverse = s == 0.f ? 0.f : __builtin_amdgcn_rcpf(s);
    const float low = inverse * (1.f - kUnsure), high = inverse * (1.f + kUnsure);
    float q[8], r[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      q[i] = v[i] * low;
      r[i] = v[i] * high;
    }
    b.codes = e2m1_word(q);
    unsure |= b.codes != e2m1_word(r);
    unsure |= pair(unsure);
    if (b.scale == 0) b.codes = 0u;
    if (unsure) {
      double w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = silu_f64((double)g[i] * al) * ((double)u[i] * al) * scale;
      b = encode_f64(w);
    }
    return b;
  }
};

// ---- where rows lie ------------------------------------------------------------
// The last of `count` parts whose start is at most v, 0 at the least.
__device__ inline int last_at_most(const int32_t* starts, int count, int v) {
  int low = 0, high = count;  // starts[low] <= v < starts[high]
  while (high - low > 1) {
    const int mid = (low + high) / 2;
    if (starts[mid] <= v) low = mid;
    else high = mid;
  }
  return low;
}

// Rows in batches of m (offsets null), or sorted by expert.
struct Rows {
  const int32_t *offsets, *atoms;
  int experts;
  int64_t rows, m;  // all of them, of a batch

  // Expert (or batch) of a row, its atom row and its row in that.
  __device__ inline void find(int64_t row, int& expert, int64_t& atom, int& r) const {
    if (offsets == nullptr) {
      const int64_t batch = row / m, at = row % m;
      expert = 0;
      atom = batch * ceil_div64(m, kAtomRows) + at / kAtomRows;
      r = (int)(at % kAtomRows);
    } else {
      expert = last_at_most(offsets, experts, (int)row);
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
    expert = last_at_most(atoms, experts, (int)atom);
    const int at = ((int)atom - atoms[expert]) * kAtomRows, first = offsets[expert] + at;
    count = min(kAtomRows, offsets[expert + 1] - first);
    if (first < 0 || (int64_t)first + count > rows) count = 0;  // not a plan's offsets: no rows rather than others' memory
    return first;
  }
};

// The scales of an atom's row, in the eight lanes that hold its halves: bytes in
// the order of the blocks.
__device__ inline uint32_t scale_word(uint32_t scale, int kh) {
  uint32_t v = scale << (kh / 2 % 4 * 8);
  v |= (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, false);         // from the pair beside
  return v | (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x141, 0xF, 0xF, false);  // from the other four
}

// A row of halves, padded to whole atoms: half kh of row `row`, from the index of
// a thread.
struct Place {
  int64_t row;
  int kh;
};
__device__ inline Place place_of(uint32_t index, uint32_t padded) {
  return {(int64_t)(index / padded), (int)(index % padded)};
}

// Few rows: eight lanes join the scales of an atom's row to a word. 2048 gated
// rows of 2048 fp16, 19 MB, 9.8 us, of which a launch is 3.
template <class Source>
__global__ void __launch_bounds__(kRowThreads)
    nvfp4_quantize_rows_kernel(Source src, Rows rows, int blocks, uint32_t* a, uint8_t* sfa) {
  const int along = ceil_div(blocks, 4);
  const Place p = place_of(blockIdx.x * kRowThreads + threadIdx.x, along * 8);
  const int64_t end = rows.offsets == nullptr ? rows.rows : rows.offsets[rows.experts];
  if (p.row >= end) return;  // for eight lanes at a time
  int expert, r;
  int64_t atom;
  rows.find(p.row, expert, atom, r);
  uint32_t scale = 0;
  if (p.kh < 2 * blocks) {
    const Half b = src.half(p.row, expert, p.kh);
    a[p.row * 2 * blocks + p.kh] = b.codes;
    scale = b.scale;
  }
  scale = scale_word(scale, p.kh);
  if (p.kh % 8 == 0) *(uint32_t*)(sfa + (atom * along + p.kh / 8) * kAtomBytes + atom_row(r)) = scale;
}

// Many rows: a workgroup per tile of 128 rows x 256 K-elements. Codes are
// stored 128 bytes of a row at a time; the tile's scales are collected in
// shared memory and stored as the 2 KB that they are. Bound by memory, and gated
// rows by the vector instructions of the activation and of its two roundings:
// 16384 x 7168 bf16, 301 MB in 59 us, 5.1 TB/s (a block of 16 to a lane, which
// touches lines in quarters: 65 us); 16390 gated rows of 2048 fp16, 153 MB in 42 us,
// 3.6 TB/s (with every activation in fp64 104 us).
template <class Source>
__global__ void __launch_bounds__(kTileThreads)
    nvfp4_quantize_tiles_kernel(Source src, Rows rows, int blocks, uint32_t* a, uint8_t* sfa) {
  __shared__ uint32_t s_sf[kTileAtoms * kAtomBytes / 4];
  constexpr int kPassRows = kTileThreads / kTileHalves;
  const int along = ceil_div(blocks, 4), chunks = ceil_div(along, kTileAtoms);
  const int64_t atom = blockIdx.x / chunks;
  const int first_atom = blockIdx.x % chunks * kTileAtoms;
  int count, expert;
  const int64_t first = rows.first_row(atom, count, expert);
  if (count == 0) return;
  const int half = threadIdx.x % kTileHalves, kh = first_atom * 8 + half;
#pragma unroll
  for (int pass = 0; pass < kAtomRows / kPassRows; ++pass) {
    const int r = pass * kPassRows + threadIdx.x / kTileHalves;
    uint32_t scale = 0;
    if (r < count && kh < 2 * blocks) {
      const Half b = src.half(first + r, expert, kh);
      a[(first + r) * 2 * blocks + kh] = b.codes;
      scale = b.scale;
    }
    if (half % 2 == 0) ((uint8_t*)s_sf)[half / 8 * kAtomBytes + atom_row(r) + half / 2 % 4] = (uint8_t)scale;
  }
  __syncthreads();
  const int words = min(kTileAtoms, along - first_atom) * (kAtomBytes / 4);
  uint32_t* to = (uint32_t*)(sfa + (atom * along + first_atom) * kAtomBytes);
  for (int i = threadIdx.x; i < words; i += kTileThreads) to[i] = s_sf[i];
}

// Dispatch: a token's row is quantised once and its codes stored to the rows of
// all its slots, four slots at a time: each lane of four takes a slot and stores
// the codes of all four. kDirect: so are the scales, a word at a time; else they go to
// token_scales [tokens][atoms along k, padded to fours] and nvfp4_dispatch_scales_kernel lays them out.
// Bound by memory: 4096 x 7168 bf16 to 31000 rows of 64 experts, 59 MB read and
// 125 MB written in 36 us and 11 for the scales.
// Nothing is stored outside a and sfa, whatever the tables hold: a row has to be
// one of `rows`, an atom row one of `atom_rows`, and a slot's id says only where
// its row's expert is looked for first: a caller may have written other ids there
// since the plan was made.
struct Slots {
  const int32_t *ids, *slot_rows, *offsets, *atoms;
  int topk, experts, rows;
  int64_t atom_rows;

  // Of the expert that has a row, its first row and its first atom row; `id`: where to look first.
  // For all lanes of a wave that have a slot: the search is theirs together, out of the way where no lane needs it
  // (as a branch of each lane's 4096 x 7168 to one of 8 experts each 27.7 us, 25.9 so; 25.2 with the ids trusted).
  __device__ inline void find(bool named, int row, int id, int& first, int& atom) const {
    const int e = (int)min((unsigned)id, (unsigned)(experts - 1));
    const int next = offsets[e + 1];
    first = offsets[e];
    atom = atoms[e];
    if (__any(named && (row < first || row >= next))) {
      const int other = last_at_most(offsets, experts, row);
      first = offsets[other];
      atom = atoms[other];
    }
  }
};
template <int kLane> __device__ inline uint32_t of_quad(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, kLane * 0x55, 0xF, 0xF, false);
}
template <class Source, bool kDirect>
__global__ void __launch_bounds__(kRowThreads)
    nvfp4_dispatch_kernel(Source src, Slots slots, int64_t tokens, int blocks, uint32_t* a, uint8_t* sfa,
                          uint32_t* token_scales) {
  const int along = ceil_div(blocks, 4);
  const Place p = place_of(blockIdx.x * kRowThreads + threadIdx.x, along * 8);
  if (p.row >= tokens) return;  // for eight lanes at a time
  const bool there = p.kh < 2 * blocks;  // for four: k is a multiple of 32
  int j = p.kh % 4, row = -1, id = 0;
  const int64_t slot = p.row * slots.topk;
  auto next = [&] {
    if (j >= slots.topk) return;
    row = slots.slot_rows[slot + j];
    if (kDirect) id = slots.ids[slot + j];
  };
  next();
  Half b = {0u, 0u};
  if (there) b = src.half(p.row, 0, p.kh);
  const uint32_t word = scale_word(b.scale, p.kh);
  const u32x4 codes = {of_quad<0>(b.codes), of_quad<1>(b.codes), of_quad<2>(b.codes), of_quad<3>(b.codes)};
  for (; j < slots.topk; j += 4, next()) {
    const bool named = (unsigned)row < (unsigned)slots.rows;
    if (there && named) *(u32x4*)(a + (int64_t)row * 2 * blocks + p.kh / 4 * 4) = codes;
    if (kDirect && p.kh % 8 < 4) {
      int first, atom;
      slots.find(named, row, id, first, atom);
      const int at = named ? row - first : 0;
      const int64_t place = (int64_t)atom + at / kAtomRows;
      if (named && (uint64_t)place < (uint64_t)slots.atom_rows)
        *(uint32_t*)(sfa + (place * along + p.kh / 8) * kAtomBytes + atom_row(at % kAtomRows)) = word;
    }
  }
  if (!kDirect && p.kh % 8 == 0) token_scales[p.row * (ceil_div(along, 4) * 4) + p.kh / 8] = word;
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
  const int slot = r < count ? row_slots[first + r] : -1;
  const int64_t token = slot >= 0 && slot < rows.rows ? slot / topk : -1;
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
// Eight values to a thread: a wave's stores then fill whole lines at once. Bound
// by memory, four fifths of it written: 16384 x 7168 to fp16, 301 MB in 46 us, 6.6
// TB/s (a fill has 6.8).
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
  const Place p = place_of(blockIdx.x * kRowThreads + threadIdx.x, 2 * blocks);
  const int64_t end = rows.offsets == nullptr ? rows.rows : rows.offsets[rows.experts];
  if (p.row >= end) return;
  int expert, r;
  int64_t atom;
  rows.find(p.row, expert, atom, r);
  const int kb = p.kh / 2;
  float v[8];
  decode(a[p.row * 2 * blocks + p.kh], sfa[(atom * ceil_div(blocks, 4) + kb / 4) * kAtomBytes + atom_row(r) + kb % 4], v);
  store8<T>(out, p.row * row_stride + p.kh * 8, vec, v);
}

template <class T>
__global__ void __launch_bounds__(kTileThreads)
    nvfp4_dequantize_tiles_kernel(const uint32_t* a, const uint8_t* sfa, Rows rows, int blocks, void* out,
                                  int64_t row_stride, int vec) {
  __shared__ uint32_t s_sf[kTileAtoms * kAtomBytes / 4];
  constexpr int kPassRows = kTileThreads / kTileHalves;
  const int along = ceil_div(blocks, 4), chunks = ceil_div(along, kTileAtoms);
  const int64_t atom = blockIdx.x / chunks;
  const int first_atom = blockIdx.x % chunks * kTileAtoms;
  int count, expert;
  const int64_t first = rows.first_row(atom, count, expert);
  if (count == 0) return;
  const int half = threadIdx.x % kTileHalves, kh = first_atom * 8 + half;
  uint32_t codes[kAtomRows / kPassRows];
#pragma unroll
  for (int pass = 0; pass < kAtomRows / kPassRows; ++pass) {
    const int r = pass * kPassRows + threadIdx.x / kTileHalves;
    codes[pass] = r < count && kh < 2 * blocks ? __builtin_nontemporal_load(a + (first + r) * 2 * blocks + kh) : 0u;
  }
  const int words = min(kTileAtoms, along - first_atom) * (kAtomBytes / 4);
  const uint32_t* from = (const uint32_t*)(sfa + (atom * along + first_atom) * kAtomBytes);
  for (int i = threadIdx.x; i < words; i += kTileThreads) s_sf[i] = from[i];
  __syncthreads();
  if (kh >= 2 * blocks) return;
#pragma unroll
  for (int pass = 0; pass < kAtomRows / kPassRows; ++pass) {
    const int r = pass * kPassRows + threadIdx.x / kTileHalves;
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

// f(source) with the source of rows for their type and factor.
template <class Fn>
int with_rows(int dtype, const void* x, int64_t row_stride, int64_t batch_stride, int64_t m, float scale, bool vec, Fn f) {
  if (dtype == NVFP4_MOE_F32) return f(RowSource<F32, false>{x, row_stride, batch_stride, m, scale, vec});
  if (dtype == NVFP4_MOE_F16)
    return scale == 1.f ? f(RowSource<F16, true>{x, row_stride, batch_stride, m, scale, vec})
                        : f(RowSource<F16, false>{x, row_stride, batch_stride, m, scale, vec});
  return scale == 1.f ? f(RowSource<BF16, true>{x, row_stride, batch_stride, m, scale, vec})
                      : f(RowSource<BF16, false>{x, row_stride, batch_stride, m, scale, vec});
}

// Whether tiles beat rows: where an expert's (or a batch's) atoms are filled by a
// quarter, and there are enough elements for the tiles of 128 x 256 to fill the
// chip. Measured, rows - tiles: swiglu of 256 experts of 16 rows, k 2048, 18.0 -
// 19.8 us, of 32 rows 32.7 - 26.8, of 64 rows 57 - 41; quantisation of 64 batches
// of 16 rows of 7168 9.1 - 10.7, of 32 rows 14.7 - 14.0; one batch of 512 x 7168
// 4.7 - 6.6, of 1024 6.9 - 7.0, of 2048 12.7 - 10.9. Rows of a batch need no
// search for their expert on their way back: 4 x 2048 x 7168 26.7 - 27.6,
// 16 x 1024 x 7168 71 - 49, while 256 experts of 64 rows of 2048 are 33 - 23.
// 0 where rows do (or where there are more tiles than a launch can have), else the number of tiles.
int64_t tiles_that_pay(const Rows& r, int64_t batches, int blocks, bool back) {
  const int64_t elements = r.rows * blocks * 16, per = r.offsets == nullptr ? r.m : r.rows / r.experts;
  if (per < 32 || elements < (int64_t)1 << (back && r.offsets == nullptr ? 26 : 23)) return 0;
  const int64_t tiles = atom_rows(r, batches) * ceil_div(ceil_div(blocks, 4), kTileAtoms);
  return tiles <= kMaxTiles ? tiles : 0;
}

template <class Source>
int launch_quantize(const Source& src, const Rows& rows, int64_t batches, int blocks, void* a, void* sfa, hipStream_t st) {
  if (const int64_t tiles = tiles_that_pay(rows, batches, blocks, false)) {
    nvfp4_quantize_tiles_kernel<<<(unsigned)tiles, kTileThreads, 0, st>>>(src, rows, blocks, (uint32_t*)a, (uint8_t*)sfa);
  } else {
    const int64_t grid = ceil_div64(rows.rows * (ceil_div(blocks, 4) * 8), kRowThreads);
    if (grid > kMaxGrid) return NVFP4_ERR_INVALID;
    nvfp4_quantize_rows_kernel<<<(unsigned)grid, kRowThreads, 0, st>>>(src, rows, blocks, (uint32_t*)a, (uint8_t*)sfa);
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

// Scales go straight to their atoms while all of them (2 MB here) stay in an
// XCD's L2 until their lines are full; beyond, they are laid out in whole lines by
// a second launch. Measured at 8 slots a token, 7168 elements, 8 experts, one
// launch - two: 2048 slots 7.0 - 9.2 us, 4096 9.7 - 11.3, 8192 19.8 - 18.2, 16384
// 35 - 26; the number of experts makes no difference (64 of 4096 elements: 8192
// slots 10.5 - 12.8, 16384 21.7 - 20.3).
bool direct_scales(int64_t slots, int k) { return slots * k <= (int64_t)1 << 25; }

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
  return with_rows(dtype, x, row_stride, batch_stride, l > 1 ? m : 0, scale, vec, [&](auto src) {
    return launch_quantize(src, rows, l, k / 16, a, sfa, (hipStream_t)stream);
  });
}

size_t nvfp4_moe_dispatch_workspace_bytes(int64_t tokens, int topk, int k) {
  if (tokens <= 0 || topk < 1 || k <= 0 || direct_scales(tokens * topk, k)) return 0;
  return (size_t)tokens * ceil_div(k, 4 * kAtomK) * 16;
}

int nvfp4_moe_dispatch(const void* x, int dtype, int64_t tokens, int topk, int k, int64_t row_stride, float scale,
                       const int32_t* ids, const int32_t* slot_rows, const int32_t* row_slots,
                       const int32_t* offsets, const int32_t* atoms, int experts, void* a, void* sfa,
                       void* workspace, size_t workspace_bytes, void* stream) {
  if (topk < 1 || topk > NVFP4_MOE_MAX_TOPK || tokens < 0 || tokens > (int64_t)1 << 30 || tokens * topk > (int64_t)1 << 30)
    return NVFP4_ERR_INVALID;
  if (int rc = check_source(x, dtype, tokens, k, row_stride)) return rc;
  if (int rc = check_operand(tokens * topk, k, a, sfa)) return rc;
  if (offsets == nullptr) return NVFP4_ERR_INVALID;
  if (int rc = check_sorted(offsets, atoms, experts)) return rc;
  if (tokens > 0 && (ids == nullptr || slot_rows == nullptr || row_slots == nullptr)) return NVFP4_ERR_INVALID;
  if (!aligned(ids, 4) || !aligned(slot_rows, 4) || !aligned(row_slots, 4)) return NVFP4_ERR_MISALIGNED;
  if (tokens == 0 || k == 0) return NVFP4_OK;
  const size_t need = nvfp4_moe_dispatch_workspace_bytes(tokens, topk, k);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return NVFP4_ERR_WORKSPACE;
  if (need > 0 && !aligned(workspace, 256)) return NVFP4_ERR_MISALIGNED;
  const int blocks = k / 16, along = ceil_div(blocks, 4);
  const int64_t grid = ceil_div64(tokens * along * 8, kRowThreads);
  const Rows rows = {offsets, atoms, experts, tokens * topk, 0};
  const int64_t scale_grid = atom_rows(rows, 1) * ceil_div(along, kScaleAtoms);
  if (grid > kMaxGrid || scale_grid > kMaxGrid) return NVFP4_ERR_INVALID;
  const Slots slots = {ids, slot_rows, offsets, atoms, topk, experts, (int)rows.rows, atom_rows(rows, 1)};
  const hipStream_t st = (hipStream_t)stream;
  int rc = with_rows(dtype, x, row_stride, 0, 0, scale, wide_rows(x, dtype, row_stride), [&](auto src) {
    using Source = decltype(src);
    if (need == 0)
      nvfp4_dispatch_kernel<Source, true><<<(unsigned)grid, kRowThreads, 0, st>>>(src, slots, tokens, blocks, (uint32_t*)a,
                                                                                 (uint8_t*)sfa, nullptr);
    else
      nvfp4_dispatch_kernel<Source, false><<<(unsigned)grid, kRowThreads, 0, st>>>(src, slots, tokens, blocks, (uint32_t*)a,
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
  const int64_t tiles = tiles_that_pay(rows, l, blocks, true);
  const int64_t grid = tiles ? tiles : ceil_div64(rows.rows * 2 * blocks, kRowThreads);
  if (tiles == 0 && grid > kMaxGrid) return NVFP4_ERR_INVALID;
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
