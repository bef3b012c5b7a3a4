// Shared by the kernels of nvfp4_ffn.h: activations and their slopes, rows in 8
// bits, the plan's rows, and the host's argument checks.
#pragma once

#include "moe_common.h"
#include "nvfp4_ffn.h"

namespace ffn {

using namespace moe;

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef int32_t i32x4 __attribute__((ext_vector_type(4)));

// Pairs of fp32 to 16 bits, to nearest even, by the card's own conversions.
template <class T> __device__ __forceinline__ uint32_t pack16(float a, float b) {
  if constexpr (T::kId == NVFP4_MOE_F16) {
    return pack2<F16>(a, b);
  } else {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    const f32x2 v = {a, b};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
  }
}
template <class T> __device__ __forceinline__ u32x4 pack16x8(const float* v) {
  return u32x4{pack16<T>(v[0], v[1]), pack16<T>(v[2], v[3]), pack16<T>(v[4], v[5]), pack16<T>(v[6], v[7])};
}
template <class T> __device__ __forceinline__ void unpack16x8(u32x4 w, float* v) {
#pragma unroll
  for (int j = 0; j < 4; ++j) unpack2<T>(w[j], v[2 * j], v[2 * j + 1]);
}

// Where the rows sorted by expert lie: nvfp4_ffn_plan, or one expert with all rows.
struct Rows {
  const int32_t* offsets;    // NULL: one expert, rows 0 .. rows-1
  const int32_t* row_slots;  // rows are tokens' rows: row r is row row_slots[r] / topk of the operand; NULL: row r itself
  int experts, topk;
  int64_t rows, sources;     // the most rows, and the operand's rows
  int clear;                 // rows of no expert are written as 0; else left
};

// First row of expert e (experts: the rows of no expert), in 0 .. rows whatever the table holds.
__device__ inline int64_t first_row(const Rows& r, int e) {
  if (!r.offsets) return e ? r.rows : 0;
  const int64_t o = r.offsets[e];
  return o < 0 ? 0 : o > r.rows ? r.rows : o;
}
// The operand's row for row r, -1 if the tables name none.
__device__ inline int64_t source_row(const Rows& p, int64_t r) {
  if (!p.row_slots) return r;
  const int slot = p.row_slots[r];
  return slot >= 0 && slot < p.rows ? slot / p.topk : -1;
}
// The expert whose rows hold row r, `experts` where none's do.
__device__ inline int expert_of(const Rows& p, int64_t r) {
  if (!p.offsets) return 0;
  int low = 0, high = p.experts;  // the first e with offsets[e + 1] > r
  while (low < high) {
    const int mid = (low + high) / 2;
    if (p.offsets[mid + 1] > r) high = mid;
    else low = mid + 1;
  }
  return low;
}

// ---- activations --------------------------------------------------------------
// e^x by the card's 2^x: log2 e is rounded (0.23 |x| 2^-24 of the value) and so is the product (|x| 2^-24), so within
// (1.25 |x| + 2) 2^-24 of it; below 2^-126 it is 0.
__device__ __forceinline__ float fast_exp(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504f); }
// 1 / (1 + e^-z). e^-z is infinite below -88.7, where the quotient is 0.
__device__ __forceinline__ float logistic(float z) { return __builtin_amdgcn_rcpf(1.f + fast_exp(-z)); }
// The normal distribution's function below z <= 0 and e = e^(-z^2/2): with t = -z / sqrt 2 and k = 1 / (1 + 0.3 t),
// erfc(t) / 2 = e^(-t^2) k P(k), where P is the polynomial of degree 8 that is nearest to erfc(t) e^(t^2) / 2 k,
// relative to it, for t of 0 to 11 (by least squares, reweighted to even out the error; 4.4 * 10^-8 off with the
// coefficients as they are rounded here, 0.75 * 2^-24). No cancellation, so small values keep their bits: 5 instructions
// and 9 products where a library's erfc has 100.
__device__ __forceinline__ float normal_tail(float z, float e) {
  const float k = __builtin_amdgcn_rcpf(fmaf(fabsf(z), 0.3f * 0.707106781f, 1.f));
  float v = -0.064777948f;
  v = fmaf(v, k, 0.242868051f);
  v = fmaf(v, k, -0.256333172f);
  v = fmaf(v, k, 0.274103731f);
  v = fmaf(v, k, -0.0475121252f);
  v = fmaf(v, k, 0.107552357f);
  v = fmaf(v, k, 0.0741435811f);
  v = fmaf(v, k, 0.085361816f);
  v = fmaf(v, k, 0.0845937133f);
  return v * k * e;
}

// The activation (a) and, where asked for, its slope (s) at z. Infinities and far values take their limits, before
// infinity meets 0: below -104 (silu) and -15 (gelu) both are 0, beyond the slope is 1.
template <bool SLOPE> __device__ __forceinline__ void activate(float z, int kind, float& a, float& s) {
  switch (kind) {
    case NVFP4_FFN_RELU:  // NaN stays
      a = z < 0.f ? 0.f : z;
      if (SLOPE) s = z > 0.f ? 1.f : z == z ? 0.f : z;
      return;
    case NVFP4_FFN_SILU: {
      const float p = logistic(z);
      a = z < -104.f ? 0.f : z * p;
      if (SLOPE) s = z < -104.f ? 0.f : z > 104.f ? 1.f : p * fmaf(z, 1.f - p, 1.f);
      return;
    }
    case NVFP4_FFN_GELU: {
      const float e = fast_exp(z * z * -0.5f), tail = normal_tail(z, e), p = z < 0.f ? tail : 1.f - tail;
      a = z < -15.f ? 0.f : z * p;
      if (SLOPE) s = z < -15.f ? 0.f : z > 15.f ? 1.f : fmaf(z * 0.398942280f, e, p);
      return;
    }
    default:
      a = z;
      if (SLOPE) s = 1.f;
      return;
  }
}
__device__ __forceinline__ float activation(float z, int kind) {
  float a, s;
  activate<false>(z, kind, a, s);
  return a;
}
// Of eight, with one branch.
__device__ __forceinline__ void activation8(float* v, int kind) {
  switch (kind) {
    case NVFP4_FFN_RELU:
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = activation(v[j], NVFP4_FFN_RELU);
      return;
    case NVFP4_FFN_SILU:
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = activation(v[j], NVFP4_FFN_SILU);
      return;
    case NVFP4_FFN_GELU:
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = activation(v[j], NVFP4_FFN_GELU);
      return;
    default: return;
  }
}

// Of eight z their slopes, in place, and their activations (a).
template <int KIND> __device__ __forceinline__ void values_slopes(float* z, float* a) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    float v, s;
    activate<true>(z[j], KIND, v, s);
    z[j] = s;
    a[j] = v;
  }
}
__device__ __forceinline__ void values_slopes8(float* z, float* a, int kind) {
  switch (kind) {
    case NVFP4_FFN_RELU: values_slopes<NVFP4_FFN_RELU>(z, a); return;
    case NVFP4_FFN_SILU: values_slopes<NVFP4_FFN_SILU>(z, a); return;
    default: values_slopes<NVFP4_FFN_GELU>(z, a); return;
  }
}
__device__ __forceinline__ void slopes8(float* z, int kind) {
  float a[8];
  values_slopes8(z, a, kind);
}

// ---- rows in 8 bits -----------------------------------------------------------
// A block of 32 elements has the scale 2^(byte - 127): the least, from 2^-126 on,
// under which its largest element is at most 448, E4M3's largest value. Byte 255:
// the block held an infinity or NaN, and all its values are NaN.
constexpr int kBlock8 = 32;

__device__ inline uint32_t abs_bits(float v) { return __builtin_bit_cast(uint32_t, v) & 0x7FFFFFFFu; }
// The scale's byte from the bits of the largest magnitude (as integers, so that infinities and NaN are the largest).
__device__ inline uint32_t scale8(uint32_t top) {
  if (top >= 0x7F800000u) return 255;
  // top = m 2^p, 1 <= m < 2, 448 = 1.75 * 2^8: 2^(p - 8) for m <= 1.75, else 2^(p - 7)
  const int e = (int)(top >> 23) - 8 + ((top & 0x7FFFFFu) > 0x600000u);
  return e < 1 ? 1 : e;
}
// 2^(byte - 127) and its inverse; byte 1 .. 247 as scale8 gives them (247: beyond 1.75 * 2^127), or 255.
__device__ inline float scale8_value(uint32_t byte) { return __builtin_bit_cast(float, byte == 255 ? 0x7FC00000u : byte << 23); }
__device__ inline float scale8_inverse(uint32_t byte) { return __builtin_bit_cast(float, byte == 255 ? 0x7FC00000u : (254u - byte) << 23); }
// Four codes; the products are exact, so each code is rounded once (to nearest, ties to even).
__device__ inline uint32_t encode4(float a, float b, float c, float d, float inverse) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(a * inverse, b * inverse, 0, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(c * inverse, d * inverse, w, true);
  return w;
}
__device__ inline void decode4(uint32_t w, float scale, float* v) {
  const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8(w, false), b = __builtin_amdgcn_cvt_pk_f32_fp8(w, true);
  v[0] = a.x * scale;
  v[1] = a.y * scale;
  v[2] = b.x * scale;
  v[3] = b.y * scale;
}

__device__ inline uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }
__device__ inline float from_lane_xor(float v, int mask) { return __shfl_xor(v, mask, 64); }
__device__ inline uint32_t from_lane_xor(uint32_t v, int mask) { return (uint32_t)__shfl_xor((int)v, mask, 64); }

// A parameter of fp32 or of the rows' type T.
template <class T> __device__ inline float param(const void* p, int64_t i, int f32) {
  return f32 ? ((const float*)p)[i] : load1<T>(p, i);
}
template <class T> __device__ inline void param8(const void* p, int64_t i, int f32, bool vec, float* v) {
  if (f32) load8<F32>(p, i, vec, v);
  else load8<T>(p, i, vec, v);
}

// ---- host -----------------------------------------------------------------------
inline bool known_activation(int a) { return a >= NVFP4_FFN_NONE && a <= NVFP4_FFN_GELU; }
// Calls f with the tag of a 16-bit type.
template <class Fn> inline auto with_type16(int dtype, Fn f) { return dtype == NVFP4_MOE_F16 ? f(F16{}) : f(BF16{}); }
inline bool type16(int dtype) { return dtype == NVFP4_MOE_F16 || dtype == NVFP4_MOE_BF16; }

// NVFP4_OK, or why the plan is none; fills rows.
int plan_rows(const nvfp4_ffn_plan* plan, int64_t rows, bool gathered, Rows* out);
// Compute units of the current device (256 if it cannot be asked).
int compute_units();

}  // namespace ffn
