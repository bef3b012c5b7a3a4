// Shared by the kernels of nvfp4_moe.h: element types, wide loads and stores,
// the tiled scale layout, and the host's argument checks.
#pragma once

#include <hip/hip_runtime.h>

#include <stdint.h>

#include "nvfp4_moe.h"

namespace moe {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

constexpr int kAtomRows = 128;   // rows of a scale atom
constexpr int kAtomK = 64;       // its K-elements
constexpr int kAtomBytes = 512;

__host__ __device__ inline int ceil_div(int a, int b) { return (a + b - 1) / b; }
__host__ __device__ inline int64_t ceil_div64(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Byte of row r (of its 128) inside an atom; the four K-blocks follow.
__device__ inline int atom_row(int r) { return (r & 31) * 16 + ((r >> 5) & 3) * 4; }

// ---- element types --------------------------------------------------------
struct F32 { static constexpr int kBytes = 4; static constexpr int kId = NVFP4_MOE_F32; };
struct F16 { static constexpr int kBytes = 2; static constexpr int kId = NVFP4_MOE_F16; };
struct BF16 { static constexpr int kBytes = 2; static constexpr int kId = NVFP4_MOE_BF16; };

template <class T> __device__ inline void unpack2(uint32_t w, float& a, float& b);
template <> __device__ inline void unpack2<F16>(uint32_t w, float& a, float& b) {
  const f16x2 h = __builtin_bit_cast(f16x2, w);
  a = (float)h.x;
  b = (float)h.y;
}
template <> __device__ inline void unpack2<BF16>(uint32_t w, float& a, float& b) {
  a = __builtin_bit_cast(float, w << 16);
  b = __builtin_bit_cast(float, w & 0xFFFF0000u);
}

// fp32 -> bf16 bits, to nearest even; NaN stays NaN.
__device__ inline uint32_t bf16_bits(float x) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x);
  return x != x ? 0x7FC0u : (u + 0x7FFFu + ((u >> 16) & 1)) >> 16;
}
template <class T> __device__ inline uint32_t pack2(float a, float b);
template <> __device__ inline uint32_t pack2<F16>(float a, float b) {
  f16x2 h;
  h.x = (_Float16)a;
  h.y = (_Float16)b;
  return __builtin_bit_cast(uint32_t, h);
}
template <> __device__ inline uint32_t pack2<BF16>(float a, float b) { return bf16_bits(a) | (bf16_bits(b) << 16); }

// One element, at any element alignment.
template <class T> __device__ inline float load1(const void* p, int64_t i) {
  if constexpr (T::kId == NVFP4_MOE_F32) return ((const float*)p)[i];
  else if constexpr (T::kId == NVFP4_MOE_F16) return (float)((const _Float16*)p)[i];
  else return __builtin_bit_cast(float, (uint32_t)((const uint16_t*)p)[i] << 16);
}
template <class T> __device__ inline void store1(void* p, int64_t i, float v) {
  if constexpr (T::kId == NVFP4_MOE_F32) ((float*)p)[i] = v;
  else if constexpr (T::kId == NVFP4_MOE_F16) ((_Float16*)p)[i] = (_Float16)v;
  else ((uint16_t*)p)[i] = (uint16_t)bf16_bits(v);
}

// Eight elements from element i on; 16-byte loads where `vec` says that the
// address is a multiple of 16 bytes.
template <class T> __device__ inline void load8(const void* p, int64_t i, bool vec, float* v) {
  if (vec) {
    if constexpr (T::kId == NVFP4_MOE_F32) {
      const f32x4 a = *(const f32x4*)((const float*)p + i), b = *(const f32x4*)((const float*)p + i + 4);
#pragma unroll
      for (int j = 0; j < 4; ++j) { v[j] = a[j]; v[j + 4] = b[j]; }
    } else {
      const u32x4 a = *(const u32x4*)((const uint16_t*)p + i);
#pragma unroll
      for (int j = 0; j < 4; ++j) unpack2<T>(a[j], v[2 * j], v[2 * j + 1]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = load1<T>(p, i + j);
  }
}
template <class T> __device__ inline void store8(void* p, int64_t i, bool vec, const float* v) {
  if (vec) {
    if constexpr (T::kId == NVFP4_MOE_F32) {
      f32x4 a, b;
#pragma unroll
      for (int j = 0; j < 4; ++j) { a[j] = v[j]; b[j] = v[j + 4]; }
      *(f32x4*)((float*)p + i) = a;
      *(f32x4*)((float*)p + i + 4) = b;
    } else {
      u32x4 a;
#pragma unroll
      for (int j = 0; j < 4; ++j) a[j] = pack2<T>(v[2 * j], v[2 * j + 1]);
      *(u32x4*)((uint16_t*)p + i) = a;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) store1<T>(p, i + j, v[j]);
  }
}

// Eight elements as they lie in memory, for loads that are used later. They are
// read once, so the lines are not kept where one load of a wave takes whole lines;
// the two halves of eight fp32 elements share theirs.
template <class T> struct Raw8 {
  u32x4 w[T::kBytes / 2];

  __device__ inline void load(const void* p, int64_t i, bool vec) {
    const uint8_t* at = (const uint8_t*)p + i * T::kBytes;
    if (vec) {
#pragma unroll
      for (int j = 0; j < T::kBytes / 2; ++j) w[j] = T::kBytes == 2 ? __builtin_nontemporal_load((const u32x4*)at + j) : ((const u32x4*)at)[j];
    } else {
#pragma unroll
      for (int j = 0; j < 2 * T::kBytes; ++j)
        w[j / 4][j % 4] = T::kBytes == 4 ? ((const uint32_t*)at)[j]
                                         : ((const uint16_t*)at)[2 * j] | (uint32_t)((const uint16_t*)at)[2 * j + 1] << 16;
    }
  }
  __device__ inline void values(float* v) const {
    if constexpr (T::kBytes == 4) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t u = w[j / 4][j % 4];  // bit_cast of a vector's element itself takes the first one
        v[j] = __builtin_bit_cast(float, u);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) unpack2<T>(w[0][j], v[2 * j], v[2 * j + 1]);
    }
  }
};

// exp in fp32: 2^(x log2 e) with the product's rounding error taken back, so that
// the result is within about 2 ulp for every x (the plain product loses |x| *
// 2^-24) where it is a normal number; below 2^-126 it is 0. -inf gives 0, NaN gives
// NaN. With `up` (a whole number), times 2^up.
__device__ inline float exp_f32_low(float x, float t) {  // the factor that is 1 but for the rounding of t = x log2 e
  const float kLog2e = 1.44269502f, kLog2eLow = 1.92596303e-8f, kLn2 = 0.693147182f;
  // |x| beyond this over- or underflows whatever the low part; it would be inf - inf
  const float low = fabsf(x) < 200.f ? fmaf(x, kLog2eLow, fmaf(x, kLog2e, -t)) : 0.f;
  return fmaf(low, kLn2, 1.f);
}
__device__ inline float exp_f32(float x) {
  const float t = x * 1.44269502f;
  return __builtin_amdgcn_exp2f(t) * exp_f32_low(x, t);
}
__device__ inline float exp_f32(float x, float up) {
  const float t = x * 1.44269502f;
  return __builtin_amdgcn_exp2f(t + up) * exp_f32_low(x, t);
}

// Stores to shared memory by lanes of this wave are seen by its other lanes.
__device__ inline void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// ---- host -----------------------------------------------------------------
extern thread_local int t_last_hip_error;

inline int launched() {
  const hipError_t e = hipGetLastError();
  if (e == hipSuccess) return NVFP4_OK;
  t_last_hip_error = (int)e;
  return NVFP4_ERR_HIP;
}

inline int element_bytes(int dtype) { return dtype == NVFP4_MOE_F32 ? 4 : 2; }
inline bool known_type(int dtype) { return dtype >= NVFP4_MOE_F32 && dtype <= NVFP4_MOE_BF16; }
inline bool aligned(const void* p, size_t bytes) { return (uintptr_t)p % bytes == 0; }
// Rows of `stride` elements from p on can be read 16 bytes at a time.
inline bool wide_rows(const void* p, int dtype, int64_t stride) {
  return aligned(p, 16) && stride * element_bytes(dtype) % 16 == 0;
}

// Calls f with the element type's tag.
template <class Fn> inline auto with_type(int dtype, Fn f) {
  switch (dtype) {
    case NVFP4_MOE_F32: return f(F32{});
    case NVFP4_MOE_F16: return f(F16{});
    default: return f(BF16{});
  }
}

}  // namespace moe
