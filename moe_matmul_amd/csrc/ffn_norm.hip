// Root-mean-square norm of a sum with the residual, and its gradient (nvfp4_ffn.h).
//
// y = s r w, r = (mean s^2 + eps)^-1/2; with h = s r:
// ds = r (w dy - h mean(w dy h)) + dsum, dw = sum over rows of dy h.
//
// Bound by memory: a workgroup holds a row in registers between the pass that sums
// and the one that writes, so every operand is read once. Squares are summed in fp64
// (rows of elements beyond 2^63 or below 2^-75 keep their norm; the sums cost a tenth
// of the time that the loads take), everything else is fp32.
// Measured: 16384 x 7168 bf16 with a residual to 8 bits 165 to 172 us (826 MB: 4.8 to 5.0 TB/s, as a copy),
// 8195 x 4096 fp16 with a residual 47 (268 MB: 5.7 TB/s), its gradient 45 and 5 for the weight's, 1 x 7168 3.8.
#include "ffn_common.h"

namespace ffn {

struct NormArgs {
  const void *x, *residual, *weight;
  int64_t rows, x_stride, residual_stride;
  int n, weight_f32;
  float eps;
  void *sum, *y;
  uint8_t *codes, *scales;
  float* rstd;
};

// How a row's eight elements at a time are reached: one by one, whole and aligned, or so and past the caches.
constexpr int kOne = 0, kWide = 1, kStreamed = 2;

// Eight elements from column `col` on of a row that ends at n.
template <class T, int VEC> __device__ __forceinline__ void load_row8(const void* p, int64_t at, int left, float* v) {
  if constexpr (VEC == kStreamed) {
    Raw8<T> raw;
    raw.load(p, at, true);
    raw.values(v);
  } else if constexpr (VEC) {
    load8<T>(p, at, true, v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = j < left ? load1<T>(p, at + j) : 0.f;
  }
}
template <class T, int VEC> __device__ __forceinline__ void store_row8(void* p, int64_t at, int left, const float* v) {
  if constexpr (VEC == kStreamed && T::kBytes == 2) {
    __builtin_nontemporal_store(pack16x8<T>(v), (u32x4*)((uint16_t*)p + at));
  } else if constexpr (VEC && T::kBytes == 2) {
    *(u32x4*)((uint16_t*)p + at) = pack16x8<T>(v);
  } else if constexpr (VEC) {
    store8<T>(p, at, true, v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < left) store1<T>(p, at + j, v[j]);
  }
}
template <class T, int VEC>
__device__ __forceinline__ void weight_row8(const void* p, int f32, int col, int left, float* v) {
  if (!p) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = 1.f;
  } else if (f32) {
    load_row8<F32, VEC != kOne>(p, col, left, v);
  } else {
    load_row8<T, VEC != kOne>(p, col, left, v);
  }
}

// The workgroup's sum, the same in all threads. Lanes by halves, waves in order.
template <int TH> __device__ __forceinline__ double block_sum(double v, double* room) {
#pragma unroll
  for (int d = 32; d; d /= 2) v += __shfl_xor(v, d, 64);
  if constexpr (TH > 64) {
    const int wave = threadIdx.x / 64;
    __syncthreads();  // the last row's sums have been read
    if (threadIdx.x % 64 == 0) room[wave] = v;
    __syncthreads();
    v = 0;
#pragma unroll
    for (int i = 0; i < TH / 64; ++i) v += room[i];
  }
  return v;
}

// x as it is kept: rounded to T.
template <class T> __device__ __forceinline__ float rounded(float v) {
  if constexpr (T::kId == NVFP4_MOE_F32) return v;
  else if constexpr (T::kId == NVFP4_MOE_F16) return (float)(_Float16)v;
  else return (float)(__bf16)v;
}

template <class T, int TH, int C, int VEC> __global__ __launch_bounds__(TH) void norm_kernel(const NormArgs a) {
  __shared__ double room[TH / 64];
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    float s[C][8];
    double squares = 0;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int col = (c * TH + threadIdx.x) * 8, left = a.n - col;
#pragma unroll
      for (int j = 0; j < 8; ++j) s[c][j] = 0.f;
      if (left <= 0) continue;
      load_row8<T, VEC>(a.x, row * a.x_stride + col, left, s[c]);
      if (a.residual) {
        float r[8];
        load_row8<T, VEC>(a.residual, row * a.residual_stride + col, left, r);
#pragma unroll
        for (int j = 0; j < 8; ++j) s[c][j] = rounded<T>(s[c][j] + r[j]);
        store_row8<T, VEC>(a.sum, row * a.n + col, left, s[c]);
      }
    }
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int j = 0; j < 8; ++j) squares = fma((double)s[c][j], (double)s[c][j], squares);
    const double mean = block_sum<TH>(squares, room) / a.n;
    const float r = (float)(1.0 / sqrt(mean + (double)a.eps));
    if (a.rstd && threadIdx.x == 0) a.rstd[row] = r;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int col = (c * TH + threadIdx.x) * 8, left = a.n - col;
      float w[8];
      if (left > 0) weight_row8<T, VEC>(a.weight, a.weight_f32, col, left, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) s[c][j] = s[c][j] * r * (left > 0 ? w[j] : 0.f);
      if (a.codes) {  // n % 32 == 0: 32 columns are those of four threads
        uint32_t top = abs_bits(s[c][0]);
#pragma unroll
        for (int j = 1; j < 8; ++j) top = umax(top, abs_bits(s[c][j]));
        top = umax(top, from_lane_xor(top, 1));
        top = umax(top, from_lane_xor(top, 2));
        const uint32_t byte = scale8(top);
        if (left > 0) {
          const float inverse = scale8_inverse(byte);
          u32x2 q;
          q.x = encode4(s[c][0], s[c][1], s[c][2], s[c][3], inverse);
          q.y = encode4(s[c][4], s[c][5], s[c][6], s[c][7], inverse);
          const int64_t k = row * a.n + col;
          *(u32x2*)(a.codes + k) = q;
          if (col % 32 == 0) a.scales[k / 32] = (uint8_t)byte;
        }
      }
      if (a.y && left > 0) store_row8<T, VEC>(a.y, row * a.n + col, left, s[c]);
    }
  }
}

struct NormBackArgs {
  const void *dy, *s, *weight, *dsum;
  int64_t rows, dy_stride, s_stride, dsum_stride;
  int n, weight_f32;
  const float* rstd;
  void* dx;
  float* partial;  // [gridDim.x][n], or NULL
};

template <class T, int TH, int C, int VEC> __global__ __launch_bounds__(TH) void norm_back_kernel(const NormBackArgs a) {
  __shared__ double room[TH / 64];
  float dw[C][8], w[C][8];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int col = (c * TH + threadIdx.x) * 8, left = a.n - col;
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[c][j] = w[c][j] = 0.f;
    if (left > 0) weight_row8<T, VEC>(a.weight, a.weight_f32, col, left, w[c]);
  }
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    float h[C][8], d[C][8];
    const float r = a.rstd[row];
    float dot = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int col = (c * TH + threadIdx.x) * 8, left = a.n - col;
#pragma unroll
      for (int j = 0; j < 8; ++j) h[c][j] = d[c][j] = 0.f;
      if (left <= 0) continue;
      load_row8<T, VEC>(a.s, row * a.s_stride + col, left, h[c]);
      load_row8<T, VEC>(a.dy, row * a.dy_stride + col, left, d[c]);
    }
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        h[c][j] *= r;
        dw[c][j] = fmaf(d[c][j], h[c][j], dw[c][j]);
        d[c][j] *= w[c][j];
        dot = fmaf(d[c][j], h[c][j], dot);
      }
    const float mean = (float)(block_sum<TH>(dot, room) / a.n);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int col = (c * TH + threadIdx.x) * 8, left = a.n - col;
      if (left <= 0) continue;
      float g[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) g[j] = r * (d[c][j] - h[c][j] * mean);
      if (a.dsum) {
        float e[8];
        load_row8<T, VEC>(a.dsum, row * a.dsum_stride + col, left, e);
#pragma unroll
        for (int j = 0; j < 8; ++j) g[j] += e[j];
      }
      store_row8<T, VEC>(a.dx, row * a.n + col, left, g);
    }
  }
  if (!a.partial) return;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int col = (c * TH + threadIdx.x) * 8, left = a.n - col;
    if (left > 0) store_row8<F32, VEC != kOne>(a.partial, (int64_t)blockIdx.x * a.n + col, left, dw[c]);
  }
}

// Threads for a row: eight elements each as far as 1024 threads go where there are fewer
// rows than compute units (latency: 1 row of 7168), 16 to 32 each where there are more.
struct NormShape { int threads, chunks; };
static NormShape shape_of(int64_t rows, int n, int units) {
  const int eights = ceil_div(n, 8);
  int threads = 64;
  const int most = rows <= 2 * units ? 1 : 2;
  while (threads < 1024 && eights > threads * most) threads *= 2;
  int chunks = 1;
  while (eights > threads * chunks) chunks *= 2;
  return {threads, chunks};
}

// What leaves the 256 MB of the card's last cache anyway goes past it: 16384 rows of 7168 with a residual, 8-bit rows
// (826 MB) 190 us and 172; but 8195 rows of 4096 in fp16 (268 MB) 44 and 48.
constexpr double kStreamBytes = 320e6;
static int reach_of(bool vec, double bytes) { return !vec ? kOne : bytes > kStreamBytes ? kStreamed : kWide; }

template <class Fn> static int with_shape(const NormShape& s, int vec, Fn f) {
  auto by_chunks = [&](auto threads) {
    constexpr int TH = decltype(threads)::value;
    auto by_vec = [&](auto chunks) {
      if (vec == kStreamed) f(threads, chunks, std::integral_constant<int, kStreamed>{});
      else if (vec == kWide) f(threads, chunks, std::integral_constant<int, kWide>{});
      else f(threads, chunks, std::integral_constant<int, kOne>{});
    };
    if (s.chunks == 1) by_vec(std::integral_constant<int, 1>{});
    else if (s.chunks == 2) by_vec(std::integral_constant<int, 2>{});
    else if constexpr (TH == 1024) {
      if (s.chunks == 4) by_vec(std::integral_constant<int, 4>{});
      else by_vec(std::integral_constant<int, 8>{});
    }
  };
  switch (s.threads) {
    case 64: by_chunks(std::integral_constant<int, 64>{}); break;
    case 128: by_chunks(std::integral_constant<int, 128>{}); break;
    case 256: by_chunks(std::integral_constant<int, 256>{}); break;
    case 512: by_chunks(std::integral_constant<int, 512>{}); break;
    default: by_chunks(std::integral_constant<int, 1024>{}); break;
  }
  return launched();
}

constexpr int kMaxNorm = 65536;

// Workgroups of the gradient, each with sums of its own: two for each 256 threads of a compute unit's 2048.
static int64_t back_blocks(int64_t rows, int n, int units) {
  const NormShape s = shape_of(rows, n, units);
  const int64_t most = (int64_t)units * (s.threads >= 512 ? 2 : 1024 / s.threads);
  return rows < most ? rows : most;
}

static bool row_aligned(const void* p, int dtype, int64_t stride, int64_t rows) {
  return !p || (aligned(p, 16) && (rows < 2 || stride * element_bytes(dtype) % 16 == 0));
}

void add_columns(const float* partial, int64_t parts, int n, void* out, int out_type, hipStream_t stream);

}  // namespace ffn

using namespace ffn;

extern "C" {

int nvfp4_ffn_rmsnorm(const void* x, int dtype, int64_t rows, int n, int64_t x_stride, const void* residual,
                      int64_t residual_stride, const void* weight, int weight_f32, float eps, void* sum, void* y,
                      void* codes, void* scales, float* rstd, void* stream) {
  if (!known_type(dtype) || rows < 0 || rows >= (int64_t)1 << 31 || n < 1 || n > kMaxNorm || !(eps >= 0.f) ||
      !codes != !scales || (codes && n % kBlock8))
    return NVFP4_ERR_INVALID;
  if (rows == 0) return NVFP4_OK;
  if (!x || (!y && !codes && !rstd) || x_stride < n || (residual && (residual_stride < n || !sum))) return NVFP4_ERR_INVALID;
  const size_t element = element_bytes(dtype);
  if (!aligned(x, element) || !aligned(residual, element) || !aligned(sum, element) || !aligned(y, element) ||
      !aligned(weight, weight_f32 ? 4 : element) || !aligned(codes, 8) || !aligned(rstd, 4))
    return NVFP4_ERR_MISALIGNED;
  NormArgs a{x, residual, weight, rows, x_stride, residual_stride, n, weight_f32, eps, sum, y, (uint8_t*)codes, (uint8_t*)scales, rstd};
  const bool vec = n % 8 == 0 && row_aligned(x, dtype, x_stride, rows) && row_aligned(residual, dtype, residual_stride, rows) &&
                   row_aligned(sum, dtype, n, rows) && row_aligned(y, dtype, n, rows) && aligned(weight, 16);
  const double bytes = (double)rows * n * element * (1 + (residual ? 2 : 0) + (y ? 1 : 0)) + (codes ? (double)rows * n : 0);
  const int units = compute_units(), reach = reach_of(vec, bytes);
  const unsigned grid = (unsigned)(rows < 1 << 20 ? rows : 1 << 20);
  return with_type(dtype, [&](auto type) {
    using T = decltype(type);
    return with_shape(shape_of(rows, n, units), reach, [&](auto th, auto c, auto v) {
      constexpr int TH = decltype(th)::value, C = decltype(c)::value;
      norm_kernel<T, TH, C, decltype(v)::value><<<grid, TH, 0, (hipStream_t)stream>>>(a);
    });
  });
}

size_t nvfp4_ffn_rmsnorm_workspace_bytes(int64_t rows, int n) {
  if (rows < 1 || rows >= (int64_t)1 << 31 || n < 1 || n > kMaxNorm) return 0;
  return (size_t)back_blocks(rows, n, compute_units()) * n * 4;
}

int nvfp4_ffn_rmsnorm_backward(const void* dy, int64_t dy_stride, const void* s, int64_t s_stride, int dtype,
                               int64_t rows, int n, const void* weight, int weight_f32, const float* rstd,
                               const void* dsum, int64_t dsum_stride, void* dx, void* dweight, void* workspace,
                               size_t workspace_bytes, void* stream) {
  if (!known_type(dtype) || rows < 0 || rows >= (int64_t)1 << 31 || n < 1 || n > kMaxNorm || (dweight && !weight))
    return NVFP4_ERR_INVALID;
  const size_t element = element_bytes(dtype), weight_element = weight_f32 ? 4 : element;
  const int weight_type = weight_f32 ? NVFP4_MOE_F32 : dtype;
  if (!aligned(weight, weight_element) || !aligned(dweight, weight_element)) return NVFP4_ERR_MISALIGNED;
  if (rows == 0) {
    if (dweight) add_columns(nullptr, 0, n, dweight, weight_type, (hipStream_t)stream);
    return dweight ? launched() : NVFP4_OK;
  }
  if (!dy || !s || !rstd || !dx || dy_stride < n || s_stride < n || (dsum && dsum_stride < n)) return NVFP4_ERR_INVALID;
  if (!aligned(dy, element) || !aligned(s, element) || !aligned(dsum, element) || !aligned(dx, element) || !aligned(rstd, 4))
    return NVFP4_ERR_MISALIGNED;
  const int units = compute_units();
  const int64_t blocks = back_blocks(rows, n, units);
  if (dweight) {
    if (!workspace || workspace_bytes < (size_t)blocks * n * 4) return NVFP4_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return NVFP4_ERR_MISALIGNED;
  }
  NormBackArgs a{dy, s, weight, dsum, rows, dy_stride, s_stride, dsum_stride, n, weight_f32, rstd, dx, dweight ? (float*)workspace : nullptr};
  const bool vec = n % 8 == 0 && row_aligned(dy, dtype, dy_stride, rows) && row_aligned(s, dtype, s_stride, rows) &&
                   row_aligned(dsum, dtype, dsum_stride, rows) && row_aligned(dx, dtype, n, rows) && aligned(weight, 16);
  const int reach = reach_of(vec, (double)rows * n * element * (dsum ? 4 : 3));
  const int rc = with_type(dtype, [&](auto type) {
    using T = decltype(type);
    return with_shape(shape_of(rows, n, units), reach, [&](auto th, auto c, auto v) {
      constexpr int TH = decltype(th)::value, C = decltype(c)::value;
      norm_back_kernel<T, TH, C, decltype(v)::value><<<(unsigned)blocks, TH, 0, (hipStream_t)stream>>>(a);
    });
  });
  if (rc || !dweight) return rc;
  add_columns((const float*)workspace, blocks, n, dweight, weight_type, (hipStream_t)stream);
  return launched();
}

}  // extern "C"
