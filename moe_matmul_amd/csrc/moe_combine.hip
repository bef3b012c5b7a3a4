// The combine: weighted sums of the experts' rows of every token, and its
// gradients.
#include "moe_common.h"

namespace moe {
namespace {

constexpr int kThreads = 256;

struct CombineArgs {
  const void* c;
  int64_t c_stride, c_rows, tokens, out_stride, dy_stride;
  const int32_t *slot_rows, *ids;
  const float *weights, *alpha;
  const void* residual;
  void* out;
  const void* dy;
  void* dc;
  float* dweights;
  int topk, n, experts, chunks, c_vec, out_vec, dy_vec;
};

// A token's slots, one to a lane: row, weight and expert's factor. Slots that add
// nothing have a negative row and factors of 0: -1, or where they have a row but
// no expert, -2 - row (it gets gradients of 0).
struct Slot {
  int64_t row;
  float weight, factor;
};
__device__ inline Slot slot_of(const CombineArgs& a, int64_t token, int lane) {
  Slot s = {-1, 0.f, 0.f};
  if (lane < a.topk) {
    const int64_t slot = token * a.topk + lane;
    const int id = a.ids == nullptr ? 0 : a.ids[slot];
    const int64_t row = a.slot_rows == nullptr ? slot : a.slot_rows[slot];
    const float weight = a.weights == nullptr ? 1.f : a.weights[slot];
    if (row >= 0 && row < a.c_rows) {
      if (id >= 0 && id < a.experts) s = {row, weight, a.alpha == nullptr ? 1.f : a.alpha[id]};
      else s.row = -2 - row;
    }
  }
  return s;
}
// Slot j of a wave's token, for the whole wave. Called where all lanes are active:
// what a lane holds is computed by that lane.
__device__ inline int64_t row_of(const Slot& s, int j) {
  const uint32_t low = __builtin_amdgcn_readlane((int)(uint32_t)s.row, j), high = __builtin_amdgcn_readlane((int)(s.row >> 32), j);
  return (int64_t)((uint64_t)high << 32 | low);
}
__device__ inline float lane_value(float v, int j) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), j));
}

// A wave takes 512 columns of a token, eight to a lane; its rows are read at
// once and added in slot order. Bound by memory: each row of c is read once, in
// whole lines that are not kept. 8192 tokens of 8 rows of 7168 fp16, one in 20
// dropped, to bf16: 1.01 GB in 169 us, 6.0 TB/s (a copy, half of it written, 4.9;
// with one row under way at a time 177 us).
template <class C, class Out, int K>
__global__ void __launch_bounds__(kThreads) nvfp4_moe_combine_kernel(CombineArgs a) {
  const uint32_t wave = blockIdx.x * (kThreads / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int64_t token = wave / (uint32_t)a.chunks;
  const int lane = threadIdx.x & 63, col = (int)(wave % (uint32_t)a.chunks) * 512 + lane * 8;
  if (token >= a.tokens) return;
  const Slot slot = slot_of(a, token, lane);
  const float gain = slot.weight * slot.factor;
  const bool mine = col < a.n;
  float sum[8];
  if (a.residual != nullptr && mine) {
    load8<Out>(a.residual, token * a.out_stride + col, a.out_vec, sum);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) sum[i] = 0.f;
  }
  for (int from = 0; from < a.topk; from += K) {
    Raw8<C> v[K];
#pragma unroll
    for (int j = 0; j < K; ++j) {
      const int64_t row = row_of(slot, from + j);  // negative from topk on
      v[j] = Raw8<C>{};
      if (row >= 0 && mine) v[j].load(a.c, row * a.c_stride + col, a.c_vec);
    }
#pragma unroll
    for (int j = 0; j < K; ++j) {
      const float w = lane_value(gain, from + j);
      float x[8];
      v[j].values(x);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[i] = fmaf(w, x[i], sum[i]);
    }
  }
  if (mine) store8<Out>(a.out, token * a.out_stride + col, a.out_vec, sum);
}

// A workgroup per token: dy is read once, its rows of c once, dc written once.
// The sums of d weights go thread by thread, then lanes, then waves: always in
// the same order. Bound by memory, half of it written: 4099 tokens of 4 rows of
// 4096 fp16, 302 MB in 63 us, 4.8 TB/s.
template <class C, class Dy, int K>
__global__ void __launch_bounds__(kThreads) nvfp4_moe_combine_backward_kernel(CombineArgs a) {
  __shared__ float s_sum[K][kThreads / 64];
  const int64_t token = blockIdx.x;
  const int lane = threadIdx.x & 63;
  const Slot slot = slot_of(a, token, lane);
  const float gain = slot.weight * slot.factor;
  int64_t row[K];
  float w[K], sum[K];
#pragma unroll
  for (int j = 0; j < K; ++j) {
    row[j] = row_of(slot, j);  // negative from topk on
    w[j] = lane_value(gain, j);
    sum[j] = 0.f;
  }
  for (int col = threadIdx.x * 8; col < a.n; col += kThreads * 8) {
    Raw8<Dy> raw;
    Raw8<C> v[K];
    raw.load(a.dy, token * a.dy_stride + col, a.dy_vec);
#pragma unroll
    for (int j = 0; j < K; ++j)
      if (row[j] >= 0) v[j].load(a.c, row[j] * a.c_stride + col, a.c_vec);
    float dy[8];
    raw.values(dy);
#pragma unroll
    for (int j = 0; j < K; ++j) {
      if (row[j] < 0) {
        const float zeros[8] = {};
        if (row[j] < -1) store8<C>(a.dc, (-2 - row[j]) * a.c_stride + col, a.c_vec, zeros);
        continue;
      }
      float x[8], d[8];
      v[j].values(x);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        sum[j] = fmaf(dy[i], x[i], sum[j]);
        d[i] = w[j] * dy[i];
      }
      store8<C>(a.dc, row[j] * a.c_stride + col, a.c_vec, d);
    }
  }
#pragma unroll
  for (int j = 0; j < K; ++j) {
    float s = sum[j];
    for (int d = 1; d < 64; d *= 2) s += __shfl_xor(s, d);
    if (lane == 0) s_sum[j][threadIdx.x / 64] = s;
  }
  __syncthreads();
  if ((int)threadIdx.x < a.topk) {
    float s = 0.f;
    for (int i = 0; i < kThreads / 64; ++i) s += s_sum[threadIdx.x][i];
    a.dweights[token * a.topk + threadIdx.x] = slot.row >= 0 ? s * slot.factor : 0.f;
  }
}

// p: dy or out, rows of `dtype` `stride` apart.
int check_combine(const CombineArgs& a, int c_dtype, int dtype, int64_t stride, const void* p) {
  if (!known_type(c_dtype) || !known_type(dtype)) return NVFP4_ERR_INVALID;
  if (a.tokens < 0 || a.tokens >= (int64_t)1 << 30 || a.topk < 1 || a.topk > NVFP4_MOE_MAX_TOPK) return NVFP4_ERR_INVALID;
  if (a.n < 0 || a.n % 8 || a.c_stride < a.n || stride < a.n) return NVFP4_ERR_INVALID;
  if (a.c_stride > (int64_t)1 << 30 || stride > (int64_t)1 << 30) return NVFP4_ERR_INVALID;
  if (a.alpha != nullptr && (a.ids == nullptr || a.experts < 1)) return NVFP4_ERR_INVALID;
  if (a.c_rows < 0 || (a.slot_rows == nullptr && a.tokens * a.topk > a.c_rows)) return NVFP4_ERR_INVALID;
  if (a.tokens > 0 && a.n > 0 && (p == nullptr || (a.c_rows > 0 && a.c == nullptr))) return NVFP4_ERR_INVALID;
  if (!aligned(a.slot_rows, 4) || !aligned(a.ids, 4) || !aligned(a.weights, 4) || !aligned(a.alpha, 4))
    return NVFP4_ERR_MISALIGNED;
  if (!aligned(a.c, element_bytes(c_dtype)) || !aligned(p, element_bytes(dtype))) return NVFP4_ERR_MISALIGNED;
  return NVFP4_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int nvfp4_moe_combine(const void* c, int c_dtype, int64_t c_stride, int64_t c_rows, int64_t tokens, int topk, int n,
                      const int32_t* slot_rows, const float* weights, const float* alpha, const int32_t* ids,
                      int experts, const void* residual, void* out, int out_dtype, int64_t out_stride, void* stream) {
  CombineArgs a = {};
  a.c = c;
  a.c_stride = c_stride;
  a.c_rows = c_rows;
  a.tokens = tokens;
  a.out_stride = out_stride;
  a.slot_rows = slot_rows;
  a.ids = ids;
  a.experts = alpha == nullptr && experts <= 0 ? INT32_MAX : experts;
  a.weights = weights;
  a.alpha = alpha;
  a.residual = residual;
  a.out = out;
  a.topk = topk;
  a.n = n;
  if (int rc = check_combine(a, c_dtype, out_dtype, out_stride, out)) return rc;
  if (!aligned(residual, element_bytes(out_dtype))) return NVFP4_ERR_MISALIGNED;
  if (tokens == 0 || n == 0) return NVFP4_OK;
  a.chunks = ceil_div(n, 512);
  a.c_vec = wide_rows(c, c_dtype, c_stride);
  a.out_vec = wide_rows(out, out_dtype, out_stride) && aligned(residual, 16);
  const int64_t blocks = ceil_div64(tokens * a.chunks, kThreads / 64);
  if (blocks >= (int64_t)1 << 24) return NVFP4_ERR_INVALID;
  const hipStream_t st = (hipStream_t)stream;
  return with_type(c_dtype, [&](auto t) {
    return with_type(out_dtype, [&](auto u) {
      using C = decltype(t);
      using O = decltype(u);
      if (topk <= 1) nvfp4_moe_combine_kernel<C, O, 1><<<(unsigned)blocks, kThreads, 0, st>>>(a);
      else if (topk <= 2) nvfp4_moe_combine_kernel<C, O, 2><<<(unsigned)blocks, kThreads, 0, st>>>(a);
      else if (topk <= 4) nvfp4_moe_combine_kernel<C, O, 4><<<(unsigned)blocks, kThreads, 0, st>>>(a);
      else nvfp4_moe_combine_kernel<C, O, 8><<<(unsigned)blocks, kThreads, 0, st>>>(a);
      return launched();
    });
  });
}

int nvfp4_moe_combine_backward(const void* dy, int dy_dtype, int64_t dy_stride, const void* c, int c_dtype,
                               int64_t c_stride, int64_t c_rows, int64_t tokens, int topk, int n,
                               const int32_t* slot_rows, const float* weights, const float* alpha, const int32_t* ids,
                               int experts, void* dc, float* dweights, void* stream) {
  CombineArgs a = {};
  a.c = c;
  a.c_stride = c_stride;
  a.c_rows = c_rows;
  a.tokens = tokens;
  a.dy = dy;
  a.dy_stride = dy_stride;
  a.slot_rows = slot_rows;
  a.ids = ids;
  a.experts = alpha == nullptr && experts <= 0 ? INT32_MAX : experts;
  a.weights = weights;
  a.alpha = alpha;
  a.dc = dc;
  a.dweights = dweights;
  a.topk = topk;
  a.n = n;
  if (int rc = check_combine(a, c_dtype, dy_dtype, dy_stride, dy)) return rc;
  if (tokens > 0 && (dweights == nullptr || (n > 0 && c_rows > 0 && dc == nullptr))) return NVFP4_ERR_INVALID;
  if (tokens >= (int64_t)1 << 24) return NVFP4_ERR_INVALID;
  if (!aligned(dc, element_bytes(c_dtype)) || !aligned(dweights, 4)) return NVFP4_ERR_MISALIGNED;
  if (tokens == 0) return NVFP4_OK;
  a.c_vec = wide_rows(c, c_dtype, c_stride) && aligned(dc, 16);
  a.dy_vec = wide_rows(dy, dy_dtype, dy_stride);
  const hipStream_t st = (hipStream_t)stream;
  return with_type(c_dtype, [&](auto t) {
    return with_type(dy_dtype, [&](auto u) {
      using C = decltype(t);
      using D = decltype(u);
      if (topk <= 2) nvfp4_moe_combine_backward_kernel<C, D, 2><<<(unsigned)tokens, kThreads, 0, st>>>(a);
      else if (topk <= 4) nvfp4_moe_combine_backward_kernel<C, D, 4><<<(unsigned)tokens, kThreads, 0, st>>>(a);
      else if (topk <= 8) nvfp4_moe_combine_backward_kernel<C, D, 8><<<(unsigned)tokens, kThreads, 0, st>>>(a);
      else nvfp4_moe_combine_backward_kernel<C, D, 16><<<(unsigned)tokens, kThreads, 0, st>>>(a);
      return launched();
    });
  });
}

}  // extern "C"
