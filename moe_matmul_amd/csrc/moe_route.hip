// Routing: scores, choice of experts and weights of every token, and the
// gradient of the weights with respect to the logits.
#include "moe_common.h"

namespace moe {

thread_local int t_last_hip_error = 0;

namespace {

constexpr int kThreads = 256;
constexpr double kLargest = 1e300;  // choice values are held within +-this, so that a key stays finite
constexpr int kIndexMask = NVFP4_MOE_MAX_EXPERTS - 1;

// ---- keys: a choice value and its expert in one fp64 ------------------------
// The nine low mantissa bits of the value hold the index such that of two equal
// values the lower index has the larger key. So one max and one min order two
// candidates with their indices, and no two keys of a token are equal.
__device__ inline double make_key(double v, int e) {
  v = fmin(fmax(v, -kLargest), kLargest) + 0.0;  // -0 counts as 0
  uint64_t u = __builtin_bit_cast(uint64_t, v) & ~(uint64_t)kIndexMask;
  u |= (int64_t)u < 0 ? (uint64_t)e : (uint64_t)(kIndexMask - e);
  return __builtin_bit_cast(double, u);
}
__device__ inline double no_key() { return -__builtin_inf(); }
__device__ inline int key_index(double key) {
  const uint64_t u = __builtin_bit_cast(uint64_t, key);
  const int low = (int)(u & kIndexMask);
  return key == no_key() ? -1 : (int64_t)u < 0 ? low : kIndexMask - low;
}
__device__ inline double key_value(double key) {
  return key == no_key() ? key
                         : __builtin_bit_cast(double, __builtin_bit_cast(uint64_t, key) & ~(uint64_t)kIndexMask);
}

// ---- exp and sigmoid in fp64 -------------------------------------------------
// 2^n times the Taylor series of e^r, |r| <= ln 2 / 2: 13 terms leave 2^-53 / 4.
__device__ inline double exp_f64(double x) {
  x = fmin(fmax(x, -700.0), 700.0);
  const double n = __builtin_rint(x * 1.4426950408889634);
  double r = fma(-n, 6.93147180369123816490e-01, x);
  r = fma(-n, 1.90821492927058770002e-10, r);
  double p = 1.0 / 479001600;
  p = fma(p, r, 1.0 / 39916800);
  p = fma(p, r, 1.0 / 3628800);
  p = fma(p, r, 1.0 / 362880);
  p = fma(p, r, 1.0 / 40320);
  p = fma(p, r, 1.0 / 5040);
  p = fma(p, r, 1.0 / 720);
  p = fma(p, r, 1.0 / 120);
  p = fma(p, r, 1.0 / 24);
  p = fma(p, r, 1.0 / 6);
  p = fma(p, r, 0.5);
  p = fma(p, r, 1.0);
  p = fma(p, r, 1.0);
  return __builtin_ldexp(p, (int)n);
}
__device__ inline double inverse_f64(double d) {
  double r = __builtin_amdgcn_rcp(d);
  r = fma(fma(-d, r, 1.0), r, r);
  return fma(fma(-d, r, 1.0), r, r);
}

// ---- sorted lists in registers -------------------------------------------------
__device__ inline void order(double& a, double& b) {  // a the larger
  const double x = fmax(a, b), y = fmin(a, b);
  a = x;
  b = y;
}
// Odd-even merge sort, falling.
template <int N> __device__ inline void sort_falling(double (&v)[N]) {
#pragma unroll
  for (int p = 1; p < N; p *= 2) {
#pragma unroll
    for (int k = p; k >= 1; k /= 2) {
#pragma unroll
      for (int j = k % p; j <= N - 1 - k; j += 2 * k) {
#pragma unroll
        for (int i = 0; i < k; ++i)
          if (i + j + k < N && (i + j) / (2 * p) == (i + j + k) / (2 * p)) order(v[i + j], v[i + j + k]);
      }
    }
  }
}
// The K largest of two falling lists, falling: the larger of each pair of one
// list and the other reversed form a bitonic sequence.
template <int K> __device__ inline void merge_falling(double (&list)[K], const double (&other)[K]) {
#pragma unroll
  for (int i = 0; i < K; ++i) list[i] = fmax(list[i], other[K - 1 - i]);
#pragma unroll
  for (int k = K / 2; k >= 1; k /= 2) {
#pragma unroll
    for (int i = 0; i < K; ++i)
      if ((i & k) == 0) order(list[i], list[i + k]);
  }
}

template <int kCtrl> __device__ inline double from_lane(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t low = __builtin_amdgcn_mov_dpp((int)(uint32_t)u, kCtrl, 0xF, 0xF, false);
  const uint32_t high = __builtin_amdgcn_mov_dpp((int)(uint32_t)(u >> 32), kCtrl, 0xF, 0xF, false);
  return __builtin_bit_cast(double, (uint64_t)high << 32 | low);
}
constexpr int kXor1 = 0xB1, kXor2 = 0x4E;           // quad permutations
constexpr int kMirror8 = 0x141, kMirror16 = 0x140;  // lane i <-> 7 - i, 15 - i

template <int K, int kCtrl> __device__ inline void merge_with(double (&list)[K]) {
  double other[K];
#pragma unroll
  for (int i = 0; i < K; ++i) other[i] = from_lane<kCtrl>(list[i]);
  merge_falling(list, other);
}
template <int K> __device__ inline void merge_across(double (&list)[K], int distance) {
  double other[K];
#pragma unroll
  for (int i = 0; i < K; ++i) other[i] = __shfl_xor(list[i], distance);
  merge_falling(list, other);
}
// Every lane of a token's `lanes` gets the K largest of all of them.
template <int K> __device__ inline void merge_lanes(double (&list)[K], int lanes) {
  if (lanes > 1) merge_with<K, kXor1>(list);
  if (lanes > 2) merge_with<K, kXor2>(list);
  if (lanes > 4) merge_with<K, kMirror8>(list);
  if (lanes > 8) merge_with<K, kMirror16>(list);
  if (lanes > 16) merge_across<K>(list, 16);
  if (lanes > 32) merge_across<K>(list, 32);
}

template <class V, class Op> __device__ inline V across(V v, int lanes, Op op) {
  for (int d = 1; d < lanes; d *= 2) v = op(v, __shfl_xor(v, d));
  return v;
}
__device__ inline float max_across(float v, int lanes) {
  return across(v, lanes, [](float a, float b) { return fmaxf(a, b); });
}
template <class V> __device__ inline V sum_across(V v, int lanes) {
  return across(v, lanes, [](V a, V b) { return a + b; });
}

// ---- which experts a lane holds --------------------------------------------
// `lanes` lanes share a token. Each holds up to NC chunks of eight experts:
// chunk c is experts base + c * step .. + 7, those below end.
struct Share {
  int base, step, end;
};

struct RouteArgs {
  const void* logits;
  int64_t tokens, row_stride;
  const float* bias;
  int32_t* ids;
  float* weights;
  int experts, dtype, vec;
  int lanes;      // per token
  int per;        // experts of a group
  int lanes_of;   // lanes that share a group (1 where a lane has whole groups)
  int groups_of;  // groups that a lane has (1 where lanes share one)
  nvfp4_moe_choice how;
};

__device__ inline Share share_of(const RouteArgs& a, int lane) {
  Share s;
  if (a.how.groups == 1) {
    s.base = lane * 8;
    s.step = a.lanes * 8;
    s.end = a.experts;
  } else if (a.lanes_of > 1) {
    const int g = lane / a.lanes_of, part = (a.per + a.lanes_of - 1) / a.lanes_of, at = lane % a.lanes_of * part;
    s.base = g * a.per + at;
    s.step = 8;
    s.end = g < a.how.groups ? g * a.per + min(a.per, at + part) : 0;
  } else {
    s.base = lane * a.groups_of * a.per;
    s.step = 8;
    s.end = min(a.experts, (lane + 1) * a.groups_of * a.per);
  }
  return s;
}

// A lane's logits; NaN past its share (its own NaNs are noted first).
template <class T, int NC>
__device__ inline void load_share(const void* row, const Share& s, bool vec, float (&x)[NC * 8]) {
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int e = s.base + c * s.step;
    float v[8];
    if (e + 8 <= s.end) {
      load8<T>(row, e, vec && e % 8 == 0, v);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = e + j < s.end ? load1<T>(row, e + j) : -__builtin_inff();
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) x[c * 8 + j] = v[j];
  }
}
template <int NC>
__device__ inline void load_logits(const void* logits, int dtype, int64_t at, const Share& s, bool vec,
                                   float (&x)[NC * 8]) {
  if (dtype == NVFP4_MOE_F32) load_share<F32, NC>((const float*)logits + at, s, vec, x);
  else if (dtype == NVFP4_MOE_F16) load_share<F16, NC>((const uint16_t*)logits + at, s, vec, x);
  else load_share<BF16, NC>((const uint16_t*)logits + at, s, vec, x);
}
__device__ inline float load_logit(const void* logits, int dtype, int64_t at) {
  return dtype == NVFP4_MOE_F32   ? load1<F32>(logits, at)
         : dtype == NVFP4_MOE_F16 ? load1<F16>(logits, at)
                                  : load1<BF16>(logits, at);
}

__device__ inline bool poisons(float x, int score) {
  return x != x || (score == NVFP4_MOE_SOFTMAX && x == __builtin_inff());
}

// Routing. A token's logits are read once into the registers of `lanes` lanes;
// each lane keeps the K largest keys of its experts in a sorted list (sort a
// chunk, merge it in: two instructions for each comparison), and the lanes'
// lists are merged in log2(lanes) steps. kScores: the choice goes by scores
// (a bias or groups), which are then computed in fp64; else by the logits.
template <int K, int NC, bool kScores>
__global__ void __launch_bounds__(kThreads) nvfp4_moe_route_kernel(RouteArgs a) {
  __shared__ double s_best[kScores ? kThreads : 1][2];
  __shared__ double s_group[kScores ? kThreads / 4 : 1][kScores ? NVFP4_MOE_MAX_GROUPS : 1];
  const int lane = threadIdx.x & (a.lanes - 1), local = threadIdx.x / a.lanes;
  const int64_t mine = (int64_t)blockIdx.x * (kThreads / a.lanes) + local;
  const int64_t token = mine < a.tokens ? mine : a.tokens - 1;  // lanes past the end repeat the last token
  const Share s = share_of(a, lane);
  float x[NC * 8];
  load_logits<NC>(a.logits, a.dtype, token * a.row_stride, s, a.vec, x);

  bool bad = false;
  float top = -__builtin_inff();
#pragma unroll
  for (int i = 0; i < NC * 8; ++i) {
    bad |= poisons(x[i], a.how.score);
    top = fmaxf(top, x[i]);  // passes over NaN
  }
  const uint64_t lanes_mask = (a.lanes == 64 ? ~0ull : (1ull << a.lanes) - 1) << (threadIdx.x & 63 & ~(a.lanes - 1));
  bad = (__ballot(bad) & lanes_mask) != 0;

  const bool softmax = a.how.score == NVFP4_MOE_SOFTMAX;
  float total = 1.f;  // of e^(x - top) over all experts
  double list[K];
  if constexpr (!kScores) {
    if (softmax && !a.how.renormalize) {
      top = max_across(top, a.lanes);
      const float from = top == -__builtin_inff() ? 0.f : top;
      total = 0.f;
#pragma unroll
      for (int i = 0; i < NC * 8; ++i) total += exp_f32(x[i] - from);
      total = sum_across(total, a.lanes);
    }
#pragma unroll
    for (int i = 0; i < K; ++i) list[i] = no_key();
#pragma unroll
    for (int at = 0; at < NC * 8; at += K) {
      double part[K];
#pragma unroll
      for (int i = 0; i < K; ++i) {
        const int n = at + i;
        const bool there = n < NC * 8 && x[n < NC * 8 ? n : 0] > -__builtin_inff();  // not for NaN
        part[i] = there ? make_key((double)x[n < NC * 8 ? n : 0], s.base + n / 8 * s.step + n % 8) : no_key();
      }
      sort_falling(part);
      merge_falling(list, part);
    }
  } else {
    double v[NC * 8];
    if (softmax) {
      top = max_across(top, a.lanes);
      const double from = top == -__builtin_inff() ? 0.0 : (double)fminf(top, 3.4e38f);
      double sum = 0.0;
#pragma unroll
      for (int i = 0; i < NC * 8; ++i) {
        v[i] = exp_f64((double)x[i] - from);
        sum += x[i] > -__builtin_inff() ? v[i] : 0.0;
      }
      sum = sum_across(sum, a.lanes);
      total = (float)sum;
      const double inverse = inverse_f64(sum > 0.0 ? sum : 1.0);
#pragma unroll
      for (int i = 0; i < NC * 8; ++i) v[i] *= inverse;
    } else {
#pragma unroll
      for (int i = 0; i < NC * 8; ++i) v[i] = inverse_f64(1.0 + exp_f64(-(double)x[i]));
    }
#pragma unroll
    for (int i = 0; i < NC * 8; ++i) {
      const int e = s.base + i / 8 * s.step + i % 8;
      if (a.bias != nullptr) v[i] += e < s.end ? (double)a.bias[e] : 0.0;
      const bool there = x[i] > -__builtin_inff() && v[i] > -__builtin_inf();  // neither for NaN
      v[i] = there ? make_key(v[i], e) : no_key();
    }
    if (a.how.groups > 1) {
      // The best two of each lane, or the values of each lane's groups, then a
      // group's rank: how many groups are better.
      auto worth = [&](double first, double second) {
        const double f = key_value(first), g = key_value(second);
        return a.how.group_best == 1 || g == no_key() ? f : f + g;
      };
      if (a.groups_of == 1) {
        double one = no_key(), two = no_key();
#pragma unroll
        for (int i = 0; i < NC * 8; ++i) {
          two = fmax(two, fmin(one, v[i]));
          one = fmax(one, v[i]);
        }
        s_best[threadIdx.x][0] = one;
        s_best[threadIdx.x][1] = two;
        __syncthreads();
        for (int g = lane; g < a.how.groups; g += a.lanes) {
          double first = no_key(), second = no_key();
          for (int q = 0; q < a.lanes_of; ++q) {
            const int from = threadIdx.x - lane + g * a.lanes_of + q;
            const double p = s_best[from][0], r = s_best[from][1];
            second = fmax(fmax(second, r), fmin(first, p));
            first = fmax(first, p);
          }
          s_group[local][g] = worth(first, second);
        }
      } else {
        for (int q = 0; q < a.groups_of; ++q) {
          const int g = lane * a.groups_of + q;
          if (g >= a.how.groups) break;
          double one = no_key(), two = no_key();
#pragma unroll
          for (int i = 0; i < NC * 8; ++i) {
            const double w = i / a.per == q ? v[i] : no_key();
            two = fmax(two, fmin(one, w));
            one = fmax(one, w);
          }
          s_group[local][g] = worth(one, two);
        }
      }
      __syncthreads();
      for (int q = 0; q < a.groups_of; ++q) {
        const int g = a.groups_of == 1 ? lane / a.lanes_of : lane * a.groups_of + q;
        const double w = g < a.how.groups ? s_group[local][g] : no_key();
        int better = 0;
        for (int o = 0; o < a.how.groups; ++o) {
          const double u = s_group[local][o];
          better += u > w || (u == w && o < g);
        }
#pragma unroll
        for (int i = 0; i < NC * 8; ++i) {
          const bool of = a.groups_of == 1 || i / a.per == q;
          if (of && better >= a.how.topk_groups) v[i] = no_key();
        }
      }
    }
#pragma unroll
    for (int i = 0; i < K; ++i) list[i] = no_key();
#pragma unroll
    for (int at = 0; at < NC * 8; at += K) {
      double part[K];
#pragma unroll
      for (int i = 0; i < K; ++i) part[i] = at + i < NC * 8 ? v[at + i < NC * 8 ? at + i : 0] : no_key();
      sort_falling(part);
      merge_falling(list, part);
    }
  }
  merge_lanes(list, a.lanes);

  // lane j < topk has slot j
  double key = no_key();
#pragma unroll
  for (int i = 0; i < K; ++i) key = i == lane ? list[i] : key;
  const int id = lane < a.how.topk ? key_index(key) : -1;
  const float chosen = id >= 0 ? load_logit(a.logits, a.dtype, token * a.row_stride + id) : -__builtin_inff();
  float w;
  if (softmax) {
    const float from = a.how.renormalize ? max_across(chosen, a.lanes) : top;
    w = exp_f32(chosen - (from == -__builtin_inff() ? 0.f : from));
  } else {
    w = id >= 0 ? 1.f / (1.f + exp_f32(-chosen)) : 0.f;
  }
  if (a.how.renormalize) total = sum_across(w, a.lanes);
  else if (!softmax) total = 1.f;
  w = w / (total == 0.f ? 1.f : total) * a.how.scale;
  if (id < 0) w = 0.f;
  else if (bad) w = __builtin_nanf("");
  if (lane < a.how.topk && mine < a.tokens) {
    a.ids[token * a.how.topk + lane] = id;
    a.weights[token * a.how.topk + lane] = w;
  }
}

struct RouteBackwardArgs {
  const void* logits;
  int64_t tokens, row_stride;
  const int32_t* ids;
  const float* dweights;
  void* dlogits;
  int64_t out_stride;
  int experts, dtype, vec, out_vec;
  int lanes;
  nvfp4_moe_choice how;
};

template <class T, int NC>
__device__ inline void store_share(void* row, const Share& s, bool vec, const float (&x)[NC * 8]) {
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int e = s.base + c * s.step;
    if (e + 8 <= s.end) {
      store8<T>(row, e, vec, x + c * 8);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (e + j < s.end) store1<T>(row, e + j, x[c * 8 + j]);
    }
  }
}

// d logits. With dp = scale * dw of the chosen experts (0 elsewhere), S the sum
// of the chosen scores and q = s / S:
//   renormalised: ds = (dp - sum dp q) / S, else ds = dp
//   softmax: dx = s (ds - sum ds s) (renormalised, the sum is 0 and dx = q (dp - sum dp q))
//   sigmoid: dx = ds s (1 - s)
// Only the softmax that is not renormalised has a gradient for experts that
// were not chosen, and only it reads the whole row. The chosen experts' values
// go to their lanes through shared memory; every lane then writes its share.
template <int NC>
__global__ void __launch_bounds__(kThreads) nvfp4_moe_route_backward_kernel(RouteBackwardArgs a) {
  __shared__ float s_dp[NC * 8][kThreads];
  const int lane = threadIdx.x & (a.lanes - 1);
  const int64_t mine = (int64_t)blockIdx.x * (kThreads / a.lanes) + threadIdx.x / a.lanes;
  const int64_t token = mine < a.tokens ? mine : a.tokens - 1;
  const bool softmax = a.how.score == NVFP4_MOE_SOFTMAX, dense = softmax && !a.how.renormalize;
  const Share s = {lane * 8, a.lanes * 8, a.experts};
#pragma unroll
  for (int i = 0; i < NC * 8; ++i) s_dp[i][threadIdx.x] = 0.f;

  int id = -1;
  float dw = 0.f, chosen = -__builtin_inff();
  if (lane < a.how.topk) {
    id = a.ids[token * a.how.topk + lane];
    if (id >= a.experts) id = -1;
    if (id >= 0) {
      dw = a.dweights[token * a.how.topk + lane] * a.how.scale;
      chosen = load_logit(a.logits, a.dtype, token * a.row_stride + id);
    }
  }
  float x[NC * 8], p, from = 0.f;
  if (dense) {
    load_logits<NC>(a.logits, a.dtype, token * a.row_stride, s, a.vec, x);
    float top = -__builtin_inff(), total = 0.f;
#pragma unroll
    for (int i = 0; i < NC * 8; ++i) top = fmaxf(top, x[i]);
    top = max_across(top, a.lanes);
    from = top == -__builtin_inff() ? 0.f : top;
#pragma unroll
    for (int i = 0; i < NC * 8; ++i) {
      x[i] = exp_f32(x[i] - from);
      total += x[i];
    }
    total = sum_across(total, a.lanes);
    total = total == 0.f ? 1.f : total;
    const float inverse = 1.f / total;
#pragma unroll
    for (int i = 0; i < NC * 8; ++i) x[i] *= inverse;
    p = id >= 0 ? exp_f32(chosen - from) * inverse : 0.f;
  } else if (softmax) {
    from = max_across(chosen, a.lanes);
    p = id >= 0 ? exp_f32(chosen - (from == -__builtin_inff() ? 0.f : from)) : 0.f;
  } else {
    p = id >= 0 ? 1.f / (1.f + exp_f32(-chosen)) : 0.f;
  }
  float total = 1.f, q = p;
  if (a.how.renormalize) {
    total = sum_across(p, a.lanes);
    total = total == 0.f ? 1.f : total;
    q = p / total;
  }
  const float dot = sum_across(id >= 0 ? dw * q : 0.f, a.lanes);
  float give;  // to the chosen expert's lane
  if (dense) give = dw;
  else if (softmax) give = q * (dw - dot);
  else give = (a.how.renormalize ? (dw - dot) / total : dw) * p * (1.f / (1.f + exp_f32(chosen)));
  __syncthreads();
  if (id >= 0) {
    const int chunk = id / 8, owner = (threadIdx.x & ~(a.lanes - 1)) + (chunk & (a.lanes - 1));
    s_dp[chunk / a.lanes * 8 + id % 8][owner] = give;
  }
  __syncthreads();
  float out[NC * 8];
#pragma unroll
  for (int i = 0; i < NC * 8; ++i) {
    const float got = s_dp[i][threadIdx.x];
    out[i] = dense ? x[i] * (got - dot) : got;
  }
  if (mine < a.tokens) {
    if (a.dtype == NVFP4_MOE_F32) store_share<F32, NC>((float*)a.dlogits + token * a.out_stride, s, a.out_vec, out);
    else if (a.dtype == NVFP4_MOE_F16) store_share<F16, NC>((uint16_t*)a.dlogits + token * a.out_stride, s, a.out_vec, out);
    else store_share<BF16, NC>((uint16_t*)a.dlogits + token * a.out_stride, s, a.out_vec, out);
  }
}

int check_choice(const nvfp4_moe_choice* how, int experts) {
  if (how == nullptr || experts < 1 || experts > NVFP4_MOE_MAX_EXPERTS) return NVFP4_ERR_INVALID;
  if (how->score != NVFP4_MOE_SOFTMAX && how->score != NVFP4_MOE_SIGMOID) return NVFP4_ERR_INVALID;
  if (how->groups < 1 || how->groups > NVFP4_MOE_MAX_GROUPS || experts % how->groups) return NVFP4_ERR_INVALID;
  if (how->topk_groups < 1 || how->topk_groups > how->groups) return NVFP4_ERR_INVALID;
  if (how->group_best < 1 || how->group_best > 2) return NVFP4_ERR_INVALID;
  if (how->topk < 1 || how->topk > NVFP4_MOE_MAX_TOPK) return NVFP4_ERR_INVALID;
  if (how->topk > how->topk_groups * (experts / how->groups)) return NVFP4_ERR_INVALID;
  return NVFP4_OK;
}

int check_rows(const void* p, int dtype, int64_t tokens, int experts, int64_t stride) {
  if (!known_type(dtype) || tokens < 0 || tokens >= (int64_t)1 << 26 || stride < experts) return NVFP4_ERR_INVALID;
  if (stride > (int64_t)1 << 40) return NVFP4_ERR_INVALID;
  if (tokens > 0 && p == nullptr) return NVFP4_ERR_INVALID;
  return aligned(p, element_bytes(dtype)) ? NVFP4_OK : NVFP4_ERR_MISALIGNED;
}

int at_least_pow2(int v) {
  int p = 1;
  while (p < v) p *= 2;
  return p;
}

// Lanes of a token: enough that every slot has one and none holds more than 32
// experts, and more where there are too few tokens to fill the chip.
int widen(int lanes, int64_t tokens, int experts) {
  while (lanes < 64 && tokens * lanes < 256 * 1024 && lanes * 8 < experts) lanes *= 2;
  return lanes;
}

// Chunks of eight experts of the fullest lane, and how groups lie on lanes.
int lay_out(RouteArgs& a) {
  const int groups = a.how.groups;
  a.per = a.experts / groups;
  a.lanes_of = a.groups_of = 1;
  if (groups == 1) return ceil_div(ceil_div(a.experts, 8), a.lanes);
  if (a.lanes >= groups) a.lanes_of = a.lanes / groups;
  else a.groups_of = ceil_div(groups, a.lanes);
  return ceil_div(a.groups_of > 1 ? a.groups_of * a.per : ceil_div(a.per, a.lanes_of), 8);
}

template <int K, int NC> void launch_route(const RouteArgs& a, bool scores, int64_t blocks, hipStream_t stream) {
  if (scores) nvfp4_moe_route_kernel<K, NC, true><<<dim3((unsigned)blocks), kThreads, 0, stream>>>(a);
  else nvfp4_moe_route_kernel<K, NC, false><<<dim3((unsigned)blocks), kThreads, 0, stream>>>(a);
}
template <int K> void launch_route(const RouteArgs& a, int chunks, bool scores, int64_t blocks, hipStream_t stream) {
  if (chunks <= 1) launch_route<K, 1>(a, scores, blocks, stream);
  else if (chunks <= 2) launch_route<K, 2>(a, scores, blocks, stream);
  else launch_route<K, 4>(a, scores, blocks, stream);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int nvfp4_moe_last_hip_error(void) { return t_last_hip_error; }

int nvfp4_moe_route(const void* logits, int dtype, int64_t tokens, int experts, int64_t row_stride,
                    const float* bias, const nvfp4_moe_choice* choice, int32_t* ids, float* weights,
                    void* stream) {
  if (int rc = check_choice(choice, experts)) return rc;
  if (int rc = check_rows(logits, dtype, tokens, experts, row_stride)) return rc;
  if (tokens > 0 && (ids == nullptr || weights == nullptr)) return NVFP4_ERR_INVALID;
  if (!aligned(ids, 4) || !aligned(weights, 4) || !aligned(bias, 4)) return NVFP4_ERR_MISALIGNED;
  if (tokens == 0) return NVFP4_OK;
  RouteArgs a = {};
  a.logits = logits;
  a.tokens = tokens;
  a.row_stride = row_stride;
  a.bias = bias;
  a.ids = ids;
  a.weights = weights;
  a.experts = experts;
  a.dtype = dtype;
  a.vec = wide_rows(logits, dtype, row_stride);
  a.how = *choice;
  a.lanes = widen(at_least_pow2(choice->topk < 4 ? 4 : choice->topk), tokens, experts);
  int chunks = lay_out(a);
  while (chunks > 4) {
    a.lanes *= 2;
    chunks = lay_out(a);
  }
  const bool scores = bias != nullptr || choice->groups > 1;
  const int64_t blocks = ceil_div64(tokens, kThreads / a.lanes);
  const hipStream_t st = (hipStream_t)stream;
  if (choice->topk <= 2) launch_route<2>(a, chunks, scores, blocks, st);
  else if (choice->topk <= 4) launch_route<4>(a, chunks, scores, blocks, st);
  else if (choice->topk <= 8) launch_route<8>(a, chunks, scores, blocks, st);
  else launch_route<16>(a, chunks, scores, blocks, st);
  return launched();
}

int nvfp4_moe_route_backward(const void* logits, int dtype, int64_t tokens, int experts, int64_t row_stride,
                             const nvfp4_moe_choice* choice, const int32_t* ids, const float* dweights,
                             void* dlogits, int64_t dlogits_stride, void* stream) {
  if (int rc = check_choice(choice, experts)) return rc;
  if (int rc = check_rows(logits, dtype, tokens, experts, row_stride)) return rc;
  if (int rc = check_rows(dlogits, dtype, tokens, experts, dlogits_stride)) return rc;
  if (tokens > 0 && (ids == nullptr || dweights == nullptr)) return NVFP4_ERR_INVALID;
  if (!aligned(ids, 4) || !aligned(dweights, 4)) return NVFP4_ERR_MISALIGNED;
  if (tokens == 0) return NVFP4_OK;
  RouteBackwardArgs a = {};
  a.logits = logits;
  a.tokens = tokens;
  a.row_stride = row_stride;
  a.ids = ids;
  a.dweights = dweights;
  a.dlogits = dlogits;
  a.out_stride = dlogits_stride;
  a.experts = experts;
  a.dtype = dtype;
  a.vec = wide_rows(logits, dtype, row_stride);
  a.out_vec = wide_rows(dlogits, dtype, dlogits_stride);
  a.how = *choice;
  a.lanes = widen(at_least_pow2(choice->topk < 4 ? 4 : choice->topk), tokens, experts);
  while (ceil_div(experts, 8 * a.lanes) > 4) a.lanes *= 2;
  const int chunks = ceil_div(experts, 8 * a.lanes);
  const dim3 grid((unsigned)ceil_div64(tokens, kThreads / a.lanes));
  const hipStream_t st = (hipStream_t)stream;
  if (chunks <= 1) nvfp4_moe_route_backward_kernel<1><<<grid, kThreads, 0, st>>>(a);
  else if (chunks <= 2) nvfp4_moe_route_backward_kernel<2><<<grid, kThreads, 0, st>>>(a);
  else nvfp4_moe_route_backward_kernel<4><<<grid, kThreads, 0, st>>>(a);
  return launched();
}

}  // extern "C"
