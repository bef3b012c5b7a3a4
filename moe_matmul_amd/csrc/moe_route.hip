// Routing: scores, choice of experts and weights of every token, and the
// gradient of the weights with respect to the logits.
#include "moe_common.h"

#include <type_traits>

namespace moe {

thread_local int t_last_hip_error = 0;

namespace {

constexpr int kThreads = 256;
constexpr double kLargest = 0x1p+1000;  // choice values are held within +-this, so that a key stays finite
constexpr int kIndexMask = NVFP4_MOE_MAX_EXPERTS - 1;
constexpr int kLeastLanes = 4;  // of a token
constexpr int64_t kLogitLanes = 64 * 1024, kScoreLanes = 256 * 1024;  // in all, that fill the chip

// ---- keys: a choice value and its expert in one number ------------------------
// The low bits hold the index such that of two equal values the lower index has
// the larger key. So one max and one min order two candidates with their
// indices, and no two keys of a token are equal.

// fp64 values in fp64, the index in the nine low mantissa bits. Values lie within
// +-kLargest (whose low bits are 0), which is also the key of no candidate: fp32
// logits keep their order exactly, scores to 2^-43.
struct Wide {
  typedef double Key;
  static __device__ inline Key none() { return -kLargest; }
  static __device__ inline Key make(double v, int e) {  // NaN and -inf: none
    v = fmin(fmax(v, -kLargest), kLargest) + 0.0;       // -0 counts as 0
    uint64_t u = __builtin_bit_cast(uint64_t, v) & ~(uint64_t)kIndexMask;
    u |= (int64_t)u < 0 ? (uint64_t)e : (uint64_t)(kIndexMask - e);
    return __builtin_bit_cast(double, u);
  }
  // fp32 logits have no low bits to clear
  static __device__ inline Key of_logit(float x, int e) {
    const double v = fmin(fmax((double)(x + 0.f), -kLargest), kLargest);
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    return __builtin_bit_cast(double, u | ((int64_t)u < 0 ? (uint64_t)e : (uint64_t)(kIndexMask - e)));
  }
  static __device__ inline int index(Key key) {
    const uint64_t u = __builtin_bit_cast(uint64_t, key);
    const int low = (int)(u & kIndexMask);
    return !there(key) ? -1 : (int64_t)u < 0 ? low : kIndexMask - low;
  }
  static __device__ inline bool there(Key key) { return key > -0.9 * kLargest; }
  static __device__ inline double value(Key key) {
    return __builtin_bit_cast(double, __builtin_bit_cast(uint64_t, key) & ~(uint64_t)kIndexMask);
  }
  static __device__ inline Key larger(Key a, Key b) { return fmax(a, b); }
  static __device__ inline Key smaller(Key a, Key b) { return fmin(a, b); }
};

// 16-bit logits: their bits, mapped so that they order as whole numbers, over the index.
struct Narrow {
  typedef uint32_t Key;
  static __device__ inline Key none() { return 0u; }
  // `bits`: of the logit, fp16 or bf16; `infinity`: of +inf in that type
  static __device__ inline Key of_bits(uint32_t bits, uint32_t infinity, int e) {
    if (bits == 0x8000u) bits = 0;  // -0 counts as 0
    const uint32_t order = bits & 0x8000u ? ~bits & 0xFFFFu : bits | 0x8000u;
    const bool candidate = (bits & 0x7FFFu) <= infinity && bits != (0x8000u | infinity);  // neither NaN nor -inf
    return candidate ? order << 16 | (uint32_t)(kIndexMask - e) : 0u;
  }
  static __device__ inline int index(Key key) { return key == 0 ? -1 : kIndexMask - (int)(key & 0xFFFFu); }
  static __device__ inline Key larger(Key a, Key b) { return max(a, b); }
  static __device__ inline Key smaller(Key a, Key b) { return min(a, b); }
};

// ---- exp and sigmoid in fp64 -------------------------------------------------
// 2^n times the Taylor series of e^r, |r| <= ln 2 / 2: 13 terms leave r^13 / 13!, at
// most 1.5 * 2^-53.
// r = x - n ln 2 with ln 2 in two parts (Cody and Waite): its first 42 bits, times
// which an n of up to 11 bits is exact, and the rest.
__device__ inline double exp_f64(double x) {
  x = fmin(fmax(x, -700.0), 700.0);
  const double n = __builtin_rint(x * 1.4426950408889634);
  double r = fma(-n, 0x1.62e42fefa38p-1, x);
  r = fma(-n, 0x1.ef35793c7673p-45, r);
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

// sigmoid(x) / e^from = e^(x - from) / (1 + e^x) of logits x and from, both below 0
// or from 0. For scores that leave fp32's range while their ratios are ordinary
// numbers: those whose sum is below kSmallSum, of which a score's own rounding in
// fp32's last steps would be more than 2^-126, and those below kSmallLogit.
// What the difference of the logits loses (half an ulp of up to 700) is put back,
// and results below 2^-126 are kept (v_exp and v_rcp give 0). What is 0 in fp64 is 0.
constexpr float kSmallLogit = -64.f, kLeastLogit = -708.f, kSmallSum = 0x1p-10f;
__device__ inline float sigmoid_over_exp(float x, float from) {
  const float d = x - from, lost = (x - d) - from, up = d < -80.f ? 0x1p64f : 1.f;
  const float e = exp_f32(d, d < -80.f ? 64.f : 0.f);
  return x >= kLeastLogit ? fmaf(e, lost, e) / ((1.f + exp_f32(x)) * up) : 0.f;
}

// ---- sorted lists in registers -------------------------------------------------
template <class W> __device__ inline void order(typename W::Key& a, typename W::Key& b) {  // a the larger
  const typename W::Key x = W::larger(a, b), y = W::smaller(a, b);
  a = x;
  b = y;
}
// Odd-even merge sort, falling.
template <class W, int N> __device__ inline void sort_falling(typename W::Key (&v)[N]) {
#pragma unroll
  for (int p = 1; p < N; p *= 2) {
#pragma unroll
    for (int k = p; k >= 1; k /= 2) {
#pragma unroll
      for (int j = k % p; j <= N - 1 - k; j += 2 * k) {
#pragma unroll
        for (int i = 0; i < k; ++i)
          if (i + j + k < N && (i + j) / (2 * p) == (i + j + k) / (2 * p)) order<W>(v[i + j], v[i + j + k]);
      }
    }
  }
}
// The K largest of two falling lists, falling: the larger of each pair of one
// list and the other reversed form a bitonic sequence.
template <class W, int K>
__device__ inline void merge_falling(typename W::Key (&list)[K], const typename W::Key (&other)[K]) {
#pragma unroll
  for (int i = 0; i < K; ++i) list[i] = W::larger(list[i], other[K - 1 - i]);
#pragma unroll
  for (int k = K / 2; k >= 1; k /= 2) {
#pragma unroll
    for (int i = 0; i < K; ++i)
      if ((i & k) == 0) order<W>(list[i], list[i + k]);
  }
}
// The K largest of N keys, falling.
template <class W, int K, int N>
__device__ inline void keep_largest(const typename W::Key (&v)[N], typename W::Key (&list)[K]) {
#pragma unroll
  for (int at = 0; at < N; at += K) {
    typename W::Key part[K];
#pragma unroll
    for (int i = 0; i < K; ++i) part[i] = at + i < N ? v[at + i < N ? at + i : 0] : W::none();
    sort_falling<W, K>(part);
    if (at == 0) {
#pragma unroll
      for (int i = 0; i < K; ++i) list[i] = part[i];
    } else {
      merge_falling<W, K>(list, part);
    }
  }
}

template <int kCtrl> __device__ inline uint32_t lane_bits(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, kCtrl, 0xF, 0xF, false);
}
template <int kCtrl, class V> __device__ inline V from_lane(V v) {
  if constexpr (sizeof(V) == 8) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    return __builtin_bit_cast(V, (uint64_t)lane_bits<kCtrl>((uint32_t)(u >> 32)) << 32 | lane_bits<kCtrl>((uint32_t)u));
  } else {
    return __builtin_bit_cast(V, lane_bits<kCtrl>(__builtin_bit_cast(uint32_t, v)));
  }
}
constexpr int kXor1 = 0xB1, kXor2 = 0x4E;           // quad permutations
constexpr int kMirror8 = 0x141, kMirror16 = 0x140;  // lane i <-> 7 - i, 15 - i

template <class W, int K, int kCtrl> __device__ inline void merge_with(typename W::Key (&list)[K]) {
  typename W::Key other[K];
#pragma unroll
  for (int i = 0; i < K; ++i) other[i] = from_lane<kCtrl>(list[i]);
  merge_falling<W, K>(list, other);
}
template <class W, int K> __device__ inline void merge_across(typename W::Key (&list)[K], int distance) {
  typename W::Key other[K];
#pragma unroll
  for (int i = 0; i < K; ++i) other[i] = __shfl_xor(list[i], distance);
  merge_falling<W, K>(list, other);
}
// Every lane of a token's `lanes` gets the K largest of all of them.
template <class W, int K> __device__ inline void merge_lanes(typename W::Key (&list)[K], int lanes) {
  if (lanes > 1) merge_with<W, K, kXor1>(list);
  if (lanes > 2) merge_with<W, K, kXor2>(list);
  if (lanes > 4) merge_with<W, K, kMirror8>(list);
  if (lanes > 8) merge_with<W, K, kMirror16>(list);
  if (lanes > 16) merge_across<W, K>(list, 16);
  if (lanes > 32) merge_across<W, K>(list, 32);
}

// op over the values of a token's `lanes` (a power of two), in all of them; in a fixed order.
template <class V, class Op> __device__ inline V across(V v, int lanes, Op op) {
  if (lanes > 1) v = op(v, from_lane<kXor1>(v));
  if (lanes > 2) v = op(v, from_lane<kXor2>(v));
  if (lanes > 4) v = op(v, from_lane<kMirror8>(v));
  if (lanes > 8) v = op(v, from_lane<kMirror16>(v));
  if (lanes > 16) v = op(v, __shfl_xor(v, 16));
  if (lanes > 32) v = op(v, __shfl_xor(v, 32));
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
  int experts, dtype, vec, bias_vec;
  int lanes, lane_bits;  // per token, and their logarithm
  int per;               // experts of a group
  int part;              // of these, a lane's where lanes share one
  int lanes_of;          // lanes that share a group (1 where a lane has whole groups)
  int inverse_of;        // 2^16 / lanes_of, rounded up
  int groups_of;         // groups that a lane has (1 where lanes share one)
  nvfp4_moe_choice how;
};

// The group that a lane has a part of: lane / lanes_of, for lanes below 64.
__device__ inline int group_of(const RouteArgs& a, int lane) { return (lane * a.inverse_of) >> 16; }

__device__ inline Share share_of(const RouteArgs& a, int lane) {
  Share s;
  if (a.how.groups == 1) {
    s.base = lane * 8;
    s.step = a.lanes * 8;
    s.end = a.experts;
  } else if (a.lanes_of > 1) {
    const int g = group_of(a, lane), at = (lane - g * a.lanes_of) * a.part;
    s.base = g * a.per + at;
    s.step = 8;
    s.end = g < a.how.groups ? g * a.per + min(a.per, at + a.part) : 0;
  } else {
    s.base = lane * a.groups_of * a.per;
    s.step = 8;
    s.end = min(a.experts, (lane + 1) * a.groups_of * a.per);
  }
  return s;
}

// A lane's logits; -inf past its share.
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

// Whether the choice goes by the logits (as 32-bit keys where they have 16 bits),
// by scores (a bias), or by scores in groups.
enum Mode { kLogits16, kLogits32, kScores, kGroups };

// How many groups precede group g of a token, by worth and then by index.
__device__ inline int rank_of(const double* worth, int groups, int g) {
  const double w = worth[g];
  int before = 0;
  for (int o = 0; o < groups; ++o) before += worth[o] > w || (worth[o] == w && o < g);
  return before;
}

__device__ inline void best_two(double v, double& one, double& two) {
  two = fmax(two, fmin(one, v));
  one = fmax(one, v);
}

// The choice by scores in fp32, as 23-bit fixed-point numbers below the token's
// largest choice value (0 for one that is 1 or more below it, and for none) over
// the index: half the instructions of the fp64 choice. In units of 2^-22 a number is off the exact
// value by 1 for the score (e^-x within (|x| + 2) 2^-24, times s (1 - s); its sum
// and reciprocal), 1 for the sum with a bias (values up to 5), 1.75 for the
// difference and its truncation; with softmax by as much for the
// score, and 11 more for the sum of up to 512 terms (a factor that all scores
// share). Returns whether the list is that of the exact values: no two
// neighbours in it and no candidate next to its end are as near to each other as
// two such errors.
constexpr uint32_t kSigmoidMargin = 8, kSoftmaxMargin = 32;
template <int K, int NC>
__device__ inline bool choose_fp32(const RouteArgs& a, const Share& s, const float (&x)[NC * 8],
                                   const float (&bias)[NC * 8], float from, float inverse, uint32_t (&list)[K]) {
  const bool softmax = a.how.score == NVFP4_MOE_SOFTMAX;
  const uint32_t margin = softmax ? kSoftmaxMargin : kSigmoidMargin;
  float value[NC * 8], top = -__builtin_inff();
#pragma unroll
  for (int i = 0; i < NC * 8; ++i) {
    const float e = __builtin_amdgcn_exp2f((softmax ? x[i] - from : -x[i]) * 1.44269502f);
    value[i] = (softmax ? e * inverse : __builtin_amdgcn_rcpf(1.f + e)) + bias[i];
    value[i] = x[i] > -__builtin_inff() ? value[i] : -__builtin_inff();  // not for NaN
    top = fmaxf(top, value[i]);
  }
  top = max_across(top, a.lanes);
  bool sure = fabsf(top) <= 4.f;  // not for a token without candidates
  uint32_t v[NC * 8];
#pragma unroll
  for (int i = 0; i < NC * 8; ++i) {
    const int e = s.base + i / 8 * s.step + i % 8;
    const float fixed = fmaxf(fmaf(value[i], 0x1p22f, 0x1p22f - top * 0x1p22f), 0.f);  // 0 for NaN
    v[i] = (uint32_t)fminf(fixed, 0x1p22f) << 9 | (uint32_t)(kIndexMask - e);
  }
  keep_largest<Narrow, K, NC * 8>(v, list);
  merge_lanes<Narrow, K>(list, a.lanes);
  uint32_t last = 0;  // the last chosen
#pragma unroll
  for (int i = 0; i < K; ++i) {
    last = i < a.how.topk ? list[i] : last;
    if (i + 1 < K) sure &= i + 1 >= a.how.topk || list[i] - list[i + 1 < K ? i + 1 : i] > (margin + 1) << 9;
  }
  sure &= last >> 9 > margin;
  const uint32_t near = last - (margin << 9);
  int count = 0;
#pragma unroll
  for (int i = 0; i < NC * 8; ++i) count += (v[i] | kIndexMask) >= near;
  return sure && sum_across(count, a.lanes) == a.how.topk;
}

// The same in fp64, for any values.
template <int K, int NC, bool kGrouped>
__device__ inline void choose_fp64(const RouteArgs& a, const Share& s, int lane, const float (&x)[NC * 8],
                                   const float (&bias)[NC * 8], float top, double (*s_best)[2], double* s_worth,
                                   double (&list)[K]) {
  double v[NC * 8];
  if (a.how.score == NVFP4_MOE_SOFTMAX) {
    const double from = top == -__builtin_inff() ? 0.0 : (double)fminf(top, 3.4e38f);
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < NC * 8; ++i) {
      v[i] = exp_f64((double)x[i] - from);
      sum += x[i] > -__builtin_inff() ? v[i] : 0.0;
    }
    sum = sum_across(sum, a.lanes);
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
    v[i] = x[i] > -__builtin_inff() ? Wide::make(v[i] + bias[i], e) : Wide::none();  // none for a NaN logit, too
  }
  if constexpr (kGrouped) {
    auto worth = [&](double one, double two) {
      return a.how.group_best == 1 || !Wide::there(two) ? Wide::value(one) : Wide::value(one) + Wide::value(two);
    };
    if (a.groups_of == 1) {
      double one = Wide::none(), two = Wide::none();
#pragma unroll
      for (int i = 0; i < NC * 8; ++i) best_two(v[i], one, two);
      s_best[threadIdx.x][0] = one;
      s_best[threadIdx.x][1] = two;
      wave_sync();
      for (int g = lane; g < a.how.groups; g += a.lanes) {
        one = two = Wide::none();
        for (int q = 0; q < a.lanes_of; ++q) {
          const int at = threadIdx.x - lane + g * a.lanes_of + q;
          two = fmax(s_best[at][1], two);
          best_two(s_best[at][0], one, two);
        }
        s_worth[g] = worth(one, two);
      }
    } else {
      for (int q = 0; q < a.groups_of; ++q) {
        const int g = lane * a.groups_of + q;
        if (g >= a.how.groups) break;
        double one = Wide::none(), two = Wide::none();
#pragma unroll
        for (int i = 0; i < NC * 8; ++i) best_two(i / a.per == q ? v[i] : Wide::none(), one, two);
        s_worth[g] = worth(one, two);
      }
    }
    wave_sync();
    for (int q = 0; q < a.groups_of; ++q) {
      const int g = a.groups_of == 1 ? group_of(a, lane) : lane * a.groups_of + q;
      const int before = g < a.how.groups ? rank_of(s_worth, a.how.groups, g) : a.how.groups;
#pragma unroll
      for (int i = 0; i < NC * 8; ++i)
        if ((a.groups_of == 1 || i / a.per == q) && before >= a.how.topk_groups) v[i] = Wide::none();
    }
  }
  keep_largest<Wide, K, NC * 8>(v, list);
  merge_lanes<Wide, K>(list, a.lanes);
}

// Routing. A token's logits are read once into the registers of `lanes` lanes;
// each lane keeps the K largest keys of its experts in a sorted list (sort K,
// merge them in: two instructions for each comparison), and the lanes' lists are
// merged in log2(lanes) steps. Bound by these instructions, not by the logits.
// A choice by scores is made in fp32, and again in fp64 by a wave that holds a
// token for which fp32 cannot tell (one token of 256 experts in 600); in groups in fp64 at once, as
// with sums of groups to compare in both the registers no longer suffice, and the
// few waves that go twice end last. In fp32 first - in fp64, sigmoid scores of bf16
// logits with bias: 40000 x 64 9.1 - 9.6 us, 131072 x 64 19.2 - 21.8, 24000 x 128 10.4 -
// 11.5; in 4 of 8 groups, when both were tried, 131072 x 256 92 - 89, in 2 of 4 groups
// 65536 x 128 33 - 29. By logits: 65537 x 64 in fp32, softmax, 6 chosen, 10.2 us (17 MB
// read and 3 written, 4 us of a copy's rate; a launch is 3). 16384 tokens of 256
// grouped scores 14.9 us, one token 5.5 us.
template <int K, int NC, Mode kMode>
__global__ void __launch_bounds__(kThreads, NC > 2 ? 2 : 4) nvfp4_moe_route_kernel(RouteArgs a) {
  extern __shared__ double s_worth[];  // [tokens][groups]
  __shared__ double s_best[kMode == kGroups ? kThreads : 1][2];
  constexpr bool kByScore = kMode == kScores || kMode == kGroups;
  const int lane = threadIdx.x & (a.lanes - 1), local = threadIdx.x >> a.lane_bits;
  const int64_t mine = (int64_t)blockIdx.x * (kThreads >> a.lane_bits) + local;
  const int64_t token = mine < a.tokens ? mine : a.tokens - 1;  // lanes past the end repeat the last token
  const Share s = share_of(a, lane);
  float x[NC * 8];
  load_logits<NC>(a.logits, a.dtype, token * a.row_stride, s, a.vec, x);

  bool bad = false;
  float top = -__builtin_inff();
#pragma unroll
  for (int i = 0; i < NC * 8; ++i) {
    bad |= x[i] != x[i];
    top = fmaxf(top, x[i]);  // passes over NaN
  }
  bad |= a.how.score == NVFP4_MOE_SOFTMAX && top == __builtin_inff();
  const uint64_t lanes_mask = (a.lanes == 64 ? ~0ull : (1ull << a.lanes) - 1) << (threadIdx.x & 63 & ~(a.lanes - 1));
  bad = (__ballot(bad) & lanes_mask) != 0;

  const bool softmax = a.how.score == NVFP4_MOE_SOFTMAX;
  float total = 1.f;  // of e^(x - top) over all experts
  if (softmax && (kByScore || !a.how.renormalize)) {
    top = max_across(top, a.lanes);
    const float from = top == -__builtin_inff() ? 0.f : top;
    total = 0.f;
    // the plain product's error, |x - top| 2^-24 of a term, is small where the term is not
#pragma unroll
    for (int i = 0; i < NC * 8; ++i) {
      const float e = __builtin_amdgcn_exp2f((x[i] - from) * 1.44269502f);
      total += kByScore && x[i] != x[i] ? 0.f : e;
    }
    total = sum_across(total, a.lanes);
  }
  int chosen_ids[K];
  if constexpr (kByScore) {
    float bias[NC * 8];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int e = s.base + c * s.step;
      float b[8] = {};
      if (a.bias != nullptr) {
        if (e + 8 <= s.end) {
          load8<F32>(a.bias, e, a.bias_vec && e % 4 == 0, b);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) b[j] = e + j < s.end ? a.bias[e + j] : 0.f;
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) bias[c * 8 + j] = b[j];
    }
    bool sure = false;
    if constexpr (kMode == kScores) {
      uint32_t list[K];
      sure = choose_fp32<K, NC>(a, s, x, bias, top, 1.f / total, list);
#pragma unroll
      for (int i = 0; i < K; ++i) chosen_ids[i] = kIndexMask - (int)(list[i] & kIndexMask);
    }
    if (__any(!sure)) {
      double exact[K];  // a wave's own parts of s_best and s_worth
      choose_fp64<K, NC, kMode == kGroups>(a, s, lane, x, bias, top, s_best, s_worth + local * a.how.groups, exact);
#pragma unroll
      for (int i = 0; i < K; ++i) chosen_ids[i] = Wide::index(exact[i]);
    }
  } else {
    typedef typename std::conditional<kMode == kLogits16, Narrow, Wide>::type W;
    typename W::Key v[NC * 8], list[K];
    const bool half = a.dtype == NVFP4_MOE_F16;
#pragma unroll
    for (int i = 0; i < NC * 8; ++i) {
      const int e = s.base + i / 8 * s.step + i % 8;
      if constexpr (kMode == kLogits16) {
        const uint32_t bits = half ? (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)x[i]) : __builtin_bit_cast(uint32_t, x[i]) >> 16;
        v[i] = Narrow::of_bits(bits, half ? 0x7C00u : 0x7F80u, e);
      } else {
        v[i] = Wide::of_logit(x[i], e);
      }
    }
    keep_largest<W, K, NC * 8>(v, list);
    merge_lanes<W, K>(list, a.lanes);
#pragma unroll
    for (int i = 0; i < K; ++i) chosen_ids[i] = W::index(list[i]);
  }

  // slot j belongs to lane j % lanes: slots of a lane are K / lanes at most
  constexpr int kLaneSlots = K > kLeastLanes ? K / kLeastLanes : 1;
  int ids[kLaneSlots];
  float chosen[kLaneSlots], w[kLaneSlots], largest = -__builtin_inff();
#pragma unroll
  for (int q = 0; q < kLaneSlots; ++q) {
    const int slot = q * a.lanes + lane;
    ids[q] = -1;
#pragma unroll
    for (int i = 0; i < K; ++i) ids[q] = i == slot && i < a.how.topk ? chosen_ids[i] : ids[q];
    chosen[q] = ids[q] >= 0 ? load_logit(a.logits, a.dtype, token * a.row_stride + ids[q]) : -__builtin_inff();
    largest = fmaxf(largest, chosen[q]);
  }
  const int share = a.lanes < K ? a.lanes : K;  // lanes that have a slot
  if (softmax && a.how.renormalize) top = max_across(largest, share);
  const float from = top == -__builtin_inff() ? 0.f : top;
  float sum = 0.f;
  bool small = false;
#pragma unroll
  for (int q = 0; q < kLaneSlots; ++q) {
    if (softmax) w[q] = exp_f32(chosen[q] - from);
    else w[q] = ids[q] >= 0 ? __builtin_amdgcn_rcpf(1.f + exp_f32(-chosen[q])) : 0.f;
    sum += w[q];
    small |= ids[q] >= 0 && chosen[q] < kSmallLogit;
  }
  if (a.how.renormalize) total = sum_across(sum, share);
  else if (!softmax) total = 1.f;
  if (!softmax && __any(small || (lane < share && total < kSmallSum))) {
    largest = max_across(largest, share);
    const float over = total < kSmallSum ? largest : 0.f;
    sum = 0.f;
#pragma unroll
    for (int q = 0; q < kLaneSlots; ++q) {
      if (over < 0.f || chosen[q] < kSmallLogit) w[q] = ids[q] >= 0 ? sigmoid_over_exp(chosen[q], over) : 0.f;
      sum += w[q];
    }
    if (a.how.renormalize) total = sum_across(sum, share);
  }
  const float factor = total == 0.f ? a.how.scale : a.how.scale / total;
#pragma unroll
  for (int q = 0; q < kLaneSlots; ++q) {
    const int slot = q * a.lanes + lane;
    float y = w[q] * factor;
    if (ids[q] < 0) y = 0.f;
    else if (bad) y = __builtin_nanf("");
    if (slot < a.how.topk && mine < a.tokens) {
      a.ids[token * a.how.topk + slot] = ids[q];
      a.weights[token * a.how.topk + slot] = y;
    }
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
//   sigmoid: dx = ds s (1 - s) (renormalised, dx = q (dp - sum dp q) (1 - s))
// q is formed from scores over a common factor, so that S may lie below fp32's range.
// Only the softmax that is not renormalised has a gradient for experts that
// were not chosen, and only it reads the whole row. The chosen experts' values
// go to their lanes through shared memory; every lane then writes its share.
// Bound by memory and the launch: 65537 x 64 fp32 logits of a dense softmax,
// 34 MB and 3 MB of ids and dw, 10.4 us (7.5 us at a copy's rate, 3 a launch).
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
    const float over = a.how.renormalize ? fminf(max_across(chosen, a.lanes), 0.f) : 0.f;
    if (id < 0) p = 0.f;
    else if (over < 0.f || chosen < kSmallLogit) p = sigmoid_over_exp(chosen, over);
    else p = 1.f / (1.f + exp_f32(-chosen));
  }
  float q = p;
  if (a.how.renormalize) {
    const float total = sum_across(p, a.lanes);
    q = total == 0.f ? 0.f : p / total;
  }
  const float dot = sum_across(id >= 0 ? dw * q : 0.f, a.lanes);
  float give;  // to the chosen expert's lane
  if (dense) give = dw;
  else if (softmax) give = q * (dw - dot);
  else give = q * (dw - (a.how.renormalize ? dot : 0.f)) * (1.f / (1.f + exp_f32(chosen)));
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

// Lanes of a token: as few as hold its logits in registers, as the lanes' merged lists are the same work in each of
// them, but more where there are too few tokens to fill the chip (15000 tokens x
// 256 fp32 logits: 8.0 us with 8 lanes, 8.8 with 16; 16384 x 256 scores, which take
// longer before the merges: 14.7 us with 8, 12.4 with 16, in groups 16.3 and 16.0).
int widen(int lanes, int64_t tokens, int experts, int64_t enough) {
  while (lanes < 64 && tokens * lanes < enough && lanes * 8 < experts) lanes *= 2;
  return lanes;
}

// Chunks of eight experts of the fullest lane, and how groups lie on lanes.
int lay_out(RouteArgs& a) {
  const int groups = a.how.groups;
  a.per = a.experts / groups;
  a.lanes_of = a.groups_of = 1;
  a.lane_bits = __builtin_ctz(a.lanes);
  if (groups == 1) return ceil_div(ceil_div(a.experts, 8), a.lanes);
  if (a.lanes >= groups) a.lanes_of = a.lanes / groups;
  else a.groups_of = ceil_div(groups, a.lanes);
  a.inverse_of = ceil_div(1 << 16, a.lanes_of);
  a.part = ceil_div(a.per, a.lanes_of);
  return ceil_div(a.groups_of > 1 ? a.groups_of * a.per : a.part, 8);
}

template <int K, int NC> void launch_route(const RouteArgs& a, Mode mode, int64_t blocks, hipStream_t stream) {
  const dim3 grid((unsigned)blocks);
  const size_t shared = a.how.groups > 1 ? sizeof(double) * (kThreads / a.lanes) * a.how.groups : 0;
  if (mode == kGroups) nvfp4_moe_route_kernel<K, NC, kGroups><<<grid, kThreads, shared, stream>>>(a);
  else if (mode == kScores) nvfp4_moe_route_kernel<K, NC, kScores><<<grid, kThreads, 0, stream>>>(a);
  else if (mode == kLogits16) nvfp4_moe_route_kernel<K, NC, kLogits16><<<grid, kThreads, 0, stream>>>(a);
  else nvfp4_moe_route_kernel<K, NC, kLogits32><<<grid, kThreads, 0, stream>>>(a);
}
template <int K> void launch_route(const RouteArgs& a, int chunks, Mode mode, int64_t blocks, hipStream_t stream) {
  if (chunks <= 1) launch_route<K, 1>(a, mode, blocks, stream);
  else if (chunks <= 2) launch_route<K, 2>(a, mode, blocks, stream);
  else launch_route<K, 4>(a, mode, blocks, stream);
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
  const Mode mode = choice->groups > 1         ? kGroups
                    : bias != nullptr          ? kScores
                    : dtype == NVFP4_MOE_F32   ? kLogits32
                                               : kLogits16;
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
  a.bias_vec = aligned(bias, 16);
  a.how = *choice;
  a.lanes = widen(kLeastLanes, tokens, experts, mode == kScores || mode == kGroups ? kScoreLanes : kLogitLanes);
  int chunks = lay_out(a);
  while (chunks > 4) {
    a.lanes *= 2;
    chunks = lay_out(a);
  }
  const int64_t blocks = ceil_div64(tokens, kThreads / a.lanes);
  const hipStream_t st = (hipStream_t)stream;
  if (choice->topk <= 2) launch_route<2>(a, chunks, mode, blocks, st);
  else if (choice->topk <= 4) launch_route<4>(a, chunks, mode, blocks, st);
  else if (choice->topk <= 8) launch_route<8>(a, chunks, mode, blocks, st);
  else launch_route<16>(a, chunks, mode, blocks, st);
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
  a.lanes = widen(at_least_pow2(choice->topk < 4 ? 4 : choice->topk), tokens, experts, kScoreLanes);
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
