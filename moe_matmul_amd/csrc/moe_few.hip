// The experts' products of a few tokens: NVFP4 weights, fp16 or bf16
// activations, one output row per (token, expert) slot.
#include "moe_common.h"

namespace moe {
namespace {

constexpr int kWaves = 8;
constexpr int kThreads = 64 * kWaves;
constexpr int kStep = 128;       // K-elements of a step: 32 (16 bytes of codes) for each of a wave's four lane groups
constexpr int kStageItems = 4;   // 16-byte pieces of x that a lane stages at a time

struct FewArgs {
  const void* x;
  int64_t x_stride;
  const int32_t* ids;
  const uint8_t *b, *sfb;
  const float* alpha;
  void* out;
  int slots, topk, per_slot, experts, n, k, x_vec, out_dtype;
  int columns;  // of out
  int tiles;    // workgroups of a slot
};

// Eight codes of one dword times their scale, as f16: both factors and the
// product (at most 2 + 4 significant bits, 2^-10 .. 2688) are exact in f16.
__device__ inline f16x8 dequant8(uint32_t w, _Float16 s) {
  const f16x2 ss = {s, s};
  const f16x2 p0 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.f, 0) * ss;
  const f16x2 p1 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.f, 1) * ss;
  const f16x2 p2 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.f, 2) * ss;
  const f16x2 p3 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.f, 3) * ss;
  return f16x8{p0.x, p0.y, p1.x, p1.y, p2.x, p2.y, p3.x, p3.y};
}

// What a lane reads for one K-step: 32 codes of each of its weight rows, and the
// scale words of those rows.
template <int SUB> struct Weights {
  u32x4 codes[SUB];
  uint32_t scales[SUB];
};

// A lane's weight rows of a tile: SUB of them, 32 apart, so that (from a row
// that is a multiple of 32 * SUB, plus 0 .. 31) their scales lie side by side in
// the tiled layout.
template <int SUB> struct Operand {
  const uint8_t* codes[SUB];   // at this lane's K offset
  const uint8_t* scales[SUB];  // the words of this lane's first atom

  __device__ inline void at(const FewArgs& a, int expert, int row0, int lane) {
    const int group = lane / 16, kt = ceil_div(a.k, kAtomK);
    const int64_t atom0 = (int64_t)expert * ceil_div(a.n, kAtomRows);
#pragma unroll
    for (int s = 0; s < SUB; ++s) {
      const int row = min(row0 + 32 * s + lane % 16, a.n - 1);  // columns past n are computed and dropped
      codes[s] = a.b + ((int64_t)expert * a.n + row) * (a.k / 2) + group * 16;
      scales[s] = a.sfb + ((atom0 + row / kAtomRows) * kt + group / 2) * kAtomBytes + atom_row(row % kAtomRows);
    }
  }
  __device__ inline Weights<SUB> load(const FewArgs& a, int step, int lane) const {
    Weights<SUB> w;
    const bool there = step * kStep + lane / 16 * 32 < a.k;
    const int64_t code = (int64_t)step * (kStep / 2), scale = (int64_t)step * (kStep / kAtomK) * kAtomBytes;
#pragma unroll
    for (int s = 0; s < SUB; ++s) {
      w.codes[s] = there ? *(const u32x4*)(codes[s] + code) : u32x4{0u, 0u, 0u, 0u};
      w.scales[s] = there ? *(const uint32_t*)(scales[s] + scale) : 0u;
    }
    return w;
  }
};

// A workgroup computes a tile of weight rows (SWIGLU: the tile's rows of both
// halves) for all slots of one expert, MT of them at a time; its eight waves
// split K. The first slot of an expert does the work of all of them, the others
// leave at once, so no order of slots has to be made before. Weights go from
// memory to registers, two steps ahead; a wave's part of x goes through its own
// shared memory, as f16. bf16 rows are scaled by a power of two for that, which
// brings the largest of a wave's part of a row to 2^14 .. 2^15: all elements down
// to 2^-32 of it keep their eight bits, and what smaller ones lose is below
// 2^-39 of it, far under the rounding of the fp32 sums. Waves' sums are joined
// in shared memory, in wave order.
template <class X, int SUB, bool SWIGLU, int MT>
__global__ void __launch_bounds__(kThreads) nvfp4_few_tokens_kernel(FewArgs a) {
  constexpr int kStageK = kStageItems * 64 * 8 / MT;           // K-elements of a stage
  constexpr int kStageRow = kStageK + 8;                       // padded: rows start in different banks
  constexpr int kHalves = SWIGLU ? 2 : 1;
  constexpr int kStageBytes = kWaves * MT * kStageRow * 2;
  constexpr int kTileN = 16 * SUB;
  constexpr int kSumBytes = kWaves * MT * kTileN * 4;
  __shared__ __attribute__((aligned(16))) uint8_t s_shared[kStageBytes > kSumBytes ? kStageBytes : kSumBytes];
  __shared__ uint16_t s_slots[NVFP4_MOE_MAX_FEW_SLOTS];
  __shared__ float s_unscale[kWaves][MT];
  __shared__ int s_count;

  const int slot = blockIdx.x / a.tiles, tile = blockIdx.x % a.tiles;
  const int wave = threadIdx.x / 64, lane = threadIdx.x & 63;
  // tile -> its first weight row: runs of 16 rows that are 32 apart, within 32 * SUB rows
  const int row0 = tile / 2 * (32 * SUB) + tile % 2 * 16;
  const int expert = a.ids[slot];
  if ((unsigned)expert >= (unsigned)a.experts) {
    for (int i = threadIdx.x; i < kTileN; i += kThreads) {
      const int col = row0 + i / 16 * 32 + i % 16;
      if (col >= a.columns) continue;
      const int64_t at = (int64_t)slot * a.columns + col;
      if (a.out_dtype == NVFP4_MOE_F32) store1<F32>(a.out, at, 0.f);
      else store1<F16>(a.out, at, 0.f);  // zero has the same bits in bf16
    }
    return;
  }
  // the slots of this expert, in order
  if (wave == 0) {
    int count = 0;
    for (int i0 = 0; i0 < a.slots; i0 += 64) {
      const bool mine = i0 + lane < a.slots && a.ids[i0 + lane] == expert;
      const uint64_t all = __ballot(mine);
      if (mine) s_slots[count + __popcll(all & ((1ull << lane) - 1))] = (uint16_t)(i0 + lane);
      count += __popcll(all);
    }
    if (lane == 0) s_count = count;
  }
  __syncthreads();
  const int count = s_count;
  if (s_slots[0] != slot) return;

  Operand<SUB> operand[kHalves];
#pragma unroll
  for (int h = 0; h < kHalves; ++h) operand[h].at(a, expert, row0 + h * (a.n / 2), lane);
  const int steps = ceil_div(a.k, kStep), first = steps * wave / kWaves, last = steps * (wave + 1) / kWaves;
  _Float16* stage = (_Float16*)s_shared + wave * MT * kStageRow;

  for (int from = 0; from < count; from += MT) {
    const int rows = min(MT, count - from);
    // this lane's pieces of a stage: piece p is 8 elements, kStageK / 8 pieces to a row
    int64_t base[kStageItems];
    int piece_k[kStageItems];
#pragma unroll
    for (int i = 0; i < kStageItems; ++i) {
      const int p = i * 64 + lane, r = p / (kStageK / 8);
      const int s = s_slots[from + min(r, rows - 1)];
      base[i] = (int64_t)(a.per_slot ? s : s / a.topk) * a.x_stride;
      piece_k[i] = p % (kStageK / 8) * 8;
    }
    auto load_piece = [&](int i, int k0) {
      const int k = k0 + piece_k[i];
      u32x4 v = {0u, 0u, 0u, 0u};
      if (k < a.k) {
        const uint16_t* p = (const uint16_t*)a.x + base[i] + k;
        if (a.x_vec) {
          v = *(const u32x4*)p;
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) v[j] = p[2 * j] | (uint32_t)p[2 * j + 1] << 16;
        }
      }
      return v;
    };
    const int k_end = last * kStep;
    float scale[kStageItems];
    if constexpr (X::kId == NVFP4_MOE_BF16) {
      uint32_t top[kStageItems] = {};
      for (int k0 = first * kStep; k0 < k_end; k0 += kStageK) {
#pragma unroll
        for (int i = 0; i < kStageItems; ++i) {
          const u32x4 v = k0 + piece_k[i] < k_end ? load_piece(i, k0) : u32x4{0u, 0u, 0u, 0u};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t low = v[j] & 0x7FFFu, high = v[j] >> 16 & 0x7FFFu;
            top[i] = max(top[i], max(low < 0x7F80u ? low : 0u, high < 0x7F80u ? high : 0u));
          }
        }
      }
#pragma unroll
      for (int i = 0; i < kStageItems; ++i) {
        for (int d = 1; d < kStageK / 8 && d < 64; d *= 2) top[i] = max(top[i], (uint32_t)__shfl_xor((int)top[i], d));
        // 2^(14 - exponent of the largest), within what fp32 has
        const int up = min(max(127 + 14 + 127 - (int)(top[i] >> 7), 1), 253);
        scale[i] = __builtin_bit_cast(float, (uint32_t)up << 23);
        const int p = i * 64 + lane;
        if (p % (kStageK / 8) == 0) s_unscale[wave][p / (kStageK / 8)] = __builtin_bit_cast(float, (uint32_t)(254 - up) << 23);
      }
    }

    f32x4 sum[kHalves][SUB];
#pragma unroll
    for (int h = 0; h < kHalves; ++h)
#pragma unroll
      for (int s = 0; s < SUB; ++s) sum[h][s] = f32x4{0.f, 0.f, 0.f, 0.f};
    Weights<SUB> next[kHalves];
#pragma unroll
    for (int h = 0; h < kHalves; ++h) next[h] = operand[h].load(a, first, lane);

    for (int k0 = first * kStep; k0 < k_end; k0 += kStageK) {
      // stage x as f16; the wave's reads of the stage before are done (they were waited for by their MFMAs)
#pragma unroll
      for (int i = 0; i < kStageItems; ++i) {
        u32x4 v = load_piece(i, k0);
        if constexpr (X::kId == NVFP4_MOE_BF16) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float lo, hi;
            unpack2<BF16>(v[j], lo, hi);
            v[j] = pack2<F16>(lo * scale[i], hi * scale[i]);
          }
        }
        *(u32x4*)(stage + (i * 64 + lane) / (kStageK / 8) * kStageRow + piece_k[i]) = v;
      }
      wave_sync();
      const int here = min(kStageK, k_end - k0) / kStep;
      for (int t = 0; t < here; ++t) {
        Weights<SUB> w[kHalves];
        const int step = k0 / kStep + t;
#pragma unroll
        for (int h = 0; h < kHalves; ++h) {
          w[h] = next[h];
          if (step + 1 < last) next[h] = operand[h].load(a, step + 1, lane);
        }
        f16x8 xs[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          xs[j] = *(const f16x8*)(stage + lane % 16 % MT * kStageRow + t * kStep + lane / 16 * 32 + j * 8);
#pragma unroll
        for (int h = 0; h < kHalves; ++h)
#pragma unroll
          for (int s = 0; s < SUB; ++s) {
            const f16x2 sc = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w[h].scales[s] >> (lane / 16 % 2 * 16), 1.f, false);
#pragma unroll
            for (int j = 0; j < 4; ++j)
              sum[h][s] = __builtin_amdgcn_mfma_f32_16x16x32_f16(xs[j], dequant8(w[h].codes[s][j], j < 2 ? sc.x : sc.y),
                                                               sum[h][s], 0, 0, 0);
          }
      }
      wave_sync();
    }

    // join the waves: lane has rows lane / 16 * 4 + i of column lane % 16
    float total[kHalves][(MT * kTileN + kThreads - 1) / kThreads];
    float* sums = (float*)s_shared;  // [wave][row][column]
#pragma unroll
    for (int h = 0; h < kHalves; ++h) {
      __syncthreads();
#pragma unroll
      for (int s = 0; s < SUB; ++s)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = lane / 16 * 4 + i;
          if (r < MT) {
            const float u = X::kId == NVFP4_MOE_BF16 ? s_unscale[wave][r] : 1.f;
            sums[(wave * MT + r) * kTileN + s * 16 + lane % 16] = sum[h][s][i] * u;
          }
        }
      __syncthreads();
#pragma unroll
      for (int o = 0; o * kThreads < MT * kTileN; ++o) {
        const int at = o * kThreads + threadIdx.x;
        float t = 0.f;
        if (at < MT * kTileN)
          for (int w = 0; w < kWaves; ++w) t += sums[w * MT * kTileN + at];
        total[h][o] = t;
      }
    }
    const float alpha = a.alpha == nullptr ? 1.f : a.alpha[expert];
#pragma unroll
    for (int o = 0; o * kThreads < MT * kTileN; ++o) {
      const int at = o * kThreads + threadIdx.x, r = at / kTileN, c = at % kTileN;
      const int col = row0 + c / 16 * 32 + c % 16;
      if (at >= MT * kTileN || r >= rows || col >= a.columns) continue;
      float y = total[0][o] * alpha;
      if constexpr (SWIGLU) y = y / (1.f + exp_f32(-y)) * (total[kHalves - 1][o] * alpha);
      const int64_t to = (int64_t)s_slots[from + r] * a.columns + col;
      if (a.out_dtype == NVFP4_MOE_F32) store1<F32>(a.out, to, y);
      else if (a.out_dtype == NVFP4_MOE_F16) store1<F16>(a.out, to, y);
      else store1<BF16>(a.out, to, y);
    }
    __syncthreads();
  }
}

template <class X, int SUB, bool SWIGLU> void launch_few(const FewArgs& a, int64_t tokens, hipStream_t st) {
  const unsigned grid = (unsigned)a.slots * a.tiles;
  if (tokens <= 4) nvfp4_few_tokens_kernel<X, SUB, SWIGLU, 4><<<grid, kThreads, 0, st>>>(a);
  else nvfp4_few_tokens_kernel<X, SUB, SWIGLU, 16><<<grid, kThreads, 0, st>>>(a);
}
template <class X, bool SWIGLU> void launch_few(FewArgs& a, int64_t tokens, hipStream_t st) {
  // wide tiles where they still fill the chip
  const int sub = (int64_t)a.slots * ceil_div(a.columns, 64) >= 256 ? 4 : (int64_t)a.slots * ceil_div(a.columns, 32) >= 256 ? 2 : 1;
  a.tiles = ceil_div(a.columns, 32 * sub) * 2;
  if (sub == 4) launch_few<X, 4, SWIGLU>(a, tokens, st);
  else if (sub == 2) launch_few<X, 2, SWIGLU>(a, tokens, st);
  else launch_few<X, 1, SWIGLU>(a, tokens, st);
}
template <class X> void launch_few(FewArgs& a, int64_t tokens, int swiglu, hipStream_t st) {
  if (swiglu) launch_few<X, true>(a, tokens, st);
  else launch_few<X, false>(a, tokens, st);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" int nvfp4_moe_few_tokens(const void* x, int dtype, int64_t x_stride, int per_slot, const int32_t* ids,
                                    int64_t tokens, int topk, int experts, int n, int k, const void* b,
                                    const void* sfb, const float* alpha, int swiglu, void* out, int out_dtype,
                                    void* stream) {
  if (dtype != NVFP4_MOE_F16 && dtype != NVFP4_MOE_BF16) return NVFP4_ERR_INVALID;
  if (!known_type(out_dtype)) return NVFP4_ERR_INVALID;
  if (tokens < 0 || topk < 1 || topk > NVFP4_MOE_MAX_TOPK || tokens > NVFP4_MOE_MAX_FEW_SLOTS ||
      tokens * topk > NVFP4_MOE_MAX_FEW_SLOTS)
    return NVFP4_ERR_INVALID;
  if (experts < 1 || experts > NVFP4_MOE_MAX_EXPERTS) return NVFP4_ERR_INVALID;
  if (n < 0 || n % (swiglu ? 16 : 8) || n > 1 << 20 || k < 0 || k % 32 || k > 1 << 22) return NVFP4_ERR_INVALID;
  if (x_stride < k || x_stride > (int64_t)1 << 40) return NVFP4_ERR_INVALID;
  const bool work = tokens > 0 && n > 0;
  if (work && (ids == nullptr || out == nullptr)) return NVFP4_ERR_INVALID;
  if (work && k > 0 && (x == nullptr || b == nullptr || sfb == nullptr)) return NVFP4_ERR_INVALID;
  if (!aligned(x, 2) || !aligned(ids, 4) || !aligned(b, 16) || !aligned(sfb, 16) || !aligned(alpha, 4) ||
      !aligned(out, element_bytes(out_dtype)))
    return NVFP4_ERR_MISALIGNED;
  if (!work) return NVFP4_OK;
  FewArgs a = {};
  a.x = x;
  a.x_stride = x_stride;
  a.ids = ids;
  a.b = (const uint8_t*)b;
  a.sfb = (const uint8_t*)sfb;
  a.alpha = alpha;
  a.out = out;
  a.slots = (int)(tokens * topk);
  a.topk = topk;
  a.per_slot = per_slot != 0;
  a.experts = experts;
  a.n = n;
  a.k = k;
  a.x_vec = wide_rows(x, dtype, x_stride);
  a.out_dtype = out_dtype;
  a.columns = swiglu ? n / 2 : n;
  if (dtype == NVFP4_MOE_F16) launch_few<F16>(a, tokens, swiglu, (hipStream_t)stream);
  else launch_few<BF16>(a, tokens, swiglu, (hipStream_t)stream);
  return launched();
}
