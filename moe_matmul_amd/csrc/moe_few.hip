// The experts' products of a few tokens: NVFP4 weights, fp16 or bf16
// activations, one output row per (token, expert) slot.
#include "moe_common.h"

namespace moe {
namespace {

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr int kStep = 256;    // K-elements of a step: 128 bytes of a weight row, and four scale atoms
constexpr int kStepBytes = kStep / 2;
constexpr int kPieces = kStepBytes / 16;  // 16-byte pieces of a row's step
// Steps of weights in flight, in registers, and waves of a SIMD that the registers
// have to allow. 13 tokens of 2 of 8 experts of 7168 x 2048: 21.5 us, with three steps
// 27.8, with four waves 24.1; one token of 8 experts of 4096 x 7168 with SwiGLU 28.2 us,
// 33.8 and 35.4, as registers spill; with two waves the same.
constexpr int kDepth = 2;
constexpr int kMinWaves = 3;
constexpr int kHold = 4;      // pieces of x that a thread has under way
constexpr int kMaxRows = 16;  // slots of a pass: rows of the matrix instruction
constexpr int kStageElements = 16384;  // of x in shared memory, at most (32 KB)
// Waves that share the columns before any share K, three for four SIMDs: sharing K
// gains where the columns leave SIMDs idle only. Alone - shared: a token of 2 experts
// of 2048 x 7168 25.5 - 12.8 us; 4 tokens of 8 of 32 experts of 4096 x 7168 with SwiGLU
// 67 - 92.
constexpr int kEnoughWaves = 768;
constexpr int kPad = 8;       // elements after a staged row: rows start in different banks

// a stage of shared memory holds kDepth steps of every row of a pass, at least
static_assert(kMaxRows * kDepth * kStep <= kStageElements, "a stage would hold no whole round of steps");

struct FewArgs {
  const void* x;
  int64_t x_stride;
  const int32_t* ids;
  const uint8_t *b, *sfb;
  const float* alpha;
  void* out;
  int slots, topk, per_slot, experts, n, k, x_vec, out_dtype;
  int columns;    // of out
  int tiles;      // workgroups of an expert
  int by_expert;  // a workgroup's expert is its number (else that of the slot of that number)
  int stage;      // elements of x that fit in shared memory, with their padding
  int rows;       // slots of a pass: 1, 2, 4, 8 or 16
  int slots_at;   // where the slots of the expert lie after that, in bytes
  int k_waves;    // waves that share K; the others of a workgroup have other columns
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

// What a lane reads for one K-step of U runs of 16 weight rows: codes as they
// lie in memory, eight lanes to the 128 bytes of a row, and the word of four
// scales of the row and atom that the lane multiplies.
template <int U> struct Weights {
  u32x4 codes[U][2];
  uint32_t scales[U];
};

// N words at an address that is a multiple of their size.
template <int N> __device__ inline void load_words(const uint8_t* p, uint32_t* w) {
  typedef uint32_t words __attribute__((ext_vector_type(N)));
  const words v = *(const words*)p;
#pragma unroll
  for (int i = 0; i < N; ++i) w[i] = v[i];
}

// A wave's weight rows: H halves of SUB runs of 16 rows. The runs of a half are
// 32 rows apart, where the tiled layout has their scales side by side. The
// matrix instruction wants a run's row lane % 16 in a lane, K-elements lane / 16
// * 64 .. + 63 of the step; loaded like that, a quarter of a wave would touch 16
// cache lines for 16 bytes each, and the address unit, not memory, would set
// the pace (16 x 16-byte pieces a load: 3.3 TB/s). So rows are loaded whole
// lines at a time and change lanes through shared memory.
template <int H, int SUB> struct Operand {
  static constexpr int U = H * SUB;
  const uint8_t *codes, *scales;       // of the expert
  uint32_t row_at[U][2], scale_at[U];  // bytes: of the rows that this lane loads (lane / 8 and + 8), and multiplies
  int last_code, last_atom, lane;
  bool apart;  // a half does not begin at a multiple of 32 * SUB rows: its runs' scales do not lie together

  // Lanes past the end of K read its end; x is 0 there, and scales() makes their scales 0.
  __device__ inline Weights<U> load(int step) const {
    Weights<U> w;
    const uint32_t code = min(step * kStepBytes + lane % 8 * 16, last_code);
    const uint32_t scale = min(step * (kStep / kAtomK) + lane / 16, last_atom) * kAtomBytes;
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < 2; ++i) w.codes[u][i] = __builtin_nontemporal_load((const u32x4*)(codes + (row_at[u][i] + code)));
    if (H == 1 || !apart) {
#pragma unroll
      for (int h = 0; h < H; ++h) load_words<SUB>(scales + (scale_at[h * SUB] + scale), w.scales + h * SUB);
    } else {
#pragma unroll
      for (int u = 0; u < U; ++u) load_words<1>(scales + (scale_at[u] + scale), w.scales + u);
    }
    return w;
  }
  // Which bytes of a scale word lie within K.
  __device__ inline uint32_t scale_mask(int step) const {
    const int atom = step * (kStep / kAtomK) + lane / 16;
    return atom < last_atom ? ~0u : atom > last_atom ? 0u : last_code % (kAtomK / 2) == 0 ? 0xFFFFu : ~0u;
  }
};

// Where the 16-byte piece p of row r of a run's step lies in shared memory, in
// pieces: without bank conflicts for the eight lanes that write a row, and for
// 16 lanes that read a piece of 16 rows.
__device__ inline int piece_at(int r, int p) { return r * kPieces + (p ^ (r / 2 & 7)); }

__device__ inline void store_any(void* out, int dtype, int64_t at, float y) {
  if (dtype == NVFP4_MOE_F32) store1<F32>(out, at, y);
  else if (dtype == NVFP4_MOE_F16) store1<F16>(out, at, y);
  else store1<BF16>(out, at, y);
}

// The largest of a wave's values, in lane 63: along rows of 16 lanes, then from row to row.
template <int kCtrl> __device__ inline uint32_t max_from(uint32_t v) {
  return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, kCtrl, 0xF, 0xF, true));
}
__device__ inline uint32_t wave_max(uint32_t v) {
  v = max_from<0x111>(v);  // row_shr 1, 2, 4, 8
  v = max_from<0x112>(v);
  v = max_from<0x114>(v);
  v = max_from<0x118>(v);
  v = max_from<0x142>(v);  // row_bcast 15, 31
  return max_from<0x143>(v);
}

// The exponent field of the power of two that brings a row's largest element to
// 2^14 .. 2^15, within what fp32 has.
__device__ inline int scale_up(uint32_t top) { return min(max(127 + 14 + 127 - (int)(top >> 7), 1), 253); }

// A workgroup computes some columns of all slots of one expert, `rows` of them
// at a time; its four waves split the columns, K, or both. The workgroups find
// the expert's slots themselves, so no order of slots has to be made before.
// Bound by reading the weights: a token of 8 experts of 4096 x 7168 with SwiGLU, 132
// MB in 28 us, 4.7 TB/s (reads alone reach 6.4 here); 13 tokens of 2 of 8 experts of
// 7168 x 2048, 66 MB in 21.5 us, 3.1 TB/s, of which about 7 pass before the first weights
// arrive and after the last.
//
// Weights go from memory to registers, kDepth steps ahead, the first of them
// before anything else is read but the expert's number. x is staged in shared
// memory as f16. bf16 rows are scaled by a power of two for that, which
// brings the largest element of a row so far to 2^14 .. 2^15: elements down to
// 2^-32 of it keep their eight bits, and what smaller ones lose is below 2^-39
// of it, far under the rounding of the fp32 sums. Sums over waves are formed in
// wave order.
template <class X, int U, bool SWIGLU>
__global__ void __launch_bounds__(kThreads, kMinWaves) nvfp4_few_tokens_kernel(FewArgs a) {
  constexpr int H = SWIGLU ? 2 : 1, SUB = U / H;
  constexpr bool kScaled = X::kId == NVFP4_MOE_BF16;
  extern __shared__ __attribute__((aligned(16))) uint8_t s_shared[];
  __shared__ u32x4 s_codes[kWaves][U * 16 * kPieces];
  __shared__ uint32_t s_top[kMaxRows];  // a row's largest element so far, without its sign

  uint16_t* s_slots = (uint16_t*)(s_shared + a.slots_at);

  const int which = blockIdx.x / a.tiles, tile = blockIdx.x % a.tiles;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x & 63;
  const int k_wave = wave % a.k_waves;
  // a wave's tile number -> its first weight row: runs of 16 rows, 32 apart, within 32 * SUB rows
  const int wave_tile = tile * (kWaves / a.k_waves) + wave / a.k_waves;
  const int row0 = wave_tile / 2 * (32 * SUB) + wave_tile % 2 * 16;
  const int expert = a.by_expert ? which : a.ids[which];

  // a slot without an expert gives zeros: from its own workgroups, or from those of expert 0
  auto zero_slot = [&](int slot) {
    for (int i = lane; i < 16 * SUB; i += 64) {
      const int col = row0 + i / 16 * 32 + i % 16;
      if (k_wave == 0 && col < a.columns) store_any(a.out, a.out_dtype, (int64_t)slot * a.columns + col, 0.f);
    }
  };
  if (!a.by_expert && (unsigned)expert >= (unsigned)a.experts) {
    zero_slot(which);
    return;
  }

  // Weights: rows past n are read from the last row, computed and dropped.
  Operand<H, SUB> operand;
  operand.last_code = a.k / 2 - 16;
  operand.last_atom = ceil_div(a.k, kAtomK) - 1;
  operand.lane = lane;
  operand.apart = a.n / H % (32 * SUB) != 0;
  const int kt = ceil_div(a.k, kAtomK);
  operand.codes = a.b + (int64_t)expert * a.n * (a.k / 2);
  operand.scales = a.sfb + (int64_t)expert * ceil_div(a.n, kAtomRows) * kt * kAtomBytes;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int run = (row0 < a.columns ? row0 : 0) + u % SUB * 32 + u / SUB * (a.n / H);
#pragma unroll
    for (int i = 0; i < 2; ++i) operand.row_at[u][i] = (uint32_t)min(run + i * 8 + lane / 8, a.n - 1) * (a.k / 2);
    // scales of runs that lie together are padded to whole atoms: their rows may pass n
    const int row = H == 2 && operand.apart ? min(run + lane % 16, a.n - 1) : run + lane % 16;
    operand.scale_at[u] = (uint32_t)(row / kAtomRows * kt) * kAtomBytes + atom_row(row % kAtomRows);
  }
  // This wave's K-steps, and where its weights go ahead.
  const int steps = ceil_div(a.k, kStep);
  const int first = steps * k_wave / a.k_waves, last = steps * (k_wave + 1) / a.k_waves;
  Weights<U> ahead[kDepth];
  auto prefetch = [&] {
#pragma unroll
    for (int d = 0; d < kDepth; ++d) ahead[d] = operand.load(min(first + d, steps - 1));
  };
  if (steps > 0) prefetch();

  // the slots of this expert, in order
  int count = 0, first_slot = -1;
  for (int i0 = 0; i0 < a.slots; i0 += 64) {
    const int id = i0 + lane < a.slots ? a.ids[i0 + lane] : a.experts;
    const bool mine = id == expert;
    const uint64_t all = __ballot(mine);
    if (a.by_expert && which == 0) {
      uint64_t none = __ballot(i0 + lane < a.slots && (unsigned)id >= (unsigned)a.experts);
      for (; none != 0; none &= none - 1) zero_slot(i0 + __builtin_ctzll(none));
    }
    if (all == 0) continue;
    if (first_slot < 0) {
      first_slot = i0 + __builtin_ctzll(all);
      // only the first slot's workgroups do the work
      if (!a.by_expert && first_slot != which) return;
    }
    if (wave == 0 && mine) s_slots[count + __popcll(all & ((1ull << lane) - 1))] = (uint16_t)(i0 + lane);
    count += __popcll(all);
  }
  if (count == 0) return;
  if (threadIdx.x < kMaxRows) s_top[threadIdx.x] = 0;
  __syncthreads();

  // A stage holds the next `part` steps of every K-wave, for the slots of a pass.
  int row_space = 1;
  while (row_space < a.rows && row_space < count) row_space *= 2;
  const int most = ceil_div(ceil_div(steps, a.k_waves), kDepth) * kDepth;
  const int part = min(a.stage / (row_space * a.k_waves * kStep) / kDepth * kDepth, most);
  const int pieces = a.k_waves * part * (kStep / 8), stage_row = pieces * 8 + kPad;
  const int row_waves = row_space < kWaves ? kWaves / row_space : 1, turns = ceil_div(pieces, 64 * row_waves);
  _Float16* stage = (_Float16*)s_shared;

  for (int from = 0; from < count; from += a.rows) {
    const int rows = min(a.rows, count - from);
    f32x4 sum[U];
    int up[4] = {253, 253, 253, 253};  // scales of this lane's rows so far
#pragma unroll
    for (int u = 0; u < U; ++u) sum[u] = f32x4{0.f, 0.f, 0.f, 0.f};
    int step = first;
    for (int done = 0; done < most; done += part) {
      // x, in pieces of 8 elements. A row's pieces go to `row_waves` waves, 64 at a time. bf16 rows are gone through
      // twice: for their largest elements, and to be scaled. In between, a thread's pieces stay in registers if they
      // are kHold or fewer; else they are read again (from a cache).
      const int part_pieces = part * (kStep / 8);
      const bool held = turns * ceil_div(rows * row_waves, kWaves) <= kHold;
      u32x4 v[kHold];
      auto each_piece = [&](bool load, auto&& use) {  // use(row, piece, its elements)
        int row = wave / row_waves, turn = 0;
        while (row < rows) {
          const int row_before = row, turn_before = turn;
          if (load) {
#pragma unroll
            for (int h = 0; h < kHold; ++h) {
              const int i = (turn * row_waves + wave % row_waves) * 64 + lane;
              const int w = (i >= part_pieces) + (i >= 2 * part_pieces) + (i >= 3 * part_pieces);  // its K-wave
              const int k = (steps * w / a.k_waves + done) * kStep + (i - w * part_pieces) * 8;
              v[h] = u32x4{0u, 0u, 0u, 0u};
              if (row < rows && i < pieces && k < a.k) {
                const int slot = s_slots[from + row];
                const uint16_t* x = (const uint16_t*)a.x + (int64_t)(a.per_slot ? slot : slot / a.topk) * a.x_stride;
                if (a.x_vec) {
                  v[h] = *(const u32x4*)(x + k);
                } else {
#pragma unroll
                  for (int j = 0; j < 4; ++j) v[h][j] = x[k + 2 * j] | (uint32_t)x[k + 2 * j + 1] << 16;
                }
              }
              if (++turn == turns) {
                turn = 0;
                row += kWaves / row_waves;
              }
            }
          }
          row = row_before;
          turn = turn_before;
#pragma unroll
          for (int h = 0; h < kHold; ++h) {
            if (row < rows) use(row, (turn * row_waves + wave % row_waves) * 64 + lane, v[h]);
            if (++turn == turns) {
              turn = 0;
              row += kWaves / row_waves;
            }
          }
        }
      };
      if constexpr (kScaled) {
        each_piece(true, [&](int r, int, u32x4 v) {
          uint32_t top = 0;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t low = v[j] & 0x7FFFu, high = v[j] >> 16 & 0x7FFFu;  // infinities and NaNs do not count
            top = max(top, max(low < 0x7F80u ? low : 0u, high < 0x7F80u ? high : 0u));
          }
          top = wave_max(top);
          if (lane == 63) atomicMax(&s_top[r], top);
        });
        __syncthreads();
      }
      each_piece(!kScaled || !held, [&](int r, int i, u32x4 v) {
        if (i >= pieces) return;
        if constexpr (kScaled) {
          const float scale = __builtin_bit_cast(float, (uint32_t)scale_up(s_top[r]) << 23);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float lo, hi;
            unpack2<BF16>(v[j], lo, hi);
            v[j] = pack2<F16>(lo * scale, hi * scale);
          }
        }
        *(u32x4*)(stage + r * stage_row + i * 8) = v;
      });
      __syncthreads();
      if constexpr (kScaled) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = lane / 16 * 4 + i;
          if (r >= rows) continue;
          const int now = scale_up(s_top[r]);
          if (done > 0) {
            const float down = __builtin_bit_cast(float, (uint32_t)max(127 + now - up[i], 0) << 23);
#pragma unroll
            for (int u = 0; u < U; ++u) sum[u][i] *= down;
          }
          up[i] = now;
        }
      }
      // rows from `rows` on hold whatever was there: their sums are dropped
      const _Float16* mine = stage + (lane % 16 & (row_space - 1)) * stage_row + (k_wave * part - first - done) * kStep +
                             lane / 16 * 64;
      u32x4* turn = s_codes[wave];
      auto multiply = [&](int at, const Weights<U>& w) {
        const uint32_t mask = operand.scale_mask(at);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int i = 0; i < 2; ++i) turn[u * 16 * kPieces + piece_at(i * 8 + lane / 8, lane % 8)] = w.codes[u][i];
        wave_sync();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          f16x8 xs[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) xs[j] = *(const f16x8*)(mine + at * kStep + h * 32 + j * 8);
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const u32x4 c = turn[u * 16 * kPieces + piece_at(lane % 16, lane / 16 * 2 + h)];
            const f16x2 sc = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((w.scales[u] & mask) >> (h * 16), 1.f, false);
#pragma unroll
            for (int j = 0; j < 4; ++j)
              sum[u] = __builtin_amdgcn_mfma_f32_16x16x32_f16(xs[j], dequant8(c[j], j < 2 ? sc.x : sc.y), sum[u], 0, 0, 0);
          }
        }
        wave_sync();
      };
      // whole rounds always load (the last step again at the end), so that what is waited for is known when compiled
      const int end = min(first + done + part, last);
      for (; step + kDepth <= end; step += kDepth) {
#pragma unroll
        for (int d = 0; d < kDepth; ++d) {
          multiply(step + d, ahead[d]);
          ahead[d] = operand.load(min(step + d + kDepth, last - 1));
        }
      }
      if (end == last) {
#pragma unroll
        for (int d = 0; d + 1 < kDepth; ++d)
          if (step + d < last) multiply(step + d, ahead[d]);
        step = last;
      }
      __syncthreads();  // the stage has been read
    }
    if (from + a.rows < count && steps > 0) prefetch();
    if (kScaled && threadIdx.x < kMaxRows) s_top[threadIdx.x] = 0;  // read again after the next barrier only

    // lane has rows lane / 16 * 4 + i of column lane % 16 of its runs
    // the factor's mantissa and exponent: a sum's own power of two is taken out together with the latter, so that what is
    // between them does not leave fp32's range where the result does not
    const float alpha = a.alpha == nullptr ? 1.f : a.alpha[expert], alpha_part = __builtin_amdgcn_frexp_mantf(alpha);
    const int alpha_exp = __builtin_amdgcn_frexp_expf(alpha);
    float* sums = (float*)s_shared;  // [wave][run][row][column]
    if (a.k_waves > 1) {
      if (k_wave > 0) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (lane / 16 * 4 + i < rows) sums[((wave * U + u) * kMaxRows + lane / 16 * 4 + i) * 16 + lane % 16] = sum[u][i];
      }
      __syncthreads();
    }
    if (k_wave == 0) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = lane / 16 * 4 + i;
        if (r >= rows) continue;
        float y[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          y[u] = sum[u][i];
          for (int w = 1; w < a.k_waves; ++w) y[u] += sums[(((wave + w) * U + u) * kMaxRows + r) * 16 + lane % 16];
          y[u] = kScaled ? __builtin_ldexpf(y[u] * alpha_part, alpha_exp + 127 - up[i]) : y[u] * alpha;
        }
#pragma unroll
        for (int u = 0; u < SUB; ++u) {
          const int col = row0 + u * 32 + lane % 16;
          float out = y[u];
          if constexpr (SWIGLU) out = out / (1.f + exp_f32(-out)) * y[SUB + u];
          if (col < a.columns) store_any(a.out, a.out_dtype, (int64_t)s_slots[from + r] * a.columns + col, out);
        }
      }
    }
    __syncthreads();
  }
}

template <class X, int U, bool SWIGLU> int launch_few(FewArgs& a, int64_t tokens, hipStream_t st) {
  constexpr int SUB = SWIGLU ? U / 2 : U;
  const int wave_tiles = ceil_div(a.columns, 32 * SUB) * 2, used = a.by_expert ? a.experts : a.slots;
  const int steps = ceil_div(a.k, kStep);
  // a token's experts differ as a rule: then an expert has at most a slot of each token (else it takes more passes)
  a.rows = 1;
  while (a.rows < kMaxRows && a.rows < tokens) a.rows *= 2;
  // K is split over the waves until there are enough waves to fill the chip, or a wave's steps get few
  a.k_waves = 1;
  while (a.k_waves < kWaves && (int64_t)used * wave_tiles * a.k_waves < kEnoughWaves && steps >= 4 * a.k_waves &&
         2 * a.rows * a.k_waves * kDepth * kStep <= kStageElements)
    a.k_waves *= 2;
  a.tiles = ceil_div(wave_tiles, kWaves / a.k_waves);
  a.stage = a.rows * a.k_waves * ceil_div(ceil_div(steps, a.k_waves), kDepth) * kDepth * kStep;
  if (a.stage > kStageElements) a.stage = kStageElements;
  const size_t sums = (size_t)kWaves * U * kMaxRows * 16 * 4, staged = ((size_t)a.stage + kMaxRows * kPad) * 2;
  a.slots_at = (int)(a.k_waves > 1 && sums > staged ? sums : staged);
  const size_t shared = a.slots_at + ((size_t)a.slots * 2 + 15) / 16 * 16;
  nvfp4_few_tokens_kernel<X, U, SWIGLU><<<(unsigned)(used * a.tiles), kThreads, shared, st>>>(a);
  return launched();
}
template <class X> int launch_few(FewArgs& a, int64_t tokens, int swiglu, hipStream_t st) {
  return swiglu ? launch_few<X, 2, true>(a, tokens, st) : launch_few<X, 2, false>(a, tokens, st);
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
  if ((int64_t)n * (k / 2) >= (int64_t)1 << 31) return NVFP4_ERR_INVALID;
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
  a.by_expert = a.experts < a.slots;
  return dtype == NVFP4_MOE_F16 ? launch_few<F16>(a, tokens, swiglu, (hipStream_t)stream)
                                : launch_few<BF16>(a, tokens, swiglu, (hipStream_t)stream);
}
