// Entry points of the products of nvfp4_ffn.h: argument checks, the choice of tiles
// and of parts of k, and the kernel that adds the parts.
#include <math.h>

#include "ffn_gemm.h"

namespace moe {
thread_local int t_last_hip_error = 0;
}

namespace ffn {

int run_few(const Product& p, int dtype, bool gated, hipStream_t stream);
int run_forward(Product& p, const Tiling& t, int dtype, bool gated, hipStream_t stream);
int run_dx(Product& p, const Tiling& t, int dtype, hipStream_t stream);
int run_dw(Product& p, const Tiling& t, int dtype, hipStream_t stream);

constexpr int kMaxSide = 1 << 20;          // n and k
constexpr int64_t kMaxStride = 1 << 22;    // of the products' rows: see reachable
constexpr int64_t kMaxBytes = 0x7FFFFFFF;  // of what one resource reaches

int compute_units() {
  static thread_local int units[16];  // by device
  int device = 0;
  if (hipGetDevice(&device) != hipSuccess || device < 0 || device >= 16) return 256;
  if (!units[device]) {
    int n = 0;
    units[device] = hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, device) == hipSuccess && n > 0 ? n : 256;
  }
  return units[device];
}

int plan_rows(const nvfp4_ffn_plan* plan, int64_t rows, bool gathered, Rows* out) {
  *out = Rows{nullptr, nullptr, 1, 1, rows, rows, 0};
  if (!plan) return NVFP4_OK;
  if (plan->experts < 1 || plan->experts > NVFP4_MOE_MAX_EXPERTS || !plan->offsets) return NVFP4_ERR_INVALID;
  if (!aligned(plan->offsets, 4)) return NVFP4_ERR_MISALIGNED;
  out->offsets = plan->offsets;
  out->experts = plan->experts;
  if (!gathered) return NVFP4_OK;
  if (plan->topk < 1 || plan->topk > NVFP4_MOE_MAX_TOPK || rows % plan->topk || !plan->row_slots) return NVFP4_ERR_INVALID;
  if (!aligned(plan->row_slots, 4)) return NVFP4_ERR_MISALIGNED;
  out->row_slots = plan->row_slots;
  out->topk = plan->topk;
  out->sources = rows / plan->topk;
  return NVFP4_OK;
}

// The tiles and parts of k that take least by a model of the kernels' times in microseconds: a round of tiles over the
// compute units (two small ones to a unit) has a fixed part and one for every 64 k, fitted to products that fill whole
// rounds (4096 x 4096 x 2048 and 8192: 256 x 256 59 and 205, 256 x 128 64 and 241, 128 x 128 66 and 259; 5120 x 4096 and
// 2048 columns: 320 x 256 73 and 278, 320 x 128 43 and 142; 64 x 4096 x 7168 in 4 and 8 parts of 64 x 128: 14 and 12).
// The tallest tiles are for rows that leave a part of a round in all others: 5120 x 4096 x 2048 89 at best without
// them, 73 with; by experts, two tiles of 320 hold the 512 rows that they have on the average and the some more that
// half of them have (eight of 2048 x 4096, 3900 rows: gradient of rows 97 without them, 76 with). A tile that is not
// filled takes kEmpty of its time for its loads. Parts are written and read at some 4 TB/s, in a launch of their own;
// by experts they cost more, as rows that are not there have parts too. Against the best tile that there is the choice
// loses up to a tenth, in small products a fifth.
static Tiling choose_tiling(int64_t rows, int cols, int64_t k, int experts, bool over_k, int units, double* time) {
  static const double kFixed[kShapes] = {7, 8, 9, 4, 10, 10}, kStage[kShapes] = {0.97, 0.92, 1.6, 0.7, 1.03, 2.2};
  static const double kAlone[kShapes] = {0.64, 1, 1, 0.57, 1, 1}, kEmpty = 0.4;
  const double e = over_k ? experts : 1;
  const double stages = (double)ceil_div64(k > 0 ? k : 1, 64);
  Tiling best{0, 1};
  double least = 1e30;
  // the weights' (or rows') own bytes
  const double streamed = 5 + (double)cols * k * 2 * (over_k ? e : experts < rows ? experts : rows) / 5e6;
  for (int shape = 0; shape < (over_k ? kShapesOverK : kShapes); ++shape) {
    const int bm = tile_rows(shape), bn = tile_cols(shape);
    // rows of tiles, and how much of their height is used
    double high, fill;
    if (!over_k && experts > 1) {
      // experts have about as many rows (half of them more: what a standard deviation more needs)
      const double some = (double)(experts < rows ? experts : rows), each = rows / some, of_each = ceil((each + sqrt(each)) / bm);
      high = of_each * some;
      fill = ceil(each / of_each / 32) * 32 / bm;
    } else {
      const double all = ceil((double)rows / bm), even = even_rows((uint32_t)rows, bm), last = (rows - (all - 1) * even) / even;
      high = all - 1 + (last > 0.4 ? last : 0.4);
      fill = even / bm;
    }
    const double stage = kStage[shape] * (kEmpty + (1 - kEmpty) * (fill < 1 ? fill : 1));
    const double latency = !over_k && experts > 1 ? 0.5 : 0;  // a stage of weights that no other tile has read: from memory
    const double tiles = high * ceil_div(cols, bn) * e;
    // (of more than the largest tiles can cover, launch_product tells)
    if (shape != 2 && ((double)rows / bm + experts + 1) * ceil_div(cols, bn) * e + 8 * kXcds > kMostTiles) continue;
    for (int splits = 1; splits <= 16; splits += splits < 4 ? 1 : splits < 8 ? 2 : 4) {
      if (splits > 1 && stages / splits < 4) break;
      const double all = tiles * splits, room = shape != 0 && shape != 3 ? units : 2.0 * units;
      const double whole = floor(all / room), rest = all - whole * room;
      const double part = stages / splits;
      double t = whole * (kFixed[shape] + part * fmax(stage, latency));
      if (rest > 0.01) {
        // units that are alone on the memory and the power are faster: a stage of 160 tiles of 256 x 256 takes 1.07; two
        // small tiles of a unit share it until there are fewer than units
        const double r = rest / units;
        const double alone = r > 1 ? 1 : kAlone[shape] * (room > units ? 1 : bn == 128 ? 0.66 + 0.34 * r : r > 0.5 ? 0.2 + 0.8 * r : 0.6);
        t += kFixed[shape] + part * fmax(latency, stage * alone);
      }
      t = t < streamed ? streamed + 0.05 * t : 1.05 * t;  // (where the weights' bytes bound all, the least work)
      if (splits > 1) t += (experts > 1 ? 5 + splits : 4 + 0.5 * splits) + (double)rows * cols * e * 4 * 2 * splits / 4e6;
      if (t < least) {
        least = t;
        best = Tiling{shape, splits};
      }
    }
  }
  *time = least;
  return best;
}

// ---- how a product is computed ------------------------------------------------------
enum Kind { kForward = NVFP4_FFN_FORWARD, kForwardCodes = NVFP4_FFN_FORWARD_CODES, kDx = NVFP4_FFN_DX, kDw = NVFP4_FFN_DW };

// Whether the kernel of few rows is the faster one: for up to so many rows (8 rows, against 64 x 128 tiles and parts of
// k: 4096 x 7168 17.8 and 23 us, 28672 x 4096 53 and 70; more than 8 read the weights twice). By experts their mean
// counts, as one with more than 8 rows takes several passes: 8 experts of 2 x 1024 x 4096, 4 rows each on the average 33
// and 38, 6 rows 46 and 39. Their sum counts too, as they may all be one expert's, whose passes wait for one another: 64
// experts of 2 x 1024 x 2048, 64 rows of any experts 76 and 86, of one 43 and 19; 256 rows 117 and 114, 151 and 19; 256
// experts of 2 x 512 x 2048, 256 rows 139 and 154, 154 and 22; 1024 rows 223 and 233, 582 and 25.
constexpr int kFewRows = 8, kFewRowsOfExpert = 4, kFewRowsOfExperts = 64;
static bool few_rows(Kind kind, int64_t rows, int experts) {
  const int by_experts = kFewRowsOfExpert * experts < kFewRowsOfExperts ? kFewRowsOfExpert * experts : kFewRowsOfExperts;
  return kind == kForward && rows <= (experts > 1 ? by_experts : kFewRows);
}

// Rows row0 .. row0 + rows - 1 of the output, by few rows or by tiles.
struct Part {
  int64_t row0, rows;
  bool few;
  Tiling tiling;
};

// One part, or two: whole tiles and the rows that are left over, where those would take a round of tiles of their own.
static int choose_parts(Kind kind, int64_t rows, int cols, int64_t k, int experts, int units, Part* parts) {
  const bool over_k = kind == kDw;
  auto one = [&](int64_t row0, int64_t n, Part* part) {
    *part = Part{row0, n, few_rows(kind, n, experts), Tiling{0, 1}};
    if (part->few) return 4 + (double)cols * k * 2 / 5e6;
    double time;
    part->tiling = choose_tiling(n, cols, k, experts ? experts : 1, over_k, units, &time);
    return time;
  };
  const double whole = one(0, rows, parts);
  const int64_t left = rows % 256, main = rows - left;
  if (!experts && main && left && left <= 128) {
    Part two[2];
    if (one(0, main, two) + one(main, left, two + 1) + 6 < whole) {
      parts[0] = two[0];
      parts[1] = two[1];
      return 2;
    }
  }
  return 1;
}

static size_t parts_workspace(const Part* parts, int count, int cols, int experts_out) {
  size_t most = 0;
  for (int i = 0; i < count; ++i)
    if (!parts[i].few && parts[i].tiling.splits > 1) {
      const size_t need = (size_t)parts[i].tiling.splits * parts[i].rows * experts_out * cols * 4;
      if (need > most) most = need;
    }
  return most;
}

// ---- the parts of k ---------------------------------------------------------------
// A thread adds the parts of eight columns (of g and of u) in their order. Bound by
// reading them: 4 bytes an element and part.
template <class T, bool GATED, bool OVER_K> __global__ __launch_bounds__(256) void parts_kernel(const Product p, int64_t rows) {
  const int wide = (GATED ? p.ep.inner : p.n) / 8;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t row = i / wide;
  const int col = (int)(i % wide) * 8;
  bool in = row < rows;
  int e = 0;
  if (!OVER_K && in && p.rows.offsets) {
    e = expert_of(p.rows, row);
    in = e < p.rows.experts || p.rows.clear;
  }
  const bool live = OVER_K || !p.rows.offsets || e < p.rows.experts;
  float v[8] = {}, u[8] = {};
  if (in && live) {
    for (int s = 0; s < p.splits; ++s) {
      const float* from = p.partial + s * p.partial_step + row * p.n;
      float w[8];
      load8<F32>(from, col, true, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] += w[j];
      if constexpr (GATED) {
        load8<F32>(from, p.ep.inner + col, true, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) u[j] += w[j];
      }
    }
  }
  if constexpr (GATED) {
    if (p.ep.residual) {
      if (in) finish_gated_dz<T>(p.ep, row, col, v, u, *(const u32x4*)((const uint16_t*)p.ep.residual + row * p.ep.ldr + col));
      return;
    }
    if (p.ep.codes) finish_codes(p.ep, row, col, in, v, u);  // (inner % 32 == 0: a row's lanes come in fours)
    if (in) finish_gated<T>(p.ep, row, col, v, u);
  } else {
    if (!in) return;
    float b[8] = {}, r[8] = {};
    if (p.ep.bias && live) param8<T>(p.ep.bias, (int64_t)e * p.n + col, p.ep.bias_f32, true, b);
    if (p.ep.residual && live) load8<T>(p.ep.residual, row * p.ep.ldr + col, true, r);
    finish_linear<T>(p.ep, p.n, row, col, v, b, r);
  }
}

static int finish_splits(const Product& p, int dtype, bool gated, bool over_k, hipStream_t stream) {
  const int64_t rows = over_k ? p.m * p.rows.experts : p.m;
  const int64_t blocks = ceil_div64(rows * ((gated ? p.ep.inner : p.n) / 8), 256);
  if (blocks > 0x7FFFFF) return NVFP4_ERR_INVALID;
  with_type16(dtype, [&](auto type) {
    using T = decltype(type);
    const dim3 grid((unsigned)blocks);
    hipStream_t s = stream;
    if (gated) parts_kernel<T, true, false><<<grid, 256, 0, s>>>(p, rows);
    else if (over_k) parts_kernel<T, false, true><<<grid, 256, 0, s>>>(p, rows);
    else parts_kernel<T, false, false><<<grid, 256, 0, s>>>(p, rows);
    return 0;
  });
  return launched();
}

// ---- checks ---------------------------------------------------------------------------
static bool side_ok(int v) { return v >= 8 && v <= kMaxSide && v % 8 == 0; }
static bool rows_ok(int64_t rows) { return rows >= 0 && rows < ((int64_t)1 << 31); }
static bool stride_ok(int64_t stride, int width) { return stride >= width && stride < kMaxStride; }
static bool wide16(const void* p) { return aligned(p, 16); }

static int check_workspace(const void* ws, size_t have, size_t need) {
  if (!need) return NVFP4_OK;
  if (!ws || have < need) return NVFP4_ERR_WORKSPACE;
  return aligned(ws, 256) ? NVFP4_OK : NVFP4_ERR_MISALIGNED;
}

// Rows of A with k inside are reached by signed 32-bit offsets from their tile's first: the last one's 128 bytes of a
// stage have to end within what a resource reaches. 256 rows do at any stride that is taken. At strides from 2^31 / 319
// bytes on 320 do not, and their tiles give way to those of 256 rows and the same width; the parts of k, and so the
// workspace, stay. (Gathered rows lie within that reach of their operand's first, dw has k outside.)
constexpr bool within_reach(int high, int64_t stride) { return (high - 1) * stride * 2 + 128 <= kMaxBytes; }
static_assert(within_reach(256, kMaxStride), "the tiles that others give way to");
static Tiling reachable(Tiling t, Kind kind, const Product& p) {
  const bool by_stride = kind != kDw && !p.rows.row_slots;
  if (by_stride && tile_rows(t.shape) > 256 && !within_reach(tile_rows(t.shape), p.lda)) t.shape = tile_cols(t.shape) == 256 ? 2 : 1;
  return t;
}

// Enqueues the parts of a checked product; `workspace` holds what parts_workspace says.
static int run_product(Kind kind, const Product& whole, bool gated, int dtype, void* workspace, size_t workspace_bytes, void* stream) {
  Part parts[2];
  const int e = whole.rows.experts, cols = whole.n;
  const int64_t k = kind == kDw ? whole.rows.rows / e : whole.k;
  const int count = choose_parts(kind, whole.m, cols, k, whole.rows.offsets ? e : 0, compute_units(), parts);
  if (const int rc = check_workspace(workspace, workspace_bytes, parts_workspace(parts, count, cols, kind == kDw ? e : 1))) return rc;
  for (int i = 0; i < count; ++i) {
    const Part& part = parts[i];
    Product p = whole;
    if (count > 1) {  // dense
      const int64_t r = part.row0;
      p.m = part.rows;
      auto skip = [](auto& at, int64_t bytes) {
        if (at) at = (std::decay_t<decltype(at)>)((uintptr_t)at + bytes);
      };
      skip(p.a, kind == kDw ? r * 2 : r * p.lda * 2);
      skip(p.ep.y, r * p.ep.ldy * (p.ep.y_f32 ? 4 : 2));
      skip(p.ep.z, r * p.n * 2);
      skip(p.ep.residual, r * p.ep.ldr * 2);
      skip(p.ep.kept, r * p.n * 2);
      skip(p.ep.codes, r * p.n);
      skip(p.ep.scales, r * p.n / 32);
      if (kind != kDw) p.rows.rows = p.rows.sources = part.rows;
    }
    p.partial = (float*)workspace;
    p.partial_step = p.m * (kind == kDw ? e : 1) * cols;
    int rc;
    hipStream_t s = (hipStream_t)stream;
    const Tiling tiling = reachable(part.tiling, kind, p);
    if (part.few) rc = run_few(p, dtype, gated, s);
    else if (kind == kDx) rc = run_dx(p, tiling, dtype, s);
    else if (kind == kDw) rc = run_dw(p, tiling, dtype, s);
    else rc = run_forward(p, tiling, dtype, gated, s);
    if (!rc && !part.few && part.tiling.splits > 1) rc = finish_splits(p, dtype, gated, kind == kDw, s);
    if (rc) return rc;
  }
  return NVFP4_OK;
}

static size_t product_workspace(Kind kind, int64_t rows, int cols, int64_t k, int experts) {
  Part parts[2];
  const int count = choose_parts(kind, rows, cols, k, experts, compute_units(), parts);
  return parts_workspace(parts, count, cols, kind == kDw && experts ? experts : 1);
}

}  // namespace ffn

using namespace ffn;

extern "C" {

int nvfp4_ffn_last_hip_error(void) { return t_last_hip_error; }

size_t nvfp4_ffn_product_workspace_bytes(int64_t rows, int n, int k, int experts) {
  if (rows < 1 || !rows_ok(rows) || !side_ok(n) || !side_ok(k) || experts > NVFP4_MOE_MAX_EXPERTS) return 0;
  const int e = experts < 1 ? 0 : experts;
  size_t most = 0;
  for (const Kind kind : {kForward, kForwardCodes, kDx}) {
    const size_t need = product_workspace(kind, rows, n, k, e);
    if (need > most) most = need;
  }
  return most;
}

size_t nvfp4_ffn_dw_workspace_bytes(int64_t rows, int n, int k, int experts) {
  if (rows < 1 || !rows_ok(rows) || !side_ok(n) || !side_ok(k) || experts > NVFP4_MOE_MAX_EXPERTS) return 0;
  return product_workspace(kDw, n, k, experts < 1 ? rows : rows / experts, experts < 1 ? 0 : experts);
}

int nvfp4_ffn_product_parts(int kind, int64_t rows, int n, int k, int experts, int32_t* out) {
  if (kind < kForward || kind > kDw || rows < 1 || !rows_ok(rows) || !side_ok(n) || !side_ok(k) || experts < 0 ||
      experts > NVFP4_MOE_MAX_EXPERTS || !out)
    return 0;
  Part parts[2];
  const int units = compute_units();
  const int count = kind == kDw   ? choose_parts(kDw, n, k, experts ? rows / experts : rows, experts, units, parts)
                    : kind == kDx ? choose_parts(kDx, rows, k, n, experts, units, parts)
                                  : choose_parts((Kind)kind, rows, n, k, experts, units, parts);
  for (int i = 0; i < count; ++i) {
    const int shape = parts[i].tiling.shape;
    out[4 * i] = (int32_t)parts[i].rows;
    out[4 * i + 1] = parts[i].few ? 0 : tile_rows(shape);
    out[4 * i + 2] = parts[i].few ? 0 : tile_cols(shape);
    out[4 * i + 3] = parts[i].few ? 1 : parts[i].tiling.splits;
  }
  return count;
}

int nvfp4_ffn_linear(const void* x, int64_t x_stride, const void* w, const void* bias, int bias_f32, int act,
                     const void* residual, int64_t residual_stride, void* z, void* y, int dtype, int64_t rows, int n,
                     int k, const nvfp4_ffn_plan* plan, int clear, void* workspace, size_t workspace_bytes, void* stream) {
  if (!type16(dtype) || !known_activation(act) || !rows_ok(rows) || !side_ok(n) || !side_ok(k)) return NVFP4_ERR_INVALID;
  Product p{};
  if (const int rc = plan_rows(plan, rows, false, &p.rows)) return rc;
  if (rows == 0) return NVFP4_OK;
  if (!x || !w || !y || !stride_ok(x_stride, k) || (residual && residual_stride < n) || (int64_t)n * k * 2 > kMaxBytes)
    return NVFP4_ERR_INVALID;
  if (!wide16(x) || !wide16(w) || !wide16(y) || !wide16(bias) || !wide16(z) || !wide16(residual) || x_stride % 8 ||
      (residual && residual_stride % 8))
    return NVFP4_ERR_MISALIGNED;
  p.a = x; p.b = w; p.lda = x_stride; p.ldb = k; p.m = rows; p.n = n; p.k = k; p.b_step = (int64_t)n * k;
  p.rows.clear = clear != 0;
  p.ep.y = y; p.ep.ldy = n; p.ep.bias = bias; p.ep.bias_f32 = bias_f32; p.ep.act = act;
  p.ep.residual = residual; p.ep.ldr = residual_stride; p.ep.z = z;
  return run_product(kForward, p, false, dtype, workspace, workspace_bytes, stream);
}

int nvfp4_ffn_gated(const void* x, int64_t x_stride, const void* w, int act, void* h, void* kept, void* codes,
                    void* scales, int dtype, int64_t rows, int inner, int k, const nvfp4_ffn_plan* plan, int clear,
                    void* workspace, size_t workspace_bytes, void* stream) {
  if (!type16(dtype) || !known_activation(act) || act == NVFP4_FFN_NONE || !rows_ok(rows) || !side_ok(inner) ||
      !side_ok(k) || 2 * inner > kMaxSide || !codes != !scales || (codes && inner % kBlock8))
    return NVFP4_ERR_INVALID;
  Product p{};
  if (const int rc = plan_rows(plan, rows, plan != nullptr, &p.rows)) return rc;
  if (rows == 0) return NVFP4_OK;
  if (!x || !w || !h || !stride_ok(x_stride, k) || (int64_t)2 * inner * k * 2 > kMaxBytes) return NVFP4_ERR_INVALID;
  if (plan && p.rows.sources * x_stride * 2 > kMaxBytes) return NVFP4_ERR_INVALID;
  if (!wide16(x) || !wide16(w) || !wide16(h) || !wide16(kept) || !aligned(codes, 8) || x_stride % 8) return NVFP4_ERR_MISALIGNED;
  p.a = x; p.b = w; p.lda = x_stride; p.ldb = k; p.m = rows; p.n = 2 * inner; p.k = k; p.b_step = (int64_t)2 * inner * k;
  p.rows.clear = clear != 0;
  p.ep.y = h; p.ep.ldy = inner; p.ep.act = act; p.ep.inner = inner; p.ep.kept = kept;
  p.ep.codes = (uint8_t*)codes; p.ep.scales = (uint8_t*)scales;
  return run_product(codes ? kForwardCodes : kForward, p, true, dtype, workspace, workspace_bytes, stream);
}

int nvfp4_ffn_gated_again(const void* dh, int64_t dh_stride, const void* x, int64_t x_stride, const void* w, int act,
                          void* dz, int dtype, int64_t rows, int inner, int k, const nvfp4_ffn_plan* plan,
                          void* workspace, size_t workspace_bytes, void* stream) {
  if (!type16(dtype) || !known_activation(act) || act == NVFP4_FFN_NONE || !rows_ok(rows) || !side_ok(inner) ||
      !side_ok(k) || 2 * inner > kMaxSide)
    return NVFP4_ERR_INVALID;
  Product p{};
  if (const int rc = plan_rows(plan, rows, plan != nullptr, &p.rows)) return rc;
  if (rows == 0) return NVFP4_OK;
  if (!dh || !x || !w || !dz || dh_stride < inner || !stride_ok(x_stride, k) || (int64_t)2 * inner * k * 2 > kMaxBytes) return NVFP4_ERR_INVALID;
  if (plan && p.rows.sources * x_stride * 2 > kMaxBytes) return NVFP4_ERR_INVALID;
  if (!wide16(dh) || !wide16(x) || !wide16(w) || !wide16(dz) || x_stride % 8 || dh_stride % 8) return NVFP4_ERR_MISALIGNED;
  p.a = x; p.b = w; p.lda = x_stride; p.ldb = k; p.m = rows; p.n = 2 * inner; p.k = k; p.b_step = (int64_t)2 * inner * k;
  p.ep.y = dz; p.ep.ldy = 2 * inner; p.ep.act = act; p.ep.inner = inner;
  p.ep.residual = dh; p.ep.ldr = dh_stride;
  return run_product(kForward, p, true, dtype, workspace, workspace_bytes, stream);
}

int nvfp4_ffn_linear_dx_ex(const void* dz, int64_t dz_stride, const void* w, void* dx, int dx_f32, int dtype, int64_t rows,
                           int n, int k, const nvfp4_ffn_plan* plan, int clear, void* workspace, size_t workspace_bytes,
                           void* stream) {
  if (!type16(dtype) || !rows_ok(rows) || !side_ok(n) || !side_ok(k)) return NVFP4_ERR_INVALID;
  Product p{};
  if (const int rc = plan_rows(plan, rows, false, &p.rows)) return rc;
  if (rows == 0) return NVFP4_OK;
  if (!dz || !w || !dx || !stride_ok(dz_stride, n) || (int64_t)n * k * 2 > kMaxBytes) return NVFP4_ERR_INVALID;
  if (!wide16(dz) || !wide16(w) || !wide16(dx) || dz_stride % 8) return NVFP4_ERR_MISALIGNED;
  // the reduction is over n, the output's columns are k
  p.a = dz; p.b = w; p.lda = dz_stride; p.ldb = k; p.m = rows; p.n = k; p.k = n; p.b_step = (int64_t)n * k;
  p.rows.clear = clear != 0;
  p.ep.y = dx; p.ep.ldy = k; p.ep.y_f32 = dx_f32;
  return run_product(kDx, p, false, dtype, workspace, workspace_bytes, stream);
}

int nvfp4_ffn_linear_dx(const void* dz, int64_t dz_stride, const void* w, void* dx, int dtype, int64_t rows, int n, int k,
                        const nvfp4_ffn_plan* plan, int clear, void* workspace, size_t workspace_bytes, void* stream) {
  return nvfp4_ffn_linear_dx_ex(dz, dz_stride, w, dx, 0, dtype, rows, n, k, plan, clear, workspace, workspace_bytes, stream);
}

int nvfp4_ffn_linear_dw(const void* dz, int64_t dz_stride, const void* x, int64_t x_stride, void* dw, int dw_f32, int dtype,
                        int64_t rows, int n, int k, const nvfp4_ffn_plan* plan, void* workspace, size_t workspace_bytes,
                        void* stream) {
  if (!type16(dtype) || !rows_ok(rows) || !side_ok(n) || !side_ok(k) || !dw) return NVFP4_ERR_INVALID;
  Product p{};
  if (const int rc = plan_rows(plan, rows, false, &p.rows)) return rc;
  if ((rows && (!dz || !x)) || (rows && (!stride_ok(dz_stride, n) || !stride_ok(x_stride, k))) || (int64_t)n * k * 2 > kMaxBytes)
    return NVFP4_ERR_INVALID;
  if (!wide16(dz) || !wide16(x) || !wide16(dw) || (rows && (dz_stride % 8 || x_stride % 8))) return NVFP4_ERR_MISALIGNED;
  p.a = dz; p.b = x; p.lda = dz_stride; p.ldb = x_stride; p.m = n; p.n = k; p.k = 0;
  p.ep.y = dw; p.ep.ldy = k; p.ep.y_f32 = dw_f32;
  return run_product(kDw, p, false, dtype, workspace, workspace_bytes, stream);
}

}  // extern "C"
