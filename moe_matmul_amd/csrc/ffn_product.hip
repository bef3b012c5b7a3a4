// Entry points of the products of nvfp4_ffn.h: argument checks, the choice of tiles
// and of parts of k, and the kernel that adds the parts.
#include <math.h>

#include "ffn_gemm.h"

namespace moe {
thread_local int t_last_hip_error = 0;
}

namespace ffn {

int run_forward(Product& p, const Tiling& t, int dtype, bool gated, hipStream_t stream);
int run_dx(Product& p, const Tiling& t, int dtype, hipStream_t stream);
int run_dw(Product& p, const Tiling& t, int dtype, hipStream_t stream);

constexpr int kMaxSide = 1 << 20;          // n and k
constexpr int64_t kMaxStride = 1 << 22;    // a tile's offsets stay below 2^31 bytes
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
// compute units (two small ones to a unit) has a fixed part and one for every 64 k, measured on products that
// fill whole rounds (4096 x 4096 x 2048 and 8192: 59 and 214, 64 and 241, 66 and 259 for 256 x 256, 256 x 128 and
// 128 x 128); a last row of tiles that is mostly empty costs about two fifths of a whole one; parts are written and
// read at some 4 TB/s, in a launch of their own.
Tiling choose_tiling(int64_t rows, int cols, int64_t k, int experts, bool over_k, int units) {
  static const double kFixed[3] = {7, 8, 9}, kStage[3] = {0.97, 0.92, 1.6}, kAlone[3] = {0.62, 0.92, 1.6};
  const double e = over_k ? experts : 1;
  const double stages = (double)ceil_div64(k > 0 ? k : 1, 64);
  Tiling best{0, 1};
  double least = 1e30;
  for (int shape = 0; shape < 3; ++shape) {
    const int bm = shape ? 256 : 128, bn = shape == 2 ? 256 : 128;
    const double tail = (double)(rows % bm) / bm;
    double high = rows / bm + (tail > 0 ? (tail > 0.4 ? tail : 0.4) : 0);
    if (!over_k && experts > 1) {
      // every expert has a last row of tiles, half full
      const double some = (double)(experts < rows ? experts : rows);
      high = (double)rows / bm + 0.4 * some;
      if (high < some) high = some;
    }
    const double tiles = high * ceil_div(cols, bn) * e;
    for (int splits = 1; splits <= 16; splits += splits < 4 ? 1 : splits < 8 ? 2 : 4) {
      if (splits > 1 && stages / splits < 4) break;
      const double all = tiles * splits, room = shape ? units : 2.0 * units;
      const double whole = floor(all / room), rest = all - whole * room;
      const double part = stages / splits;
      double t = whole * (kFixed[shape] + part * kStage[shape]);
      if (rest > 0.01) t += kFixed[shape] + part * (rest <= units ? kAlone[shape] : kStage[shape]);
      if (splits > 1) t += 4 + (double)rows * cols * e * 4 * 2 * splits / 4e6;
      if (t < least) {
        least = t;
        best = Tiling{shape, splits};
      }
    }
  }
  return best;
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

int finish_splits(const Product& p, int dtype, bool gated, bool over_k, void* stream) {
  const int64_t rows = over_k ? p.m * p.rows.experts : p.m;
  const int64_t blocks = ceil_div64(rows * ((gated ? p.ep.inner : p.n) / 8), 256);
  if (blocks > 0x7FFFFF) return NVFP4_ERR_INVALID;
  with_type16(dtype, [&](auto type) {
    using T = decltype(type);
    const dim3 grid((unsigned)blocks);
    hipStream_t s = (hipStream_t)stream;
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

static size_t workspace_of(const Tiling& t, int64_t rows, int64_t cols) {
  return t.splits > 1 ? (size_t)t.splits * rows * cols * 4 : 0;
}

static int check_workspace(const void* ws, size_t have, size_t need) {
  if (!need) return NVFP4_OK;
  if (!ws || have < need) return NVFP4_ERR_WORKSPACE;
  return aligned(ws, 256) ? NVFP4_OK : NVFP4_ERR_MISALIGNED;
}

}  // namespace ffn

using namespace ffn;

extern "C" {

int nvfp4_ffn_last_hip_error(void) { return t_last_hip_error; }

size_t nvfp4_ffn_product_workspace_bytes(int64_t rows, int n, int k, int experts) {
  if (rows < 1 || !rows_ok(rows) || !side_ok(n) || !side_ok(k) || experts > NVFP4_MOE_MAX_EXPERTS) return 0;
  return workspace_of(choose_tiling(rows, n, k, experts < 1 ? 1 : experts, false, compute_units()), rows, n);
}

size_t nvfp4_ffn_dw_workspace_bytes(int64_t rows, int n, int k, int experts) {
  if (rows < 1 || !rows_ok(rows) || !side_ok(n) || !side_ok(k) || experts > NVFP4_MOE_MAX_EXPERTS) return 0;
  const int e = experts < 1 ? 1 : experts;
  return workspace_of(choose_tiling(n, k, rows / e, e, true, compute_units()), (int64_t)e * n, k);
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
  const Tiling t = choose_tiling(rows, n, k, p.rows.experts, false, compute_units());
  if (const int rc = check_workspace(workspace, workspace_bytes, workspace_of(t, rows, n))) return rc;
  p.a = x; p.b = w; p.lda = x_stride; p.ldb = k; p.m = rows; p.n = n; p.k = k; p.b_step = (int64_t)n * k;
  p.rows.clear = clear != 0;
  p.partial = (float*)workspace; p.partial_step = rows * n;
  p.ep.y = y; p.ep.ldy = n; p.ep.bias = bias; p.ep.bias_f32 = bias_f32; p.ep.act = act;
  p.ep.residual = residual; p.ep.ldr = residual_stride; p.ep.z = z;
  const int rc = run_forward(p, t, dtype, false, (hipStream_t)stream);
  return rc || t.splits == 1 ? rc : finish_splits(p, dtype, false, false, stream);
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
  const Tiling t = choose_tiling(rows, 2 * inner, k, p.rows.experts, false, compute_units());
  if (const int rc = check_workspace(workspace, workspace_bytes, workspace_of(t, rows, 2 * inner))) return rc;
  p.a = x; p.b = w; p.lda = x_stride; p.ldb = k; p.m = rows; p.n = 2 * inner; p.k = k; p.b_step = (int64_t)2 * inner * k;
  p.rows.clear = clear != 0;
  p.partial = (float*)workspace; p.partial_step = rows * 2 * inner;
  p.ep.y = h; p.ep.ldy = inner; p.ep.act = act; p.ep.inner = inner; p.ep.kept = kept;
  p.ep.codes = (uint8_t*)codes; p.ep.scales = (uint8_t*)scales;
  const int rc = run_forward(p, t, dtype, true, (hipStream_t)stream);
  return rc || t.splits == 1 ? rc : finish_splits(p, dtype, true, false, stream);
}

int nvfp4_ffn_linear_dx(const void* dz, int64_t dz_stride, const void* w, void* dx, int dtype, int64_t rows, int n, int k,
                        const nvfp4_ffn_plan* plan, int clear, void* workspace, size_t workspace_bytes, void* stream) {
  if (!type16(dtype) || !rows_ok(rows) || !side_ok(n) || !side_ok(k)) return NVFP4_ERR_INVALID;
  Product p{};
  if (const int rc = plan_rows(plan, rows, false, &p.rows)) return rc;
  if (rows == 0) return NVFP4_OK;
  if (!dz || !w || !dx || !stride_ok(dz_stride, n) || (int64_t)n * k * 2 > kMaxBytes) return NVFP4_ERR_INVALID;
  if (!wide16(dz) || !wide16(w) || !wide16(dx) || dz_stride % 8) return NVFP4_ERR_MISALIGNED;
  const Tiling t = choose_tiling(rows, k, n, p.rows.experts, false, compute_units());
  if (const int rc = check_workspace(workspace, workspace_bytes, workspace_of(t, rows, k))) return rc;
  // the reduction is over n, the output's columns are k
  p.a = dz; p.b = w; p.lda = dz_stride; p.ldb = k; p.m = rows; p.n = k; p.k = n; p.b_step = (int64_t)n * k;
  p.rows.clear = clear != 0;
  p.partial = (float*)workspace; p.partial_step = rows * k;
  p.ep.y = dx; p.ep.ldy = k;
  const int rc = run_dx(p, t, dtype, (hipStream_t)stream);
  return rc || t.splits == 1 ? rc : finish_splits(p, dtype, false, false, stream);
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
  Tiling t{0, 1};
  if (rows) t = choose_tiling(n, k, rows / p.rows.experts, p.rows.experts, true, compute_units());
  const int64_t out_rows = (int64_t)p.rows.experts * n;
  if (const int rc = check_workspace(workspace, workspace_bytes, workspace_of(t, out_rows, k))) return rc;
  p.a = dz; p.b = x; p.lda = dz_stride; p.ldb = x_stride; p.m = n; p.n = k; p.k = 0;
  p.partial = (float*)workspace; p.partial_step = out_rows * k;
  p.ep.y = dw; p.ep.ldy = k; p.ep.y_f32 = dw_f32;
  const int rc = run_dw(p, t, dtype, (hipStream_t)stream);
  return rc || t.splits == 1 ? rc : finish_splits(p, dtype, false, true, stream);
}

}  // extern "C"
