// Operators on rows around the products of nvfp4_ffn.h: rows to 8 bits and back,
// tokens' rows at their slots' rows, gradients of activations with their column sums.
// All bound by memory: a thread takes eight adjacent elements. Measured, bf16: 16390 x 2048 to 8 bits 17.9 us and back
// 16.5 (102 MB each: 5.7 and 6.2 TB/s); gather to 3900 rows of 4096 10.8; gated_dz of 4099 x 2 x 2048 from 8 bits 14.4
// (68 MB); linear_dz of 2051 x 4104 with silu and column sums 15.6 and 4.6 (51 MB: a floor of 10).
#include "ffn_common.h"

namespace ffn {

// ---- 8 bits -------------------------------------------------------------------
template <class T> __global__ __launch_bounds__(256) void quantize8_kernel(const void* x, int64_t eights, int wide, int64_t stride, bool vec,
                                                                           uint8_t* codes, uint8_t* scales) {
  const int64_t step = (int64_t)gridDim.x * 256;
  for (int64_t base = (int64_t)blockIdx.x * 256; base < eights; base += step) {
    const int64_t i = base + threadIdx.x;
    float v[8] = {};
    // rows without gaps are one long row
    if (i < eights) load8<T>(x, stride == (int64_t)wide * 8 ? i * 8 : i / wide * stride + i % wide * 8, vec, v);
    uint32_t top = abs_bits(v[0]);
#pragma unroll
    for (int j = 1; j < 8; ++j) top = umax(top, abs_bits(v[j]));
    top = umax(top, from_lane_xor(top, 1));
    top = umax(top, from_lane_xor(top, 2));
    if (i >= eights) continue;
    const uint32_t byte = scale8(top);
    const float inverse = scale8_inverse(byte);
    u32x2 q;
    q.x = encode4(v[0], v[1], v[2], v[3], inverse);
    q.y = encode4(v[4], v[5], v[6], v[7], inverse);
    *(u32x2*)(codes + i * 8) = q;
    if (i % 4 == 0) scales[i / 4] = (uint8_t)byte;
  }
}

// Eight values of a row in 8 bits; i counts eights of all rows.
__device__ __forceinline__ void values8(const uint8_t* codes, const uint8_t* scales, int64_t i, float* v) {
  const u32x2 q = *(const u32x2*)(codes + i * 8);
  const float scale = scale8_value(scales[i / 4]);
  decode4(q.x, scale, v);
  decode4(q.y, scale, v + 4);
}

template <class T> __global__ __launch_bounds__(256) void dequantize8_kernel(const uint8_t* codes, const uint8_t* scales, int64_t eights, int wide,
                                                                             void* out, int64_t stride, bool vec) {
  const int64_t step = (int64_t)gridDim.x * 256;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < eights; i += step) {
    float v[8];
    values8(codes, scales, i, v);
    const int64_t at = stride == (int64_t)wide * 8 ? i * 8 : i / wide * stride + i % wide * 8;
    if (vec && T::kBytes == 2) *(u32x4*)((uint16_t*)out + at) = pack16x8<T>(v);
    else store8<T>(out, at, vec, v);
  }
}

// ---- tokens' rows at their slots' rows ------------------------------------------------
template <class T, bool EIGHT>
__global__ __launch_bounds__(256) void gather_kernel(const void* x, int64_t stride, const uint8_t* codes, const uint8_t* scales,
                                                     int wide, Rows p, void* out) {
  const int64_t rows = first_row(p, p.experts);
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    const int64_t from = source_row(p, row);
    if (from < 0) continue;
    for (int c = threadIdx.x; c < wide; c += 256) {
      if constexpr (EIGHT) {
        float v[8];
        values8(codes, scales, from * wide + c, v);
        ((u32x4*)out)[row * wide + c] = pack16x8<T>(v);
      } else {
        ((u32x4*)out)[row * wide + c] = *(const u32x4*)((const uint16_t*)x + from * stride + c * 8);
      }
    }
  }
}

// ---- gradients of activations -----------------------------------------------------------
constexpr int kChunkRows = 64;   // rows whose columns a workgroup sums
constexpr int kChunkCols = 256;  // its columns: 32 lanes of eight

// The chunk `index` of kChunkRows rows, counted over all experts: its rows; false: no such chunk. As the plan may
// leave no more than one part of a chunk to each expert, there are rows / 64 + experts at most.
__device__ __forceinline__ bool find_chunk(const Rows& p, int64_t index, int lane, int64_t& row, int64_t& end) {
  int64_t before = 0;
  for (int c = 0; c < p.experts; c += 64) {
    const int e = c + lane;
    const int64_t lo = e < p.experts ? first_row(p, e) : 0, hi = e < p.experts ? first_row(p, e + 1) : 0;
    const int chunks = hi > lo ? (int)((hi - lo + kChunkRows - 1) / kChunkRows) : 0;
    int upto = chunks;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int v = __shfl_up(upto, d, 64);
      if (lane >= d) upto += v;
    }
    const uint64_t found = __ballot(before + upto > index);
    if (found) {
      const int src = __builtin_ctzll(found);
      row = (int64_t)__shfl((int)lo, src, 64) + (index - before - __shfl(upto - chunks, src, 64)) * kChunkRows;
      end = min(row + kChunkRows, (int64_t)__shfl((int)hi, src, 64));
      return true;
    }
    before += __shfl(upto, 63, 64);
  }
  return false;
}

// dz = dy act'(z), and with `partial` [chunks][n] the columns' sums of the chunk's rows: each thread every eighth row
// of eight columns, the eight threads of a column in order.
template <class T> __global__ __launch_bounds__(256) void linear_dz_kernel(const void* dy, int64_t dy_stride, const void* z, int act, void* dz,
                                                                           int n, Rows p, int64_t chunks, float* partial) {
  __shared__ float room[8][kChunkCols];
  const int64_t chunk = blockIdx.y + (int64_t)blockIdx.z * gridDim.y;
  int64_t row, end;
  // (tables that do not fit together may name more chunks than there is room for)
  if (chunk >= chunks || !find_chunk(p, chunk, threadIdx.x & 63, row, end)) return;
  const int col = blockIdx.x * kChunkCols + threadIdx.x % 32 * 8, first = threadIdx.x / 32;
  float sum[8] = {};
  if (col < n) {
    // the loads of four rows are under way together
    for (int64_t r0 = row + first; r0 < end; r0 += 32) {
      u32x4 d4[4], z4[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int64_t r = r0 + 8 * u;
        if (r >= end) continue;
        d4[u] = *(const u32x4*)((const uint16_t*)dy + r * dy_stride + col);
        if (act != NVFP4_FFN_NONE) z4[u] = *(const u32x4*)((const uint16_t*)z + r * n + col);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int64_t r = r0 + 8 * u;
        if (r >= end) continue;
        float d[8];
        unpack16x8<T>(d4[u], d);
        if (act != NVFP4_FFN_NONE) {
          float v[8];
          unpack16x8<T>(z4[u], v);
          slopes8(v, act);
#pragma unroll
          for (int j = 0; j < 8; ++j) d[j] *= v[j];
        }
        if (dz) *(u32x4*)((uint16_t*)dz + r * n + col) = pack16x8<T>(d);
#pragma unroll
        for (int j = 0; j < 8; ++j) sum[j] += d[j];
      }
    }
  }
  if (!partial) return;
#pragma unroll
  for (int j = 0; j < 8; ++j) room[first][threadIdx.x % 32 * 8 + j] = sum[j];
  __syncthreads();
  const int at = blockIdx.x * kChunkCols + threadIdx.x;
  if (at < n) {
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) v += room[i][threadIdx.x];
    partial[chunk * n + at] = v;
  }
}

template <class T, bool EIGHT>
__global__ __launch_bounds__(256) void gated_dz_kernel(const void* dh, int64_t dh_stride, const void* kept, const uint8_t* codes,
                                                       const uint8_t* scales, int act, void* dz, int inner, Rows p) {
  const int64_t rows = first_row(p, p.offsets ? p.experts : 1);
  const int wide = inner / 8;
  const int64_t eights = rows * wide, step = (int64_t)gridDim.x * 256;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < eights; i += step) {
    const int64_t row = i / wide;
    const int c = (int)(i - row * wide);
    float d[8], g[8], u[8];
    load8<T>(dh, row * dh_stride + c * 8, true, d);
    if constexpr (EIGHT) {
      values8(codes, scales, row * 2 * wide + c, g);
      values8(codes, scales, row * 2 * wide + wide + c, u);
    } else {
      load8<T>(kept, (row * 2 * wide + c) * 8, true, g);
      load8<T>(kept, (row * 2 * wide + wide + c) * 8, true, u);
    }
    float a[8];
    values_slopes8(g, a, act);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      g[j] *= d[j] * u[j];
      u[j] = d[j] * a[j];
    }
    ((u32x4*)dz)[row * 2 * wide + c] = pack16x8<T>(g);
    ((u32x4*)dz)[row * 2 * wide + wide + c] = pack16x8<T>(u);
  }
}

// ---- sums of parts ------------------------------------------------------------------------
// out[e][col] = the sum of the parts of expert e, 32 columns a workgroup: 32 threads for each column, four interleaved
// chains each, so that few loads wait for one another (1024 parts of 4096: 8 threads took 11 us). Without a plan one
// expert has all `parts`.
constexpr int kAddThreads = 1024, kAddRows = kAddThreads / 32;
__global__ __launch_bounds__(kAddThreads) void add_columns_kernel(const float* partial, int64_t parts, int n, Rows p, void* out, int type) {
  __shared__ float room[kAddRows][33];
  const int col = blockIdx.x * 32 + threadIdx.x % 32, first = threadIdx.x / 32, e = blockIdx.y;
  int64_t begin = 0, end = parts;
  if (p.offsets) {
    // chunks of the experts before, and of this one
    int64_t before = 0;
    for (int i = threadIdx.x & 63; i < e; i += 64) {
      const int64_t lo = first_row(p, i), hi = first_row(p, i + 1);
      before += hi > lo ? (hi - lo + kChunkRows - 1) / kChunkRows : 0;
    }
#pragma unroll
    for (int d = 32; d; d /= 2) before += __shfl_xor((long long)before, d, 64);
    const int64_t lo = first_row(p, e), hi = first_row(p, e + 1);
    begin = min(before, parts);
    end = min(begin + (hi > lo ? (hi - lo + kChunkRows - 1) / kChunkRows : 0), parts);
  }
  float v[4] = {};
  if (col < n) {
    int64_t i = begin + first;
    for (; i + 3 * kAddRows < end; i += 4 * kAddRows) {
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] += partial[(i + kAddRows * j) * n + col];
    }
    for (; i < end; i += kAddRows) v[0] += partial[i * n + col];
  }
  room[first][threadIdx.x % 32] = (v[0] + v[1]) + (v[2] + v[3]);
  __syncthreads();
  if (threadIdx.x >= 32 || col >= n) return;
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < kAddRows; ++i) sum += room[i][threadIdx.x];
  const int64_t at = (int64_t)e * n + col;
  if (type == NVFP4_MOE_F32) store1<F32>(out, at, sum);
  else if (type == NVFP4_MOE_F16) store1<F16>(out, at, sum);
  else store1<BF16>(out, at, sum);
}

void add_columns(const float* partial, int64_t parts, int n, void* out, int out_type, hipStream_t stream) {
  add_columns_kernel<<<dim3(ceil_div(n, 32), 1), kAddThreads, 0, stream>>>(partial, parts, n, Rows{nullptr, nullptr, 1, 1, 0, 0, 0}, out, out_type);
}

// Workgroups of 256 threads for `items` threads' work, as many as keep the card full.
static unsigned blocks_for(int64_t items) {
  const int64_t most = (int64_t)1 << 20, n = ceil_div64(items, 256);
  return (unsigned)(n < most ? n : most);
}
static bool rows_ok(int64_t rows) { return rows >= 0 && rows < (int64_t)1 << 31; }
static bool width_ok(int n, int step) { return n >= step && n <= 1 << 20 && n % step == 0; }
// Chunks of so many rows, with a plan (experts, else 0) the most there can be.
static int64_t chunks_of(int64_t rows, int experts) {
  return experts ? rows / kChunkRows + (experts < rows ? experts : rows) : ceil_div64(rows, kChunkRows);
}

}  // namespace ffn

using namespace ffn;

extern "C" {

int nvfp4_ffn_quantize8(const void* x, int dtype, int64_t rows, int n, int64_t x_stride, void* codes, void* scales,
                        void* stream) {
  if (!known_type(dtype) || !rows_ok(rows) || !width_ok(n, kBlock8)) return NVFP4_ERR_INVALID;
  if (rows == 0) return NVFP4_OK;
  if (!x || !codes || !scales || x_stride < n) return NVFP4_ERR_INVALID;
  if (!aligned(x, element_bytes(dtype)) || !aligned(codes, 8)) return NVFP4_ERR_MISALIGNED;
  if (rows == 1) x_stride = n;
  const int64_t eights = rows * (n / 8);
  with_type(dtype, [&](auto type) {
    quantize8_kernel<decltype(type)><<<blocks_for(eights), 256, 0, (hipStream_t)stream>>>(
        x, eights, n / 8, x_stride, wide_rows(x, dtype, x_stride), (uint8_t*)codes, (uint8_t*)scales);
    return 0;
  });
  return launched();
}

int nvfp4_ffn_dequantize8(const void* codes, const void* scales, int64_t rows, int n, void* out, int dtype,
                          int64_t out_stride, void* stream) {
  if (!known_type(dtype) || !rows_ok(rows) || !width_ok(n, kBlock8)) return NVFP4_ERR_INVALID;
  if (rows == 0) return NVFP4_OK;
  if (!out || !codes || !scales || out_stride < n) return NVFP4_ERR_INVALID;
  if (!aligned(out, element_bytes(dtype)) || !aligned(codes, 8)) return NVFP4_ERR_MISALIGNED;
  if (rows == 1) out_stride = n;
  const int64_t eights = rows * (n / 8);
  with_type(dtype, [&](auto type) {
    dequantize8_kernel<decltype(type)><<<blocks_for(eights), 256, 0, (hipStream_t)stream>>>(
        (const uint8_t*)codes, (const uint8_t*)scales, eights, n / 8, out, out_stride, wide_rows(out, dtype, out_stride));
    return 0;
  });
  return launched();
}

int nvfp4_ffn_gather(const void* x, int64_t x_stride, const void* codes, const void* scales, int dtype, int64_t tokens,
                     int n, const nvfp4_ffn_plan* plan, void* out, void* stream) {
  if (!type16(dtype) || !rows_ok(tokens) || !plan || plan->topk < 1 || plan->topk > NVFP4_MOE_MAX_TOPK ||
      !rows_ok(tokens * plan->topk) || !width_ok(n, x ? 8 : kBlock8))
    return NVFP4_ERR_INVALID;
  const int64_t rows = tokens * plan->topk;
  Rows p;
  if (const int rc = plan_rows(plan, rows, true, &p)) return rc;
  if (rows == 0) return NVFP4_OK;
  if (!out || (x ? x_stride < n : !codes || !scales)) return NVFP4_ERR_INVALID;
  if (!aligned(out, 16) || (x ? !aligned(x, 16) || x_stride % 8 : !aligned(codes, 8))) return NVFP4_ERR_MISALIGNED;
  const unsigned grid = (unsigned)(rows < 1 << 20 ? rows : 1 << 20);
  with_type16(dtype, [&](auto type) {
    using T = decltype(type);
    if (x) gather_kernel<T, false><<<grid, 256, 0, (hipStream_t)stream>>>(x, x_stride, nullptr, nullptr, n / 8, p, out);
    else gather_kernel<T, true><<<grid, 256, 0, (hipStream_t)stream>>>(nullptr, 0, (const uint8_t*)codes, (const uint8_t*)scales, n / 8, p, out);
    return 0;
  });
  return launched();
}

size_t nvfp4_ffn_dz_workspace_bytes(int64_t rows, int n, int experts) {
  if (rows < 1 || !rows_ok(rows) || !width_ok(n, 8) || experts > NVFP4_MOE_MAX_EXPERTS) return 0;
  return (size_t)chunks_of(rows, experts < 1 ? 0 : experts) * n * 4;
}

int nvfp4_ffn_linear_dz(const void* dy, int64_t dy_stride, const void* z, int act, void* dz, void* dbias, int bias_f32,
                        int dtype, int64_t rows, int n, const nvfp4_ffn_plan* plan, void* workspace,
                        size_t workspace_bytes, void* stream) {
  if (!type16(dtype) || act < NVFP4_FFN_NONE || act > NVFP4_FFN_GELU || !rows_ok(rows) || !width_ok(n, 8)) return NVFP4_ERR_INVALID;
  Rows p;
  if (const int rc = plan_rows(plan, rows, false, &p)) return rc;
  if (!aligned(dbias, bias_f32 ? 4 : 2)) return NVFP4_ERR_MISALIGNED;
  const int bias_type = bias_f32 ? NVFP4_MOE_F32 : dtype;
  if (rows == 0) {
    if (!dbias) return NVFP4_OK;
    p.offsets = nullptr;  // an empty sum for every expert
    add_columns_kernel<<<dim3(ceil_div(n, 32), p.experts), kAddThreads, 0, (hipStream_t)stream>>>(nullptr, 0, n, p, dbias, bias_type);
    return launched();
  }
  if (!dy || dy_stride < n || (act != NVFP4_FFN_NONE && (!z || !dz))) return NVFP4_ERR_INVALID;
  if (!aligned(dy, 16) || dy_stride % 8 || !aligned(z, 16) || !aligned(dz, 16)) return NVFP4_ERR_MISALIGNED;
  const int64_t chunks = chunks_of(rows, p.offsets ? p.experts : 0);
  if (dbias) {
    if (!workspace || workspace_bytes < (size_t)chunks * n * 4) return NVFP4_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return NVFP4_ERR_MISALIGNED;
  } else if (!dz) {
    return NVFP4_OK;
  }
  const unsigned high = 32768, grid_y = (unsigned)(chunks < high ? chunks : high);
  const dim3 grid(ceil_div(n, kChunkCols), grid_y, (unsigned)ceil_div64(chunks, grid_y));
  with_type16(dtype, [&](auto type) {
    linear_dz_kernel<decltype(type)><<<grid, 256, 0, (hipStream_t)stream>>>(dy, dy_stride, z, act, dz, n, p, chunks,
                                                                           dbias ? (float*)workspace : nullptr);
    return 0;
  });
  if (const int rc = launched()) return rc;
  if (!dbias) return NVFP4_OK;
  add_columns_kernel<<<dim3(ceil_div(n, 32), p.experts), kAddThreads, 0, (hipStream_t)stream>>>((const float*)workspace, chunks, n, p, dbias, bias_type);
  return launched();
}

int nvfp4_ffn_gated_dz(const void* dh, int64_t dh_stride, const void* kept, const void* codes, const void* scales, int act,
                       void* dz, int dtype, int64_t rows, int inner, const nvfp4_ffn_plan* plan, void* stream) {
  if (!type16(dtype) || act <= NVFP4_FFN_NONE || act > NVFP4_FFN_GELU || !rows_ok(rows) || !width_ok(inner, kept ? 8 : kBlock8))
    return NVFP4_ERR_INVALID;
  Rows p;
  if (const int rc = plan_rows(plan, rows, false, &p)) return rc;
  if (rows == 0) return NVFP4_OK;
  if (!dh || !dz || dh_stride < inner || (!kept && (!codes || !scales))) return NVFP4_ERR_INVALID;
  if (!aligned(dh, 16) || dh_stride % 8 || !aligned(dz, 16) || !aligned(kept, 16) || (!kept && !aligned(codes, 8))) return NVFP4_ERR_MISALIGNED;
  const unsigned grid = blocks_for(rows * (inner / 8));
  with_type16(dtype, [&](auto type) {
    using T = decltype(type);
    if (kept) gated_dz_kernel<T, false><<<grid, 256, 0, (hipStream_t)stream>>>(dh, dh_stride, kept, nullptr, nullptr, act, dz, inner, p);
    else gated_dz_kernel<T, true><<<grid, 256, 0, (hipStream_t)stream>>>(dh, dh_stride, nullptr, (const uint8_t*)codes, (const uint8_t*)scales, act, dz, inner, p);
    return 0;
  });
  return launched();
}

}  // extern "C"
