// The plan: slots sorted by expert (a stable counting sort), the row offsets
// and scale-atom offsets of the experts, and the group tables of the products.
#include "moe_common.h"

namespace moe {
namespace {

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / 64;
constexpr int kBins = NVFP4_MOE_MAX_EXPERTS;
// A workgroup places at least kOneBlockSlots slots. Up to kOnePassSlots each of
// them counts all slots itself (2800 slots: 5 us, of which a launch is 4); beyond,
// a launch of its own for the counts is faster (65536 slots of 256 experts: 11 us
// with, 18 without). More than kMaxBlocks cost more in counts to add up than they save.
constexpr int kOneBlockSlots = 1024;
constexpr int kOnePassSlots = 8192;
constexpr int kMaxBlocks = 128;

struct PlanArgs {
  const int32_t* ids;
  int slots, experts, id_bits;  // id_bits: bits that tell the bins 0 .. experts apart
  int block_slots, blocks;
  int32_t *offsets, *atoms, *slot_rows, *row_slots;
  int32_t* slot_ids;  // or null
  int32_t* counts;  // [blocks][experts], of every block's slots; null where every block counts all slots
  int num_products;
  nvfp4_moe_product products[NVFP4_MOE_MAX_PRODUCTS];
};

__device__ inline int bin_of(int id, int experts) { return (unsigned)id < (unsigned)experts ? id : -1; }

// Slots of this block per expert, and of each wave's part of them in s_wave.
__device__ inline void count_block(const PlanArgs& a, int from, int to, int (*s_wave)[kBins]) {
  for (int i = threadIdx.x; i < kWaves * a.experts; i += kThreads) s_wave[i / a.experts][i % a.experts] = 0;
  __syncthreads();
  const int wave = threadIdx.x / 64, part = ceil_div(ceil_div(to - from, kWaves), 64) * 64;
  const int begin = from + wave * part, end = min(to, begin + part);
  for (int i = begin + (int)(threadIdx.x & 63); i < end; i += 64) {
    const int e = bin_of(a.ids[i], a.experts);
    if (e >= 0) atomicAdd(&s_wave[wave][e], 1);  // whole numbers: the order does not matter
  }
  __syncthreads();
}

// First pass of a long plan: every block's counts.
__global__ void __launch_bounds__(kThreads) nvfp4_moe_count_kernel(PlanArgs a) {
  __shared__ int s_wave[kWaves][kBins];
  const int from = blockIdx.x * a.block_slots, to = min(a.slots, from + a.block_slots);
  count_block(a, from, to, s_wave);
  for (int e = threadIdx.x; e < a.experts; e += kThreads) {
    int n = 0;
    for (int w = 0; w < kWaves; ++w) n += s_wave[w][e];
    a.counts[(int64_t)blockIdx.x * a.experts + e] = n;
  }
}

// Slots from .. to - 1 per expert.
__device__ inline void count_slots(const PlanArgs& a, int from, int to, int* bins) {
#pragma unroll 8
  for (int i = from + (int)threadIdx.x; i < to; i += kThreads) {
    const int e = bin_of(a.ids[i], a.experts);
    if (e >= 0) atomicAdd(&bins[e], 1);
  }
}

// Sums up to and with each bin, by one wave.
__device__ inline void scan_bins(int* x, int lane) {
  constexpr int kPart = kBins / 64;
  int v[kPart], sum = 0;
#pragma unroll
  for (int i = 0; i < kPart; ++i) {
    sum += x[lane * kPart + i];
    v[i] = sum;
  }
  int before = sum;  // of the lanes up to this one
  for (int d = 1; d < 64; d *= 2) {
    const int u = __shfl_up(before, d);
    before += lane >= d ? u : 0;
  }
  before -= sum;
#pragma unroll
  for (int i = 0; i < kPart; ++i) x[lane * kPart + i] = before + v[i];
}

// Second pass: the place of every slot. A wave walks its slots in order, 64 at
// a time; lanes of one expert find each other with one ballot per bit of the
// id, and a lane's rank among them is the number of such lanes before it.
__global__ void __launch_bounds__(kThreads) nvfp4_moe_place_kernel(PlanArgs a) {
  __shared__ int s_wave[kWaves][kBins];
  __shared__ int s_rows[kBins], s_atoms[kBins];  // after the scan: sums up to and with the bin
  const int from = blockIdx.x * a.block_slots, to = min(a.slots, from + a.block_slots);
  const bool all = a.blocks > 1 && a.counts == nullptr;
  if (all && threadIdx.x < kBins) s_rows[threadIdx.x] = s_atoms[threadIdx.x] = 0;
  count_block(a, from, to, s_wave);
  if (all) {
    count_slots(a, 0, from, s_rows);            // slots before this block
    count_slots(a, to, a.slots, s_atoms);       // and after it
    __syncthreads();
  }
  const int e = threadIdx.x;
  int total = 0, before = 0;  // slots of expert e in all blocks, in the blocks before
  if (e < a.experts) {
    if (a.counts == nullptr) {
      before = all ? s_rows[e] : 0;
      total = before + (all ? s_atoms[e] : 0);
#pragma unroll
      for (int w = 0; w < kWaves; ++w) total += s_wave[w][e];
    } else {
#pragma unroll 8
      for (int b = 0; b < a.blocks; ++b) {
        const int n = a.counts[(int64_t)b * a.experts + e];
        total += n;
        before += b < (int)blockIdx.x ? n : 0;
      }
    }
  }
  if (e < kBins) {
    s_rows[e] = total;
    s_atoms[e] = ceil_div(total, kAtomRows);
  }
  __syncthreads();
  if (threadIdx.x < 128) scan_bins(threadIdx.x < 64 ? s_rows : s_atoms, threadIdx.x & 63);
  __syncthreads();
  const int rows = s_rows[kBins - 1];
  if (e < a.experts) {
    const int row = s_rows[e] - total, atom = s_atoms[e] - ceil_div(total, kAtomRows);
    int at = row + before;
    for (int w = 0; w < kWaves; ++w) {
      const int n = s_wave[w][e];
      s_wave[w][e] = at;
      at += n;
    }
    if (blockIdx.x == 0) {
      a.offsets[e] = row;
      a.atoms[e] = atom;
      if (e == 0) {
        a.offsets[a.experts] = rows;
        a.atoms[a.experts] = s_atoms[kBins - 1];
      }
      for (int i = 0; i < a.num_products; ++i) {
        const nvfp4_moe_product& p = a.products[i];
        const int64_t kt = (p.k + kAtomK - 1) / kAtomK, b_sf = (int64_t)((p.n + kAtomRows - 1) / kAtomRows) * kt * kAtomBytes;
        int32_t* size = (int32_t*)p.sizes + 4 * e;
        size[0] = total;
        size[1] = p.n;
        size[2] = p.k;
        size[3] = 1;
        uint64_t* abc = (uint64_t*)p.abc + 3 * e;
        abc[0] = p.a + (uint64_t)row * (p.k / 2);
        abc[1] = p.b + (uint64_t)e * p.n * (p.k / 2);
        abc[2] = p.c + (uint64_t)row * p.n * 2;
        uint64_t* sf = (uint64_t*)p.sf + 2 * e;
        sf[0] = p.sfa + (uint64_t)atom * kt * kAtomBytes;
        sf[1] = p.sfb + (uint64_t)e * b_sf;
      }
    }
  }
  __syncthreads();
  // no slot has these rows
  for (int64_t i = (int64_t)rows + blockIdx.x * kThreads + threadIdx.x; i < a.slots; i += (int64_t)a.blocks * kThreads)
    a.row_slots[i] = -1;

  const int wave = threadIdx.x / 64, lane = threadIdx.x & 63, part = ceil_div(ceil_div(to - from, kWaves), 64) * 64;
  const int begin = from + wave * part, end = min(to, begin + part);
  for (int i0 = begin; i0 < end; i0 += 64) {
    const int i = i0 + lane;
    const int bin = i < end ? bin_of(a.ids[i], a.experts) : -1;
    uint64_t same = __ballot(bin >= 0);
    for (int b = 0; b < a.id_bits; ++b) {
      const uint64_t set = __ballot((bin >> b) & 1);
      same &= (bin >> b) & 1 ? set : ~set;
    }
    if (bin >= 0) {
      const int rank = __popcll(same & ((1ull << lane) - 1));
      const int row = s_wave[wave][bin] + rank;
      a.slot_rows[i] = row;
      a.row_slots[row] = i;
      // the last of the lanes moves the counter on; a wave's reads of it come before, in order
      if (same >> lane == 1) s_wave[wave][bin] = row + 1;
    } else if (i < end) {
      a.slot_rows[i] = -1;
    }
    if (a.slot_ids != nullptr && i < end) a.slot_ids[i] = bin;
    wave_sync();
  }
}

// A plan of no slots.
__global__ void nvfp4_moe_empty_plan_kernel(PlanArgs a) {
  for (int e = threadIdx.x; e <= a.experts; e += blockDim.x) a.offsets[e] = a.atoms[e] = 0;
  for (int i = 0; i < a.num_products; ++i) {
    for (int e = threadIdx.x; e < a.experts; e += blockDim.x) {
      const nvfp4_moe_product& p = a.products[i];
      const int64_t kt = (p.k + kAtomK - 1) / kAtomK, b_sf = (int64_t)((p.n + kAtomRows - 1) / kAtomRows) * kt * kAtomBytes;
      int32_t* size = (int32_t*)p.sizes + 4 * e;
      size[0] = 0;
      size[1] = p.n;
      size[2] = p.k;
      size[3] = 1;
      uint64_t *abc = (uint64_t*)p.abc + 3 * e, *sf = (uint64_t*)p.sf + 2 * e;
      abc[0] = p.a;
      abc[1] = p.b + (uint64_t)e * p.n * (p.k / 2);
      abc[2] = p.c;
      sf[0] = p.sfa;
      sf[1] = p.sfb + (uint64_t)e * b_sf;
    }
  }
}

// Slots of a block: at most kMaxBlocks blocks, whole waves' rounds.
int block_slots(int64_t slots) {
  const int64_t even = ceil_div64(slots, kMaxBlocks);
  return (int)(ceil_div64(even < kOneBlockSlots ? kOneBlockSlots : even, kThreads) * kThreads);
}

bool plan_sizes(int64_t tokens, int topk, int experts) {
  return tokens >= 0 && tokens < (int64_t)1 << 31 && topk >= 1 && topk <= NVFP4_MOE_MAX_TOPK && experts >= 1 &&
         experts <= NVFP4_MOE_MAX_EXPERTS && tokens * topk <= (int64_t)1 << 30;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t nvfp4_moe_plan_workspace_bytes(int64_t tokens, int topk, int experts) {
  if (!plan_sizes(tokens, topk, experts) || tokens * topk <= kOnePassSlots) return 0;
  return (size_t)ceil_div64(tokens * topk, block_slots(tokens * topk)) * experts * sizeof(int32_t);
}

size_t nvfp4_moe_sf_bytes(int64_t rows, int experts, int k) {
  if (rows < 0 || rows >= (int64_t)1 << 31 || experts < 1 || experts > NVFP4_MOE_MAX_EXPERTS || k < 0) return 0;
  // every expert that has rows may leave all but one row of its last atom empty
  const int64_t used = rows < experts ? rows : experts;
  return (size_t)((rows - used) / kAtomRows + used) * ((k + kAtomK - 1) / kAtomK) * kAtomBytes;
}

int nvfp4_moe_plan(const int32_t* ids, int64_t tokens, int topk, int experts, int32_t* offsets, int32_t* atoms,
                   int32_t* slot_rows, int32_t* row_slots, const nvfp4_moe_product* products, int num_products,
                   void* workspace, size_t workspace_bytes, void* stream) {
  return nvfp4_moe_plan_ex(ids, tokens, topk, experts, offsets, atoms, slot_rows, row_slots, nullptr, products, num_products,
                           workspace, workspace_bytes, stream);
}

int nvfp4_moe_plan_ex(const int32_t* ids, int64_t tokens, int topk, int experts, int32_t* offsets, int32_t* atoms,
                      int32_t* slot_rows, int32_t* row_slots, int32_t* slot_ids, const nvfp4_moe_product* products,
                      int num_products, void* workspace, size_t workspace_bytes, void* stream) {
  if (!plan_sizes(tokens, topk, experts) || offsets == nullptr || atoms == nullptr) return NVFP4_ERR_INVALID;
  if (tokens > 0 && (ids == nullptr || slot_rows == nullptr || row_slots == nullptr)) return NVFP4_ERR_INVALID;
  if (num_products < 0 || num_products > NVFP4_MOE_MAX_PRODUCTS || (num_products > 0 && products == nullptr))
    return NVFP4_ERR_INVALID;
  if (!aligned(ids, 4) || !aligned(offsets, 4) || !aligned(atoms, 4) || !aligned(slot_rows, 4) || !aligned(row_slots, 4) ||
      !aligned(slot_ids, 4))
    return NVFP4_ERR_MISALIGNED;
  PlanArgs a = {};
  for (int i = 0; i < num_products; ++i) {
    const nvfp4_moe_product& p = products[i];
    if (p.n < 0 || p.k < 0 || p.n % 8 || p.k % 32) return NVFP4_ERR_INVALID;
    if (!p.sizes || !p.abc || !p.sf) return NVFP4_ERR_INVALID;
    if ((p.sizes | p.abc | p.sf | p.a | p.b | p.c | p.sfa | p.sfb) % 16) return NVFP4_ERR_MISALIGNED;
    a.products[i] = p;
  }
  const size_t need = nvfp4_moe_plan_workspace_bytes(tokens, topk, experts);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return NVFP4_ERR_WORKSPACE;
  if (need > 0 && !aligned(workspace, 256)) return NVFP4_ERR_MISALIGNED;
  a.ids = ids;
  a.slots = (int)(tokens * topk);
  a.experts = experts;
  while (experts >> a.id_bits) ++a.id_bits;
  a.block_slots = block_slots(a.slots);
  a.blocks = a.slots ? (int)ceil_div64(a.slots, a.block_slots) : 0;
  a.offsets = offsets;
  a.atoms = atoms;
  a.slot_rows = slot_rows;
  a.row_slots = row_slots;
  a.slot_ids = slot_ids;
  a.counts = need > 0 ? (int32_t*)workspace : nullptr;
  a.num_products = num_products;
  const hipStream_t st = (hipStream_t)stream;
  if (a.slots == 0) {
    nvfp4_moe_empty_plan_kernel<<<1, 256, 0, st>>>(a);
    return launched();
  }
  if (a.counts != nullptr) {
    nvfp4_moe_count_kernel<<<a.blocks, kThreads, 0, st>>>(a);
    if (int rc = launched()) return rc;
  }
  nvfp4_moe_place_kernel<<<a.blocks, kThreads, 0, st>>>(a);
  return launched();
}

}  // extern "C"
