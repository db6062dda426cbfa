// The plan of a product grouped by expert: the groups' bounds held to the rows, the table of the
// tiles of rows, and the tensor maps that end with a group.  Made by blocks of the kernel that also
// packs operands (grouped.cu), or by a product's kernel for itself (grouped_gemm.cu).
#pragma once

#include "common.cuh"
#include "grouped.h"

namespace moe {

constexpr int kRowChunk = 8;    // tiles of rows that share the weights' tiles in L2
constexpr int kMostGroups = 1024;
constexpr int kWideRows = 256, kWideStep = 32;  // rows of a tile of grouped_wide_kernel

// The plan in shared memory of a kernel that plans for itself (bound null: the plan kernel's).
struct Table {
  int* bound;  // [groups + 1]
  int* first;  // [groups + 1]: first tile of rows of each group, then their number
};

// The last group whose first tile is not past tile i (so one that has tiles).
__device__ __forceinline__ int group_of_tile(const int* first, int groups, int i) {
  int lo = 0, hi = groups;
  while (hi - lo > 1) {
    const int m = (lo + hi) >> 1;
    if (first[m] <= i) lo = m;
    else hi = m;
  }
  return lo;
}

// Tile i of rows as the table of tiles has it.
__device__ __forceinline__ int4 table_entry(const Table& t, int groups, int i, int tile_rows) {
  const int g = group_of_tile(t.first, groups, i);
  const int first = t.first[g], tiles = t.first[g + 1] - first;
  const int chunk = first + (i - first) / kRowChunk * kRowChunk;
  // rows of the group's tiles: even shares, where a tile need not be full
  const int size = t.bound[g + 1] - t.bound[g];
  const int rows = tile_rows == kWideRows
                       ? ((size + tiles - 1) / tiles + kWideStep - 1) / kWideStep * kWideStep
                       : tile_rows;
  return make_int4(g, t.bound[g] + (chunk - first) * rows, chunk,
                   min(kRowChunk, first + tiles - chunk) | rows << 4);
}

// Reads the offsets (at most 1025) and makes them ascend within 0..rows: a running maximum, so that
// bad ones cannot lead a kernel out of its buffers; `report`: one block tells of them through the
// error word.  Then the groups' first tiles.  Every thread of the block calls it; PER groups a
// thread; scratch: 32 ints.
template <int PER>
__device__ __forceinline__ void make_table(const int32_t* offsets, int rows, int groups,
                                           int tile_rows, const Table& t, int* scratch, bool report,
                                           unsigned* err) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int start = min(max(offsets[0], 0), rows);
  int given[PER], bound[PER];
  int most = start;
#pragma unroll
  for (int k = 0; k < PER; ++k) {
    const int g = tid * PER + k;
    given[k] = g < groups ? offsets[g + 1] : start;
    most = max(most, min(max(given[k], 0), rows));
    bound[k] = most;
  }
  int before = most;  // running maximum over the threads up to this one
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int n = __shfl_up_sync(0xffffffffu, before, o);
    if (lane >= o) before = max(before, n);
  }
  if (lane == 31) scratch[warp] = before;
  before = __shfl_up_sync(0xffffffffu, before, 1);
  if (lane == 0) before = start;
  __syncthreads();
  for (int w = 0; w < warp; ++w) before = max(before, scratch[w]);
  bool bad = tid == 0 && offsets[0] != start;
#pragma unroll
  for (int k = 0; k < PER; ++k) {
    const int g = tid * PER + k;
    bound[k] = max(bound[k], before);
    if (g < groups) {
      t.bound[g + 1] = bound[k];
      bad |= given[k] != bound[k];
    }
  }
  if (tid == 0) t.bound[0] = start;
  if (report && bad) report_error(err, MOE_DEVERR_BOUNDS);
  __syncthreads();
  int tiles[PER], sum = 0;
#pragma unroll
  for (int k = 0; k < PER; ++k) {
    const int g = tid * PER + k;
    tiles[k] = g < groups ? (t.bound[g + 1] - t.bound[g] + tile_rows - 1) / tile_rows : 0;
    sum += tiles[k];
  }
  int total;
  int at = block_exclusive_scan(sum, scratch, &total);
#pragma unroll
  for (int k = 0; k < PER; ++k) {
    const int g = tid * PER + k;
    if (g < groups) t.first[g] = at;
    at += tiles[k];
  }
  if (tid == 0) t.first[groups] = total;
  __syncthreads();
}

constexpr int kPlanThreads = 256;

struct PlanTask {
  const int32_t* offsets;
  GroupPlan plan;
  int rows, groups, tile_rows;
  int blocks;  // of kPlanThreads, 0: no plan
  unsigned* err;
  CUtensorMap tm_a, tm_b;  // whole operands of the weight gradient
};

// Fills in the task; with `weight_grad` (may be null) its operands' maps are made, too.  False where
// those cannot be encoded.
bool group_plan_task(const int32_t* offsets, int rows, int groups, int tile_rows,
                     const GroupPlan& plan, const GroupedProduct* weight_grad, unsigned* err,
                     PlanTask* task);

// Every block makes the table for itself; they share its tiles and the groups' tensor maps, and
// block 0 writes the bounds.
__device__ __forceinline__ void plan_block(const PlanTask& p, int block) {
  __shared__ int s_bound[kMostGroups + 1], s_first[kMostGroups + 1];
  __shared__ int scratch[32];
  __shared__ alignas(128) uint32_t s_map[kPlanThreads / 32][32];
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const Table table{s_bound, s_first};
  make_table<kMostGroups / kPlanThreads>(p.offsets, p.rows, p.groups, p.tile_rows, table, scratch,
                                         block == 0, p.err);
  const int total = s_first[p.groups];
  if (block == 0) {
    if (t == 0) *p.plan.count = total;
    for (int g = t; g <= p.groups; g += kPlanThreads) p.plan.bounds[g] = s_bound[g];
  }
  for (int i = block * kPlanThreads + t; i < total; i += p.blocks * kPlanThreads)
    p.plan.tiles[i] = table_entry(table, p.groups, i, p.tile_rows);
  if (p.plan.maps == nullptr) return;
  constexpr int kWarps = kPlanThreads / 32;
  for (int i = block * kWarps + warp; i < 2 * p.groups; i += p.blocks * kWarps) {
    const CUtensorMap* from = i & 1 ? &p.tm_b : &p.tm_a;
    s_map[warp][lane] = reinterpret_cast<const uint32_t*>(from)[lane];
    __syncwarp();
    const uint32_t sm = smem_u32(s_map[warp]);
    if (lane == 0) {
      // (a map with no rows is never used)
      asm volatile("tensormap.replace.tile.global_dim.shared::cta.b1024.b32 [%0], 1, %1;" ::"r"(sm),
                   "r"(max(s_bound[(i >> 1) + 1], 1))
                   : "memory");
    }
    __syncwarp();
    asm volatile(
        "tensormap.cp_fenceproxy.global.shared::cta.tensormap::generic.release.gpu.sync.aligned "
        "[%0], [%1], 128;" ::"l"(reinterpret_cast<uint64_t>(
            static_cast<CUtensorMap*>(p.plan.maps) + i)),
        "r"(sm)
        : "memory");
    __syncwarp();
  }
}

}  // namespace moe
