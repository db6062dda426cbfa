// The matrix products grouped by expert on the 5th-generation tensor cores: the forward, the
// gradient of its input and the gradient of the weights, over groups of rows whose sizes are known
// on the device only.
//
//   forward          C_r  = sum_k A[r,k] B_g[f,k]      rows r of group g; reduction over inputs
//   input gradient   C_r  = sum_n A[r,n] B_g[n,f]      the same rows; reduction over outputs
//   weight gradient  C_g  = sum_r A[r,n] B[r,f]        reduction over the group's rows
//
// Two persistent kernels (grouped_kernel in several forms): TMA loads either operand layout in
// 128-byte swizzled boxes (k-contiguous, or row-contiguous for the weights of the input gradient and
// both operands of the weight gradient) and the descriptors name the layout, so nothing is transposed
// in memory.
//  - Tiles of rows start at a group's first row and run over its end; the rows past it belong to
//    the next group (a row of the result depends on its own row of A alone) and are not stored.
//  - The reduction of the weight gradient must end with the group: what follows may be another
//    group's infinity or NaN, so masking one operand would not do.  Every group has its own pair
//    of tensor maps, copies of the call's maps whose number of rows is the group's end: TMA then
//    fills the rest of the block that the end cuts with zeros.  The plan kernel writes them; the
//    blocks before the last use the call's own.
//  - A float32 result leaves the tensor core every 256 values (many rows a group, one part: 512;
//    float32 operands, six products per value: 64), a bf16 one every 16384 (two parts: 8192), and
//    is added up in registers: the tensor core truncates its additions.
//
// Kernels, by the mean number of rows a group has (known on the host: rows and groups):
//  - grouped_wide_kernel, over 64: CTA pairs, 256 features x up to 256 rows (see there).  8192
//    tokens of 8 experts of 128, 2048 -> 2 x 768 with SwiGLU: 288 us, 1,430 TFLOP/s, the tensor pipe
//    77% busy; rows that fill their tiles (8 groups of 1024, 14336 <-> 4096) run at 1,800 to 1,900;
//  - grouped_kernel<1, 32 or 64, .., swapped>, to 32 and to 64: single CTAs, the weights on the
//    side of 128, bound by the weights' read (512 rows over 119 of 128 groups, 768 -> 2048: 6.0 TB/s).
//    They plan for themselves: a launch of its own took 1.8 us of one token's 15.4.  (rows / groups is
//    what the buffers hold: 8 rows of 128 groups take 10.6 us in buffers of 8 to 4096 rows, 16.5 in
//    those of 9000 and more, with the weights in L2);
//  - grouped_kernel<2, 256, 1 or 2, ..>: CTA pairs for bf16 weight gradients, 256 x 256 tiles.  Bound
//    by writing: 805 MB take 201 us by themselves here, 356 us with 412 GFLOP, 226 without the stores;
//    two parts (825 GFLOP) 517;
//  - grouped_kernel<1, 128, 3, 3>: float32 operands in three parts, all three products.
// The kernels on CTA pairs hold a tile's sums in 128 registers of an epilogue thread's 168 and spill
// around them (108 bytes in the wide one, 140 in the weight gradients').
#include <algorithm>
#include <cstring>
#include <type_traits>

#include "common.cuh"
#include "grouped.h"
#include "grouped_plan.cuh"
#include "linear_act.cuh"
#include "tc_operand.cuh"

namespace moe {
namespace {

constexpr int BK = 64;
// K-blocks per accumulator: of a bf16 result, of a float one, of a float one of many rows a group, of
// float operands.  An accumulator of values of one sign falls short by up to 6.2e-9 of its size per
// value: 1.6e-6 over 256 values, 3.2e-6 over 512.  Few rows wait for the weights' read, so every 256
// values cost them nothing (63.1 us and 63.3, 512 rows of 119 groups, 768 -> 2048); in the wide kernel
// they would cost a forward of 65536 rows of these 253 -> 323 us.  With dz in three parts, whose
// products are added up in the same accumulator, the error would be 1.7e-6 in relative L2 after 512
// values, after 256 8.1e-7 (1,485 and 1,527 us for the gradients of 8192 tokens' gate/up).  Float32
// operands every 64 values: 1.0e-7 of the result in the root mean square, 5.9e-7 every 128, for 1 to
// 6% of the time.
constexpr int kMaxChunk = 256, kFloatChunk = 4, kWideFloatChunk = 8, kPartsChunk = 1;

// PA, PB: bf16 parts per value on the A and on the B side.
template <int CTAS, int BN, int PA, int PB, bool SWAP>
struct GroupedCfg {
  static constexpr int kEpiWarps = 8;
  static constexpr int kThreads = 64 + 32 * kEpiWarps;
  static constexpr int kBRows = BN / CTAS;
  static constexpr int kABytes = 128 * BK * 2, kBBytes = kBRows * BK * 2;
  static constexpr int kStageBytes = PA * kABytes + PB * kBBytes;
  static constexpr int kStgBytes = SWAP ? 0 : kEpiWarps * 4096;  // 32 rows of 128 bytes per warp
  static constexpr int kBarBytes = 256;
  // the groups' bounds and first tiles, where the kernel plans for itself
  static constexpr int kTableBytes = SWAP ? 2 * (kMostGroups + 4) * 4 + 128 : 0;
  static constexpr int kRaw =
      (232448 - 1024 - kBarBytes - kStgBytes - kTableBytes) / kStageBytes;
  static constexpr int kStages = kRaw > 12 ? 12 : kRaw;
  static constexpr int kSmem = 1024 + kStages * kStageBytes + kStgBytes + kBarBytes + kTableBytes;
  static constexpr int kTmemCols = 2 * BN;
  static constexpr int kTileRows = SWAP ? BN : 128 * CTAS;
  static constexpr int kTileFeatures = SWAP ? 128 : BN;
  static_assert(8 * (2 * kStages + 5) + 8 <= kBarBytes, "barrier region");
};

struct GroupedParams {
  CUtensorMap tm_a, tm_b;  // as the sides of the tile: with swapped sides A is the weights
  CUtensorMap tm_c, tm_z;
  CUtensorMap tm_rows[3];  // wide kernel: B's map with boxes of 64, 32 and 16 rows (tm_b: 128)
  int w_blocks;            // swapped sides, swiglu: tm_a takes both halves' blocks of 16 rows
  GroupPlan plan;
  GroupedKind kind;
  int groups, total_rows, num_kb, chunk;
  int tiles_a;       // weight gradient: tiles along the rows of C_g
  int tiles_b;       // tiles along the features
  int feat_step;     // features of C per tile
  int quads;         // swapped sides: the tile's rows of weights, in 32
  int rows;          // weight gradient: rows of C_g
  int features, swiglu;
  int a_mn, b_mn;
  int a_step, b_step;  // third coordinate per plane (weights: groups, activations: 1)
  void* c;
  void* z;
  long long ldc, c_group, ldz;
  int c_f32, tma_c, tma_z, vec_c, vec_z;
  unsigned* err;
};

// The products of a launch: one, or both gradients of a float32 layer, whose tiles follow one another
// (517 rows of 7 groups, 333 -> 201: 33 tiles of dx and 84 of dw; one after the other 43 us a call
// instead of 27.5).
template <int N>
struct GroupedJobs {
  GroupedParams p[N];
  int count;
};

struct Tile {
  int group, row0, row_end, feat0;
  int rows;        // of the tile (forward and input gradient)
  int k0, num_kb;  // first row of the reduction (weight gradient), k-blocks
  int cut_kb;      // the block that the group's end cuts (weight gradient), or -1
};

__device__ __forceinline__ int total_tiles(const GroupedParams& p, const Table& table) {
  if (p.kind == GroupedKind::kWeightGrad) return p.groups * p.tiles_a * p.tiles_b;
  return (table.bound != nullptr ? table.first[p.groups] : *p.plan.count) * p.tiles_b;
}

// What tile idx's place is read from, to be loaded while the tile before it is worked on: the
// table's entry of its rows, or (weight gradient) the ends of its group.
template <typename Cfg>
__device__ __forceinline__ int4 fetch_tile(const GroupedParams& p, const Table& table, int idx) {
  if (table.bound != nullptr)
    return table_entry(table, p.groups, idx / p.tiles_b, Cfg::kTileRows);
  if (p.kind != GroupedKind::kWeightGrad) return p.plan.tiles[idx / p.tiles_b];
  const int g = idx / (p.tiles_a * p.tiles_b);
  return make_int4(p.plan.bounds[g], p.plan.bounds[g + 1], g, 0);
}

// Tiles of up to kRowChunk tiles of rows of a group share every tile of features in turn.
// row_end is not set in a ragged product: row_end_of.
template <typename Cfg>
__device__ __forceinline__ Tile tile_at(const GroupedParams& p, int idx, const int4& e) {
  Tile t;
  if (p.kind != GroupedKind::kWeightGrad) {
    const int in = idx - e.z * p.tiles_b;
    const int tiles = e.w & 15, f = in / tiles;
    t.group = e.x;
    t.rows = e.w >> 4;
    t.row0 = e.y + (in - f * tiles) * t.rows;
    t.row_end = 0;
    t.feat0 = f * p.feat_step;
    t.k0 = 0;
    t.num_kb = p.num_kb;
    t.cut_kb = -1;
  } else {
    const int per = p.tiles_a * p.tiles_b;
    t.group = e.z;
    t.rows = 0;
    const int in = idx - t.group * per;
    const int c = in / (kRowChunk * p.tiles_b);
    const int rest = in - c * kRowChunk * p.tiles_b;
    const int h = min(kRowChunk, p.tiles_a - c * kRowChunk);
    const int f = rest / h;
    t.row0 = (c * kRowChunk + rest - f * h) * Cfg::kTileRows;
    t.row_end = p.rows;
    t.feat0 = f * p.feat_step;
    t.k0 = e.x;
    const int size = e.y - t.k0;
    t.num_kb = (size + BK - 1) / BK;
    t.cut_kb = size % BK != 0 ? t.num_kb - 1 : -1;
  }
  return t;
}

__device__ __forceinline__ int row_end_of(const GroupedParams& p, const Table& table,
                                          const Tile& t) {
  if (table.bound != nullptr) return table.bound[t.group + 1];
  return p.kind == GroupedKind::kWeightGrad ? p.rows : p.plan.bounds[t.group + 1];
}

// ------------------------------------------------------------------- loading ----

template <int CTAS>
__device__ __forceinline__ void load_box(uint32_t dst, const void* map, uint32_t bar, int c0,
                                         int c1, int c2) {
  if constexpr (CTAS == 2) tma_load_3d_pair(dst, map, bar, c0, c1, c2);
  else tma_load_3d(dst, map, bar, c0, c1, c2);
}

// One k-block (from k on) of ROWS operand rows from row on.
template <int CTAS, int ROWS>
__device__ __forceinline__ void load_rows(uint32_t dst, const void* map, uint32_t bar, int mn,
                                          int row, int k, int third) {
  if (!mn) {
    load_box<CTAS>(dst, map, bar, k, row, third);
  } else {
#pragma unroll
    for (int c = 0; c < ROWS; c += 64) load_box<CTAS>(dst + c * 128u, map, bar, row + c, k, third);
  }
}

__device__ __forceinline__ void acquire_map(const void* map) {
  asm volatile("fence.proxy.tensormap::generic.acquire.gpu [%0], 128;" ::"l"(
                   reinterpret_cast<uint64_t>(map))
               : "memory");
}

// ------------------------------------------------------------------- storing ----

__device__ __forceinline__ void tma_store_3d(const void* map, uint32_t src, int c0, int c1,
                                             int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
          reinterpret_cast<uint64_t>(map)),
      "r"(src), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}
__device__ __forceinline__ void bulk_commit() {
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}
__device__ __forceinline__ void bulk_wait_read_but_one() {
  asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
}
__device__ __forceinline__ void bulk_wait() {
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}
__device__ __forceinline__ void fence_async_shared() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// tcgen05.ld into floats; the values are there after tmem_ld_wait.  keep and after_wait hold their
// uses behind that wait, which does not name the registers.
__device__ __forceinline__ void tmem_ld_columns(uint32_t addr, float (&v)[32]) {
  tmem_ld_32x32b_x32(addr, reinterpret_cast<uint32_t (&)[32]>(v));
}
__device__ __forceinline__ void tmem_ld_columns(uint32_t addr, float (&v)[16]) {
  tmem_ld_32x32b_x16(addr, reinterpret_cast<uint32_t (&)[16]>(v));
}
__device__ __forceinline__ float after_wait(float v) {
  asm volatile("" : "+f"(v));
  return v;
}
__device__ __forceinline__ void tmem_ld_fragments(uint32_t addr, float (&v)[32], int at) {
  uint32_t r[16];
  tmem_ld_16x256b_x4(addr, r);
#pragma unroll
  for (int q = 0; q < 16; ++q) v[at + q] = __uint_as_float(r[q]);
}
template <int A, int B>
__device__ __forceinline__ void keep(float (&v)[A][B]) {
#pragma unroll
  for (int i = 0; i < A; ++i)
#pragma unroll
    for (int q = 0; q < B; ++q) asm volatile("" : "+f"(v[i][q]));
}

// A staged piece: rows of 128 bytes, the 16-byte parts of row r at part ^ (r & 7), which is TMA's
// 128-byte swizzle.  (Rows of 64 bytes leave no faster than those of 128: half the rate.)
// A lane's own row: 32 floats, or 32 values in bf16 from part c0 on.
__device__ __forceinline__ void stage_f32(uint8_t* stg, int lane, const float (&v)[32]) {
#pragma unroll
  for (int c = 0; c < 8; ++c)
    *reinterpret_cast<float4*>(stg + lane * 128 + ((c ^ (lane & 7)) << 4)) =
        make_float4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void stage_bf16(uint8_t* stg, int lane, int c0, const float (&v)[32]) {
#pragma unroll
  for (int c = 0; c < 4; ++c)
    *reinterpret_cast<uint4*>(stg + lane * 128 + (((c0 + c) ^ (lane & 7)) << 4)) =
        make_uint4(pack2(v[8 * c], v[8 * c + 1]), pack2(v[8 * c + 2], v[8 * c + 3]),
                   pack2(v[8 * c + 4], v[8 * c + 5]), pack2(v[8 * c + 6], v[8 * c + 7]));
}

// Where a piece of an output goes: rows of a group's matrix (C, third = the group), or of one half
// of z, whose map has the halves before the rows (third = the half).
struct Out {
  const CUtensorMap* map;
  char* base;  // of the group or half
  long long ld;
  int cols, third, is_z, tma, vec;
};

// Rows first.. of a staged piece (`count` of them) to memory, eight lanes to a row.
template <typename T>
__device__ __forceinline__ void copy_rows(const Out& o, const uint8_t* stg, int lane, int first,
                                          int count, int row0, int row_end, int col) {
  constexpr int N = 16 / static_cast<int>(sizeof(T));
  const int part = lane & 7, c = col + part * N;
  const int n = min(N, o.cols - c);
#pragma unroll 1
  for (int r = first + (lane >> 3); r < first + count; r += 4) {
    if (row0 + r >= row_end || n <= 0) break;
    const uint8_t* src = stg + r * 128 + ((part ^ (r & 7)) << 4);
    T* dst = reinterpret_cast<T*>(o.base) + static_cast<long long>(row0 + r) * o.ld + c;
    if (o.vec && n == N) {
      *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(src);
    } else {
      for (int q = 0; q < n; ++q) dst[q] = reinterpret_cast<const T*>(src)[q];
    }
  }
}

// Whether TMA may take a piece from column col on: it clips columns past the end in 16-byte steps
// only, so a row that ends inside one is left to the lanes.
template <typename T>
__device__ __forceinline__ bool tma_takes(const Out& o, int col) {
  constexpr int N = 16 / static_cast<int>(sizeof(T));
  return o.tma && (col + 8 * N <= o.cols || o.cols % N == 0);
}

// A warp's staged piece to rows row0.. (below row_end) and columns col.. of the output: by TMA
// where all 32 rows are the group's, else by the lanes.
template <typename T>
__device__ __forceinline__ void put_piece(const Out& o, uint8_t* stg, int lane, int row0,
                                          int row_end, int col, bool whole) {
  if (whole && tma_takes<T>(o, col)) {
    fence_async_shared();
    __syncwarp();
    if (lane == 0) {
      tma_store_3d(o.map, smem_u32(stg), col, o.is_z ? o.third : row0, o.is_z ? row0 : o.third);
      bulk_commit();
    }
    return;
  }
  __syncwarp();
  copy_rows<T>(o, stg, lane, 0, 32, row0, row_end, col);
}

// Sixteen rows of the wide kernel's fragments in float: rows 8 j0.. of the 32, 16 or 32 lanes, lane
// f of them at float f0 + f of a row of the piece.
__device__ __forceinline__ void put_f32(uint8_t* at, int lane, int f0, const float (&v)[32], int j0,
                                        int first_row, int lanes) {
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    if (16 * half >= lanes) break;
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {  // e & 1: the row, e >> 1: lanes 8 on
        const int f = f0 + 16 * half + 8 * (e >> 1) + (lane >> 2);
        const int row = first_row + 8 * j + 2 * (lane & 3) + (e & 1);
        *reinterpret_cast<float*>(at + row * 128 + (((f >> 2) ^ (row & 7)) << 4) +
                                  (f & 3) * 4) = v[16 * half + 4 * (j0 + j) + e];
      }
  }
}

// -------------------------------------------------------------------- kernel ----

// Products that a launch takes, by the parts of A.
template <int PA>
constexpr int kMostJobs = PA == 3 ? 2 : 1;

// A float32 product lets the next launch start at its end.  At its start the blocks of the next call's
// packing would all come to lie on the SMs that its tiles leave idle, and pack from there: 517 rows
// of 7 groups, 333 -> 201, gradients 32.6 us a call, with the trigger at the end 27.5.
template <int PA>
constexpr bool kLateTrigger = PA == 3;

template <int CTAS, int BN, int PA, int PB, bool SWAP>
__global__ void __launch_bounds__(GroupedCfg<CTAS, BN, PA, PB, SWAP>::kThreads, 1)
    grouped_kernel(const __grid_constant__ GroupedJobs<kMostJobs<PA>> jobs) {
  using Cfg = GroupedCfg<CTAS, BN, PA, PB, SWAP>;
  constexpr int S = Cfg::kStages;
  // what a kernel of this form is launched for
  static_assert(SWAP ? CTAS == 1 && PA == 1 : (CTAS == 2 && PB == 1) || (PA == 3 && PB == 3), "form");
  auto is_weight_grad = [](const GroupedParams& p) {  // CTA pairs: always; swapped sides: never
    return CTAS == 2 || (!SWAP && p.kind == GroupedKind::kWeightGrad);
  };
  auto with_swiglu = [](const GroupedParams& p) { return CTAS == 1 && p.swiglu != 0; };
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* stg_all = smem + S * Cfg::kStageBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(stg_all + Cfg::kStgBytes);
  const uint32_t bar0 = smem_u32(bars);
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (S + s); };
  auto tfull_bar = [&](int a) { return bar0 + 8u * (2 * S + a); };
  auto tempty_bar = [&](int a) { return bar0 + 8u * (2 * S + 2 + a); };
  const uint32_t mma_done_bar = bar0 + 8u * (2 * S + 4);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * S + 5);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = CTAS == 2 ? cluster_ctarank() : 0;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(tfull_bar(a), 1);
      mbar_init(tempty_bar(a), CTAS * Cfg::kEpiWarps);
    }
    mbar_init(mma_done_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&jobs.p[0].tm_a);
    tma_prefetch_desc(&jobs.p[0].tm_b);
    if (!SWAP && jobs.p[0].tma_c) tma_prefetch_desc(&jobs.p[0].tm_c);
  }
  if (warp == 1) {
    if constexpr (CTAS == 2) {
      tmem_alloc_pair(smem_u32(tmem_slot), Cfg::kTmemCols);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(smem_u32(tmem_slot), Cfg::kTmemCols);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (CTAS == 2) cluster_sync_all();  // the peer's barriers exist before use
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  // (CTA pairs run in stream order, without overlap on either side)
  if constexpr (CTAS == 1) {
    grid_dep_wait();
    if constexpr (!kLateTrigger<PA>) grid_dep_trigger();
  }
  unsigned* const err = jobs.p[0].err;
  Table table{nullptr, nullptr};
  if constexpr (SWAP) {
    const GroupedParams& p = jobs.p[0];
    if (p.plan.offsets != nullptr) {
      int* room = reinterpret_cast<int*>(stg_all + Cfg::kStgBytes + Cfg::kBarBytes);
      table.bound = room + 32;
      table.first = table.bound + kMostGroups + 4;
      constexpr int kPer = (kMostGroups + Cfg::kThreads - 1) / Cfg::kThreads;
      make_table<kPer>(p.plan.offsets, p.total_rows, p.groups, Cfg::kTileRows, table, room,
                       blockIdx.x == 0, err);
    }
  }

  // tiles of the first product, and of all
  const int total0 = total_tiles(jobs.p[0], table);
  int total = total0;
  if constexpr (kMostJobs<PA> == 2) {
    if (jobs.count == 2) total += total_tiles(jobs.p[1], table);
  }
  // The product of tile *idx, which becomes its number in that product.
  auto job_of = [&](int* idx) -> const GroupedParams& {
    if constexpr (kMostJobs<PA> == 2) {
      if (*idx >= total0) {
        *idx -= total0;
        return jobs.p[1];
      }
    }
    return jobs.p[0];
  };
  auto fetch = [&](int idx) {
    const GroupedParams& p = job_of(&idx);
    return fetch_tile<Cfg>(p, table, idx);
  };
  const int first = static_cast<int>(blockIdx.x) / CTAS;
  const int step = static_cast<int>(gridDim.x) / CTAS;

  if (warp == 0) {
    // ------------------------------------------------------------ producer ----
    const bool leader = elect_one_sync();
    int stage = 0, issued = 0;  // (issued stops counting at S)
    uint32_t phase = 0;
    if (leader) {
      bool ok = true;
      int4 entry = first < total ? fetch(first) : int4{};
      for (int idx = first; ok && idx < total; idx += step) {
        int at = idx;
        const GroupedParams& p = job_of(&at);
        const Tile t = tile_at<Cfg>(p, at, entry);
        if (idx + step < total) entry = fetch(idx + step);
        const CUtensorMap* tm_a = &p.tm_a;
        const CUtensorMap* tm_b = &p.tm_b;
        int a_row = t.row0 + static_cast<int>(rank) * 128, a_third = 0;
        int b_row = t.feat0 + static_cast<int>(rank) * Cfg::kBRows, b_third = 0;
        if constexpr (SWAP) {
          a_row = t.feat0;
          b_row = t.row0;
          a_third = t.group;
        } else if (!is_weight_grad(p)) {
          b_third = t.group;
        }
        for (int kb = 0; kb < t.num_kb; ++kb) {
          if (!mbar_wait(empty_bar(stage), phase ^ 1u, abort_flag, err)) {
            ok = false;
            break;
          }
          if (kb == t.cut_kb) {
            tm_a = static_cast<const CUtensorMap*>(p.plan.maps) + 2 * t.group;
            tm_b = tm_a + 1;
            acquire_map(tm_a);
            acquire_map(tm_b);
          }
          const uint32_t fb = CTAS == 2 ? mapa_shared(full_bar(stage), 0) : full_bar(stage);
          const uint32_t dst = smem_u32(smem) + stage * Cfg::kStageBytes;
          const int bytes = SWAP ? PA * p.quads * 4096 + PB * Cfg::kBBytes : CTAS * Cfg::kStageBytes;
          if (rank == 0) mbar_arrive_expect_tx(full_bar(stage), static_cast<uint32_t>(bytes));
          const int k = t.k0 + kb * BK;
#pragma unroll
          for (int pl = 0; pl < PA; ++pl) {
            const uint32_t da = dst + pl * Cfg::kABytes;
            const int ta = a_third + pl * p.a_step;
            if constexpr (SWAP) {
              if (p.w_blocks) {  // 16 gate rows, then the same 16 up rows, for each 32 lanes
                tma_load_5d(da, tm_a, fb, k, 0, 0, a_row >> 4, ta);
              } else if (p.swiglu) {
                for (int q = 0; q < p.quads; ++q) {
                  load_box<CTAS>(da + q * 4096u, tm_a, fb, k, a_row + 16 * q, ta);
                  load_box<CTAS>(da + q * 4096u + 2048u, tm_a, fb, k, p.features + a_row + 16 * q,
                                 ta);
                }
              } else if (p.quads > 2) {
                load_rows<CTAS, 128>(da, tm_a, fb, p.a_mn, a_row, k, ta);
              } else {
                load_rows<CTAS, 64>(da, tm_a, fb, p.a_mn, a_row, k, ta);
              }
            } else {
              load_rows<CTAS, 128>(da, tm_a, fb, p.a_mn, a_row, k, ta);
            }
          }
#pragma unroll
          for (int pl = 0; pl < PB; ++pl) {
            const uint32_t db = dst + PA * Cfg::kABytes + pl * Cfg::kBBytes;
            const int tb = b_third + pl * p.b_step;
            if constexpr (SWAP) {
              load_box<CTAS>(db, tm_b, fb, k, b_row, tb);
            } else if (with_swiglu(p)) {  // gate and up halves of the tile
              load_box<CTAS>(db, tm_b, fb, k, b_row, tb);
              load_box<CTAS>(db + Cfg::kBBytes / 2, tm_b, fb, k, p.features + b_row, tb);
            } else {
              load_rows<CTAS, Cfg::kBRows>(db, tm_b, fb, p.b_mn, b_row, k, tb);
            }
          }
          issued = min(issued + 1, S);
          if (++stage == S) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
    }
    __syncwarp();
    // (both CTAs' loads complete on the even CTA's barriers)
    drain_stages<S>(leader, lane, stage, phase, issued, empty_bar, full_bar, rank == 0, abort_flag,
                    err);
  } else if (warp == 1) {
    // ----------------------------------------------------------------- MMA ----
    if (rank == 0 && elect_one_sync()) {
      auto commit = [&](uint32_t bar) {
        if constexpr (CTAS == 2) tc_commit_pair(bar, 0x3);
        else tc_commit(bar);
      };
      int stage = 0;
      uint32_t phase = 0;
      int local = 0;  // accumulators filled
      bool ok = true;
      int4 entry = first < total ? fetch(first) : int4{};
      for (int idx = first; ok && idx < total; idx += step) {
        int at = idx;
        const GroupedParams& p = job_of(&at);
        const int num_kb = tile_at<Cfg>(p, at, entry).num_kb;
        const uint32_t idesc = idesc_bf16_f32(128 * CTAS, BN) |
                               (static_cast<uint32_t>(p.a_mn) << 15) |
                               (static_cast<uint32_t>(p.b_mn) << 16);
        const uint32_t a_step = p.a_mn ? 2048u : 32u, b_step = p.b_mn ? 2048u : 32u;
        if (idx + step < total) entry = fetch(idx + step);
        for (int kb = 0; ok && kb < num_kb; ++local) {
          const int acc = local & 1;
          if (!mbar_wait(tempty_bar(acc), (static_cast<uint32_t>(local >> 1) & 1u) ^ 1u, abort_flag,
                         err)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t d = tmem_base + static_cast<uint32_t>(acc * BN);
          const int end = min(num_kb, kb + p.chunk);
          uint32_t accumulate = 0;
          for (; kb < end; ++kb) {
            if (!mbar_wait(full_bar(stage), phase, abort_flag, err)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t a_base = smem_u32(smem) + stage * Cfg::kStageBytes;
            const uint32_t b_base = a_base + PA * Cfg::kABytes;
            // smallest products first; of three parts each, those above 2^-24
            constexpr bool kThree = PA == 3 && PB == 3;
            constexpr int kTerms = kThree ? 6 : PA * PB;
            constexpr int pa[6] = {2, 1, 0, 1, 0, 0}, pb[6] = {0, 1, 2, 0, 1, 0};
            static_assert(kThree || PA == 1 || PB == 1, "parts");
#pragma unroll
            for (int q = 0; q < kTerms; ++q) {
              const int qa = kThree ? pa[q] : PA - 1 - (PA > 1 ? q : 0);
              const int qb = kThree ? pb[q] : PB - 1 - (PB > 1 ? q : 0);
#pragma unroll
              for (int kk = 0; kk < BK / 16; ++kk) {
                const uint64_t da = operand_desc(a_base + qa * Cfg::kABytes + kk * a_step, p.a_mn);
                const uint64_t db = operand_desc(b_base + qb * Cfg::kBBytes + kk * b_step, p.b_mn);
                if constexpr (CTAS == 2) tc_mma_bf16_pair(d, da, db, idesc, accumulate);
                else tc_mma_bf16(d, da, db, idesc, accumulate);
                accumulate = 1u;
              }
            }
            commit(empty_bar(stage));
            if (++stage == S) {
              stage = 0;
              phase ^= 1u;
            }
          }
          if (ok) commit(tfull_bar(acc));
        }
      }
      if (!ok || *abort_flag) {
        if constexpr (CTAS == 2) tc_commit_pair(mma_done_bar, 0x1);
        else tc_commit(mma_done_bar);
        volatile int no_abort = 0;
        mbar_wait(mma_done_bar, 0, &no_abort, err);
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue ----
    const int quad = warp & 3, part = (warp - 2) >> 2;
    constexpr int W = BN / (Cfg::kEpiWarps / 4);  // columns of the accumulator that a warp takes
    constexpr int P = W >= 32 ? 32 : W;           // columns per load
    constexpr int NP = W / P;
    int local = 0;  // accumulators read
    float sum[NP][P];
    int4 entry = first < total ? fetch(first) : int4{};
    for (int idx = first; idx < total; idx += step) {
      int at = idx;
      const GroupedParams& p = job_of(&at);
      Tile t = tile_at<Cfg>(p, at, entry);
      t.row_end = row_end_of(p, table, t);
      if (idx + step < total) entry = fetch(idx + step);
      bool ok = true;
      if (t.num_kb == 0) {
#pragma unroll
        for (int i = 0; i < NP; ++i)
#pragma unroll
          for (int q = 0; q < P; ++q) sum[i][q] = 0.f;
      }
      for (int kb = 0; kb < t.num_kb; kb += p.chunk, ++local) {
        const bool ready = mbar_wait(tfull_bar(local & 1), static_cast<uint32_t>(local >> 1) & 1u,
                                     abort_flag, err);
        ok = !__any_sync(0xffffffffu, !ready);
        if (!ok) break;
        tc_fence_after();
        const uint32_t acc = tmem_base + (static_cast<uint32_t>(quad * 32) << 16) +
                             static_cast<uint32_t>((local & 1) * BN);
        // with swiglu (sides not swapped) the first half of a warp's columns are the gate's
        auto column = [&](int i) {
          return !SWAP && with_swiglu(p) ? (i / ((NP + 1) / 2)) * W + part * (W / 2) +
                                         (i % ((NP + 1) / 2)) * P
                                   : part * W + i * P;
        };
        if (kb == 0) {  // straight into the sums, all on their way at once
#pragma unroll
          for (int i = 0; i < NP; ++i) tmem_ld_columns(acc + column(i), sum[i]);
          tmem_ld_wait();
          keep(sum);
        } else {
#pragma unroll
          for (int i = 0; i < NP; ++i) {
            float r[P];
            tmem_ld_columns(acc + column(i), r);
            tmem_ld_wait();
#pragma unroll
            for (int q = 0; q < P; ++q) sum[i][q] += after_wait(r[q]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if constexpr (CTAS == 2) mbar_arrive_cluster(mapa_shared(tempty_bar(local & 1), 0));
          else mbar_arrive(tempty_bar(local & 1));
        }
      }
      if (!ok) break;

      if constexpr (SWAP) {
        // lanes are features, columns are rows of the groups
        if (quad >= p.quads) continue;  // (lanes whose weights were not loaded)
        const int f = p.swiglu ? t.feat0 + quad * 16 + (lane & 15) : t.feat0 + quad * 32 + lane;
#pragma unroll
        for (int q = 0; q < W; ++q) {
          const int row = t.row0 + part * W + q;
          if (row >= t.row_end) break;
          float v = sum[q / P][q % P];
          if (p.swiglu) {
            const float other = __shfl_xor_sync(0xffffffffu, v, 16);
            if (p.z != nullptr && f < p.features) {
              const long long at = static_cast<long long>(row) * p.ldz + (lane >> 4) * p.features + f;
              static_cast<__nv_bfloat16*>(p.z)[at] = __float2bfloat16_rn(v);
            }
            v = act_value<true>(MOE_ACT_SILU, v) * other;
          }
          if (f < p.features && (!p.swiglu || lane < 16)) {
            const long long at = static_cast<long long>(row) * p.ldc + f;
            if (p.c_f32) static_cast<float*>(p.c)[at] = v;
            else static_cast<__nv_bfloat16*>(p.c)[at] = __float2bfloat16_rn(v);
          }
        }
      } else {
        uint8_t* stg = stg_all + (warp - 2) * 4096;
        const int row0 = t.row0 + static_cast<int>(rank) * 128 + quad * 32;
        if (row0 >= t.row_end) continue;
        const bool weight_grad = is_weight_grad(p);
        // rows past a weight's last are clipped by TMA, those past a group's end would not be
        const bool whole = weight_grad || row0 + 32 <= t.row_end;
        Out oc{&p.tm_c, static_cast<char*>(p.c), p.ldc, p.features, 0, 0, p.tma_c, p.vec_c};
        if (weight_grad) {
          oc.third = t.group;
          oc.base += static_cast<long long>(t.group) * p.c_group * (p.c_f32 ? 4 : 2);
        }
        // N times 32 columns, sum[I0..], to columns col.. of the output: float in three-part
        // products, else bf16
        auto emit = [&](const Out& o, int col, auto i0, auto n) {
          constexpr int I0 = decltype(i0)::value, N = decltype(n)::value;
          using T = std::conditional_t<PA == 3, float, __nv_bfloat16>;
#pragma unroll
          for (int i = 0; i < N; ++i) {
            if (col + 32 * i >= o.cols) break;
            if (PA != 3 && i % 2 != 0) continue;
            if (lane == 0) bulk_wait_read();  // the last piece has left the staging
            __syncwarp();
            if constexpr (PA == 3) {
              stage_f32(stg, lane, sum[I0 + i]);
            } else {
              stage_bf16(stg, lane, 0, sum[I0 + i]);
              stage_bf16(stg, lane, 4, sum[I0 + (i + 1) % N]);
            }
            put_piece<T>(o, stg, lane, row0, t.row_end, col + 32 * i, whole);
          }
        };
        using std::integral_constant;
        constexpr integral_constant<int, 0> zero{};
        constexpr integral_constant<int, NP / 2> mid{};
        constexpr integral_constant<int, NP> all{};
        if (!with_swiglu(p)) {
          emit(oc, t.feat0 + part * W, zero, all);
        } else if constexpr (CTAS == 1) {
          const int col = t.feat0 + part * (W / 2);
          if (p.z != nullptr) {
            Out oz{&p.tm_z, static_cast<char*>(p.z), p.ldz, p.features, 0, 1, p.tma_z, p.vec_z};
            emit(oz, col, zero, mid);
            oz.third = 1;
            oz.base += static_cast<long long>(p.features) * 4;
            emit(oz, col, mid, mid);
          }
#pragma unroll
          for (int i = 0; i < NP / 2; ++i)
#pragma unroll
            for (int q = 0; q < P; ++q)
              sum[i][q] = act_value<false>(MOE_ACT_SILU, sum[i][q]) * sum[i + NP / 2][q];
          emit(oc, col, zero, mid);
        }
      }
    }
    if (!SWAP && lane == 0) bulk_wait();
  }
  if constexpr (CTAS == 1 && kLateTrigger<PA>) grid_dep_trigger();
  tc_fence_before();
  __syncthreads();
  if constexpr (CTAS == 2) cluster_sync_all();  // no peer still reads or arrives here
  tc_fence_after();
  if (warp == 1) {
    if constexpr (CTAS == 2) tmem_dealloc_pair(tmem_base, Cfg::kTmemCols);
    else tmem_dealloc(tmem_base, Cfg::kTmemCols);
  }
  __syncwarp();
  if constexpr (CTAS == 2) cluster_sync_all();  // the pair gives its TMEM back before either leaves
}

// ------------------------------------------- weights on the side of 256 (pairs) ----

// The forward and the input gradient of groups with many rows.  A CTA pair's tile is 256 features
// (the weights are the MMA's A side) times a group's share of up to 256 rows in steps of 32: the
// MMA's N follows the group, so a group of 524 rows costs three tiles of 192 instead of three of
// 256.  Per stage 16 KB of weights and up to 16 KB (three parts: 48 KB) of rows in each CTA.
//
// The accumulator has features in its lanes and rows in its columns.  The epilogue reads it in 16 x
// 8 fragments and stores them transposed (stmatrix), 32 rows at a time, into 128-byte rows that TMA
// takes to memory; four warps (one per 32 lanes) share a piece, two such sets take turns.  With
// swiglu every 32 lanes are 16 gate features and the same 16 up features, so a thread has both.
template <int PB>
struct WideCfg {
  static constexpr int kEpiWarps = 8;
  static constexpr int kThreads = 64 + 32 * kEpiWarps;
  static constexpr int kABytes = 128 * BK * 2, kBBytes = 128 * BK * 2;
  static constexpr int kStageBytes = kABytes + PB * kBBytes;
  // a set's staging: two pieces of 32 rows x 128 features in bf16, or one in float
  static constexpr int kSetBytes = 16384;
  static constexpr int kStgBytes = kEpiWarps / 4 * kSetBytes;
  static constexpr int kBarBytes = 256;
  static constexpr int kStages = (232448 - 1024 - kBarBytes - kStgBytes) / kStageBytes;
  static constexpr int kSmem = 1024 + kStages * kStageBytes + kStgBytes + kBarBytes;
  static constexpr int kTileRows = kWideRows, kTileFeatures = 256;
  static constexpr int kTmemCols = 512;
};

// Four 8 x 8 matrices of 16-bit values, transposed: thread t holds of matrix i the values
// (row 2 (t % 4), column t / 4) and (row 2 (t % 4) + 1, column t / 4) in r[i] and gives, for
// i = t / 8, the address of row t % 8.
__device__ __forceinline__ void stmatrix_x4_trans(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                                  uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr),
               "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}

// Whether `ok` holds in all of the 128 threads that call it with barrier `id`.
__device__ __forceinline__ bool all_of_set(int id, bool ok) {
  uint32_t all;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 q, %1, 0;\n\t"
      "bar.red.and.pred p, %2, 128, q;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(all)
      : "r"(ok ? 1u : 0u), "r"(id)
      : "memory");
  return all != 0;
}

template <int PB>
__global__ void __launch_bounds__(WideCfg<PB>::kThreads, 1)
    grouped_wide_kernel(const __grid_constant__ GroupedParams p) {
  using Cfg = WideCfg<PB>;
  constexpr int S = Cfg::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* stg_all = smem + S * Cfg::kStageBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(stg_all + Cfg::kStgBytes);
  const uint32_t bar0 = smem_u32(bars);
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (S + s); };
  auto tfull_bar = [&](int a) { return bar0 + 8u * (2 * S + a); };
  auto tempty_bar = [&](int a) { return bar0 + 8u * (2 * S + 2 + a); };
  const uint32_t mma_done_bar = bar0 + 8u * (2 * S + 4);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * S + 5);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(tfull_bar(a), 1);
      mbar_init(tempty_bar(a), 2 * Cfg::kEpiWarps);
    }
    mbar_init(mma_done_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&p.tm_a);
    tma_prefetch_desc(&p.tm_b);
    if (p.tma_c) tma_prefetch_desc(&p.tm_c);
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(tmem_slot), Cfg::kTmemCols);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // the peer's barriers exist before anything arrives on them
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  const Table table{nullptr, nullptr};
  const int total = total_tiles(p, table);
  const int first = static_cast<int>(blockIdx.x) >> 1, step = static_cast<int>(gridDim.x) >> 1;

  if (warp == 0) {
    // ------------------------------------------------------------ producer ----
    const bool leader = elect_one_sync();
    int stage = 0, issued = 0;  // (issued stops counting at S)
    uint32_t phase = 0;
    if (leader) {
      bool ok = true;
      int4 entry = first < total ? fetch_tile<Cfg>(p, table, first) : int4{};
      for (int idx = first; ok && idx < total; idx += step) {
        const Tile t = tile_at<Cfg>(p, idx, entry);
        if (idx + step < total) entry = fetch_tile<Cfg>(p, table, idx + step);
        const int mine = t.rows >> 1;  // rows that this CTA loads
        const int x_row = t.row0 + rank * mine;
        const int w_row = t.feat0 + rank * (p.swiglu ? 64 : 128);
        // one box, of 16 to 128 rows: several smaller ones for the exact share cost more than the
        // rows they save (8192 rows in 8 groups, 14336 -> 4096: 648 us and 603)
        const int size = mine > 64 ? 0 : mine > 32 ? 1 : mine > 16 ? 2 : 3;
        const CUtensorMap* rows_map = size == 0 ? &p.tm_b : &p.tm_rows[size - 1];
        const uint32_t bytes = static_cast<uint32_t>(2 * (Cfg::kABytes + PB * ((128 >> size) * 128)));
        for (int kb = 0; kb < t.num_kb; ++kb) {
          if (!mbar_wait(empty_bar(stage), phase ^ 1u, abort_flag, p.err)) {
            ok = false;
            break;
          }
          const uint32_t fb = mapa_shared(full_bar(stage), 0);
          const uint32_t da = smem_u32(smem) + stage * Cfg::kStageBytes, db = da + Cfg::kABytes;
          if (rank == 0) mbar_arrive_expect_tx(full_bar(stage), bytes);
          const int k = kb * BK;
          if (p.w_blocks) {
            tma_load_5d_pair(da, &p.tm_a, fb, k, 0, 0, w_row >> 4, t.group);
          } else if (p.swiglu) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              tma_load_3d_pair(da + q * 4096u, &p.tm_a, fb, k, w_row + 16 * q, t.group);
              tma_load_3d_pair(da + q * 4096u + 2048u, &p.tm_a, fb, k, p.features + w_row + 16 * q,
                               t.group);
            }
          } else {
            load_rows<2, 128>(da, &p.tm_a, fb, p.a_mn, w_row, k, t.group);
          }
#pragma unroll
          for (int pl = 0; pl < PB; ++pl) {
            tma_load_3d_pair(db + pl * Cfg::kBBytes, rows_map, fb, k, x_row, pl);
          }
          issued = min(issued + 1, S);
          if (++stage == S) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
    }
    __syncwarp();
    // (both CTAs' loads complete on the even CTA's barriers)
    drain_stages<S>(leader, lane, stage, phase, issued, empty_bar, full_bar, rank == 0, abort_flag,
                    p.err);
  } else if (warp == 1) {
    // ----------------------------------------------------------------- MMA ----
    if (rank == 0 && elect_one_sync()) {
      const uint32_t a_step = p.a_mn ? 2048u : 32u;
      int stage = 0;
      uint32_t phase = 0;
      int local = 0;  // accumulators filled
      bool ok = true;
      int4 entry = first < total ? fetch_tile<Cfg>(p, table, first) : int4{};
      for (int idx = first; ok && idx < total; idx += step) {
        const Tile t = tile_at<Cfg>(p, idx, entry);
        if (idx + step < total) entry = fetch_tile<Cfg>(p, table, idx + step);
        const uint32_t idesc = idesc_bf16_f32(256, 0) | (static_cast<uint32_t>(p.a_mn) << 15) |
                               (static_cast<uint32_t>(t.rows >> 3) << 17);
        for (int kb = 0; ok && kb < t.num_kb; ++local) {
          const int acc = local & 1;
          if (!mbar_wait(tempty_bar(acc), (static_cast<uint32_t>(local >> 1) & 1u) ^ 1u, abort_flag,
                         p.err)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t d = tmem_base + static_cast<uint32_t>(acc * 256);
          const int end = min(t.num_kb, kb + p.chunk);
          uint32_t accumulate = 0;
          for (; kb < end; ++kb) {
            if (!mbar_wait(full_bar(stage), phase, abort_flag, p.err)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t a_base = smem_u32(smem) + stage * Cfg::kStageBytes;
            const uint32_t b_base = a_base + Cfg::kABytes;
#pragma unroll
            for (int pl = PB - 1; pl >= 0; --pl) {  // the smaller part first
#pragma unroll
              for (int kk = 0; kk < BK / 16; ++kk) {
                tc_mma_bf16_pair(d, operand_desc(a_base + kk * a_step, p.a_mn),
                                 operand_desc(b_base + pl * Cfg::kBBytes + kk * 32u, 0), idesc,
                                 accumulate);
                accumulate = 1u;
              }
            }
            tc_commit_pair(empty_bar(stage), 0x3);
            if (++stage == S) {
              stage = 0;
              phase ^= 1u;
            }
          }
          if (ok) tc_commit_pair(tfull_bar(acc), 0x3);
        }
      }
      if (!ok || *abort_flag) {
        tc_commit_pair(mma_done_bar, 0x1);
        volatile int no_abort = 0;
        mbar_wait(mma_done_bar, 0, &no_abort, p.err);
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue ----
    const int quad = warp & 3, set = (warp - 2) >> 2;
    constexpr int kSets = Cfg::kEpiWarps / 4, NS = 8 / kSets;  // steps of 32 rows per set
    uint8_t* const stg_set = stg_all + set * Cfg::kSetBytes;
    uint8_t* stg = stg_set;
    const bool big = p.c_f32 && !p.swiglu;  // one piece at a time
    int turn = 0;
    const bool issuer = threadIdx.x == static_cast<unsigned>(64 + set * 128);
    auto meet = [&] { asm volatile("bar.sync %0, 128;" ::"r"(set + 1) : "memory"); };
    int local = 0;  // accumulators read
    int4 entry = first < total ? fetch_tile<Cfg>(p, table, first) : int4{};
    for (int idx = first; idx < total; idx += step) {
      Tile t = tile_at<Cfg>(p, idx, entry);
      t.row_end = row_end_of(p, table, t);
      if (idx + step < total) entry = fetch_tile<Cfg>(p, table, idx + step);
      // per 32 rows: lanes 0-15, then 16-31, as tmem_ld_16x256b_x4 has them
      float sum[NS][32];
      bool ok = true;
      for (int kb = 0; kb < t.num_kb; kb += p.chunk, ++local) {
        const bool ready = mbar_wait(tfull_bar(local & 1), static_cast<uint32_t>(local >> 1) & 1u,
                                     abort_flag, p.err);
        ok = !__any_sync(0xffffffffu, !ready);
        if (!ok) break;
        tc_fence_after();
        const uint32_t acc = tmem_base + (static_cast<uint32_t>(quad * 32) << 16) +
                             static_cast<uint32_t>((local & 1) * 256 + set * 32);
        if (kb == 0) {  // straight into the sums
#pragma unroll
          for (int i = 0; i < NS; ++i)
            if ((kSets * i + set) * 32 < t.rows) {
              tmem_ld_fragments(acc + i * kSets * 32, sum[i], 0);
              tmem_ld_fragments(acc + i * kSets * 32 + (16u << 16), sum[i], 16);
            }
          tmem_ld_wait();
          keep(sum);
        } else {
#pragma unroll
          for (int i = 0; i < NS; ++i)
            if ((kSets * i + set) * 32 < t.rows) {
              uint32_t lo[16], hi[16];
              tmem_ld_16x256b_x4(acc + i * kSets * 32, lo);
              tmem_ld_16x256b_x4(acc + i * kSets * 32 + (16u << 16), hi);
              tmem_ld_wait();
#pragma unroll
              for (int q = 0; q < 16; ++q) {
                sum[i][q] += after_wait(__uint_as_float(lo[q]));
                sum[i][16 + q] += after_wait(__uint_as_float(hi[q]));
              }
            }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(mapa_shared(tempty_bar(local & 1), 0));
      }
      // a set's warps meet below, so they give up together
      if (!all_of_set(set + 1, ok)) break;
      const int mat = lane >> 3, in = lane & 7;
      Out oc{&p.tm_c, static_cast<char*>(p.c), p.ldc, p.features, 0, 0, p.tma_c, p.vec_c};
      // the staging is free of the store that used it last
      auto begin = [&] {
        if (issuer) {
          if (big) bulk_wait_read();
          else bulk_wait_read_but_one();
        }
        meet();
        if (!big) stg = stg_set + (turn++ & 1) * 8192;
      };
      // Boxes of 128 bytes x 32 rows to columns col0, col0 + width, ...
      auto finish = [&](const Out& o, int boxes, int row0, int col0, auto type, bool halves) {
        using T = decltype(type);
        constexpr int kWidth = 128 / static_cast<int>(sizeof(T));
        const bool whole = row0 + 32 <= t.row_end;
        fence_async_shared();
        meet();
        for (int b = 0; b < boxes; ++b) {
          Out ob = o;
          int col = col0 + b * kWidth;
          if (halves) {  // box b is z's half b
            col = col0;
            ob.third = b;
            ob.base += b * static_cast<long long>(o.cols) * static_cast<long long>(sizeof(T));
          }
          if (col >= o.cols) continue;
          uint8_t* at = stg + b * 4096;
          if (whole && tma_takes<T>(o, col)) {
            if (issuer)
              tma_store_3d(o.map, smem_u32(at), col, o.is_z ? ob.third : row0,
                           o.is_z ? row0 : ob.third);
          } else {
            copy_rows<T>(ob, at, lane, quad * 8, 8, row0, t.row_end, col);
          }
        }
        if (issuer) bulk_commit();
      };
      // four matrices of 8 rows x 8 lanes: this thread addresses `row` of one of them, whose lanes
      // are the row's 16-byte part `part` in box `box`
      auto put_bf16 = [&](int box, int part, int row, uint32_t a, uint32_t b, uint32_t c,
                          uint32_t d) {
        stmatrix_x4_trans(smem_u32(stg) + box * 4096u + row * 128u +
                              (static_cast<uint32_t>(part ^ (row & 7)) << 4),
                          a, b, c, d);
      };
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        const int row0 = t.row0 + (kSets * i + set) * 32;
        if ((kSets * i + set) * 32 >= t.rows || row0 >= t.row_end) continue;
        float(&v)[32] = sum[i];
        auto put_all = [&](auto place) {  // 32 rows x 32 lanes in bf16
#pragma unroll
          for (int j = 0; j < 4; ++j)
            place(8 * j + in, pack2(v[4 * j], v[4 * j + 1]), pack2(v[4 * j + 2], v[4 * j + 3]),
                  pack2(v[16 + 4 * j], v[17 + 4 * j]), pack2(v[18 + 4 * j], v[19 + 4 * j]));
        };
        if (!p.swiglu) {
          const int col0 = t.feat0 + rank * 128;
          if (!p.c_f32) {
            begin();
            put_all([&](int row, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
              put_bf16(quad >> 1, (quad & 1) * 4 + mat, row, a, b, c, d);
            });
            finish(oc, 2, row0, col0, __nv_bfloat16{}, false);
          } else {
            begin();
#pragma unroll
            for (int h = 0; h < 2; ++h)
              put_f32(stg + quad * 4096, lane, 0, v, 2 * h, 16 * h, 32);
            finish(oc, 4, row0, col0, float{}, false);
          }
        } else {
          const int col0 = t.feat0 + rank * 64;
          if (p.z != nullptr) {
            Out oz{&p.tm_z, static_cast<char*>(p.z), p.ldz, p.features, 0, 1, p.tma_z, p.vec_z};
            begin();
            put_all([&](int row, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
              put_bf16(mat >> 1, quad * 2 + (mat & 1), row, a, b, c, d);
            });
            finish(oz, 2, row0, col0, __nv_bfloat16{}, true);
          }
#pragma unroll
          for (int q = 0; q < 16; ++q) v[q] = act_value<true>(MOE_ACT_SILU, v[q]) * v[16 + q];
          begin();
          if (!p.c_f32) {
#pragma unroll
            for (int j = 0; j < 4; j += 2)  // 16 rows x 16 features
              put_bf16(0, quad * 2 + (mat & 1), 8 * (j + (mat >> 1)) + in,
                       pack2(v[4 * j], v[4 * j + 1]), pack2(v[4 * j + 2], v[4 * j + 3]),
                       pack2(v[4 * j + 4], v[4 * j + 5]), pack2(v[4 * j + 6], v[4 * j + 7]));
            finish(oc, 1, row0, col0, __nv_bfloat16{}, false);
          } else {
#pragma unroll
            for (int h = 0; h < 2; ++h)
              put_f32(stg + (quad >> 1) * 4096, lane, (quad & 1) * 16, v, 2 * h, 16 * h, 16);
            finish(oc, 2, row0, col0, float{}, false);
          }
        }
      }
    }
    if (issuer) bulk_wait();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // no peer still reads this CTA's shared memory or arrives on it
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem_base, Cfg::kTmemCols);
  __syncwarp();
  cluster_sync_all();  // the pair gives its TMEM back before either CTA leaves
}

// ---------------------------------------------------------------------- host ----

inline int ceil_div(long long a, int b) { return static_cast<int>((a + b - 1) / b); }

bool encode(CUtensorMap* m, bool f32, const void* base, const cuuint64_t (&dims)[3],
            const cuuint64_t (&strides)[2], int box0, int box1, int box2) {
  auto fn = encode_fn();
  if (fn == nullptr) return false;
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(box0), static_cast<cuuint32_t>(box1),
                             static_cast<cuuint32_t>(box2)};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
            const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// An operand as [third][outer][inner] with boxes of 64 inner elements x box_rows.
bool operand_map(CUtensorMap* m, const void* base, long long inner, long long outer,
                 long long third, long long ld, long long third_stride, int box_rows) {
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(outer),
                              static_cast<cuuint64_t>(third)};
  const cuuint64_t strides[2] = {
      static_cast<cuuint64_t>(ld) * 2,
      static_cast<cuuint64_t>(third > 1 ? third_stride : ld * outer) * 2};
  return encode(m, false, base, dims, strides, BK, box_rows, 1);
}

// A swiglu layer's weights as [groups][blocks of 16][halves][16][inner], boxes of some blocks of both
// halves: 16 gate rows, the same 16 up rows, and so on.
bool halves_map(CUtensorMap* m, const GroupedProduct& g, int blocks) {
  auto fn = encode_fn();
  if (fn == nullptr) return false;
  const cuuint64_t ld = static_cast<cuuint64_t>(g.ldb) * 2, half = ld * g.features;
  const cuuint64_t dims[5] = {static_cast<cuuint64_t>(g.depth), 16, 2,
                              static_cast<cuuint64_t>(g.features / 16),
                              static_cast<cuuint64_t>(g.groups)};
  const cuuint64_t strides[4] = {ld, half, 16 * ld, 2 * half};
  const cuuint32_t box[5] = {BK, 16, 2, static_cast<cuuint32_t>(blocks), 1}, estr[5] = {1, 1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(g.b), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// An operand of the weight gradient, row-contiguous: [parts][rows][inner], boxes of 64 x 64.
bool rows_map(CUtensorMap* m, const GroupedProduct& g, bool a) {
  return a ? operand_map(m, g.a, g.rows, g.total_rows, g.a_parts, g.lda, g.a_plane, BK)
           : operand_map(m, g.b, g.features, g.total_rows, g.b_parts, g.ldb, g.b_plane, BK);
}

// An output as dims[2] x dims[1] x dims[0] values with strides (in values) of the outer two, boxes
// of 128 bytes x 32 rows, the rows dimension `row_dim`; false if TMA cannot take it.
bool output_map(CUtensorMap* m, bool f32, const void* base, const long long (&dims)[3],
                const long long (&ld)[2], int row_dim) {
  const long long sz = f32 ? 4 : 2;
  if ((reinterpret_cast<uintptr_t>(base) & 15u) != 0 || ld[0] * sz % 16 != 0 || ld[1] * sz % 16 != 0)
    return false;
  const cuuint64_t d[3] = {static_cast<cuuint64_t>(dims[0]), static_cast<cuuint64_t>(dims[1]),
                           static_cast<cuuint64_t>(dims[2])};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(ld[0] * sz),
                                 static_cast<cuuint64_t>(ld[1] * sz)};
  return encode(m, f32, base, d, strides, static_cast<int>(128 / sz), row_dim == 1 ? 32 : 1,
                row_dim == 2 ? 32 : 1);
}

inline bool vec_ok(const void* p, long long ld, int bytes) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ld * bytes % 16 == 0;
}

// How a kernel's tile lies: rows and features of it, and the boxes that its operands are loaded in.
struct TileShape {
  int rows, features;        // of a tile (swiglu: twice the features of C)
  bool swap;                 // the weights are operand A
  int x_box, w_box, w_box_swiglu;
  int ctas, threads, smem;
  bool staged;               // C and z leave by TMA
};

template <typename Cfg, int CTAS, int BN, bool SWAP>
constexpr TileShape plain_shape() {
  return TileShape{Cfg::kTileRows, Cfg::kTileFeatures, SWAP, SWAP ? BN : 128,
                   SWAP ? 128 : Cfg::kBRows,
                   SWAP ? 16 : Cfg::kBRows / 2,
                   CTAS, Cfg::kThreads, Cfg::kSmem, !SWAP};
}
template <int PB>
constexpr TileShape wide_shape() {
  using Cfg = WideCfg<PB>;
  return TileShape{kWideRows, Cfg::kTileFeatures, true, 128, 128, 16, 2, Cfg::kThreads, Cfg::kSmem,
                   true};
}

// Rows of weights in a tile of swapped sides, in 32: fewer than 128 where the tiles then still go
// round the SMs once, so that more of them stream (one token's 8 experts of 2 x 768: 96 tiles of 128
// rows 14.1 us, 128 of 96 rows 13.8; with the weights in L2 11.7 and 11.0).  There are no more groups
// with rows than rows.
int tile_quads(const GroupedProduct& g, int num_sms) {
  const long long active = std::min(g.groups, g.total_rows);
  const bool mn = g.kind == GroupedKind::kInputGrad;  // boxes of 64
  for (int q = 2; q < 4; ++q) {
    if (mn && q == 3) continue;
    if (active * ceil_div(g.features, (g.swiglu ? 16 : 32) * q) <= num_sms) return q;
  }
  return 4;
}

// Fills in what depends on the tiles, and how many there can be.
cudaError_t lay_out(const TileShape& ts, GroupedParams* p, const GroupedProduct& g,
                    long long* tiles) {
  const bool weight_grad = g.kind == GroupedKind::kWeightGrad;
  const long long rows = g.total_rows;
  if (!weight_grad) {
    // sides: activations k-contiguous, weights k-contiguous or (input gradient) row-contiguous
    const bool mn = g.kind == GroupedKind::kInputGrad;
    const long long w_rows = mn ? g.depth : g.swiglu ? 2ll * g.features : g.features;
    const long long w_inner = mn ? g.features : g.depth;
    const int w_box = mn         ? BK
                      : g.swiglu ? ts.w_box_swiglu
                      : p->quads ? 32 * p->quads
                                 : ts.w_box;
    CUtensorMap* tx = ts.swap ? &p->tm_b : &p->tm_a;
    CUtensorMap* tw = ts.swap ? &p->tm_a : &p->tm_b;
    if (!operand_map(tx, g.a, g.depth, rows, g.a_parts, g.lda, g.a_plane, ts.x_box))
      return cudaErrorInvalidValue;
    if (p->w_blocks ? !halves_map(tw, g, p->quads ? p->quads : 4)
                    : !operand_map(tw, g.b, w_inner, w_rows,
                                   static_cast<long long>(g.b_parts) * g.groups, g.ldb,
                                   g.ldb * w_rows, w_box))
      return cudaErrorInvalidValue;
    (ts.swap ? p->a_mn : p->b_mn) = mn;
    p->a_step = ts.swap ? g.groups : 1;
    p->b_step = ts.swap ? 1 : g.groups;
    p->num_kb = ceil_div(g.depth, BK);
  } else {
    if (!rows_map(&p->tm_a, g, true) || !rows_map(&p->tm_b, g, false)) return cudaErrorInvalidValue;
    p->a_mn = p->b_mn = 1;
    p->a_step = p->b_step = 1;
    p->tiles_a = ceil_div(g.rows, ts.rows);
  }
  p->feat_step = p->quads ? (g.swiglu ? 16 : 32) * p->quads
                          : g.swiglu ? ts.features / 2 : ts.features;
  p->tiles_b = ceil_div(g.features, p->feat_step);
  if (ts.staged) {
    const long long c_rows = weight_grad ? g.rows : rows;
    p->tma_c = output_map(&p->tm_c, g.c_f32, g.c, {g.features, c_rows, weight_grad ? g.groups : 1},
                          {g.ldc, weight_grad ? g.c_group : g.ldc * c_rows}, 1);
    p->tma_z = g.z != nullptr && output_map(&p->tm_z, g.z_f32, g.z, {g.features, 2, rows},
                                            {g.features, g.ldz}, 2);
  }
  p->vec_c = vec_ok(g.c, g.ldc, g.c_f32 ? 4 : 2) &&
             (!weight_grad || g.c_group * (g.c_f32 ? 4 : 2) % 16 == 0);
  p->vec_z = vec_ok(g.z, g.ldz, g.z_f32 ? 4 : 2) && g.features * (g.z_f32 ? 4 : 2) % 16 == 0;
  *tiles =
      weight_grad ? static_cast<long long>(g.groups) * p->tiles_a * p->tiles_b
                  : static_cast<long long>(grouped_max_tiles(g.total_rows, g.groups, ts.rows)) *
                        p->tiles_b;
  return cudaSuccess;
}

// Up to `tiles` tiles.
template <typename K, typename P>
cudaError_t launch(K kernel, const TileShape& ts, std::atomic<unsigned long long>* done,
                   const P& params, long long tiles, int num_sms, cudaStream_t s) {
  if (tiles >= (1ll << 31) - num_sms) return cudaErrorInvalidValue;
  const cudaError_t e = allow_smem(kernel, ts.smem, done);
  if (e != cudaSuccess) return e;
  const int slots = num_sms / ts.ctas;
  const unsigned grid = static_cast<unsigned>(tiles < slots ? tiles : slots) * ts.ctas;
  cudaLaunchConfig_t lc;
  std::memset(&lc, 0, sizeof(lc));
  lc.gridDim = dim3(grid);
  lc.blockDim = dim3(static_cast<unsigned>(ts.threads));
  lc.dynamicSmemBytes = static_cast<size_t>(ts.smem);
  lc.stream = s;
  cudaLaunchAttribute attr[1];
  if (ts.ctas == 2) {  // in stream order, without overlap with its neighbours
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
  } else {
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
  }
  lc.attrs = attr;
  lc.numAttrs = 1;
  return count_launch(cudaLaunchKernelEx(&lc, kernel, params));
}

GroupedParams params_of(const GroupedProduct& g, const GroupPlan& plan, unsigned* err) {
  GroupedParams p;
  std::memset(&p, 0, sizeof(p));
  p.plan = plan;
  p.kind = g.kind;
  p.groups = g.groups;
  p.total_rows = g.total_rows;
  p.rows = g.rows;
  p.features = g.features;
  p.swiglu = g.swiglu;
  p.c = g.c;
  p.z = g.z;
  p.ldc = g.ldc;
  p.c_group = g.c_group;
  p.ldz = g.ldz;
  p.c_f32 = g.c_f32;
  p.err = err;
  p.chunk = g.b_parts == 3 ? kPartsChunk : g.c_f32 ? kFloatChunk : kMaxChunk / g.a_parts;
  return p;
}

struct Launch {
  const GroupPlan& plan;
  unsigned* err;
  int num_sms;
  cudaStream_t s;
};

template <int CTAS, int BN, int PA, int PB, bool SWAP>
cudaError_t launch_plain(const GroupedProduct* g, int n, const Launch& l) {
  static std::atomic<unsigned long long> done{0};
  using Cfg = GroupedCfg<CTAS, BN, PA, PB, SWAP>;
  constexpr TileShape ts = plain_shape<Cfg, CTAS, BN, SWAP>();
  GroupedJobs<kMostJobs<PA>> jobs;
  std::memset(&jobs, 0, sizeof(jobs));
  jobs.count = n;
  long long all = 0;
  for (int i = 0; i < n; ++i) {
    GroupedParams& p = jobs.p[i];
    p = params_of(g[i], l.plan, l.err);
    p.quads = SWAP ? tile_quads(g[i], l.num_sms) : 0;
    p.w_blocks = SWAP && g[i].swiglu && g[i].features % 16 == 0;
    long long tiles = 0;
    const cudaError_t e = lay_out(ts, &p, g[i], &tiles);
    if (e != cudaSuccess) return e;
    all += tiles;
  }
  return launch(grouped_kernel<CTAS, BN, PA, PB, SWAP>, ts, &done, jobs, all, l.num_sms, l.s);
}
template <int PB>
cudaError_t launch_wide(const GroupedProduct& g, const Launch& l) {
  static std::atomic<unsigned long long> done{0};
  GroupedParams p = params_of(g, l.plan, l.err);
  for (int b = 0; b < 3; ++b)
    if (!operand_map(&p.tm_rows[b], g.a, g.depth, g.total_rows, g.a_parts, g.lda, g.a_plane,
                     64 >> b))
      return cudaErrorInvalidValue;
  p.w_blocks = g.swiglu && g.features % 16 == 0;
  if (g.c_f32 && PB == 1) p.chunk = kWideFloatChunk;
  long long tiles = 0;
  const cudaError_t e = lay_out(wide_shape<PB>(), &p, g, &tiles);
  if (e != cudaSuccess) return e;
  return launch(grouped_wide_kernel<PB>, wide_shape<PB>(), &done, p, tiles, l.num_sms, l.s);
}

}  // namespace

int grouped_tile_rows(int total_rows, int groups, bool f32) {
  if (f32) return 128;
  const long long mean = (static_cast<long long>(total_rows) + groups - 1) / groups;
  return mean <= 32 ? 32 : mean <= 64 ? 64 : kWideRows;
}

bool grouped_plans_itself(int tile_rows, bool f32) { return !f32 && tile_rows < kWideRows; }

size_t grouped_max_tiles(int total_rows, int groups, int tile_rows) {
  return static_cast<size_t>(total_rows / tile_rows) +
         static_cast<size_t>(std::min(groups, total_rows));
}

bool group_plan_task(const int32_t* offsets, int rows, int groups, int tile_rows,
                     const GroupPlan& plan, const GroupedProduct* wg, unsigned* err, PlanTask* t) {
  std::memset(t, 0, sizeof(*t));
  t->offsets = offsets;
  t->plan = plan;
  t->rows = rows;
  t->groups = groups;
  t->tile_rows = tile_rows;
  t->err = err;
  // 256 tiles of rows a block, up to 16 of them; a map a warp
  const size_t tiles = grouped_max_tiles(rows, groups, tile_rows) / kPlanThreads + 1;
  t->blocks = static_cast<int>(std::min<size_t>(tiles, 16));
  if (wg == nullptr) {
    t->plan.maps = nullptr;
    return true;
  }
  t->blocks = std::max(t->blocks, ceil_div(2ll * groups, kPlanThreads / 32));
  return rows_map(&t->tm_a, *wg, true) && rows_map(&t->tm_b, *wg, false);
}

cudaError_t launch_grouped_products(const GroupedProduct* g, int n, const GroupPlan& plan,
                                    unsigned* err, int num_sms, cudaStream_t s) {
  const Launch l{plan, err, num_sms, s};
  if (n > 0 && g[0].b_parts == 3) return launch_plain<1, 128, 3, 3, false>(g, n, l);
  cudaError_t e = cudaSuccess;
  for (int i = 0; i < n && e == cudaSuccess; ++i) {
    const bool parts = g[i].a_parts > 1;  // two for a weight gradient, three for an input gradient
    if (g[i].kind == GroupedKind::kWeightGrad) {
      e = parts ? launch_plain<2, 256, 2, 1, false>(&g[i], 1, l)
                : launch_plain<2, 256, 1, 1, false>(&g[i], 1, l);
      continue;
    }
    switch (grouped_tile_rows(g[i].total_rows, g[i].groups, false)) {
      case 32:
        e = parts ? launch_plain<1, 32, 1, 3, true>(&g[i], 1, l)
                  : launch_plain<1, 32, 1, 1, true>(&g[i], 1, l);
        break;
      case 64:
        e = parts ? launch_plain<1, 64, 1, 3, true>(&g[i], 1, l)
                  : launch_plain<1, 64, 1, 1, true>(&g[i], 1, l);
        break;
      default:
        e = parts ? launch_wide<3>(g[i], l) : launch_wide<1>(g[i], l);
    }
  }
  return e;
}

}  // namespace moe
