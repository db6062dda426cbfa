// The matrix product of the linear layers on the 5th-generation tensor cores: tcgen05.mma fed
// by TMA, accumulators in TMEM, bias / activation / residual in the epilogue.
//
// The forward and both gradients are one product with differently laid out operands: y = x w^T
// has both reduction-contiguous, dx = dz w has w row-contiguous, dw = dz^T x both.  TMA loads
// either layout in 128-byte swizzled boxes, and the matrix descriptors and the instruction
// descriptor name the layout, so nothing is transposed in memory:
//   k-contiguous: a box of 64 k x R rows; 8-row atoms of 1024 bytes follow one another along
//                 the rows; a step of 16 k advances 32 bytes inside the atom;
//   row-contiguous: boxes of 64 rows x 64 k (8 KB); atoms of 8 k follow one another, the next
//                 64 rows are one box on; a step of 16 k advances two atoms (2 KB).
//
// Two kernels:
//  - linear_pair_kernel: persistent CTA pairs (cta_group::2), 256 x 256 tiles, for products
//    with tiles enough to fill the GPU.  It is launched in stream order without overlap with
//    its neighbours' prologue or tail, and a CTA leaves only after every commit that it asked
//    for has arrived and its peer has given back its TMEM, so nothing of one launch can reach
//    into the next;
//  - linear_tile_kernel: one BA x BN tile per CTA or per cluster, whose CTAs take slices of
//    the reduction and exchange partial tiles through distributed shared memory, summed in
//    rank order (deterministic).  For few output rows the operands are swapped, so that the
//    weights are on the BA side and the tokens on a side of 16, 32 or 64.  BA = 64 runs the
//    same 128-row MMA with only the first 64 rows loaded (a row of the result depends on its
//    own row of A alone): a product bound by streaming one operand then has twice the CTAs to
//    stream it.  It takes two independent products (the two gradients of a layer) in one
//    launch, so that the second fills the SMs that the first leaves idle.  Its epilogue warps add the accumulator into registers every `chunk` k-blocks
//    (float32 results): the tensor core truncates each addition (over 7168 products the mean
//    error is 8e-6 of the result's size, against 2e-7 for rounded additions).  Bound by the
//    stream of the larger operand and by latency (64 x 7168 -> 2048: 11.5 us, 5.8 of them
//    streaming at 5.3 TB/s), float32 by shared memory: a 128 x 128 MMA reads 8 KB and its share
//    of the loads writes 4 KB, 96 clocks for 64 of work (2048 x 4096 -> 4096: 365 us).
#include <algorithm>
#include <atomic>
#include <cstring>
#include <mutex>
#include <type_traits>

#include "common.cuh"
#include "linear.h"
#include "linear_act.cuh"
#include "tc_operand.cuh"

namespace moe {
namespace {

constexpr int BK = 64;        // bf16 elements per k-block: one 128-byte swizzle row
constexpr int kThreads = 192; // TMA warp, MMA warp, four epilogue warps
// k-blocks that one accumulator takes for a bf16 result, 16384 values.  The tensor core truncates
// its additions, which leaves a sum of values of one sign low by 6.2e-9 of its size per value
// (measured from 64 K to 1 M values): 1.0e-4 here, against the result's own rounding of 1.7e-3.
// DW of 524288 rows in one accumulator would be off by 3.2e-3.
constexpr int kMaxChunk = 256;

struct Epilogue {
  void* c;
  const float* bias;
  const void* res;
  void* z;
  long long ldc, ldr, ldz;
  int rows, cols;
  int act;
  int c_f32;
  int vec_c, vec_r, vec_z, vec_bias;  // 16-byte accesses allowed
  int wide16;  // bf16 results: c and z allow 32-byte accesses, res and bias 16-byte ones
};

struct Job {
  CUtensorMap tm_a, tm_b;
  Epilogue epi;
  int a_mn, b_mn;
  int num_kb;
  int tiles_a;  // tiles along the side of operand A
  int tiles_b;
  int swap;     // operand A carries the output columns (tile kernel)
  // Column sums to finish (a bias gradient): sum_out[i] = sum_s sum_parts[s][i] over the
  // output rows i, taken by the tiles of the first column of tiles; or null
  const float* sum_parts;
  float* sum_out;
  int sum_slices;
};

struct GemmParams {
  Job job[2];
  unsigned* err;
  int first;  // tiles of job[0]; the rest are job[1]'s
  int total;
  int chunk;  // k-blocks between register additions (tile kernel)
};

// The slices of row i's sum, in column_sum_kernel's order: every eighth slice, then the eight
// partial sums.
__device__ __forceinline__ void finish_sum(const Job& job, int i) {
  if (i >= job.epi.rows) return;
  float part[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
  for (int s = 0; s < job.sum_slices; s += 8) {
#pragma unroll
    for (int w = 0; w < 8; ++w)
      if (s + w < job.sum_slices)
        part[w] += __ldg(job.sum_parts + static_cast<size_t>(s + w) * job.epi.rows + i);
  }
  float total = 0.f;
#pragma unroll
  for (int w = 0; w < 8; ++w) total += part[w];
  job.sum_out[i] = total;
}

// ------------------------------------------------------------------ epilogue ----

__device__ __forceinline__ void unpack_bf16(const uint4& u, float (&v)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

// n <= 8 values at p[0..], with 16-byte accesses when `vec` and n == 8.
__device__ __forceinline__ void load_n(const float* p, int n, bool vec, float (&v)[8]) {
  if (vec && n == 8) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    return;
  }
#pragma unroll
  for (int q = 0; q < 8; ++q) v[q] = q < n ? p[q] : 0.f;
}
__device__ __forceinline__ void load_n(const __nv_bfloat16* p, int n, bool vec, float (&v)[8]) {
  if (vec && n == 8) {
    unpack_bf16(*reinterpret_cast<const uint4*>(p), v);
    return;
  }
#pragma unroll
  for (int q = 0; q < 8; ++q) v[q] = q < n ? __bfloat162float(p[q]) : 0.f;
}
__device__ __forceinline__ void store_n(float* p, int n, bool vec, const float (&v)[8]) {
  if (vec && n == 8) {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    return;
  }
#pragma unroll
  for (int q = 0; q < 8; ++q)
    if (q < n) p[q] = v[q];
}
__device__ __forceinline__ void store_n(__nv_bfloat16* p, int n, bool vec, const float (&v)[8]) {
  if (vec && n == 8) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    return;
  }
#pragma unroll
  for (int q = 0; q < 8; ++q)
    if (q < n) p[q] = __float2bfloat16_rn(v[q]);
}

// Eight neighbouring outputs of row `row` from column `col` on (row < rows, col < cols).  The
// residual is read by the thread that then stores y, so the two may be one buffer.
template <typename TA>
__device__ __forceinline__ void finish8(const Epilogue& e, int row, int col, float (&v)[8]) {
  const int n = min(8, e.cols - col);
  if (e.bias != nullptr) {
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (q < n) v[q] += __ldg(e.bias + col + q);
  }
  if (e.z != nullptr)
    store_n(static_cast<TA*>(e.z) + static_cast<size_t>(row) * e.ldz + col, n, e.vec_z, v);
  act_values<sizeof(TA) == 2>(e.act, v);
  if (e.res != nullptr) {
    float r[8];
    load_n(static_cast<const TA*>(e.res) + static_cast<size_t>(row) * e.ldr + col, n, e.vec_r, r);
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q] += r[q];
  }
  const size_t at = static_cast<size_t>(row) * e.ldc + col;
  if (e.c_f32)
    store_n(static_cast<float*>(e.c) + at, n, e.vec_c, v);
  else
    store_n(static_cast<__nv_bfloat16*>(e.c) + at, n, e.vec_c, v);
}

// The outputs that a CTA of the tile kernel finishes: rows x cols (a power of two), eight
// neighbours of a row per thread at a time.  Rows that do not allow 16-byte accesses are read
// and written value by value all the same: spreading neighbouring columns over the lanes
// coalesces those, but needs an address per value, and the few warps at hand are bound by their
// instructions (float32 333 x 1001 -> 777: 26 us, against 22).
struct OutTile {
  int row0, col0, rows, cols, shift;  // cols = 8 << shift
  __device__ __forceinline__ int items() const { return rows << shift; }
  __device__ __forceinline__ int row(int item) const { return item >> shift; }
  __device__ __forceinline__ int col(int item) const { return (item & ((1 << shift) - 1)) * 8; }
};
template <typename TA>
__device__ __forceinline__ void load_addends(const Epilogue& e, const OutTile& o, int item,
                                             float (&bias)[8], float (&res)[8]) {
#pragma unroll
  for (int u = 0; u < 8; ++u) bias[u] = res[u] = 0.f;
  const int row = o.row0 + o.row(item), col = o.col0 + o.col(item);
  if (item >= o.items() || row >= e.rows || col >= e.cols) return;
  const int n = min(8, e.cols - col);
  if (e.bias != nullptr) load_n(e.bias + col, n, e.vec_bias, bias);
  if (e.res != nullptr)
    load_n(static_cast<const TA*>(e.res) + static_cast<size_t>(row) * e.ldr + col, n, e.vec_r, res);
}
// part: `split` partial tiles of o.rows x (o.cols + 4) floats, summed in order.
template <typename TA>
__device__ __forceinline__ void finish_outputs(const Epilogue& e, const OutTile& o, int item,
                                               const float* part, int split,
                                               const float (&bias)[8], const float (&res)[8]) {
  const int row = o.row0 + o.row(item), col = o.col0 + o.col(item);
  if (row >= e.rows || col >= e.cols) return;
  const float* src = part + o.row(item) * (o.cols + 4) + o.col(item);
  float v[8];
  load_n(src, 8, true, v);
  for (int s = 1; s < split; ++s) {
    float x[8];
    load_n(src + s * o.rows * (o.cols + 4), 8, true, x);
#pragma unroll
    for (int u = 0; u < 8; ++u) v[u] += x[u];
  }
  const int n = min(8, e.cols - col);
#pragma unroll
  for (int u = 0; u < 8; ++u) v[u] += bias[u];
  if (e.z != nullptr)
    store_n(static_cast<TA*>(e.z) + static_cast<size_t>(row) * e.ldz + col, n, e.vec_z, v);
  act_values<sizeof(TA) == 2>(e.act, v);
#pragma unroll
  for (int u = 0; u < 8; ++u) v[u] += res[u];
  const size_t at = static_cast<size_t>(row) * e.ldc + col;
  if (e.c_f32) store_n(static_cast<float*>(e.c) + at, n, e.vec_c, v);
  else store_n(static_cast<__nv_bfloat16*>(e.c) + at, n, e.vec_c, v);
}

// Asks L2 for the residual (and the bias) of a tile's rows, long before they are used.
template <typename TA>
__device__ __forceinline__ void prefetch_residual(const Epilogue& e, int row0, int rows, int col0,
                                                  int cols, int t, int threads) {
  const int row_end = min(row0 + rows, e.rows), col_end = min(col0 + cols, e.cols);
  if (col0 >= col_end) return;
  if (e.bias != nullptr && col0 + t * 32 < col_end)
    asm volatile("prefetch.global.L2 [%0];" ::"l"(e.bias + col0 + t * 32));
  if (e.res == nullptr) return;
  constexpr int kLine = 128 / static_cast<int>(sizeof(TA));
  const int lines = (col_end - col0 + kLine - 1) / kLine + 1;  // one more: rows start anywhere
  for (int i = t; i < (row_end - row0) * lines; i += threads) {
    const int r = i / lines, c = min((i - r * lines) * kLine, col_end - col0 - 1);
    asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const TA*>(e.res) +
                                                  static_cast<size_t>(row0 + r) * e.ldr + col0 + c));
  }
}

// Sixteen neighbouring bf16 values of a row, 32-byte aligned: one whole sector.
__device__ __forceinline__ void store16(__nv_bfloat16* p, const float (&v)[16]) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]),
               "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// Sixteen neighbouring outputs of a bf16 tile that lies wholly inside the output, whose arrays
// allow 32-byte accesses: a thread writes its own row in whole sectors, straight from the
// accumulator. Against staging through shared memory, 4096 x 128 -> 14336 with its
// result alone takes 61 us instead of 66 and the weight gradient of 64 rows at 4096 x 4096
// 18.7 instead of 24.9. Rows that are not 32-byte aligned stay staged, where neighbouring lanes
// share a row's sectors: 3999 x 1000 -> 2050 takes 113 us that way and 154 us a row per thread.
__device__ __forceinline__ void finish16_inside(const Epilogue& e, int row, int col,
                                                float (&v)[16]) {
  using TA = __nv_bfloat16;
  uint4 r[2];
  if (e.res != nullptr) {
    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const TA*>(e.res) +
                                                      static_cast<size_t>(row) * e.ldr + col);
    r[0] = src[0];
    r[1] = src[1];
  }
  if (e.bias != nullptr) {
#pragma unroll
    for (int q = 0; q < 16; q += 4) {
      const float4 b = __ldg(reinterpret_cast<const float4*>(e.bias + col + q));
      v[q] += b.x, v[q + 1] += b.y, v[q + 2] += b.z, v[q + 3] += b.w;
    }
  }
  if (e.z != nullptr) store16(static_cast<TA*>(e.z) + static_cast<size_t>(row) * e.ldz + col, v);
  act_values<true>(e.act, v);
  if (e.res != nullptr) {
    float x[8];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      unpack_bf16(r[i], x);
#pragma unroll
      for (int q = 0; q < 8; ++q) v[8 * i + q] += x[q];
    }
  }
  store16(static_cast<TA*>(e.c) + static_cast<size_t>(row) * e.ldc + col, v);
}

// finish8 for two rows (row, row + step) of a bf16 tile that lies wholly inside the output,
// with 16-byte accesses throughout: the residuals are on their way before anything is computed.
// b: the eight columns' biases.
__device__ __forceinline__ void finish8_inside(const Epilogue& e, int row, int step, int col,
                                               const float (&b)[8], float (&v)[2][8]) {
  using TA = __nv_bfloat16;
  uint4 r[2];
  if (e.res != nullptr) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      r[i] = *reinterpret_cast<const uint4*>(static_cast<const TA*>(e.res) +
                                             static_cast<size_t>(row + i * step) * e.ldr + col);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
#pragma unroll
    for (int q = 0; q < 8; ++q) v[i][q] += b[q];
    if (e.z != nullptr)
      store_n(static_cast<TA*>(e.z) + static_cast<size_t>(row + i * step) * e.ldz + col, 8, true,
              v[i]);
    act_values<true>(e.act, v[i]);
    if (e.res != nullptr) {
      float x[8];
      unpack_bf16(r[i], x);
#pragma unroll
      for (int q = 0; q < 8; ++q) v[i][q] += x[q];
    }
    store_n(static_cast<TA*>(e.c) + static_cast<size_t>(row + i * step) * e.ldc + col, 8, true,
            v[i]);
  }
}

// --------------------------------------------------------- operands in smem ----

// One k-block of `rows` (a multiple of 64 when row-contiguous) operand rows from r0 on.
__device__ __forceinline__ void load_operand(uint32_t dst, const void* map, uint32_t bar, int mn,
                                             int r0, int rows, int kb, int plane) {
  if (!mn) {
    tma_load_3d(dst, map, bar, kb * BK, r0, plane);
  } else {
    for (int c = 0; c < rows; c += 64)
      tma_load_3d(dst + c * 128u, map, bar, r0 + c, kb * BK, plane);
  }
}
__device__ __forceinline__ void load_operand_pair(uint32_t dst, const void* map, uint32_t bar,
                                                  int mn, int r0, int kb) {
  if (!mn) {
    tma_load_3d_pair(dst, map, bar, kb * BK, r0, 0);
  } else {
    tma_load_3d_pair(dst, map, bar, r0, kb * BK, 0);
    tma_load_3d_pair(dst + 8192u, map, bar, r0 + 64, kb * BK, 0);
  }
}

// ---------------------------------------------------------- one tile per CTA ----

template <int BA, int BN, int PL>
struct TileCfg {
  static constexpr int kABytes = BA * BK * 2, kBBytes = BN * BK * 2;
  static constexpr int kStageBytes = PL * (kABytes + kBBytes);
  static constexpr int kBarBytes = 256;
  // The MMA reads 128 rows from an A tile's start: with BA = 64 the second half runs on into
  // whatever follows (8 KB past the last stage at most).
  static constexpr int kSlack = BA < 128 ? 8192 : 0;
  static constexpr int kStagesRaw = (232448 - 1024 - kBarBytes - kSlack) / kStageBytes;
  static constexpr int kStages = kStagesRaw > 12 ? 12 : kStagesRaw;
  static constexpr int kSmem = 1024 + kStages * kStageBytes + kBarBytes + kSlack;
  static constexpr int kTmemCols = 2 * BN < 32 ? 32 : 2 * BN;
  // the exchanged partial tiles reuse the stages: BA x (BN + 4) floats, or BN rows of
  // BA + 4 floats per CTA of the cluster when the operands are swapped
  static_assert(BA * (BN + 4) * 4 <= kStages * kStageBytes, "partial tile");
  static_assert(BN * (BA + 4 * 8) * 4 <= kStages * kStageBytes, "swapped partial tile");
  static_assert(8 * (2 * kStages + 6) + 8 <= kBarBytes, "barrier region");
};

// Stores into the shared memory of a CTA of the cluster that count as transaction bytes on a
// barrier there (both shared::cluster addresses): the receiver waits for the bytes, so neither
// side needs a fence.
__device__ __forceinline__ void st_async_v4(uint32_t addr, uint32_t bar, float a, float b, float c,
                                            float d) {
  asm volatile(
      "st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%2, %3, %4, %5}, [%1];" ::
          "r"(addr),
      "r"(bar), "f"(a), "f"(b), "f"(c), "f"(d)
      : "memory");
}
__device__ __forceinline__ void st_async(uint32_t addr, uint32_t bar, float a) {
  asm volatile(
      "st.async.shared::cluster.mbarrier::complete_tx::bytes.f32 [%0], %2, [%1];" ::"r"(addr),
      "r"(bar), "f"(a)
      : "memory");
}
// Cluster barrier for control flow alone (no memory is published by it).
__device__ __forceinline__ void cluster_arrive_relaxed() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
}

template <int BA, int BN, int PL>
__global__ void __launch_bounds__(kThreads, 1)
    linear_tile_kernel(const __grid_constant__ GemmParams p) {
  using TA = std::conditional_t<PL == 3, float, __nv_bfloat16>;
  using Cfg = TileCfg<BA, BN, PL>;
  constexpr int S = Cfg::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S * Cfg::kStageBytes);
  const uint32_t bar0 = smem_u32(bars);
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (S + s); };
  auto tfull_bar = [&](int a) { return bar0 + 8u * (2 * S + a); };
  auto tempty_bar = [&](int a) { return bar0 + 8u * (2 * S + 2 + a); };
  const uint32_t mma_done_bar = bar0 + 8u * (2 * S + 4);
  const uint32_t xchg_bar = bar0 + 8u * (2 * S + 5);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * S + 6);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t nranks;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(nranks));
  const int split = static_cast<int>(nranks), rank = static_cast<int>(cluster_ctarank());
  int tile = static_cast<int>(blockIdx.x) / split;
  const Job& job = p.job[tile < p.first ? 0 : 1];
  if (tile >= p.first) tile -= p.first;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(tfull_bar(a), 1);
      mbar_init(tempty_bar(a), 4);
    }
    mbar_init(mma_done_bar, 1);
    mbar_init(xchg_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
    // the slices of this CTA's rows, from every CTA of the cluster
    mbar_arrive_expect_tx(xchg_bar, BA * BN * 4);
    tma_prefetch_desc(&job.tm_a);
    tma_prefetch_desc(&job.tm_b);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), Cfg::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  grid_dep_wait();
  grid_dep_trigger();

  const int a0 = (tile % job.tiles_a) * BA, b0 = (tile / job.tiles_a) * BN;
  // this CTA's slice of the reduction (empty if there are fewer k-blocks than CTAs)
  const int kb0 = static_cast<int>(static_cast<long long>(job.num_kb) * rank / split);
  const int nkb = static_cast<int>(static_cast<long long>(job.num_kb) * (rank + 1) / split) - kb0;
  const int R = BA / split;  // rows of the A side that each CTA finishes
  // the outputs that this CTA finishes; the first ones' biases and residuals are read while the
  // partial tiles are on their way
  OutTile out;
  out.row0 = job.swap ? b0 : a0 + rank * R;
  out.col0 = job.swap ? a0 + rank * R : b0;
  out.rows = job.swap ? BN : R;
  out.cols = job.swap ? R : BN;
  out.shift = __ffs(out.cols >> 3) - 1;
  float bias[8], res[8];

  if (warp == 0) {
    // ------------------------------------------------------------ producer ----
    const bool leader = elect_one_sync();
    int stage = 0, issued = 0;
    uint32_t phase = 0;
    if (leader) {
      for (int i = 0; i < nkb; ++i) {
        if (!mbar_wait(empty_bar(stage), phase ^ 1u, abort_flag, p.err)) break;
        const uint32_t dst = smem_u32(smem) + stage * Cfg::kStageBytes;
        mbar_arrive_expect_tx(full_bar(stage), Cfg::kStageBytes);
#pragma unroll
        for (int pl = 0; pl < PL; ++pl) {
          load_operand(dst + pl * Cfg::kABytes, &job.tm_a, full_bar(stage), job.a_mn, a0, BA, kb0 + i, pl);
          load_operand(dst + PL * Cfg::kABytes + pl * Cfg::kBBytes, &job.tm_b, full_bar(stage), job.b_mn,
                       b0, BN, kb0 + i, pl);
        }
        ++issued;
        if (++stage == S) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    __syncwarp();
    drain_stages<S>(leader, lane, stage, phase, issued, empty_bar, full_bar, true, abort_flag, p.err);
    cluster_arrive_relaxed();  // every CTA's stages are free, its exchange barrier is set up
    load_addends<TA>(job.epi, out, threadIdx.x, bias, res);
    __syncwarp();
    cluster_wait();
  } else if (warp == 1) {
    // ----------------------------------------------------------------- MMA ----
    if (elect_one_sync()) {
      const uint32_t idesc = idesc_bf16_f32(128, BN) | (static_cast<uint32_t>(job.a_mn) << 15) |
                             (static_cast<uint32_t>(job.b_mn) << 16);
      const uint32_t a_step = job.a_mn ? 2048u : 32u, b_step = job.b_mn ? 2048u : 32u;
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int i = 0, c = 0; ok && i < nkb; ++c) {
        const int acc = c & 1;
        if (!mbar_wait(tempty_bar(acc), (static_cast<uint32_t>(c >> 1) & 1u) ^ 1u, abort_flag, p.err)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t d = tmem_base + static_cast<uint32_t>(acc * BN);
        const int end = min(nkb, i + p.chunk);
        uint32_t accumulate = 0;
        for (; i < end; ++i) {
          if (!mbar_wait(full_bar(stage), phase, abort_flag, p.err)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a_base = smem_u32(smem) + stage * Cfg::kStageBytes;
          const uint32_t b_base = a_base + PL * Cfg::kABytes;
          // smallest products first
          constexpr int kTerms = PL == 3 ? 6 : 1;
          constexpr int pa[6] = {2, 1, 0, 1, 0, 0}, pb[6] = {0, 1, 2, 0, 1, 0};
#pragma unroll
          for (int q = 0; q < kTerms; ++q) {
            const int qa = PL == 3 ? pa[q] : 0, qb = PL == 3 ? pb[q] : 0;
#pragma unroll
            for (int kk = 0; kk < BK / 16; ++kk) {
              tc_mma_bf16(d, operand_desc(a_base + qa * Cfg::kABytes + kk * a_step, job.a_mn),
                          operand_desc(b_base + qb * Cfg::kBBytes + kk * b_step, job.b_mn), idesc,
                          accumulate);
              accumulate = 1u;
            }
          }
          tc_commit(empty_bar(stage));
          if (++stage == S) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (ok) tc_commit(tfull_bar(acc));
      }
      if (!ok || *abort_flag) {
        tc_commit(mma_done_bar);
        volatile int no_abort = 0;
        mbar_wait(mma_done_bar, 0, &no_abort, p.err);
      }
    }
    __syncwarp();
    cluster_arrive_relaxed();
    load_addends<TA>(job.epi, out, threadIdx.x, bias, res);
    __syncwarp();
    cluster_wait();
  } else {
    // ------------------------------------------------------------ epilogue ----
    const int quad = warp & 3;
    if (job.sum_parts != nullptr && rank == 0 && (job.swap ? a0 : b0) == 0 &&
        quad * 32 + lane < (job.swap ? BN : BA))
      finish_sum(job, (job.swap ? b0 : a0) + quad * 32 + lane);
    prefetch_residual<TA>(job.epi, out.row0, out.rows, out.col0, out.cols,
                          static_cast<int>(threadIdx.x) - 64, kThreads - 64);
    __syncwarp();
    float acc[BN];
#pragma unroll
    for (int j = 0; j < BN; ++j) acc[j] = 0.f;
    const int chunks = (nkb + p.chunk - 1) / p.chunk;
    for (int c = 0; c < chunks; ++c) {
      const int buf = c & 1;
      const bool ready =
          mbar_wait(tfull_bar(buf), static_cast<uint32_t>(c >> 1) & 1u, abort_flag, p.err);
      if (__any_sync(0xffffffffu, !ready)) break;
      tc_fence_after();
      const uint32_t t = tmem_base + (static_cast<uint32_t>(quad * 32) << 16) +
                         static_cast<uint32_t>(buf * BN);
      if constexpr (BN >= 32) {
#pragma unroll
        for (int j = 0; j < BN; j += 32) {
          uint32_t r[32];
          tmem_ld_32x32b_x32(t + j, r);
          tmem_ld_wait();
#pragma unroll
          for (int q = 0; q < 32; ++q) acc[j + q] += __uint_as_float(r[q]);
        }
      } else {
        uint32_t r[16];
        tmem_ld_32x32b_x16(t, r);
        tmem_ld_wait();
#pragma unroll
        for (int q = 0; q < 16; ++q) acc[q] += __uint_as_float(r[q]);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(tempty_bar(buf));
    }
    __syncwarp();
    cluster_arrive_relaxed();
    cluster_wait();
    // this CTA's partial tile, row by row to the CTA that finishes the row (itself without a
    // split: plain stores, which are faster than asynchronous ones)
    const int row = quad * 32 + lane;
    const int owner = min(row / R, split - 1), local = row - owner * R;
    const uint32_t base = mapa_shared(smem_u32(smem), static_cast<uint32_t>(owner));
    const uint32_t bar = mapa_shared(xchg_bar, static_cast<uint32_t>(owner));
    if (row >= BA) {
      // rows that were not loaded
    } else if (split == 1) {
      float* mine = reinterpret_cast<float*>(smem);
      if (!job.swap) {
#pragma unroll
        for (int j = 0; j < BN; j += 4)
          *reinterpret_cast<float4*>(mine + row * (BN + 4) + j) =
              make_float4(acc[j], acc[j + 1], acc[j + 2], acc[j + 3]);
      } else {
#pragma unroll
        for (int j = 0; j < BN; ++j) mine[j * (BA + 4) + row] = acc[j];
      }
    } else if (!job.swap) {
      const uint32_t at = base + static_cast<uint32_t>(((rank * R + local) * (BN + 4)) * 4);
#pragma unroll
      for (int j = 0; j < BN; j += 4)
        st_async_v4(at + j * 4u, bar, acc[j], acc[j + 1], acc[j + 2], acc[j + 3]);
    } else {
      const uint32_t at = base + static_cast<uint32_t>((rank * BN * (R + 4) + local) * 4);
#pragma unroll
      for (int j = 0; j < BN; ++j)
        st_async(at + static_cast<uint32_t>(j * (R + 4) * 4), bar, acc[j]);
    }
    load_addends<TA>(job.epi, out, threadIdx.x, bias, res);
  }
  __syncwarp();
  cluster_arrive_relaxed();  // this CTA's stores are on their way
  volatile int no_abort = 0;
  bool received = true;
  if (split == 1) __syncthreads();
  else received = mbar_wait<true>(xchg_bar, 0, &no_abort, p.err);

  // sum the slices in rank order and finish the outputs, the next ones' addends on their way
  if (received && *abort_flag == 0) {
    const float* part = reinterpret_cast<const float*>(smem);
    for (int it = threadIdx.x; it < out.items(); it += kThreads) {
      float next_bias[8], next_res[8];
      load_addends<TA>(job.epi, out, it + kThreads, next_bias, next_res);
      finish_outputs<TA>(job.epi, out, it, part, split, bias, res);
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        bias[u] = next_bias[u];
        res[u] = next_res[u];
      }
    }
  }
  __syncwarp();
  cluster_wait();  // no peer is still to store into this CTA's shared memory
  if (!received) mbar_wait<true>(xchg_bar, 0, &no_abort, p.err);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem_base, Cfg::kTmemCols);
}

// ------------------------------------------------------ persistent CTA pairs ----

// Eight epilogue warps, two per TMEM lane quarter with half the columns each: with four, the
// epilogue of a tile took longer than its MMAs (4096 x 4096 -> 14336 with tanh-GELU and the
// kept pre-activation: 503 us; with eight 258 us, 1,864 TFLOP/s, the tensor pipe 90% busy).
struct PairCfg {
  static constexpr int kEpiWarps = 8;
  static constexpr int kThreads = 64 + 32 * kEpiWarps;
  static constexpr int kABytes = 128 * BK * 2;  // this CTA's 128 rows of A
  static constexpr int kBBytes = 128 * BK * 2;  // this CTA's half of the 256 rows of B
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kStages = 6;
  static constexpr int kBN = 256;
  static constexpr int kTmemCols = 512;
  static constexpr int kStgRow = 20;  // floats per staged row: 16 and a pad against conflicts
  static constexpr int kStgBytes = kEpiWarps * 32 * kStgRow * 4;
  static constexpr int kBarBytes = 256;
  static constexpr int kSmem = 1024 + kStages * kStageBytes + kStgBytes + kBarBytes;
  static_assert(kSmem <= 232448, "shared memory per CTA");
};

// Tiles in chunks of 8 rows of tiles, so that the pairs at work share operand tiles in L2.
__device__ __forceinline__ void pair_tile(const Job& p, int idx, int* ta, int* tb) {
  constexpr int kSwz = 8;
  const int per = kSwz * p.tiles_b;
  const int c = idx / per, in = idx - c * per;
  const int h = min(kSwz, p.tiles_a - c * kSwz);
  *tb = in / h;
  *ta = c * kSwz + in - *tb * h;
}

struct PairParams {
  Job job;
  unsigned* err;
  int chunk;  // k-blocks per accumulator
};

// kDeep: a tile's reduction is longer than an accumulator may take (kMaxChunk); the epilogue
// warps add up the chunks in registers.
template <bool kDeep>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(PairCfg::kThreads, 1)
    linear_pair_kernel(const __grid_constant__ PairParams p) {
  using Cfg = PairCfg;
  constexpr int S = Cfg::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  float* stg_all = reinterpret_cast<float*>(smem + S * Cfg::kStageBytes);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S * Cfg::kStageBytes + Cfg::kStgBytes);
  const uint32_t bar0 = smem_u32(bars);
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (S + s); };
  auto tfull_bar = [&](int a) { return bar0 + 8u * (2 * S + a); };
  auto tempty_bar = [&](int a) { return bar0 + 8u * (2 * S + 2 + a); };
  const uint32_t mma_done_bar = bar0 + 8u * (2 * S + 4);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * S + 5);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
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
    tma_prefetch_desc(&p.job.tm_a);
    tma_prefetch_desc(&p.job.tm_b);
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

  const Job& job = p.job;
  const int total = job.tiles_a * job.tiles_b;
  const int pair = static_cast<int>(blockIdx.x >> 1), npairs = static_cast<int>(gridDim.x >> 1);

  if (warp == 0) {
    // ------------------------------------------------------------ producer ----
    const bool leader = elect_one_sync();
    int stage = 0, issued = 0;  // (issued stops counting at S)
    uint32_t phase = 0;
    if (leader) {
      bool ok = true;
      for (int idx = pair; ok && idx < total; idx += npairs) {
        int ta, tb;
        pair_tile(job, idx, &ta, &tb);
        const int a_row = ta * 256 + static_cast<int>(rank) * 128;
        const int b_row = tb * 256 + static_cast<int>(rank) * 128;
        for (int kb = 0; kb < job.num_kb; ++kb) {
          if (!mbar_wait(empty_bar(stage), phase ^ 1u, abort_flag, p.err)) {
            ok = false;
            break;
          }
          const uint32_t fb = mapa_shared(full_bar(stage), 0);
          const uint32_t dst = smem_u32(smem) + stage * Cfg::kStageBytes;
          if (rank == 0) mbar_arrive_expect_tx(full_bar(stage), 2 * Cfg::kStageBytes);
          load_operand_pair(dst, &job.tm_a, fb, job.a_mn, a_row, kb);
          load_operand_pair(dst + Cfg::kABytes, &job.tm_b, fb, job.b_mn, b_row, kb);
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
      const uint32_t idesc = idesc_bf16_f32(256, Cfg::kBN) |
                             (static_cast<uint32_t>(job.a_mn) << 15) |
                             (static_cast<uint32_t>(job.b_mn) << 16);
      const uint32_t a_step = job.a_mn ? 2048u : 32u, b_step = job.b_mn ? 2048u : 32u;
      int stage = 0;
      uint32_t phase = 0;
      int local = 0;  // accumulators filled
      bool ok = true;
      for (int idx = pair; ok && idx < total; idx += npairs) {
        for (int kb = 0; ok && kb < job.num_kb; ++local) {
          const int acc = local & 1;
          if (!mbar_wait(tempty_bar(acc), (static_cast<uint32_t>(local >> 1) & 1u) ^ 1u, abort_flag,
                         p.err)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t d = tmem_base + static_cast<uint32_t>(acc * Cfg::kBN);
          const int first = kb, end = kDeep ? min(job.num_kb, kb + p.chunk) : job.num_kb;
          for (; kb < end; ++kb) {
            if (!mbar_wait(full_bar(stage), phase, abort_flag, p.err)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t a_base = smem_u32(smem) + stage * Cfg::kStageBytes;
            const uint32_t b_base = a_base + Cfg::kABytes;
#pragma unroll
            for (int kk = 0; kk < BK / 16; ++kk)
              tc_mma_bf16_pair(d, operand_desc(a_base + kk * a_step, job.a_mn),
                               operand_desc(b_base + kk * b_step, job.b_mn), idesc,
                               kb != first || kk != 0 ? 1u : 0u);
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
    const int quad = warp & 3, half = (warp - 2) >> 2;
    float* stg = stg_all + (warp - 2) * 32 * Cfg::kStgRow;
    const bool wide = job.epi.vec_c && (job.epi.res == nullptr || job.epi.vec_r) &&
                      (job.epi.z == nullptr || job.epi.vec_z) && job.epi.vec_bias;
    int local = 0;  // accumulators read
    for (int idx = pair; idx < total; idx += npairs) {
      int ta, tb;
      pair_tile(job, idx, &ta, &tb);
      const int row0 = ta * 256 + static_cast<int>(rank) * 128 + quad * 32;
      const int col0 = tb * 256 + half * 128;
      const bool inside = wide && row0 + 32 <= job.epi.rows && col0 + 128 <= job.epi.cols;
      // 32 neighbouring columns from col0 + c on of this thread's row
      auto finish = [&](int c, const float (&r)[32]) {
        if (inside && job.epi.wide16) {
#pragma unroll
          for (int h = 0; h < 32; h += 16) {
            float v[16];
#pragma unroll
            for (int q = 0; q < 16; ++q) v[q] = r[h + q];
            finish16_inside(job.epi, row0 + lane, col0 + c + h, v);
          }
        } else {
          // staged: lane l reads back columns (l & 1) * 8 of rows l / 2 and l / 2 + 16
          const int rr = lane >> 1, cc = (lane & 1) * 8;
#pragma unroll
          for (int h = 0; h < 32; h += 16) {
#pragma unroll
            for (int q = 0; q < 16; q += 4)
              *reinterpret_cast<float4*>(stg + lane * Cfg::kStgRow + q) =
                  make_float4(r[h + q], r[h + q + 1], r[h + q + 2], r[h + q + 3]);
            __syncwarp();
            const int col = col0 + c + h + cc;
            if (inside) {
              float bias[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, v[2][8];
              if (job.epi.bias != nullptr) load_n(job.epi.bias + col, 8, true, bias);
#pragma unroll
              for (int i = 0; i < 2; ++i)
                load_n(stg + (rr + 16 * i) * Cfg::kStgRow + cc, 8, true, v[i]);
              __syncwarp();
              finish8_inside(job.epi, row0 + rr, 16, col, bias, v);
              continue;
            }
#pragma unroll 1
            for (int i = 0; i < 32; i += 16) {
              if (row0 + rr + i < job.epi.rows && col < job.epi.cols) {
                float v[8];
                load_n(stg + (rr + i) * Cfg::kStgRow + cc, 8, true, v);
                finish8<__nv_bfloat16>(job.epi, row0 + rr + i, col, v);
              }
            }
            __syncwarp();
          }
        }
        __syncwarp();
      };
      // waits for accumulator `local`, whose columns of this thread start at accumulator()
      auto filled = [&] {
        const bool ready = mbar_wait(tfull_bar(local & 1), static_cast<uint32_t>(local >> 1) & 1u,
                                     abort_flag, p.err);
        if (__any_sync(0xffffffffu, !ready)) return false;
        tc_fence_after();
        return true;
      };
      auto accumulator = [&] {
        return tmem_base + (static_cast<uint32_t>(quad * 32) << 16) +
               static_cast<uint32_t>((local & 1) * Cfg::kBN + half * 128);
      };
      auto release_accumulator = [&] {  // it is free for the tile (or chunk) after next
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(mapa_shared(tempty_bar(local & 1), 0));
        ++local;
      };
      if constexpr (kDeep) {
        float sum[4][32];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int q = 0; q < 32; ++q) sum[i][q] = 0.f;
        bool ok = true;
        for (int kb = 0; kb < job.num_kb; kb += p.chunk) {
          ok = filled();
          if (!ok) break;
          const uint32_t t = accumulator();
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t r[32];
            tmem_ld_32x32b_x32(t + i * 32, r);
            tmem_ld_wait();
#pragma unroll
            for (int q = 0; q < 32; ++q) sum[i][q] += __uint_as_float(r[q]);
          }
          release_accumulator();
        }
        if (!ok) break;
#pragma unroll
        for (int i = 0; i < 4; ++i) finish(i * 32, sum[i]);
      } else {
        if (!filled()) break;
        const uint32_t t = accumulator();
#pragma unroll 1
        for (int c = 0; c < 128; c += 32) {
          uint32_t r[32];
          tmem_ld_32x32b_x32(t + c, r);
          tmem_ld_wait();
          if (c + 32 == 128) release_accumulator();
          float v[32];
#pragma unroll
          for (int q = 0; q < 32; ++q) v[q] = __uint_as_float(r[q]);
          finish(c, v);
        }
      }
    }
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

// The operand's planes as [planes][outer][inner] with boxes of 64 inner elements x box_rows.
// What lies past an edge reads as zero.
bool operand_map(CUtensorMap* m, const void* base, int rows, int depth, int mn, long long ld,
                 int planes, long long plane, int tile_rows) {
  auto fn = encode_fn();
  if (fn == nullptr) return false;
  const cuuint64_t inner = static_cast<cuuint64_t>(mn ? rows : depth);
  const cuuint64_t outer = static_cast<cuuint64_t>(mn ? depth : rows);
  cuuint64_t dims[3] = {inner, outer, static_cast<cuuint64_t>(planes)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(ld) * 2,
                           static_cast<cuuint64_t>(planes > 1 ? plane : ld * static_cast<long long>(outer)) * 2};
  cuuint32_t box[3] = {static_cast<cuuint32_t>(BK),
                       static_cast<cuuint32_t>(mn ? BK : tile_rows), 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A cluster launch of `split` CTAs per tile.
template <int BA, int BN, int PL>
void tile_launch(int tiles, int split, cudaStream_t s, cudaLaunchConfig_t* lc,
                 cudaLaunchAttribute (&attr)[2]) {
  std::memset(lc, 0, sizeof(*lc));
  lc->gridDim = dim3(static_cast<unsigned>(tiles) * static_cast<unsigned>(split));
  lc->blockDim = dim3(kThreads);
  lc->dynamicSmemBytes = TileCfg<BA, BN, PL>::kSmem;
  lc->stream = s;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(split);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  lc->attrs = attr;
  lc->numAttrs = 2;
}

template <int BA, int BN, int PL>
cudaError_t launch_tile(const GemmParams& p, int split, cudaStream_t s) {
  auto kernel = linear_tile_kernel<BA, BN, PL>;
  static std::atomic<unsigned long long> done{0};
  cudaError_t e = allow_smem(kernel, TileCfg<BA, BN, PL>::kSmem, &done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t lc;
  cudaLaunchAttribute attr[2];
  tile_launch<BA, BN, PL>(p.total, split, s, &lc, attr);
  return count_launch(cudaLaunchKernelEx(&lc, kernel, p));
}

// Clusters of 1, 2, 4 and 8 CTAs (one CTA per SM) that the device holds at a time: fewer than
// SMs / size, as a cluster stays within one group of SMs (GB300: 152, 76, 36, 15).
struct ClusterRoom {
  int room[4];
};
const ClusterRoom& cluster_room(int num_sms) {
  static ClusterRoom rooms[64];
  static std::once_flag once[64];
  int dev = 0;
  cudaGetDevice(&dev);
  dev &= 63;
  std::call_once(once[dev], [&] {
    for (int i = 0; i < 4; ++i) {
      rooms[dev].room[i] = num_sms >> i;
      if (i == 0) continue;
      cudaLaunchConfig_t lc;
      cudaLaunchAttribute attr[2];
      auto kernel = linear_tile_kernel<128, 128, 1>;
      int n = 0;
      if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               TileCfg<128, 128, 1>::kSmem) != cudaSuccess)
        continue;
      tile_launch<128, 128, 1>(1, 1 << i, nullptr, &lc, attr);
      if (cudaOccupancyMaxActiveClusters(&n, kernel, &lc) == cudaSuccess && n > 0)
        rooms[dev].room[i] = n;
    }
    cudaGetLastError();  // leave no sticky error behind
  });
  return rooms[dev];
}

inline int ceil_div(long long a, int b) { return static_cast<int>((a + b - 1) / b); }

inline bool vec_ok(const void* p, long long ld, int bytes) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (ld * bytes) % 16 == 0;
}

// CTA pairs or single tiles.  A pair's 256 x 256 tile is two 128 x 128 tiles of work per SM; a
// pair is preferred unless the coarser tiles leave more of the GPU idle than its better reuse
// of shared memory gains.
bool prefer_pairs(const LinearGemm& g, int num_sms) {
  if (g.planes != 1 || g.c_f32) return false;
  const long long tp = static_cast<long long>(ceil_div(g.rows, 256)) * ceil_div(g.cols, 256);
  const long long tt = static_cast<long long>(ceil_div(g.rows, 128)) * ceil_div(g.cols, 128);
  const int pairs = num_sms / 2;
  const long long waves_p = (tp + pairs - 1) / pairs, waves_t = (tt + num_sms - 1) / num_sms;
  return 16 * waves_p <= 10 * waves_t && tt > num_sms;
}

// How an output and its operands lie on the tile kernel's sides.
struct Sides {
  bool swap;
  int a, b;        // rows of the A and of the B side
  int a_mn, b_mn;
};
// Few output rows: the other operand on the side of 128 (or 64) rows.
bool swap_by_rule(const LinearGemm& g) { return g.rows <= 64 && g.cols > g.rows; }
Sides sides_of(const LinearGemm& g, bool swap) {
  return swap ? Sides{true, g.cols, g.rows, g.b_mn, g.a_mn}
              : Sides{false, g.rows, g.cols, g.a_mn, g.b_mn};
}

struct TileChoice {
  int ba, bn, split;
  bool other;  // the operands lie the other way round than swap_by_rule has them
  double cost;
};

// The tile, the split of the reduction and the operands' sides, by an estimate in SM clocks: waves
// of clusters times (a CTA's k-blocks at the slower of 60 bytes per clock into shared memory and
// the MMAs, plus the pipeline's fill, the exchange of partial tiles, which moves about 13 bytes
// per clock, and the epilogue).  Against the best of all choices, timed for 22 shapes of 8 to
// 2048 rows, it loses 7% at most.
//
// A forward product may lie the other way round than the rule has it where that saves a wave:
// 185 x 1024 -> 5440 are 170 tiles of 128 x 64 one way and 129 the other (bf16 17.5 -> 13.0 us,
// float32 32.8 -> 27.6).  The gradients keep the rule, so that one asked for by itself is split
// as it is in a joint launch in more cases; their sums are the same bit for bit only then.
TileChoice choose_tile(const LinearGemm* jobs, int n, int num_sms) {
  const ClusterRoom& room = cluster_room(num_sms);
  const int planes = jobs[0].planes;
  const int terms = planes == 3 ? 6 : 1;
  const bool forward = n == 1 && !jobs[0].a_mn && !jobs[0].b_mn;
  TileChoice best{128, 128, 1, false, 1e30};
  auto consider = [&](int ba, int bn, bool other) {
    long long tiles[2] = {0, 0};
    int num_kb[2] = {0, 0};
    for (int i = 0; i < n; ++i) {
      const Sides sd = sides_of(jobs[i], swap_by_rule(jobs[i]) != other);
      if (sd.b_mn && bn < 64) return;  // row-contiguous boxes are 64 rows wide
      tiles[i] = static_cast<long long>(ceil_div(sd.a, ba)) * ceil_div(sd.b, bn);
      num_kb[i] = ceil_div(jobs[i].depth, BK);
    }
    const double load = planes * (ba + bn) * 128.0 / 60.0;
    // an MMA of 16 products: its rate, or reading 128 + bn rows of 32 bytes
    const double mma = 4.0 * terms * std::max(0.52 * bn, 32.0 + 0.25 * bn);
    for (int i = 0; i < 4; ++i) {
      const int split = 1 << i;
      if (split > num_kb[0]) continue;  // the first job is the longest
      const long long slots = room.room[i];
      auto per_tile = [&](int j) {
        return ceil_div(num_kb[j], split) * (load > mma ? load : mma) + 4000.0 +
               (split > 1 ? 500.0 + 0.3 * ba * bn : 0.0) + 0.25 * ba * bn / split;
      };
      double cost = ((tiles[0] + slots - 1) / slots) * per_tile(0);
      if (n == 2) {
        // the second job's tiles run beside the first one's last wave, then in their own
        const long long free = (slots - tiles[0] % slots) % slots;
        const long long beside = free * static_cast<long long>(per_tile(0) / per_tile(1));
        const long long rest = std::max(0ll, tiles[1] - beside);
        cost += ((rest + slots - 1) / slots) * per_tile(1);
      }
      if (other) cost *= 1.08;  // only for a clear gain
      if (cost < best.cost) best = TileChoice{ba, bn, split, other, cost};
    }
  };
  for (int other = 0; other <= (forward ? 1 : 0); ++other)
    for (int ba = 64; ba <= 128; ba *= 2)
      for (int bn = 16; bn <= 128; bn *= 2)
        if (ba == 128 || bn < 128) consider(ba, bn, other != 0);
  return best;
}

Epilogue epilogue_of(const LinearGemm& g) {
  const int ab = g.act_f32 ? 4 : 2;
  Epilogue e;
  e.c = g.c;
  e.bias = g.bias;
  e.res = g.res;
  e.z = g.z;
  e.ldc = g.ldc;
  e.ldr = g.ldr;
  e.ldz = g.ldz;
  e.rows = g.rows;
  e.cols = g.cols;
  e.act = g.act;
  e.c_f32 = g.c_f32;
  e.vec_c = vec_ok(g.c, g.ldc, g.c_f32 ? 4 : 2);
  e.vec_r = vec_ok(g.res, g.ldr, ab);
  e.vec_z = vec_ok(g.z, g.ldz, ab);
  e.vec_bias = vec_ok(g.bias, 0, 4);
  auto sector_ok = [](const void* p, long long ld) {
    return (reinterpret_cast<uintptr_t>(p) & 31u) == 0 && ld % 16 == 0;
  };
  e.wide16 = !g.c_f32 && !g.act_f32 && sector_ok(g.c, g.ldc) &&
             (g.z == nullptr || sector_ok(g.z, g.ldz)) && (g.res == nullptr || e.vec_r) &&
             e.vec_bias;
  return e;
}

cudaError_t launch_pairs(const LinearGemm& g, unsigned* err, int num_sms, cudaStream_t s) {
  PairParams p;
  std::memset(&p, 0, sizeof(p));
  p.err = err;
  Job& j = p.job;
  if (!operand_map(&j.tm_a, g.a, g.rows, g.depth, g.a_mn, g.lda, 1, 0, 128) ||
      !operand_map(&j.tm_b, g.b, g.cols, g.depth, g.b_mn, g.ldb, 1, 0, 128))
    return cudaErrorInvalidValue;
  j.epi = epilogue_of(g);
  j.a_mn = g.a_mn;
  j.b_mn = g.b_mn;
  j.num_kb = ceil_div(g.depth, BK);
  j.tiles_a = ceil_div(g.rows, 256);
  j.tiles_b = ceil_div(g.cols, 256);
  const long long tiles = static_cast<long long>(j.tiles_a) * j.tiles_b;
  if (tiles >= (1ll << 31) - num_sms) return cudaErrorInvalidValue;
  p.chunk = kMaxChunk;
  const bool deep = j.num_kb > kMaxChunk;
  auto kernel = deep ? linear_pair_kernel<true> : linear_pair_kernel<false>;
  static std::atomic<unsigned long long> done[2];
  cudaError_t e = allow_smem(kernel, PairCfg::kSmem, &done[deep]);
  if (e != cudaSuccess) return e;
  const int pairs = static_cast<int>(tiles < num_sms / 2 ? tiles : num_sms / 2);
  // a plain launch: see the top of the file
  kernel<<<dim3(2 * pairs), dim3(PairCfg::kThreads), PairCfg::kSmem, s>>>(p);
  return count_launch(cudaGetLastError());
}

cudaError_t launch_tiles(const LinearGemm* jobs, int n, const TileChoice& t, unsigned* err,
                         cudaStream_t s) {
  GemmParams p;
  std::memset(&p, 0, sizeof(p));
  p.err = err;
  long long total = 0;
  for (int i = 0; i < n; ++i) {
    const LinearGemm& g = jobs[i];
    Job& j = p.job[i];
    const Sides sd = sides_of(g, swap_by_rule(g) != t.other);
    if (!operand_map(&j.tm_a, sd.swap ? g.b : g.a, sd.a, g.depth, sd.a_mn, sd.swap ? g.ldb : g.lda,
                     g.planes, sd.swap ? g.b_plane : g.a_plane, t.ba) ||
        !operand_map(&j.tm_b, sd.swap ? g.a : g.b, sd.b, g.depth, sd.b_mn, sd.swap ? g.lda : g.ldb,
                     g.planes, sd.swap ? g.a_plane : g.b_plane, t.bn))
      return cudaErrorInvalidValue;
    j.epi = epilogue_of(g);
    j.swap = sd.swap ? 1 : 0;
    j.a_mn = sd.a_mn;
    j.b_mn = sd.b_mn;
    j.num_kb = ceil_div(g.depth, BK);
    j.tiles_a = ceil_div(sd.a, t.ba);
    j.tiles_b = ceil_div(sd.b, t.bn);
    j.sum_parts = g.sum_parts;
    j.sum_out = g.sum_out;
    j.sum_slices = g.sum_slices;
    total += static_cast<long long>(j.tiles_a) * j.tiles_b;
    if (i == 0) p.first = static_cast<int>(total);
  }
  if (total * t.split >= (1ll << 31)) return cudaErrorInvalidValue;
  p.total = static_cast<int>(total);
  // Float32 results leave the tensor core after 128 (six products per value, so the drain still
  // hides behind the MMAs) or 256 values; bf16 ones are rounded far above its error up to
  // kMaxChunk
  p.chunk = jobs[0].planes == 3 ? 2 : jobs[0].c_f32 ? 4 : kMaxChunk;
  auto go = [&](auto pl) {
    constexpr int PL = decltype(pl)::value;
    if (t.ba == 64) {
      switch (t.bn) {
        case 16: return launch_tile<64, 16, PL>(p, t.split, s);
        case 32: return launch_tile<64, 32, PL>(p, t.split, s);
        default: return launch_tile<64, 64, PL>(p, t.split, s);
      }
    }
    switch (t.bn) {
      case 16: return launch_tile<128, 16, PL>(p, t.split, s);
      case 32: return launch_tile<128, 32, PL>(p, t.split, s);
      case 64: return launch_tile<128, 64, PL>(p, t.split, s);
      default: return launch_tile<128, 128, PL>(p, t.split, s);
    }
  };
  return jobs[0].planes == 3 ? go(std::integral_constant<int, 3>{})
                             : go(std::integral_constant<int, 1>{});
}

}  // namespace

bool linear_gemm_on_pairs(const LinearGemm& g, int num_sms) { return prefer_pairs(g, num_sms); }

// What a second launch costs in the estimate's clocks: with 4000 more shapes lost by it than with
// 8000.  Two products share a launch, and with it tile and split, unless their own choices save
// more than that: a dx of few tiles and a long reduction wants a split that a dW of many tiles and
// a short one would repay with waves (70 rows, 192 -> 5312, float32: 81 us together, 27 apart; 128
// rows, 2048 -> 7168: 172 and 131).  Where the two come close the estimate can be wrong: of 24
// shapes of 8 to 1896 rows within 10% of the border on the side of two launches, 16 gain 5 to 28%
// by them (80 rows, 200 -> 4616, bf16 19.7 -> 14.2 us), three are equal and five lose 2 to 14%
// (920 rows, 1920 -> 392, float32 36.3 -> 41.5 us).
constexpr double kLaunchClocks = 8000.0;

cudaError_t launch_linear_gemms(const LinearGemm* jobs, int n, unsigned* err, int num_sms,
                                cudaStream_t s) {
  if (n == 2 && !prefer_pairs(jobs[0], num_sms) && !prefer_pairs(jobs[1], num_sms)) {
    // the longer tiles first: the shorter ones fill the last wave better
    const int longer = jobs[0].depth >= jobs[1].depth ? 0 : 1;
    const LinearGemm by_depth[2] = {jobs[longer], jobs[1 - longer]};
    const TileChoice joint = choose_tile(by_depth, 2, num_sms);
    const TileChoice apart[2] = {choose_tile(by_depth, 1, num_sms),
                                 choose_tile(by_depth + 1, 1, num_sms)};
    if (joint.cost <= apart[0].cost + apart[1].cost + kLaunchClocks)
      return launch_tiles(by_depth, 2, joint, err, s);
    for (int i = 0; i < 2; ++i) {
      const cudaError_t e = launch_tiles(by_depth + i, 1, apart[i], err, s);
      if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
  }
  for (int i = 0; i < n; ++i) {
    const cudaError_t e = prefer_pairs(jobs[i], num_sms)
                              ? launch_pairs(jobs[i], err, num_sms, s)
                              : launch_tiles(jobs + i, 1, choose_tile(jobs + i, 1, num_sms), err, s);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace moe
