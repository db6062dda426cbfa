// moe_block_norm and moe_block_norm_backward: what stands between two blocks of a transformer --
// the norm after a block's output, its gate and scales, the residual sum, and the norm before the
// next block -- in one pass over the rows.
//
// With p = x rx wp (rx the reciprocal root mean square of x) or x, g the row's gate, c the column's
// product of branch scale, channel scale and wp:
//   s = a res + g rx x c;   y = s rs wn.
// Backward, ds the gradient of s:
//   ds  = dsum + rs (dy wn - s rs^2 D1 / W),          D1 = sum of dy wn s;
//   dx  = g rx (ds c - x rx^2 D2 / W),                D2 = sum of ds c x  (no second term without
//   dgate = rx D2 (times the logistic's slope),            the norm after the block)
// and all three vectors' gradients come from two column sums, of dy s rs and of g rx ds x.
//
// A row is read once into registers, reduced twice across its threads (the second sum needs the
// first: adding up squares and cross terms in one pass would cancel where block and residual do) and
// written once; the columns' vectors stay in the threads' registers from row to row, and so do the
// column sums, which leave as one partial per block that a second launch adds up in order.
//
//  - *_rows_kernel, where a group of threads has two rows or more: rows come through a ring of bulk
//    copies in shared memory; 16384 rows of 7168 139 us, 6.7 TB/s, a copy's rate (rows loaded by the
//    threads 265 us).  The backward does 40 operations on every element and two dependent sums per
//    row: 8192 rows of 2048 46 us and 5 for the column sums, of 4096 81 us (5.0 TB/s); float32,
//    with twice the bytes for the same work, 5.4 TB/s;
//  - block_norm_kernel and block_norm_grad_kernel: few rows, the forward of rows that are not
//    multiples of 16 bytes apart and long, and rows of over 8192 columns, which are read again in
//    each pass.  One row of 7168: 4.8 us, the launch.
#include <atomic>
#include <initializer_list>

#include "common.cuh"
#include "kernels.h"
#include "operand_io.cuh"
#include "tc_operand.cuh"
#include "topk.cuh"

namespace moe {
namespace {

// Eight values of a row as they lie in memory.
template <typename T>
struct Eight;
template <>
struct Eight<__nv_bfloat16> {
  uint32_t w[4];
  __device__ __forceinline__ void zero() { w[0] = w[1] = w[2] = w[3] = 0u; }
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
  }
  __device__ __forceinline__ void set(int q, __nv_bfloat16 v) {
    const uint32_t b = __bfloat16_as_ushort(v);
    w[q >> 1] |= q & 1 ? b << 16 : b;
  }
  __device__ __forceinline__ float get(int q) const {
    return __uint_as_float(q & 1 ? w[q >> 1] & 0xffff0000u : w[q >> 1] << 16);
  }
};
template <>
struct Eight<float> {
  float v[8];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q] = 0.f;
  }
  __device__ __forceinline__ void load(const float* p) {
    const float4 a = reinterpret_cast<const float4*>(p)[0];
    const float4 b = reinterpret_cast<const float4*>(p)[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
  __device__ __forceinline__ void set(int q, float x) { v[q] = x; }
  __device__ __forceinline__ float get(int q) const { return v[q]; }
};

// Two floats in a register pair: GB300 does a multiply-add of both in one instruction.
using Pair = unsigned long long;
__device__ __forceinline__ Pair pair(float a, float b) {
  Pair r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ Pair both(float a) { return pair(a, a); }
__device__ __forceinline__ float first(Pair p) {
  float a, b;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p));
  return a;
}
__device__ __forceinline__ float second(Pair p) {
  float a, b;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p));
  return b;
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
  Pair r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
  Pair r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
template <typename T>
__device__ __forceinline__ Pair pair_of(const Eight<T>& e, int i) {
  return pair(e.get(2 * i), e.get(2 * i + 1));
}
__device__ __forceinline__ float add_up(Pair p) { return first(p) + second(p); }
__device__ __forceinline__ void spread(const Pair (&v)[4], float (&out)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    out[2 * i] = first(v[i]);
    out[2 * i + 1] = second(v[i]);
  }
}

__device__ __forceinline__ void store_eight(__nv_bfloat16* p, const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store_eight(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store_one(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void store_one(float* p, float v) { *p = v; }

struct NormParams {
  const void *x, *residual, *sum_in, *dy, *dsum;
  const float *post, *gate, *scale, *norm;
  void *sum, *y, *dx, *dresidual;
  float* dgate;
  float* parts;  // column sums: [blocks][2][width]
  long long ldx, ldr, lds, ldy, lddx, lddr;
  int rows, width, gate_kind;
  int threads;  // per row
  int depth;    // rows on their way per group of threads (ring kernels)
  float eps, residual_scale, branch_scale;
  int lost;  // fault injection: the second row of the blocks' first groups never counts as arrived
  unsigned long long wait_ns;  // after which a ring gives up
  unsigned* err;
};

// The threads of one row: eight columns each, `i` times.  Vec: neighbouring columns, 16-byte
// accesses; else every `threads`-th column.
template <bool Vec>
struct Columns {
  int t, threads, width;
  __device__ __forceinline__ int at(int i, int q) const {
    return Vec ? (i * threads + t) * 8 + q : (i * 8 + q) * threads + t;
  }
  template <typename T>
  __device__ __forceinline__ void load(const T* row, int i, Eight<T>& e) const {
    if constexpr (Vec) {
      if (at(i, 0) < width) e.load(row + at(i, 0));
      else e.zero();
    } else {
      e.zero();
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (at(i, q) < width) e.set(q, row[at(i, q)]);
    }
  }
  template <bool FULL = false, typename T>
  __device__ __forceinline__ void store(T* row, int i, const float (&v)[8]) const {
    if constexpr (Vec) {
      if (FULL || at(i, 0) < width) store_eight(row + at(i, 0), v);
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (at(i, q) < width) store_one(row + at(i, q), v[q]);
    }
  }
  // a vector's values, `none` where there is no vector
  __device__ __forceinline__ void vector(const float* p, int i, float none, float (&v)[8]) const {
#pragma unroll
    for (int q = 0; q < 8; ++q)
      v[q] = p == nullptr ? none : at(i, q) < width ? __ldca(p + at(i, q)) : 0.f;
  }
};

// Sums of N values over the threads of a row; every thread gets them.  `part`: this group's shared
// memory, 4 floats per warp.  (Halving the values among the lanes as they are added up takes half
// the instructions and two more dependent steps, and is slower: 16384 rows of 7168 177 us instead
// of 167, the backward of 8192 rows of 2048 63 instead of 59.)
template <int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float* part, int group, int threads,
                                        int warp) {
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = warp_sum(v[k]);
  if (threads == 32) return;
  const int warps = threads >> 5, lane = threadIdx.x & 31;
  if (lane == 0) {
#pragma unroll
    for (int k = 0; k < N; ++k) part[warp * N + k] = v[k];
  }
  asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(threads) : "memory");
  if (N == 4 && warps <= 8) {  // every thread adds the few warps' sums up by itself
    float4 sum = *reinterpret_cast<const float4*>(part);
#pragma unroll
    for (int w = 1; w < 8; ++w)
      if (w < warps) {
        const float4 x = *reinterpret_cast<const float4*>(part + 4 * w);
        sum.x += x.x, sum.y += x.y, sum.z += x.z, sum.w += x.w;
      }
    const float s[4] = {sum.x, sum.y, sum.z, sum.w};
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = s[k];
    return;
  }
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = warp_sum(lane < warps ? part[lane * N + k] : 0.f);
}

// The gate of a row whose entry is v, and the logistic's slope there.
__device__ __forceinline__ float gate_from(int kind, float v, float* slope) {
  *slope = 1.f;
  if (kind == MOE_GATE_NONE) return 1.f;
  if (kind == MOE_GATE_VALUE) return v;
  const float t = expf(-fabsf(v)), r = __fdividef(1.f, 1.f + t);
  *slope = t * r * r;  // of the logistic function, without the cancellation in 1 - g
  return v >= 0.f ? r : t * r;
}

__device__ __forceinline__ float gate_of(const NormParams& p, int row, float* slope) {
  return gate_from(p.gate_kind, p.gate != nullptr ? p.gate[row] : 0.f, slope);
}

__device__ __forceinline__ float root(float squares, float inv_width, float eps) {
  return rsqrtf(fmaf(squares, inv_width, eps));
}

constexpr int kMaxThreads = 1024;
constexpr int kMaxDepth = 8, kMostGroups = 16;
// Shared memory that a row takes: itself, or the 16-byte pieces that hold it.
__host__ __device__ constexpr int ring_place(int width, int value_bytes, bool aligned) {
  return aligned ? width * value_bytes : (width * value_bytes + 30 + 15) / 16 * 16;
}

// Rows on their way to a group of threads: `depth` slots of shared memory, each with the row of up
// to N arrays (null ones have no place), copied in bulk and counted on the slot's barrier.
//
// Bulk copies take whole 16 bytes.  ALIGNED rows are that; of others the 16-byte pieces that hold
// them are copied, with what they hold of the neighbouring rows.  The first and the last row have
// no neighbour on one side, so a piece that is not all theirs is left out there and its few values
// are read from the array (width >= 16: a piece reaches no further than the next row).
template <typename T, int N, bool ALIGNED>
struct Ring {
  const T* src[N];
  long long ld[N];
  uint32_t base, slot_bytes, bar0;
  uint8_t* smem;
  int width, rows, place, depth;  // place: bytes of a slot that a row takes
  unsigned long long wait_ns;
  volatile int* abort_flag;
  unsigned* err;

  __device__ __forceinline__ void issue(int row, int slot) const {
    const uint32_t bar = bar0 + 8u * slot;
    uint32_t dst = base + slot * slot_bytes;
    if constexpr (ALIGNED) {
      mbar_arrive_expect_tx(bar, slot_bytes);
#pragma unroll
      for (int a = 0; a < N; ++a)
        if (src[a] != nullptr) {
          bulk_copy_g2s(dst, src[a] + row * ld[a], static_cast<uint32_t>(place), bar);
          dst += place;
        }
    } else {
      uint32_t bytes = 0;
#pragma unroll
      for (int a = 0; a < N; ++a)
        if (src[a] != nullptr) bytes += static_cast<uint32_t>(last(a, row) - first(a, row));
      mbar_arrive_expect_tx(bar, bytes);
#pragma unroll
      for (int a = 0; a < N; ++a)
        if (src[a] != nullptr) {
          const uintptr_t from = first(a, row);
          bulk_copy_g2s(dst + static_cast<uint32_t>(from - (start(a, row) & ~kMask)),
                        reinterpret_cast<const void*>(from),
                        static_cast<uint32_t>(last(a, row) - from), bar);
          dst += place;
        }
    }
  }
  __device__ __forceinline__ bool wait(int slot, uint32_t phase) const {
    return mbar_wait(bar0 + 8u * slot, phase, abort_flag, err, wait_ns);
  }
  // The group has given up on `row`, whose slot is the next: what else was sent for must have landed
  // before the ring's memory serves something else or goes back.  One more limit for all of it.
  __device__ __forceinline__ void drain(int row, int step, int slot, uint32_t phase) const {
    volatile int late = 0;
    for (int k = 0; k < depth && row + k * step < rows; ++k) {
      mbar_wait(bar0 + 8u * slot, phase, &late, err, wait_ns);
      if (++slot == depth) {
        slot = 0;
        phase ^= 1u;
      }
    }
  }
  // The thread's columns of the slot's rows (zeros for null arrays and past the end; FULL: there
  // are none).
  template <bool FULL, typename C>
  __device__ __forceinline__ void read(int slot, int row, const C& col, int i,
                                       Eight<T> (&e)[N]) const {
    const uint8_t* from = smem + slot * slot_bytes;
    if constexpr (ALIGNED) {
      const int at = col.at(i, 0);
#pragma unroll
      for (int a = 0; a < N; ++a) {
        if (FULL || (src[a] != nullptr && at < width))
          e[a].load(reinterpret_cast<const T*>(from) + at);
        else
          e[a].zero();
        if (FULL || src[a] != nullptr) from += place;
      }
    } else {
      const bool edge = row == 0 || row == rows - 1;
#pragma unroll
      for (int a = 0; a < N; ++a) {
        e[a].zero();
        if (src[a] == nullptr) continue;
        const T* values = reinterpret_cast<const T*>(from + (start(a, row) & kMask));
        if (!edge) {
#pragma unroll
          for (int q = 0; q < 8; ++q)
            if (col.at(i, q) < width) e[a].set(q, values[col.at(i, q)]);
        } else {
          const T* array = src[a] + row * ld[a];
          const uintptr_t lo = first(a, row), hi = last(a, row);
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            const int c = col.at(i, q);
            const uintptr_t at = reinterpret_cast<uintptr_t>(array + c);
            if (c < width) e[a].set(q, at >= lo && at < hi ? values[c] : array[c]);
          }
        }
        from += place;
      }
    }
  }

 private:
  static constexpr uintptr_t kMask = 15;
  __device__ __forceinline__ uintptr_t start(int a, int row) const {
    return reinterpret_cast<uintptr_t>(src[a] + row * ld[a]);
  }
  // what is copied of a row that is not aligned
  __device__ __forceinline__ uintptr_t first(int a, int row) const {
    return row == 0 ? (start(a, row) + kMask) & ~kMask : start(a, row) & ~kMask;
  }
  __device__ __forceinline__ uintptr_t last(int a, int row) const {
    const uintptr_t end = start(a, row) + width * sizeof(T);
    return row == rows - 1 ? end & ~kMask : (end + kMask) & ~kMask;
  }
};

// Sets a group's ring up and sends for its first rows.  Every thread of the block calls it.
template <typename T, int N, bool ALIGNED>
__device__ __forceinline__ void start_ring(Ring<T, N, ALIGNED>& r, uint8_t* rings, uint64_t* bars,
                                           int width, int depth, int lost, int group, int groups,
                                           bool leader, int row, int step, int rows) {
  int arrays = 0;
#pragma unroll
  for (int a = 0; a < N; ++a) arrays += r.src[a] != nullptr;
  r.width = width;
  r.rows = rows;
  r.place = ring_place(width, static_cast<int>(sizeof(T)), ALIGNED);
  r.slot_bytes = static_cast<uint32_t>(arrays * r.place);
  r.depth = depth;
  r.smem = rings + static_cast<size_t>(group) * depth * r.slot_bytes;
  r.base = smem_u32(r.smem);
  r.bar0 = smem_u32(bars + group * kMaxDepth);
  if (leader)
    for (int k = 0; k < depth; ++k)  // (a lost slot lacks an arrival)
      mbar_init(r.bar0 + 8u * k, lost && group == 0 && k == 1 ? 2 : 1);
  fence_mbar_init();
  __syncthreads();
  grid_dep_wait();
  grid_dep_trigger();
  if (leader)
    for (int k = 0; k < depth && row + k * step < rows; ++k) r.issue(row + k * step, k);
}
// Partial sums of the warps: at most kMaxThreads / 32 of them, 4 values, two areas.
constexpr int kPartFloats = kMaxThreads / 32 * 4;

// V: columns a thread keeps, in eights; 0: rows are read again in each pass.  NT: threads at most.
template <typename T, int V, bool Vec, int NT>
__global__ void __launch_bounds__(NT)
    block_norm_kernel(const __grid_constant__ NormParams p) {
  __shared__ __align__(16) float part[2][kPartFloats];
  grid_dep_wait();
  grid_dep_trigger();
  const int group = threadIdx.x / p.threads, groups = blockDim.x / p.threads;
  const Columns<Vec> col{static_cast<int>(threadIdx.x) - group * p.threads, p.threads, p.width};
  const int n = V > 0 ? V : (p.width + 8 * p.threads - 1) / (8 * p.threads);
  const float inv_width = 1.f / static_cast<float>(p.width);
  float* mine[2] = {part[0] + group * (p.threads >> 5) * 4, part[1] + group * (p.threads >> 5) * 4};
  constexpr int R = V > 0 ? V : 1;
  float c[R][8], wn[R][8];
  auto vectors = [&](int i, float (&cv)[8], float (&nv)[8]) {
    float post[8], scale[8];
    col.vector(p.post, i, 1.f, post);
    col.vector(p.scale, i, 1.f, scale);
    col.vector(p.norm, i, 1.f, nv);
#pragma unroll
    for (int q = 0; q < 8; ++q) cv[q] = p.branch_scale * scale[q] * post[q];
  };
  if constexpr (V > 0) {
#pragma unroll
    for (int i = 0; i < V; ++i) vectors(i, c[i], wn[i]);
  }
  Eight<T> x[R], res[R];
  auto load_row = [&](int row, int i, Eight<T>& ex, Eight<T>& er) {
    col.load(static_cast<const T*>(p.x) + row * p.ldx, i, ex);
    if (p.residual != nullptr) col.load(static_cast<const T*>(p.residual) + row * p.ldr, i, er);
    else er.zero();
  };
  const int step = gridDim.x * groups;
  int row = blockIdx.x * groups + group;
  if constexpr (V > 0) {
    if (row < p.rows) {
#pragma unroll
      for (int i = 0; i < V; ++i) load_row(row, i, x[i], res[i]);
    }
  }
  for (; row < p.rows; row += step) {
    float slope;
    float f = gate_of(p, row, &slope);
    if (p.post != nullptr) {
      float sq[1] = {0.f};
#pragma unroll
      for (int i = 0; i < n; ++i) {
        if constexpr (V == 0) col.load(static_cast<const T*>(p.x) + row * p.ldx, i, x[0]);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const float v = x[V > 0 ? i : 0].get(q);
          sq[0] = fmaf(v, v, sq[0]);
        }
      }
      row_sum<1>(sq, mine[0], group, p.threads, col.t >> 5);
      f *= root(sq[0], inv_width, p.eps);
    }
    float s[R][8];
    auto make = [&](int i, const Eight<T>& ex, const Eight<T>& er, const float (&cv)[8],
                    float (&sv)[8]) {
#pragma unroll
      for (int q = 0; q < 8; ++q)
        sv[q] = fmaf(f * ex.get(q), cv[q], p.residual_scale * er.get(q));
    };
    float sq[1] = {0.f};
    if constexpr (V > 0) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        make(i, x[i], res[i], c[i], s[i]);
#pragma unroll
        for (int q = 0; q < 8; ++q) sq[0] = fmaf(s[i][q], s[i][q], sq[0]);
        // the next row is on its way while this one is reduced
        if (row + step < p.rows) load_row(row + step, i, x[i], res[i]);
        if (p.sum != nullptr) col.store(static_cast<T*>(p.sum) + row * p.lds, i, s[i]);
      }
    } else if (p.y != nullptr) {
      for (int i = 0; i < n; ++i) {
        vectors(i, c[0], wn[0]);
        load_row(row, i, x[0], res[0]);
        make(i, x[0], res[0], c[0], s[0]);
#pragma unroll
        for (int q = 0; q < 8; ++q) sq[0] = fmaf(s[0][q], s[0][q], sq[0]);
      }
    }
    float rs = 0.f;
    if (p.y != nullptr) {
      row_sum<1>(sq, mine[1], group, p.threads, col.t >> 5);
      rs = root(sq[0], inv_width, p.eps);
    }
#pragma unroll
    for (int i = 0; i < n; ++i) {
      if constexpr (V == 0) {
        vectors(i, c[0], wn[0]);
        load_row(row, i, x[0], res[0]);
        make(i, x[0], res[0], c[0], s[0]);
        if (p.sum != nullptr) col.store(static_cast<T*>(p.sum) + row * p.lds, i, s[0]);
      }
      if (p.y != nullptr) {
        float v[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] = s[V > 0 ? i : 0][q] * rs * wn[V > 0 ? i : 0][q];
        col.store(static_cast<T*>(p.y) + row * p.ldy, i, v);
      }
    }
    if (p.y == nullptr || p.post == nullptr) {
      // one reduction a row: its area must not be written again before every warp has read it
      if (p.threads > 32 && (p.y != nullptr || p.post != nullptr))
        asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(p.threads) : "memory");
    }
  }
}

// The block's column sums to its partial: the groups' sums, in order.  Every thread of the block
// calls it; columns: [groups - 1][2][width].
template <int V, typename C>
__device__ __forceinline__ void leave_columns(const NormParams& p, const C& col, float* columns,
                                              int group, int groups, const float (&sum_n)[V][8],
                                              const float (&sum_a)[V][8]) {
  float* out = p.parts + static_cast<size_t>(blockIdx.x) * 2 * p.width;
  if (group > 0) {
    float* to = columns + static_cast<size_t>(group - 1) * 2 * p.width;
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (col.at(i, q) < p.width) {
          to[col.at(i, q)] = sum_n[i][q];
          to[p.width + col.at(i, q)] = sum_a[i][q];
        }
  }
  __syncthreads();
  if (group > 0) return;
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const int at = col.at(i, q);
      if (at >= p.width) continue;
      float a = sum_n[i][q], b = sum_a[i][q];
      for (int k = 0; k + 1 < groups; ++k) {
        a += columns[static_cast<size_t>(k) * 2 * p.width + at];
        b += columns[(static_cast<size_t>(k) * 2 + 1) * p.width + at];
      }
      out[at] = a;
      out[p.width + at] = b;
    }
}

// A row's sums: of x^2, s^2 and dy wn s; then of ds c x.
template <typename T, int V, bool Vec, int NT>
__global__ void __launch_bounds__(NT)
    block_norm_grad_kernel(const __grid_constant__ NormParams p) {
  __shared__ __align__(16) float part[2][kPartFloats];
  extern __shared__ float columns[];  // V > 0: [groups - 1][2][width]
  grid_dep_wait();
  grid_dep_trigger();
  const int group = threadIdx.x / p.threads, groups = blockDim.x / p.threads;
  const Columns<Vec> col{static_cast<int>(threadIdx.x) - group * p.threads, p.threads, p.width};
  const int n = V > 0 ? V : (p.width + 8 * p.threads - 1) / (8 * p.threads);
  const float inv_width = 1.f / static_cast<float>(p.width);
  float* mine[2] = {part[0] + group * (p.threads >> 5) * 4, part[1] + group * (p.threads >> 5) * 4};
  constexpr int R = V > 0 ? V : 1;
  float* out = p.parts == nullptr ? nullptr
                                  : p.parts + static_cast<size_t>(blockIdx.x) * 2 * p.width;
  float c[R][8], wn[R][8], sum_n[R][8], sum_a[R][8];
  auto vectors = [&](int i, float (&cv)[8], float (&nv)[8]) {
    float post[8], scale[8];
    col.vector(p.post, i, 1.f, post);
    col.vector(p.scale, i, 1.f, scale);
    col.vector(p.norm, i, 0.f, nv);
#pragma unroll
    for (int q = 0; q < 8; ++q) cv[q] = p.branch_scale * scale[q] * post[q];
  };
  if constexpr (V > 0) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      vectors(i, c[i], wn[i]);
#pragma unroll
      for (int q = 0; q < 8; ++q) sum_n[i][q] = sum_a[i][q] = 0.f;
    }
  } else if (out != nullptr) {  // the block's partial sums live in memory (one group a block)
    for (int k = threadIdx.x; k < 2 * p.width; k += blockDim.x) out[k] = 0.f;
    __syncthreads();
  }
  Eight<T> x[R], s[R], dy[R], ds[R];
  auto load_one = [&](const void* base, long long ld, int row, int i, Eight<T>& e) {
    if (base != nullptr) col.load(static_cast<const T*>(base) + row * ld, i, e);
    else e.zero();
  };
  auto load_row = [&](int row, int i) {
    constexpr bool keep = V > 0;
    load_one(p.x, p.ldx, row, i, x[keep ? i : 0]);
    load_one(p.sum_in, p.lds, row, i, s[keep ? i : 0]);
    load_one(p.dy, p.ldy, row, i, dy[keep ? i : 0]);
    load_one(p.dsum, p.lds, row, i, ds[keep ? i : 0]);
    if constexpr (!keep) vectors(i, c[0], wn[0]);
  };
  const int step = gridDim.x * groups;
  for (int row = blockIdx.x * groups + group; row < p.rows; row += step) {
    float slope;
    const float g = gate_of(p, row, &slope);
    float sums[3] = {0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < n; ++i) {
      load_row(row, i);
      const int k = V > 0 ? i : 0;
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const float vx = x[k].get(q), vs = s[k].get(q);
        sums[0] = fmaf(vx, vx, sums[0]);
        sums[1] = fmaf(vs, vs, sums[1]);
        sums[2] = fmaf(dy[k].get(q) * wn[k][q], vs, sums[2]);
      }
    }
    row_sum<3>(sums, mine[0], group, p.threads, col.t >> 5);
    const float rx = p.post != nullptr ? root(sums[0], inv_width, p.eps) : 1.f;
    const float rs = p.dy != nullptr ? root(sums[1], inv_width, p.eps) : 0.f;
    const float d1 = rs * rs * (sums[2] * inv_width);
    auto grad = [&](int k, int q) {  // ds
      return fmaf(rs, fmaf(-s[k].get(q), d1, dy[k].get(q) * wn[k][q]), ds[k].get(q));
    };
    float dot[1] = {0.f};
    const bool need_dot = p.post != nullptr || p.dgate != nullptr;
    if (need_dot) {
#pragma unroll
      for (int i = 0; i < n; ++i) {
        if constexpr (V == 0) load_row(row, i);
        const int k = V > 0 ? i : 0;
#pragma unroll
        for (int q = 0; q < 8; ++q) dot[0] = fmaf(grad(k, q) * c[k][q], x[k].get(q), dot[0]);
      }
      row_sum<1>(dot, mine[1], group, p.threads, col.t >> 5);
      if (p.dgate != nullptr && col.t == 0) p.dgate[row] = rx * dot[0] * slope;
    }
    const float d2 = p.post != nullptr ? rx * rx * (dot[0] * inv_width) : 0.f;
    const float f = g * rx;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      if constexpr (V == 0) load_row(row, i);
      const int k = V > 0 ? i : 0;
      float v[8], an[8], aa[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        v[q] = grad(k, q);
        an[q] = dy[k].get(q) * s[k].get(q) * rs;
        aa[q] = f * v[q] * x[k].get(q);
        if constexpr (V > 0) {
          sum_n[i][q] += an[q];
          sum_a[i][q] += aa[q];
        } else if (out != nullptr && col.at(i, q) < p.width) {
          out[col.at(i, q)] += an[q];
          out[p.width + col.at(i, q)] += aa[q];
        }
      }
      if (p.dresidual != nullptr) {
        float r[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) r[q] = p.residual_scale * v[q];
        col.store(static_cast<T*>(p.dresidual) + row * p.lddr, i, r);
      }
      if (p.dx != nullptr) {
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] = f * fmaf(-x[k].get(q), d2, v[q] * c[k][q]);
        col.store(static_cast<T*>(p.dx) + row * p.lddx, i, v);
      }
    }
    // one reduction a row: its area must not be written again before every warp has read it
    if (!need_dot && p.threads > 32)
      asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(p.threads) : "memory");
  }
  if constexpr (V > 0) {
    if (out != nullptr) leave_columns<V>(p, col, columns, group, groups, sum_n, sum_a);
  }
}

// Eight values of a vector: in registers, or (KEEP false) in shared memory.
template <bool KEEP>
struct Vector {
  float v[KEEP ? 8 : 1];
  __device__ __forceinline__ void get(const float* p, float (&out)[8]) const {
    if constexpr (KEEP) {
#pragma unroll
      for (int q = 0; q < 8; ++q) out[q] = v[q];
    } else {
      const float4 a = reinterpret_cast<const float4*>(p)[0];
      const float4 b = reinterpret_cast<const float4*>(p)[1];
      out[0] = a.x, out[1] = a.y, out[2] = a.z, out[3] = a.w;
      out[4] = b.x, out[5] = b.y, out[6] = b.z, out[7] = b.w;
    }
  }
};

// The forward over many rows.  The first sum of the next row is taken with the second sum of the
// present one, so that a row costs one barrier.  V: eights of columns per thread; a thread's
// instructions for a row (two sums, the gate, addresses) cost as much as eight columns' own, so
// two where rows have them.
// FULL: residual, sum and y are all there and the threads' columns are the row's: the checks of
// that would be a quarter of the instructions.
template <typename T, int V, bool FULL>
__global__ void __launch_bounds__(512) block_norm_rows_kernel(const __grid_constant__ NormParams p) {
  __shared__ __align__(16) float part[2][kPartFloats];
  __shared__ uint64_t bars[kMostGroups * kMaxDepth];
  __shared__ int gave_up;
  // Each thread sees for itself whether its row arrived, but a row's threads go on, or leave,
  // together: what is left here before the barrier of the row's sums, they all read behind it (one
  // warp votes: 65536 rows of 256 31.7 us through this).
  __shared__ volatile int missing[2][kMostGroups];
  extern __shared__ __align__(128) uint8_t rings[];
  const int group = threadIdx.x / p.threads, groups = blockDim.x / p.threads;
  const Columns<true> col{static_cast<int>(threadIdx.x) - group * p.threads, p.threads, p.width};
  const int warp = col.t >> 5;
  const float inv_width = 1.f / static_cast<float>(p.width);
  const int step = gridDim.x * groups;
  int row = blockIdx.x * groups + group;
  Ring<T, 2, true> ring;
  if (threadIdx.x == 0) gave_up = 0;
  if (threadIdx.x < 2 * kMostGroups)
    missing[threadIdx.x / kMostGroups][threadIdx.x % kMostGroups] = 0;
  ring.src[0] = static_cast<const T*>(p.x);
  ring.src[1] = static_cast<const T*>(p.residual);
  ring.ld[0] = p.ldx;
  ring.ld[1] = p.ldr;
  ring.wait_ns = p.wait_ns;
  ring.abort_flag = &gave_up;
  ring.err = p.err;
  start_ring(ring, rings, bars, p.width, p.depth, p.lost, group, groups, col.t == 0, row, step,
             p.rows);
  Pair c[V][4], wn[V][4];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    float post[8], scale[8], norm[8];
    col.vector(p.post, i, 1.f, post);
    col.vector(p.scale, i, 1.f, scale);
    col.vector(p.norm, i, 1.f, norm);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      c[i][q] = pair(p.branch_scale * scale[2 * q] * post[2 * q],
                     p.branch_scale * scale[2 * q + 1] * post[2 * q + 1]);
      wn[i][q] = pair(norm[2 * q], norm[2 * q + 1]);
    }
  }
  Eight<T> cur[V][2];
  int slot = 0, area = 0;
  uint32_t phase = 0;
  float sums[2] = {0.f, 0.f};  // of s^2, of the next row's x^2
  float gate = 1.f, slope;
  // (a row's gate is loaded a row ahead of its use)
  auto gate_entry = [&](int r) { return p.gate != nullptr && r < p.rows ? p.gate[r] : 0.f; };
  float entry = gate_entry(row);
  bool ok = row < p.rows;
  auto next_row = [&](int r) {
    gate = gate_from(p.gate_kind, entry, &slope);
    entry = gate_entry(r + step);
    if (!ring.wait(slot, phase)) return false;
    Pair square = both(0.f);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      ring.template read<FULL>(slot, r, col, i, cur[i]);
      if (p.post != nullptr) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const Pair x = pair_of(cur[i][0], q);
          square = fma2(x, x, square);
        }
      }
    }
    sums[1] = add_up(square);
    return true;
  };
  auto reduce = [&](bool arrived) {
    if (!arrived) missing[area][group] = 1;
    row_sum<2>(sums, part[area] + group * (p.threads >> 5) * 2, group, p.threads, warp);
    arrived = p.threads == 32 ? __all_sync(0xffffffffu, arrived) : missing[area][group] == 0;
    area ^= 1;
    return arrived;
  };
  if (ok) ok = reduce(next_row(row));
  for (; ok; row += step) {
    const float f = p.post != nullptr ? gate * root(sums[1], inv_width, p.eps) : gate;
    // the barrier has passed, so every thread has this row out of its slot
    if (p.threads == 32) __syncwarp();
    if (col.t == 0 && row + p.depth * step < p.rows) ring.issue(row + p.depth * step, slot);
    if (++slot == p.depth) {
      slot = 0;
      phase ^= 1u;
    }
    Pair s[V][4], square = both(0.f);
    const Pair f2 = both(f), scale2 = both(p.residual_scale);
    sums[1] = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        s[i][q] = fma2(mul2(f2, pair_of(cur[i][0], q)), c[i][q],
                       mul2(scale2, pair_of(cur[i][1], q)));
        square = fma2(s[i][q], s[i][q], square);
      }
    sums[0] = add_up(square);
    const bool more = row + step < p.rows;
    bool arrived = !more || next_row(row + step);
    if (FULL || p.sum != nullptr) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float v[8];
        spread(s[i], v);
        col.template store<FULL>(static_cast<T*>(p.sum) + row * p.lds, i, v);
      }
    }
    arrived = reduce(arrived);
    if (FULL || p.y != nullptr) {
      const Pair rs = both(root(sums[0], inv_width, p.eps));
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float v[8];
#pragma unroll
        for (int q = 0; q < 4; ++q) s[i][q] = mul2(mul2(s[i][q], rs), wn[i][q]);
        spread(s[i], v);
        col.template store<FULL>(static_cast<T*>(p.y) + row * p.ldy, i, v);
      }
    }
    ok = more && arrived;
  }
  // (in the loop this cost 16384 rows of 7168 162 us instead of 142)
  __syncwarp();
  if (col.t == 0 && (missing[0][group] | missing[1][group]) != 0) ring.drain(row, step, slot, phase);
}

// The backward over many rows: the first sums of the next row are taken with the dot product of the
// present one.  V: eights of columns per thread; with two, c and wn lie in shared memory.
// FULL: every array is there and the threads' columns are the row's, as in the forward.
template <typename T, int V, int NT, bool FULL, bool ALIGNED>
__global__ void __launch_bounds__(NT) block_norm_grad_rows_kernel(
    const __grid_constant__ NormParams p) {
  __shared__ __align__(16) float part[2][kPartFloats];
  __shared__ uint64_t bars[kMostGroups * kMaxDepth];
  __shared__ int gave_up;
  __shared__ volatile int missing[2][kMostGroups];  // as in the forward
  // the rings, then (V > 1) c and wn; after the last row the groups' sums: [groups - 1][2][width]
  extern __shared__ __align__(128) uint8_t rings[];
  float* columns = reinterpret_cast<float*>(rings);
  const int group = threadIdx.x / p.threads, groups = blockDim.x / p.threads;
  const Columns<ALIGNED> col{static_cast<int>(threadIdx.x) - group * p.threads, p.threads, p.width};
  const int warp = col.t >> 5;
  const float inv_width = 1.f / static_cast<float>(p.width);
  const int step = gridDim.x * groups;
  int row = blockIdx.x * groups + group;
  Ring<T, 4, ALIGNED> ring;
  if (threadIdx.x == 0) gave_up = 0;
  if (threadIdx.x < 2 * kMostGroups)
    missing[threadIdx.x / kMostGroups][threadIdx.x % kMostGroups] = 0;
  ring.src[0] = static_cast<const T*>(p.x);
  ring.src[1] = static_cast<const T*>(p.sum_in);
  ring.src[2] = static_cast<const T*>(p.dy);
  ring.src[3] = static_cast<const T*>(p.dsum);
  ring.ld[0] = p.ldx;
  ring.ld[1] = ring.ld[3] = p.lds;
  ring.ld[2] = p.ldy;
  ring.wait_ns = p.wait_ns;
  ring.abort_flag = &gave_up;
  ring.err = p.err;
  start_ring(ring, rings, bars, p.width, p.depth, p.lost, group, groups, col.t == 0, row, step,
             p.rows);
  float* shared_c = reinterpret_cast<float*>(rings + static_cast<size_t>(groups) * p.depth *
                                                         ring.slot_bytes);
  const float* shared_w = shared_c + p.width;
  Vector<V == 1> c[V], wn[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    float post[8], scale[8], norm[8];
    col.vector(p.post, i, 1.f, post);
    col.vector(p.scale, i, 1.f, scale);
    col.vector(p.norm, i, 0.f, norm);
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const float v = p.branch_scale * scale[q] * post[q];
      if constexpr (V == 1) {
        c[i].v[q] = v;
        wn[i].v[q] = norm[q];
      } else if (col.at(i, q) < p.width) {  // (read by the thread that wrote it)
        shared_c[col.at(i, q)] = v;
        shared_c[p.width + col.at(i, q)] = norm[q];
      }
    }
  }
  Pair sum_n[V][4], sum_a[V][4];
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int q = 0; q < 4; ++q) sum_n[i][q] = sum_a[i][q] = both(0.f);
  Eight<T> cur[V][4];
  int slot = 0, area = 0;
  uint32_t phase = 0;
  float sums[4] = {0.f, 0.f, 0.f, 0.f};  // of ds c x; the next row's x^2, s^2, dy wn s
  float gate = 1.f, slope = 1.f;
  // (a row's gate is loaded a row ahead of its use)
  auto gate_entry = [&](int r) { return p.gate != nullptr && r < p.rows ? p.gate[r] : 0.f; };
  float entry = gate_entry(row);
  bool ok = row < p.rows;
  auto next_row = [&](int r, Eight<T> (&e)[V][4]) {
    gate = gate_from(p.gate_kind, entry, &slope);
    entry = gate_entry(r + step);
    if (!ring.wait(slot, phase)) return false;
    Pair xx = both(0.f), ss = xx, ds = xx;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int at = col.at(i, 0);
      ring.template read<FULL>(slot, r, col, i, e[i]);
      if (!FULL && at >= p.width) continue;
      float w[8];
      wn[i].get(shared_w + at, w);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const Pair vx = pair_of(e[i][0], q), vs = pair_of(e[i][1], q);
        xx = fma2(vx, vx, xx);
        ss = fma2(vs, vs, ss);
        ds = fma2(mul2(pair_of(e[i][2], q), pair(w[2 * q], w[2 * q + 1])), vs, ds);
      }
    }
    sums[1] = add_up(xx);
    sums[2] = add_up(ss);
    sums[3] = add_up(ds);
    return true;
  };
  auto reduce = [&](bool arrived) {
    if (!arrived) missing[area][group] = 1;
    row_sum<4>(sums, part[area] + group * (p.threads >> 5) * 4, group, p.threads, warp);
    arrived = p.threads == 32 ? __all_sync(0xffffffffu, arrived) : missing[area][group] == 0;
    area ^= 1;
    return arrived;
  };
  if (ok) ok = reduce(next_row(row, cur));
  for (; ok; row += step) {
    const float rx = p.post != nullptr ? root(sums[1], inv_width, p.eps) : 1.f;
    const float rs = FULL || p.dy != nullptr ? root(sums[2], inv_width, p.eps) : 0.f;
    const float d1 = rs * rs * (sums[3] * inv_width);
    const float f = gate * rx, gate_slope = rx * slope;
    // the barrier has passed, so every thread has this row out of its slot
    if (p.threads == 32) __syncwarp();
    if (col.t == 0 && row + p.depth * step < p.rows) ring.issue(row + p.depth * step, slot);
    if (++slot == p.depth) {
      slot = 0;
      phase ^= 1u;
    }
    Pair v[V][4], dot = both(0.f);
    const Pair rs2 = both(rs), d12 = both(-d1), f2 = both(f), scale2 = both(p.residual_scale);
    Eight<T> x[V];
    sums[1] = sums[2] = sums[3] = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int at = col.at(i, 0);
      float cv[8], w[8];
      if (!FULL && at >= p.width) continue;
      c[i].get(shared_c + at, cv);
      wn[i].get(shared_w + at, w);
      x[i] = cur[i][0];
      Pair r[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const Pair s = pair_of(cur[i][1], q), dy = pair_of(cur[i][2], q), vx = pair_of(x[i], q);
        const Pair ds = fma2(rs2, fma2(s, d12, mul2(dy, pair(w[2 * q], w[2 * q + 1]))),
                             pair_of(cur[i][3], q));
        sum_n[i][q] = fma2(mul2(dy, s), rs2, sum_n[i][q]);
        sum_a[i][q] = fma2(mul2(f2, ds), vx, sum_a[i][q]);
        r[q] = mul2(scale2, ds);
        v[i][q] = mul2(ds, pair(cv[2 * q], cv[2 * q + 1]));
        dot = fma2(v[i][q], vx, dot);
      }
      if (FULL || p.dresidual != nullptr) {
        float out[8];
        spread(r, out);
        col.template store<FULL>(static_cast<T*>(p.dresidual) + row * p.lddr, i, out);
      }
    }
    sums[0] = add_up(dot);
    const bool more = row + step < p.rows;
    const bool arrived = reduce(!more || next_row(row + step, cur));
    if (p.dgate != nullptr && col.t == 0) p.dgate[row] = gate_slope * sums[0];
    if (FULL || p.dx != nullptr) {
      const Pair d2 = both(p.post != nullptr ? -rx * rx * (sums[0] * inv_width) : 0.f);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if (!FULL && col.at(i, 0) >= p.width) continue;
        float out[8];
#pragma unroll
        for (int q = 0; q < 4; ++q) v[i][q] = mul2(f2, fma2(pair_of(x[i], q), d2, v[i][q]));
        spread(v[i], out);
        col.template store<FULL>(static_cast<T*>(p.dx) + row * p.lddx, i, out);
      }
    }
    ok = more && arrived;
  }
  __syncwarp();
  if (col.t == 0 && (missing[0][group] | missing[1][group]) != 0) ring.drain(row, step, slot, phase);
  if (p.parts == nullptr) return;
  __syncthreads();  // every group's last row has left its slot
  float n8[V][8], a8[V][8];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    spread(sum_n[i], n8[i]);
    spread(sum_a[i], a8[i]);
  }
  leave_columns<V>(p, col, columns, group, groups, n8, a8);
}

// The blocks' column sums, added in order, and the vectors' gradients: 32 columns per block, each
// of its 16 warps adds every sixteenth partial.
struct VectorParams {
  const float* parts;
  const float *post, *scale;
  float *dpost, *dscale, *dnorm;
  int blocks, width;
  float branch_scale;
};
constexpr int kVectorWarps = 16;
__global__ void __launch_bounds__(32 * kVectorWarps)
    norm_vectors_kernel(const __grid_constant__ VectorParams p) {
  __shared__ float s[2][kVectorWarps][32];
  grid_dep_wait();
  grid_dep_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float n = 0.f, a = 0.f;
  if (c < p.width) {
#pragma unroll 4
    for (int b = warp; b < p.blocks; b += kVectorWarps) {
      n += p.parts[static_cast<size_t>(b) * 2 * p.width + c];
      a += p.parts[(static_cast<size_t>(b) * 2 + 1) * p.width + c];
    }
  }
  s[0][warp][lane] = n;
  s[1][warp][lane] = a;
  __syncthreads();
  if (warp != 0 || c >= p.width) return;
  n = a = 0.f;
#pragma unroll
  for (int w = 0; w < kVectorWarps; ++w) {
    n += s[0][w][lane];
    a += s[1][w][lane];
  }
  a *= p.branch_scale;
  if (p.dnorm != nullptr) p.dnorm[c] = n;
  if (p.dscale != nullptr) p.dscale[c] = a * (p.post != nullptr ? p.post[c] : 1.f);
  if (p.dpost != nullptr) p.dpost[c] = a * (p.scale != nullptr ? p.scale[c] : 1.f);
}

// --------------------------------------------------------------------- host ----

// How rows lie on threads: `threads` per row, `groups` rows per block at a time.
struct Shape {
  int keep, threads, groups;
};
Shape shape_of(int width, int block) {
  Shape s;
  s.keep = width <= 8 * kMaxThreads ? 1 : 0;
  const int per = s.keep ? 8 : 64;
  const int threads = ((width + per - 1) / per + 31) / 32 * 32;
  s.threads = threads < kMaxThreads ? threads : kMaxThreads;
  const int groups = block / s.threads;
  // (a group of several warps has a named barrier of its own: 15 beside the block's)
  s.groups = s.keep == 0 || groups < 1 ? 1 : groups < 15 ? groups : s.threads == 32 ? 16 : 15;
  return s;
}

moe_status_t check_norm_config(const moe_block_norm_config_t* c) {
  if (c == nullptr) return MOE_ERR_INVALID_ARG;
  if (c->rows < 0 || c->rows > (1 << 30)) return MOE_ERR_INVALID_ARG;
  if (c->width < 1 || c->width > 65536) return MOE_ERR_INVALID_ARG;
  if (c->dtype != MOE_F32 && c->dtype != MOE_BF16) return MOE_ERR_INVALID_ARG;
  if (c->gate < MOE_GATE_NONE || c->gate > MOE_GATE_LOGISTIC) return MOE_ERR_INVALID_ARG;
  const float most = 3.402823466e38f;
  auto finite = [&](float v) { return v >= -most && v <= most; };
  if (!(c->eps > 0.f) || !finite(c->eps) || !finite(c->residual_scale) || !finite(c->branch_scale))
    return MOE_ERR_INVALID_ARG;
  for (long long s : {c->x_stride, c->residual_stride, c->sum_stride, c->y_stride, c->dx_stride,
                      c->dresidual_stride})
    if (s != 0 && (s < c->width || s > (1ll << 31))) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

// Blocks of the backward: their number sets that of the partial column sums.
constexpr int kGradBlock = 512;
int grad_blocks(const moe_block_norm_config_t* c, int num_sms) {
  const Shape s = shape_of(c->width, kGradBlock);
  const long long need = (static_cast<long long>(c->rows) + s.groups - 1) / s.groups;
  return static_cast<int>(need < num_sms ? need : num_sms);
}
// For the workspace's size, which must not depend on the device: no GPU has more.
constexpr int kMostSms = 160;

// The ring kernels' shape: `block` threads at most, rows of `two_from` columns and more 16 columns a
// thread.
constexpr int kRowsBlock = 512;
constexpr int kTwoEights = 512;
Shape rows_shape(int width, int two_from, int block) {
  Shape s;
  s.keep = width <= 16 * kRowsBlock;
  const int per = width < two_from ? 8 : 16;
  s.threads = ((width + per - 1) / per + 31) / 32 * 32;
  const int groups = block / s.threads;
  const int most = s.threads == 32 ? kMostGroups : kMostGroups - 1;  // (named barriers: 1 to 15)
  s.groups = groups < 1 ? 1 : groups < most ? groups : most;
  return s;
}

// The backward's.  With 16 columns a thread it would like more than the 128 registers that 512
// threads leave, so rows that fill no more than 448 threads are compiled for that many (8192 bf16
// rows of 7168: 206 us for 512 threads, 151 for 448).  Float32 rows would spill even so and have 8
// columns a thread where 512 threads reach.
//
// Unaligned rows have 8, every `threads`-th, so that a warp's 2-byte accesses lie next to one
// another, and no ring past 512 threads: 8000 bf16 rows of 2047 96 us, read directly 229; 700 rows
// 22 and 34; 3000 of 333 19 and 27.  (The forward of such rows is bound by its accesses'
// instructions either way and reads directly: 62 us through a ring, 64 without, 65536 rows of 257
// 106 and 101.)
constexpr int kGradBlock448 = 448;
int grad_two_from(int dtype, bool vec) {
  return dtype == MOE_F32 || !vec ? 8 * kRowsBlock + 1 : kTwoEights;
}
Shape grad_rows_shape(int width, int dtype, bool vec) {
  Shape s = rows_shape(width, grad_two_from(dtype, vec), kRowsBlock);
  if (!vec && (width < 16 || width > 8 * kRowsBlock)) s.keep = 0;  // (16: the ring's pieces)
  return s;
}

// Rows in a group's ring, 0: read directly (few rows a group).
constexpr int kRingBytes = 196608;
int ring_depth(const Shape& s, int rows, int blocks, int slot_bytes, int other) {
  if (!s.keep || slot_bytes == 0) return 0;
  const int fits = (kRingBytes - other) / (slot_bytes * s.groups);
  const int depth = fits < kMaxDepth ? fits : kMaxDepth;
  return depth >= 2 && rows / (blocks * s.groups) >= 2 ? depth : 0;
}

long long pick(long long s, int width) { return s != 0 ? s : width; }

NormParams params_of(const moe_block_norm_config_t* c, int threads) {
  NormParams p{};
  p.ldx = pick(c->x_stride, c->width);
  p.ldr = pick(c->residual_stride, c->width);
  p.lds = pick(c->sum_stride, c->width);
  p.ldy = pick(c->y_stride, c->width);
  p.lddx = pick(c->dx_stride, c->width);
  p.lddr = pick(c->dresidual_stride, c->width);
  p.rows = c->rows;
  p.width = c->width;
  p.gate_kind = c->gate;
  p.threads = threads;
  p.eps = c->eps;
  p.residual_scale = c->residual_scale;
  p.branch_scale = c->branch_scale;
  p.wait_ns = kWaitLimitNs;
  return p;
}

// Fault injection: a row that never counts as arrived, so a wait runs out, in 2 ms.
void maybe_lose_a_row(const char* point, NormParams* p) {
  if (p->depth == 0 || fault_point(point) == MOE_OK) return;
  p->lost = 1;
  p->wait_ns = 2000000;
}

// 16-byte accesses to every array, null ones aside.
struct Array {
  const void* p;
  long long ld;
};
bool all_vec(int width, int dtype, std::initializer_list<Array> arrays) {
  const long long bytes = static_cast<long long>(act_bytes(dtype));
  if (width % 8 != 0) return false;
  for (const Array& a : arrays)
    if (a.p != nullptr && (unaligned(a.p, 16) || a.ld * bytes % 16 != 0)) return false;
  return true;
}

template <typename K>
cudaError_t launch_rows(K kernel, const NormParams& p, unsigned blocks, unsigned threads,
                        size_t smem, std::atomic<unsigned long long>* done, cudaStream_t s) {
  if (smem > 40 * 1024) {  // (48 KB by default, of which the static part takes 2)
    const cudaError_t e = allow_smem(kernel, kRingBytes, done);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(kernel, dim3(blocks), dim3(threads), smem, s, p);
}

// Whether the threads' columns are just the row's.
bool whole_rows(const NormParams& p, int per_thread) { return p.threads * per_thread == p.width; }

template <typename T>
cudaError_t launch_forward(const NormParams& p, int keep, bool vec, unsigned blocks,
                           unsigned threads, size_t smem, cudaStream_t s) {
  static std::atomic<unsigned long long> done[4];
  if (p.depth > 0) {
    const bool there = p.residual != nullptr && p.sum != nullptr && p.y != nullptr;
    if (p.width < kTwoEights)
      return there && whole_rows(p, 8)
                 ? launch_rows(block_norm_rows_kernel<T, 1, true>, p, blocks, threads, smem,
                               &done[0], s)
                 : launch_rows(block_norm_rows_kernel<T, 1, false>, p, blocks, threads, smem,
                               &done[1], s);
    return there && whole_rows(p, 16)
               ? launch_rows(block_norm_rows_kernel<T, 2, true>, p, blocks, threads, smem, &done[2],
                             s)
               : launch_rows(block_norm_rows_kernel<T, 2, false>, p, blocks, threads, smem,
                             &done[3], s);
  }
  auto kernel = keep ? (vec ? block_norm_kernel<T, 1, true, kMaxThreads>
                            : block_norm_kernel<T, 1, false, kMaxThreads>)
                     : (vec ? block_norm_kernel<T, 0, true, kMaxThreads>
                            : block_norm_kernel<T, 0, false, kMaxThreads>);
  return launch_pdl(kernel, dim3(blocks), dim3(threads), 0, s, p);
}
template <typename T>
cudaError_t launch_backward(const NormParams& p, int keep, bool vec, unsigned blocks,
                            unsigned threads, size_t smem, cudaStream_t s) {
  static std::atomic<unsigned long long> done[7];
  if (p.depth > 0) {
    if (!vec)
      return launch_rows(block_norm_grad_rows_kernel<T, 1, 512, false, false>, p, blocks, threads,
                         smem, &done[6], s);
    const bool there = p.x != nullptr && p.dy != nullptr && p.dsum != nullptr && p.dx != nullptr &&
                       p.dresidual != nullptr;
    if (p.width < grad_two_from(sizeof(T) == 4 ? MOE_F32 : MOE_BF16, true))
      return there && whole_rows(p, 8)
                 ? launch_rows(block_norm_grad_rows_kernel<T, 1, 512, true, true>, p, blocks,
                               threads, smem, &done[0], s)
                 : launch_rows(block_norm_grad_rows_kernel<T, 1, 512, false, true>, p, blocks,
                               threads, smem, &done[1], s);
    const bool full = there && whole_rows(p, 16);
    if (threads <= kGradBlock448)
      return full ? launch_rows(block_norm_grad_rows_kernel<T, 2, kGradBlock448, true, true>, p,
                                blocks, threads, smem, &done[2], s)
                  : launch_rows(block_norm_grad_rows_kernel<T, 2, kGradBlock448, false, true>, p,
                                blocks, threads, smem, &done[3], s);
    return full ? launch_rows(block_norm_grad_rows_kernel<T, 2, 512, true, true>, p, blocks,
                              threads, smem, &done[4], s)
                : launch_rows(block_norm_grad_rows_kernel<T, 2, 512, false, true>, p, blocks,
                              threads, smem, &done[5], s);
  }
  if (keep && threads <= 512)
    return launch_pdl(vec ? block_norm_grad_kernel<T, 1, true, 512>
                          : block_norm_grad_kernel<T, 1, false, 512>,
                      dim3(blocks), dim3(threads), smem, s, p);
  auto kernel = keep ? (vec ? block_norm_grad_kernel<T, 1, true, kMaxThreads>
                            : block_norm_grad_kernel<T, 1, false, kMaxThreads>)
                     : (vec ? block_norm_grad_kernel<T, 0, true, kMaxThreads>
                            : block_norm_grad_kernel<T, 0, false, kMaxThreads>);
  return launch_pdl(kernel, dim3(blocks), dim3(threads), smem, s, p);
}

}  // namespace
}  // namespace moe

extern "C" moe_status_t moe_block_norm_workspace_size(const moe_block_norm_config_t* cfg,
                                                      size_t* bytes) {
  using namespace moe;
  moe_status_t st = fault_point("moe_block_norm_workspace_size");
  if (st != MOE_OK) return st;
  st = check_norm_config(cfg);
  if (st != MOE_OK) return st;
  if (bytes == nullptr) return MOE_ERR_INVALID_ARG;
  const size_t blocks = static_cast<size_t>(grad_blocks(cfg, kMostSms));
  *bytes = blocks * 2 * cfg->width * 4 + 16;
  return MOE_OK;
}

extern "C" moe_status_t moe_block_norm(const moe_block_norm_config_t* cfg, const void* x,
                                       const void* residual, const float* post_weight,
                                       const float* gate, const float* channel_scale,
                                       const float* norm_weight, void* sum, void* y,
                                       moe_stream_t stream) {
  using namespace moe;
  moe_status_t st = fault_point("moe_block_norm");
  if (st != MOE_OK) return st;
  st = check_norm_config(cfg);
  if (st != MOE_OK) return st;
  if (cfg->rows == 0) return MOE_OK;
  if (x == nullptr || (sum == nullptr && y == nullptr) ||
      (gate == nullptr) != (cfg->gate == MOE_GATE_NONE) ||
      (norm_weight == nullptr) != (y == nullptr))
    return MOE_ERR_INVALID_ARG;
  const size_t ab = act_bytes(cfg->dtype);
  for (const void* q : {x, residual, static_cast<const void*>(sum), static_cast<const void*>(y)})
    if (unaligned(q, ab)) return MOE_ERR_MISALIGNED;
  for (const float* q : {post_weight, gate, channel_scale, norm_weight})
    if (unaligned(q, 4)) return MOE_ERR_MISALIGNED;
  const NormParams q = params_of(cfg, 0);
  // in place, but rows elsewhere: one row's result would overwrite another's input
  if ((sum != nullptr && sum == x && q.lds != q.ldx) ||
      (sum != nullptr && sum == residual && q.lds != q.ldr))
    return MOE_ERR_INVALID_ARG;
  st = check_current_device();
  if (st != MOE_OK) return st;
  const int sms = device_num_sms();
  // one group's rows follow one another through its ring, so a block per SM; without one, blocks
  // of a few groups fill the SMs
  const bool sums = post_weight != nullptr || y != nullptr;
  const bool vec = all_vec(cfg->width, cfg->dtype,
                           {{x, q.ldx}, {residual, q.ldr}, {sum, q.lds}, {y, q.ldy}});
  const int slot = (residual != nullptr ? 2 : 1) * cfg->width * static_cast<int>(ab);
  Shape sh = rows_shape(cfg->width, kTwoEights, kRowsBlock);
  const int depth = sums && vec ? ring_depth(sh, cfg->rows, sms, slot, 0) : 0;
  long long most = sms;
  if (depth == 0) {
    sh = shape_of(cfg->width, 256);
    most = static_cast<long long>(sms) * (kMaxThreads / (sh.threads * sh.groups));
  }
  const int block = sh.threads * sh.groups;
  const long long need = (static_cast<long long>(cfg->rows) + sh.groups - 1) / sh.groups;
  NormParams p = params_of(cfg, sh.threads);
  p.depth = depth;
  maybe_lose_a_row("moe_block_norm.copy", &p);
  p.err = device_error_word();
  p.x = x;
  p.residual = residual;
  p.post = post_weight;
  p.gate = gate;
  p.scale = channel_scale;
  p.norm = norm_weight;
  p.sum = sum;
  p.y = y;
  const unsigned blocks = static_cast<unsigned>(need < most ? need : most);
  const unsigned threads = static_cast<unsigned>(block);
  const size_t smem = static_cast<size_t>(depth) * slot * sh.groups;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return status_of(cfg->dtype == MOE_BF16
                       ? launch_forward<__nv_bfloat16>(p, sh.keep, vec, blocks, threads, smem, s)
                       : launch_forward<float>(p, sh.keep, vec, blocks, threads, smem, s));
}

extern "C" moe_status_t moe_block_norm_backward(
    const moe_block_norm_config_t* cfg, const void* dy, const void* dsum, const void* x,
    const void* sum, const float* post_weight, const float* gate, const float* channel_scale,
    const float* norm_weight, void* dx, void* dresidual, float* dgate, float* dpost_weight,
    float* dchannel_scale, float* dnorm_weight, void* ws, size_t ws_bytes, moe_stream_t stream) {
  using namespace moe;
  moe_status_t st = fault_point("moe_block_norm_backward");
  if (st != MOE_OK) return st;
  st = check_norm_config(cfg);
  if (st != MOE_OK) return st;
  const size_t ab = act_bytes(cfg->dtype);
  for (const void* q : {dy, dsum, x, sum, static_cast<const void*>(dx),
                        static_cast<const void*>(dresidual)})
    if (unaligned(q, ab)) return MOE_ERR_MISALIGNED;
  for (const float* q : {post_weight, gate, channel_scale, norm_weight,
                         static_cast<const float*>(dgate), static_cast<const float*>(dpost_weight),
                         static_cast<const float*>(dchannel_scale),
                         static_cast<const float*>(dnorm_weight)})
    if (unaligned(q, 4)) return MOE_ERR_MISALIGNED;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (cfg->rows == 0) {
    if (dpost_weight == nullptr && dchannel_scale == nullptr && dnorm_weight == nullptr)
      return MOE_OK;
    st = check_current_device();
    if (st != MOE_OK) return st;
    for (float* q : {dpost_weight, dchannel_scale, dnorm_weight})
      if (q != nullptr &&
          cudaMemsetAsync(q, 0, static_cast<size_t>(cfg->width) * 4, s) != cudaSuccess)
        return MOE_ERR_CUDA;
    return MOE_OK;
  }
  const bool vectors = dpost_weight != nullptr || dchannel_scale != nullptr || dnorm_weight != nullptr;
  const bool own = dpost_weight != nullptr || dchannel_scale != nullptr || dgate != nullptr;
  if ((dy == nullptr && dsum == nullptr) ||
      (!vectors && dx == nullptr && dresidual == nullptr && dgate == nullptr) ||
      (dy != nullptr && (sum == nullptr || norm_weight == nullptr)) ||
      (gate == nullptr) != (cfg->gate == MOE_GATE_NONE) ||
      (dgate != nullptr && gate == nullptr) || (dpost_weight != nullptr && post_weight == nullptr) ||
      (dnorm_weight != nullptr && dy == nullptr) ||
      (x == nullptr && (own || (dx != nullptr && post_weight != nullptr))))
    return MOE_ERR_INVALID_ARG;
  Shape sh = shape_of(cfg->width, kGradBlock);
  NormParams p = params_of(cfg, sh.threads);
  // in place, but rows elsewhere, as in the forward
  if (dsum != nullptr && ((dx == dsum && p.lddx != p.lds) || (dresidual == dsum && p.lddr != p.lds)))
    return MOE_ERR_INVALID_ARG;
  const int sms = device_num_sms();
  const size_t need = static_cast<size_t>(grad_blocks(cfg, kMostSms)) * 2 * cfg->width * 4 + 16;
  if (vectors && (ws == nullptr || ws_bytes < need)) return MOE_ERR_WORKSPACE;
  if (vectors && unaligned(ws, 16)) return MOE_ERR_MISALIGNED;
  st = check_current_device();
  if (st != MOE_OK) return st;
  // (read only where something needs it)
  p.x = own || (dx != nullptr && post_weight != nullptr) ? x : nullptr;
  p.sum_in = dy != nullptr ? sum : nullptr;
  p.dy = dy;
  p.dsum = dsum;
  p.post = p.x != nullptr ? post_weight : nullptr;
  p.gate = gate;
  p.scale = channel_scale;
  p.norm = norm_weight;
  p.dx = dx;
  p.dresidual = dresidual;
  p.dgate = dgate;
  p.parts = vectors ? static_cast<float*>(ws) : nullptr;
  const bool vec = all_vec(cfg->width, cfg->dtype,
                           {{p.x, p.ldx}, {p.sum_in, p.lds}, {dy, p.ldy}, {dsum, p.lds},
                            {dx, p.lddx}, {dresidual, p.lddr}});
  int arrays = 0;
  for (const void* q : {p.x, p.sum_in, dy, dsum}) arrays += q != nullptr;
  const int slot = arrays * ring_place(cfg->width, static_cast<int>(ab), vec);
  const Shape rs = grad_rows_shape(cfg->width, cfg->dtype, vec);
  const int vector_bytes =  // c and wn
      vec && cfg->width >= grad_two_from(cfg->dtype, vec) ? 2 * cfg->width * 4 : 0;
  int blocks = grad_blocks(cfg, sms < kMostSms ? sms : kMostSms);
  p.depth = ring_depth(rs, cfg->rows, blocks, slot, vector_bytes);
  if (p.depth > 0) {
    sh = rs;
    p.threads = sh.threads;
    const int most = (cfg->rows + sh.groups - 1) / sh.groups;
    if (blocks > most) blocks = most;
  }
  const unsigned threads = static_cast<unsigned>(sh.threads * sh.groups);
  maybe_lose_a_row("moe_block_norm_backward.copy", &p);
  p.err = device_error_word();
  // the groups' column sums take the rings' place in the end
  const size_t column_sums =
      vectors && sh.keep ? static_cast<size_t>(sh.groups - 1) * 2 * cfg->width * 4 : 0;
  const size_t ring =
      p.depth > 0 ? static_cast<size_t>(p.depth) * slot * sh.groups + vector_bytes : 0;
  const size_t smem = ring > column_sums ? ring : column_sums;
  const unsigned grid = static_cast<unsigned>(blocks);
  const cudaError_t e =
      cfg->dtype == MOE_BF16
          ? launch_backward<__nv_bfloat16>(p, sh.keep, vec, grid, threads, smem, s)
          : launch_backward<float>(p, sh.keep, vec, grid, threads, smem, s);
  if (e != cudaSuccess) return MOE_ERR_CUDA;
  if (!vectors) return MOE_OK;
  VectorParams v{};
  v.parts = static_cast<const float*>(ws);
  v.post = post_weight;
  v.scale = channel_scale;
  v.dpost = dpost_weight;
  v.dscale = dchannel_scale;
  v.dnorm = dnorm_weight;
  v.blocks = blocks;
  v.width = cfg->width;
  v.branch_scale = cfg->branch_scale;
  return status_of(launch_pdl(norm_vectors_kernel,
                              dim3(static_cast<unsigned>((cfg->width + 31) / 32)),
                              dim3(32 * kVectorWarps), 0, s, v));
}
