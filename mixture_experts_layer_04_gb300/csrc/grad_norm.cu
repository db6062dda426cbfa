// moe_clip_grad_norm: the 2-norm over many gradients and the gradients scaled down to a largest
// norm.
//
//   norm = scale * sqrt(sum over the tensors and their elements of g^2);
//   out  = g * scale * min(1, max_norm / (norm + eps)).
//
// Two launches (per kPerLaunch tensors).  The list of tensors travels as a kernel parameter, so
// nothing is copied to the device and the call can be captured.  A tensor is cut into chunks; a
// block takes every gridDim.x-th chunk and leaves one 64-bit partial sum.  The second launch adds
// the partial sums up in order, in every block, and scales; it walks the chunks from the last to
// the first, because the last ones read are what L2 still holds.
//
// Squares: eight elements are squared and added in float, and those sums added in pairs of floats
// (an addition in 64 bits per eight bf16 elements would take two thirds of what the 64-bit units
// can do).  Where a square would leave float's range (above 2^96, or the largest element below
// 2^-55 and not 0) the eight are squared in 64 bits.
//
// Bound by memory: 150 bf16 tensors of 640 M elements 206 us (6.2 TB/s) and 393 us (6.5 TB/s), 603
// us a call, 574 at a copy's rate with the second read.  23 tensors of 300 K elements 8.1 us: two
// launches.
#include <cmath>

#include "common.cuh"
#include "kernels.h"
#include "operand_io.cuh"

namespace moe {
namespace {

constexpr int kPerLaunch = 512;  // tensors: 32 bytes each in the kernel's parameters
constexpr int kFewTensors = 64;  // a list that short has a kernel with as short a parameter
constexpr int kThreads = 512;
constexpr int kLeastChunk = 4096, kMostChunk = 32768;  // elements
// Blocks per SM: both kernels want registers for their loads (the scaling compiled for four blocks of
// 32 registers spills 268 bytes: 640 M elements 608 us a call instead of 603, 23 tensors of 300 K
// 9.7 instead of 8.1).  The short list's holds its first loads while it works the factor out, and
// spills 132 bytes even so.
constexpr int kBlocksPerSm = 2;
constexpr int kMostBlocks = 1024;

struct Entry {
  const void* grad;
  void* out;
  int first_chunk;
  int types;  // bit 0: grad is bf16, bit 1: out is bf16
};
// CAP: tensors that a launch's list has room for.  A short list's chunks name their tensors, where
// they are few, so that no block has to search for its own.
constexpr int kNamedChunks = 1024;
template <int CAP>
struct ClipParams {
  Entry e[CAP];
  long long size[CAP];
  unsigned char tensor_of[CAP <= kFewTensors ? kNamedChunks : 1];
  double* parts;
  float* norm;
  int tensors, chunks, chunk;
  int parts_before;  // partial sums of the launches before this one
  int parts_total;
  float scale, max_norm, eps;
};
static_assert(sizeof(ClipParams<kPerLaunch>) <= 32764, "kernel parameters");

template <int CAP>
__device__ __forceinline__ int find(const ClipParams<CAP>& p, int chunk) {
  if (CAP <= kFewTensors && p.chunks <= kNamedChunks) return p.tensor_of[chunk];
  int lo = 0, hi = p.tensors;
  while (hi - lo > 1) {
    const int m = (lo + hi) >> 1;
    if (p.e[m].first_chunk <= chunk) lo = m;
    else hi = m;
  }
  return lo;
}

// A chunk of a tensor of a launch's list.
struct Chunk {
  const Entry* e;
  long long at;
  int n;
};
template <int CAP>
__device__ __forceinline__ Chunk chunk_of(const ClipParams<CAP>& p, int c) {
  const int t = find(p, c);
  const long long at = static_cast<long long>(c - p.e[t].first_chunk) * p.chunk;
  const long long left = p.size[t] - at;
  return Chunk{&p.e[t], at, static_cast<int>(left < p.chunk ? left : p.chunk)};
}
__device__ __forceinline__ bool both_aligned(const void* a, const void* b) {
  return ((reinterpret_cast<uintptr_t>(a) | reinterpret_cast<uintptr_t>(b)) & 15u) == 0;
}

struct Raw8 {
  uint4 a, b;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    a = *reinterpret_cast<const uint4*>(p);
  }
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const uint4*>(p)[0];
    b = reinterpret_cast<const uint4*>(p)[1];
  }
  __device__ __forceinline__ void get(const __nv_bfloat16*, float (&v)[8]) const { unpack8(a, v); }
  __device__ __forceinline__ void get(const float*, float (&v)[8]) const {
    v[0] = __uint_as_float(a.x), v[1] = __uint_as_float(a.y), v[2] = __uint_as_float(a.z);
    v[3] = __uint_as_float(a.w), v[4] = __uint_as_float(b.x), v[5] = __uint_as_float(b.y);
    v[6] = __uint_as_float(b.z), v[7] = __uint_as_float(b.w);
  }
};
// A thread's sum: hi + lo is exact but for lo's own roundings (2^-48 of the sum), `rest` takes what
// leaves float's range.
struct Squares {
  float hi = 0.f, lo = 0.f;
  double rest = 0.0;
  // hi + lo += s + l
  __device__ __forceinline__ void join(float s, float l) {
    const float t = __fadd_rn(hi, s), b = __fsub_rn(t, hi);
    lo += l + __fadd_rn(__fsub_rn(hi, __fsub_rn(t, b)), __fsub_rn(s, b));
    hi = t;
  }
  __device__ __forceinline__ void add(const float (&v)[8]) {
    float most = 0.f, s = 0.f;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      most = fmaxf(most, fabsf(v[q]));
      s = fmaf(v[q], v[q], s);
    }
    // (a NaN is not below the limit; 2^31 such sums stay below float's largest)
    if (s < 0x1p96f && (most > 0x1p-55f || most == 0.f)) {
      join(s, 0.f);
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q)
        rest = fma(static_cast<double>(v[q]), static_cast<double>(v[q]), rest);
    }
  }
  // the block's total, in thread 0
  __device__ __forceinline__ double total() {
    __shared__ double part[kThreads / 32];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float h = __shfl_xor_sync(0xffffffffu, hi, o), l = __shfl_xor_sync(0xffffffffu, lo, o);
      join(h, l);
    }
    if (__any_sync(0xffffffffu, rest != 0.0)) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) rest += __shfl_xor_sync(0xffffffffu, rest, o);
    }
    if ((threadIdx.x & 31) == 0)
      part[threadIdx.x >> 5] = static_cast<double>(hi) + static_cast<double>(lo) + rest;
    __syncthreads();
    double sum = 0.0;
    if (threadIdx.x == 0)
      for (int w = 0; w < kThreads / 32; ++w) sum += part[w];
    return sum;
  }
};

template <typename T>
__device__ __forceinline__ void chunk_squares(const T* g, int n, Squares& sum) {
  int done = 0;
  if ((reinterpret_cast<uintptr_t>(g) & 15u) == 0) {
    const int vecs = n / 8;
    done = vecs * 8;
    constexpr int U = sizeof(T) == 2 ? 4 : 2;
    for (int i = threadIdx.x; i < vecs; i += U * kThreads) {
      Raw8 r[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (i + u * kThreads < vecs) r[u].load(g + (i + u * kThreads) * 8);
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (i + u * kThreads < vecs) {
          float v[8];
          r[u].get(g, v);
          sum.add(v);
        }
    }
  }
  for (int i = done + threadIdx.x; i < n; i += 8 * kThreads) {
    float v[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q] = i + q * kThreads < n ? to_f(g[i + q * kThreads]) : 0.f;
    sum.add(v);
  }
}

template <int CAP>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) grad_squares_kernel(
    const __grid_constant__ ClipParams<CAP> p) {
  grid_dep_wait();
  grid_dep_trigger();
  Squares sum;
  for (int c = blockIdx.x; c < p.chunks; c += gridDim.x) {
    const Chunk k = chunk_of(p, c);
    if (k.e->types & 1)
      chunk_squares(static_cast<const __nv_bfloat16*>(k.e->grad) + k.at, k.n, sum);
    else
      chunk_squares(static_cast<const float*>(k.e->grad) + k.at, k.n, sum);
  }
  const double total = sum.total();
  if (threadIdx.x == 0) p.parts[p.parts_before + blockIdx.x] = total;
}

__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
__device__ __forceinline__ void store1(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// first: the thread's first eight elements if `have`
template <int U, typename T, typename O>
__device__ __forceinline__ void chunk_scale(const T* g, O* out, int n, float f, const Raw8& first,
                                            bool have) {
  int done = 0;
  if (both_aligned(g, out)) {
    const int vecs = n / 8;
    done = vecs * 8;
    for (int i = threadIdx.x; i < vecs; i += U * kThreads) {
      Raw8 r[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (i + u * kThreads < vecs) {
          if (u == 0 && have) r[u] = first;
          else r[u].load(g + (i + u * kThreads) * 8);
        }
      have = false;
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (i + u * kThreads < vecs) {
          float v[8];
          r[u].get(g, v);
#pragma unroll
          for (int q = 0; q < 8; ++q) v[q] *= f;
          store8(out + (i + u * kThreads) * 8, v);
        }
    }
  }
  for (int i = done + threadIdx.x; i < n; i += kThreads) store1(out + i, to_f(g[i]) * f);
}

// Newton's step in 64 bits from a float estimate, which doubles its 22 bits; far from 1 the
// library's routines.
__device__ __forceinline__ bool moderate(double v) { return v > 0x1p-100 && v < 0x1p100; }
__device__ __forceinline__ double root_of(double v) {
  if (!moderate(v)) return sqrt(v);
  const double y = static_cast<double>(rsqrtf(static_cast<float>(v))), r = v * y;
  return fma(fma(-r, r, v), 0.5 * y, r);
}
__device__ __forceinline__ double quotient(double a, double b) {
  if (!moderate(a) || !moderate(b)) return a / b;
  const double y = static_cast<double>(1.f / static_cast<float>(b)), q = a * y;
  return fma(fma(-q, b, a), y, q);
}

template <int CAP>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) grad_scale_kernel(
    const __grid_constant__ ClipParams<CAP> p) {
  // A short list's first gradients are on their way while the factor is worked out.
  constexpr bool kAhead = CAP <= kFewTensors;
  constexpr int U = 2;
  int c = p.chunks - 1 - static_cast<int>(blockIdx.x);
  Chunk k{};
  Raw8 first;
  bool have = false;
  if (c >= 0) k = chunk_of(p, c);
  grid_dep_wait();
  grid_dep_trigger();
  if (kAhead && c >= 0) {
    const bool bf16 = k.e->types & 1;
    const char* g = static_cast<const char*>(k.e->grad) + k.at * (bf16 ? 2 : 4);
    const char* out = static_cast<const char*>(k.e->out) + k.at * (k.e->types & 2 ? 2 : 4);
    if (both_aligned(g, out) && static_cast<int>(threadIdx.x) < k.n / 8) {
      if (bf16) first.load(reinterpret_cast<const __nv_bfloat16*>(g) + threadIdx.x * 8);
      else first.load(reinterpret_cast<const float*>(g) + threadIdx.x * 8);
      have = true;
    }
  }
  // One warp adds the partial sums and one thread takes the root: the 64-bit units do two
  // operations a clock (in all 512 threads this took 6 us).
  __shared__ float factor;
  if (threadIdx.x < 32) {
    double total = 0.0;
    for (int i = threadIdx.x; i < p.parts_total; i += 32) total += p.parts[i];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    if (threadIdx.x == 0) {
      const double norm = root_of(total) * static_cast<double>(p.scale);
      if (p.norm != nullptr && blockIdx.x == 0) *p.norm = static_cast<float>(norm);
      // a norm that is NaN makes the factor NaN; an infinite one makes it 0, but where max_norm is
      // infinite, too: then there is nothing to clip to, and the quotient would be NaN
      const double room =
          p.max_norm < INFINITY
              ? quotient(static_cast<double>(p.max_norm), norm + static_cast<double>(p.eps))
              : norm == norm ? 1.0 : norm;
      factor = static_cast<float>(static_cast<double>(p.scale) *
                                  (room < 1.0 || room != room ? room : 1.0));
    }
  }
  __syncthreads();
  const float f = factor;
  while (c >= 0) {
    const Entry& e = *k.e;
    const long long at = k.at;
    if (f == 1.f && e.grad == e.out) {
      // in place, nothing to change
    } else if (e.types == 0) {
      chunk_scale<U>(static_cast<const float*>(e.grad) + at, static_cast<float*>(e.out) + at, k.n, f,
                  first, have);
    } else if (e.types == 1) {
      chunk_scale<U>(static_cast<const __nv_bfloat16*>(e.grad) + at, static_cast<float*>(e.out) + at,
                  k.n, f, first, have);
    } else if (e.types == 2) {
      chunk_scale<U>(static_cast<const float*>(e.grad) + at, static_cast<__nv_bfloat16*>(e.out) + at,
                  k.n, f, first, have);
    } else {
      chunk_scale<U>(static_cast<const __nv_bfloat16*>(e.grad) + at,
                  static_cast<__nv_bfloat16*>(e.out) + at, k.n, f, first, have);
    }
    c -= static_cast<int>(gridDim.x);
    if (c >= 0) k = chunk_of(p, c);
    have = false;
  }
}

// --------------------------------------------------------------------- host ----

moe_status_t check_tensors(const moe_grad_t* grads, int n) {
  if (n < 0 || n > (1 << 20) || (n > 0 && grads == nullptr)) return MOE_ERR_INVALID_ARG;
  for (int i = 0; i < n; ++i) {
    const moe_grad_t& g = grads[i];
    if (g.size < 0 || g.size > (1ll << 40)) return MOE_ERR_INVALID_ARG;
    if ((g.dtype != MOE_F32 && g.dtype != MOE_BF16) ||
        (g.out_dtype != MOE_F32 && g.out_dtype != MOE_BF16))
      return MOE_ERR_INVALID_ARG;
    if (g.size > 0 && g.grad == nullptr) return MOE_ERR_INVALID_ARG;
    if (g.out == g.grad && g.out != nullptr && g.dtype != g.out_dtype) return MOE_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(g.grad) % act_bytes(g.dtype) != 0 ||
        reinterpret_cast<uintptr_t>(g.out) % act_bytes(g.out_dtype) != 0)
      return MOE_ERR_MISALIGNED;
  }
  return MOE_OK;
}

inline long long launches_for(int n) { return n == 0 ? 1 : (n + kPerLaunch - 1) / kPerLaunch; }

template <int CAP>
moe_status_t run_clip(const moe_grad_t* grads, int n, float grad_scale, float max_norm, float eps,
                      float* norm, void* ws, cudaStream_t s) {
  const int sms = device_num_sms();
  auto blocks_of = [&](int chunks) {
    const int most = sms * kBlocksPerSm < kMostBlocks ? sms * kBlocksPerSm : kMostBlocks;
    return chunks < most ? (chunks > 0 ? chunks : 1) : most;
  };
  const long long launches = n == 0 ? 1 : (n + CAP - 1) / CAP;
  ClipParams<CAP> p;
  p.parts = static_cast<double*>(ws);
  p.scale = grad_scale;
  p.max_norm = max_norm;
  p.eps = eps;
  // chunks small enough that a short list fills the blocks (23 tensors of 300 K elements: 18.0 us
  // with 32768 elements, 9.9 with 4096), large enough that a block seldom looks for its tensor
  long long total = 0;
  for (int i = 0; i < n; ++i) total += grads[i].size;
  p.chunk = kLeastChunk;
  while (p.chunk < kMostChunk && total / p.chunk > 32ll * sms) p.chunk *= 2;
  // one batch of the list: tensors with elements, and with results where `scaling`
  auto fill = [&](long long batch, bool scaling) -> bool {
    p.tensors = 0;
    long long chunks = 0;
    const int end = static_cast<int>((batch + 1) * CAP < n ? (batch + 1) * CAP : n);
    for (int i = static_cast<int>(batch * CAP); i < end; ++i) {
      const moe_grad_t& g = grads[i];
      if (g.size == 0 || (scaling && g.out == nullptr)) continue;
      Entry& e = p.e[p.tensors];
      e.grad = g.grad;
      e.out = g.out;
      e.first_chunk = static_cast<int>(chunks);
      e.types = (g.dtype == MOE_BF16 ? 1 : 0) | (g.out_dtype == MOE_BF16 ? 2 : 0);
      const long long end_chunk = chunks + (g.size + p.chunk - 1) / p.chunk;
      if (CAP <= kFewTensors)
        for (long long c = chunks; c < end_chunk && c < kNamedChunks; ++c)
          p.tensor_of[c] = static_cast<unsigned char>(p.tensors);
      p.size[p.tensors++] = g.size;
      chunks = end_chunk;
      if (chunks >= (1ll << 30)) return false;
    }
    p.chunks = static_cast<int>(chunks);
    return true;
  };
  for (long long b = 0; b < launches; ++b)
    if (!fill(b, false)) return MOE_ERR_UNSUPPORTED;
  int parts = 0;
  for (long long b = 0; b < launches; ++b) {
    fill(b, false);
    p.norm = nullptr;
    p.parts_before = parts;
    p.parts_total = 0;
    if (p.chunks == 0) continue;
    const int blocks = blocks_of(p.chunks);
    if (launch_pdl(grad_squares_kernel<CAP>, dim3(static_cast<unsigned>(blocks)), dim3(kThreads), 0,
                   s, p) != cudaSuccess)
      return MOE_ERR_CUDA;
    parts += blocks;
  }
  // scaled last list first, for what L2 still holds; the first launch writes the norm
  float* out = norm;
  for (long long b = launches - 1; b >= 0; --b) {
    fill(b, true);
    if (p.chunks == 0 && (out == nullptr || b > 0)) continue;
    p.norm = out;
    p.parts_before = 0;
    p.parts_total = parts;
    const int blocks = blocks_of(p.chunks);
    if (launch_pdl(grad_scale_kernel<CAP>, dim3(static_cast<unsigned>(blocks)), dim3(kThreads), 0, s,
                   p) != cudaSuccess)
      return MOE_ERR_CUDA;
    out = nullptr;
  }
  return MOE_OK;
}

}  // namespace
}  // namespace moe

extern "C" moe_status_t moe_clip_grad_norm_workspace_size(int n, size_t* bytes) {
  using namespace moe;
  const moe_status_t st = fault_point("moe_clip_grad_norm_workspace_size");
  if (st != MOE_OK) return st;
  if (n < 0 || n > (1 << 20) || bytes == nullptr) return MOE_ERR_INVALID_ARG;
  *bytes = static_cast<size_t>(launches_for(n)) * kMostBlocks * sizeof(double);
  return MOE_OK;
}

extern "C" moe_status_t moe_clip_grad_norm(const moe_grad_t* grads, int n, float grad_scale,
                                           float max_norm, float eps, float* norm, void* ws,
                                           size_t ws_bytes, moe_stream_t stream) {
  using namespace moe;
  moe_status_t st = fault_point("moe_clip_grad_norm");
  if (st != MOE_OK) return st;
  st = check_tensors(grads, n);
  if (st != MOE_OK) return st;
  // (an infinite max_norm: scale alone)
  if (!(grad_scale > 0.f) || !(grad_scale < INFINITY) || !(max_norm > 0.f) || !(eps >= 0.f) ||
      !(eps < INFINITY))
    return MOE_ERR_INVALID_ARG;
  bool any_out = false;
  for (int i = 0; i < n; ++i) any_out |= grads[i].out != nullptr && grads[i].size > 0;
  if (norm == nullptr && !any_out) return MOE_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(norm) % 4 != 0) return MOE_ERR_MISALIGNED;
  if (ws == nullptr || ws_bytes < static_cast<size_t>(launches_for(n)) * kMostBlocks * sizeof(double))
    return MOE_ERR_WORKSPACE;
  if (reinterpret_cast<uintptr_t>(ws) % 16 != 0) return MOE_ERR_MISALIGNED;
  st = check_current_device();
  if (st != MOE_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return n <= kFewTensors ? run_clip<kFewTensors>(grads, n, grad_scale, max_norm, eps, norm, ws, s)
                          : run_clip<kPerLaunch>(grads, n, grad_scale, max_norm, eps, norm, ws, s);
}
