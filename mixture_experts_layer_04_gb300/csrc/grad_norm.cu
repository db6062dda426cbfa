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
// (the 64-bit units manage an addition per eight bf16 elements at two thirds of their rate, so
// they join the chunks only).  Where a square would leave float's range (above 2^120, or the
// largest element below 2^-55 and not 0) the eight are squared in 64 bits.  Bound by memory.
#include <cmath>

#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kPerLaunch = 512;   // tensors: 24 bytes each in the kernel's parameters
constexpr int kThreads = 512;
constexpr int kChunk = 32768;     // elements
constexpr int kBlocksPerSm = 4;   // of the sum, one partial sum each
constexpr int kMostBlocks = 1024;

struct Entry {
  const void* grad;
  void* out;
  int first_chunk;
  int types;  // bit 0: grad is bf16, bit 1: out is bf16
};
struct Batch {
  Entry e[kPerLaunch];
  // elements past a tensor's whole chunks are found from its size
  long long size[kPerLaunch];
};
struct ClipParams {
  Batch batch;
  double* parts;
  float* norm;
  int tensors, chunks;
  int parts_before;  // partial sums of the launches before this one
  int parts_total;
  float scale, max_norm, eps;
};
static_assert(sizeof(ClipParams) <= 32764, "kernel parameters");

__device__ __forceinline__ int find(const ClipParams& p, int chunk) {
  int lo = 0, hi = p.tensors;
  while (hi - lo > 1) {
    const int m = (lo + hi) >> 1;
    if (p.batch.e[m].first_chunk <= chunk) lo = m;
    else hi = m;
  }
  return lo;
}

__device__ __forceinline__ void unpack8(const uint4& u, float (&v)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
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
__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }

// A thread's sum over a chunk: hi + lo is exact but for lo's own roundings (2^-48 of the sum),
// `rest` takes what leaves float's range.
struct Squares {
  float hi = 0.f, lo = 0.f;
  double rest = 0.0;
  __device__ __forceinline__ void add(const float (&v)[8]) {
    float most = 0.f, s = 0.f;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      most = fmaxf(most, fabsf(v[q]));
      s = fmaf(v[q], v[q], s);
    }
    // (a NaN is not below the limit; a chunk has at most 64 such sums a thread)
    if (s < 0x1p120f && (most > 0x1p-55f || most == 0.f)) {
      const float t = __fadd_rn(hi, s), b = __fsub_rn(t, hi);
      lo += __fadd_rn(__fsub_rn(hi, __fsub_rn(t, b)), __fsub_rn(s, b));
      hi = t;
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q)
        rest = fma(static_cast<double>(v[q]), static_cast<double>(v[q]), rest);
    }
  }
  __device__ __forceinline__ double total() const {
    return static_cast<double>(hi) + static_cast<double>(lo) + rest;
  }
};

template <typename T>
__device__ __forceinline__ double chunk_squares(const T* g, int n) {
  Squares sum;
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
  return sum.total();
}

__device__ __forceinline__ double block_sum(double v) {
  __shared__ double s[kThreads / 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) v += s[w];
  return v;
}

__global__ void __launch_bounds__(kThreads) grad_squares_kernel(
    const __grid_constant__ ClipParams p) {
  grid_dep_wait();
  grid_dep_trigger();
  double sum = 0.0;
  for (int c = blockIdx.x; c < p.chunks; c += gridDim.x) {
    const int t = find(p, c);
    const long long at = static_cast<long long>(c - p.batch.e[t].first_chunk) * kChunk;
    const long long left = p.batch.size[t] - at;
    const int n = static_cast<int>(left < kChunk ? left : kChunk);
    sum += p.batch.e[t].types & 1
               ? chunk_squares(static_cast<const __nv_bfloat16*>(p.batch.e[t].grad) + at, n)
               : chunk_squares(static_cast<const float*>(p.batch.e[t].grad) + at, n);
  }
  sum = block_sum(sum);
  if (threadIdx.x == 0) p.parts[p.parts_before + blockIdx.x] = sum;
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

template <typename T, typename O>
__device__ __forceinline__ void chunk_scale(const T* g, O* out, int n, float f) {
  int done = 0;
  if (((reinterpret_cast<uintptr_t>(g) | reinterpret_cast<uintptr_t>(out)) & 15u) == 0) {
    const int vecs = n / 8;
    done = vecs * 8;
    constexpr int U = 2;
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
#pragma unroll
          for (int q = 0; q < 8; ++q) v[q] *= f;
          store8(out + (i + u * kThreads) * 8, v);
        }
    }
  }
  for (int i = done + threadIdx.x; i < n; i += kThreads) store1(out + i, to_f(g[i]) * f);
}

__global__ void __launch_bounds__(kThreads) grad_scale_kernel(
    const __grid_constant__ ClipParams p) {
  grid_dep_wait();
  grid_dep_trigger();
  double total = 0.0;
  for (int i = threadIdx.x; i < p.parts_total; i += kThreads) total += p.parts[i];
  total = block_sum(total);
  const double norm = sqrt(total) * static_cast<double>(p.scale);
  if (p.norm != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *p.norm = static_cast<float>(norm);
  if (p.chunks == 0) return;
  const double room = static_cast<double>(p.max_norm) / (norm + static_cast<double>(p.eps));
  // (a norm that is NaN makes the factor NaN; an infinite one makes it 0)
  const float f = static_cast<float>(static_cast<double>(p.scale) * (room < 1.0 || room != room ? room : 1.0));
  for (int c = p.chunks - 1 - static_cast<int>(blockIdx.x); c >= 0; c -= gridDim.x) {
    const int t = find(p, c);
    const Entry& e = p.batch.e[t];
    if (f == 1.f && e.grad == e.out) continue;  // in place, nothing to change
    const long long at = static_cast<long long>(c - e.first_chunk) * kChunk;
    const long long left = p.batch.size[t] - at;
    const int n = static_cast<int>(left < kChunk ? left : kChunk);
    switch (e.types) {
      case 0:
        chunk_scale(static_cast<const float*>(e.grad) + at, static_cast<float*>(e.out) + at, n, f);
        break;
      case 1:
        chunk_scale(static_cast<const __nv_bfloat16*>(e.grad) + at,
                    static_cast<float*>(e.out) + at, n, f);
        break;
      case 2:
        chunk_scale(static_cast<const float*>(e.grad) + at,
                    static_cast<__nv_bfloat16*>(e.out) + at, n, f);
        break;
      default:
        chunk_scale(static_cast<const __nv_bfloat16*>(e.grad) + at,
                    static_cast<__nv_bfloat16*>(e.out) + at, n, f);
    }
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
  const long long launches = launches_for(n);
  if (ws == nullptr || ws_bytes < static_cast<size_t>(launches) * kMostBlocks * sizeof(double))
    return MOE_ERR_WORKSPACE;
  if (reinterpret_cast<uintptr_t>(ws) % 16 != 0) return MOE_ERR_MISALIGNED;
  st = check_current_device();
  if (st != MOE_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int sms = device_num_sms();
  const int most = sms * kBlocksPerSm < kMostBlocks ? sms * kBlocksPerSm : kMostBlocks;
  ClipParams p;
  p.parts = static_cast<double*>(ws);
  p.scale = grad_scale;
  p.max_norm = max_norm;
  p.eps = eps;
  // one batch of the list: tensors with elements, and with results where `scaling`
  auto fill = [&](long long batch, bool scaling) -> bool {
    p.tensors = 0;
    long long chunks = 0;
    const int end = static_cast<int>((batch + 1) * kPerLaunch < n ? (batch + 1) * kPerLaunch : n);
    for (int i = static_cast<int>(batch * kPerLaunch); i < end; ++i) {
      const moe_grad_t& g = grads[i];
      if (g.size == 0 || (scaling && g.out == nullptr)) continue;
      Entry& e = p.batch.e[p.tensors];
      e.grad = g.grad;
      e.out = g.out;
      e.first_chunk = static_cast<int>(chunks);
      e.types = (g.dtype == MOE_BF16 ? 1 : 0) | (g.out_dtype == MOE_BF16 ? 2 : 0);
      p.batch.size[p.tensors++] = g.size;
      chunks += (g.size + kChunk - 1) / kChunk;
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
    const int blocks = p.chunks < most ? p.chunks : most;
    if (blocks == 0) continue;
    if (launch_pdl(grad_squares_kernel, dim3(static_cast<unsigned>(blocks)), dim3(kThreads), 0, s,
                   p) != cudaSuccess)
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
    const int blocks = p.chunks < most ? (p.chunks > 0 ? p.chunks : 1) : most;
    if (launch_pdl(grad_scale_kernel, dim3(static_cast<unsigned>(blocks)), dim3(kThreads), 0, s,
                   p) != cudaSuccess)
      return MOE_ERR_CUDA;
    out = nullptr;
  }
  return MOE_OK;
}
