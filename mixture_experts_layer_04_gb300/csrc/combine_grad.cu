// moe_combine_backward: the gradient of the gated weighted sum.
//
// Forward: y[t] = sum_k w[t,k] * o[inv[t,k]].  So d w[t,k] = <dy[t], o[inv[t,k]]> and
// d o[inv[t,k]] = w[t,k] * dy[t].  One pass: an assignment's row of o is read once, dotted
// with dy[t] in fp32 and the scaled dy[t] written to the same row of d_o.
//
// Bound by memory: T*K*H floats read, T*K*H activations written; the K assignments of a
// token are neighbouring warps, so dy[t] comes from memory once and then from L1/L2.  A warp
// walks an assignment's row eight columns per lane per step; with few assignments the row is
// split over 2 to 8 warps of the block, whose partial dots meet in shared memory (in warp
// order, so the result does not depend on timing).  8192 tokens of 2048 columns, K = 8: 122 us,
// 6.9 TB/s, the rate of a plain copy; 16 tokens 4.5 us, which is the launch.
#include <initializer_list>

#include "common.cuh"
#include "kernels.h"
#include "topk.cuh"

namespace moe {
namespace {

constexpr int kWarps = 8;

__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p));
  const float4 b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
  v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
  const uint4 u = __ldg(reinterpret_cast<const uint4*>(p));
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
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

// W warps per assignment, kWarps / W assignments per block.
template <typename TA, int W>
__global__ void __launch_bounds__(32 * kWarps)
    combine_grad_kernel(const TA* __restrict__ dy, const float* __restrict__ o,
                        const int32_t* __restrict__ inv, const float* __restrict__ w,
                        TA* __restrict__ d_o, float* __restrict__ d_w, int rows, int H, int K) {
  __shared__ float part[kWarps];
  grid_dep_wait();
  grid_dep_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int slice = warp % W;
  const long long a = static_cast<long long>(blockIdx.x) * (kWarps / W) + warp / W;
  const int r = a < rows ? inv[a] : -1;
  float acc = 0.f;
  if (r >= 0 && r < rows) {
    const float g = d_o != nullptr ? w[a] : 0.f;
    const TA* y = dy + static_cast<size_t>(a / K) * H;
    const float* src = d_w != nullptr ? o + static_cast<size_t>(r) * H : nullptr;
    TA* dst = d_o != nullptr ? d_o + static_cast<size_t>(r) * H : nullptr;
#pragma unroll 4
    for (int c = (slice * 32 + lane) * 8; c < H; c += W * 256) {
      float vy[8], vo[8];
      load8(y + c, vy);
      if (src != nullptr) {
        load8(src + c, vo);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc = fmaf(vy[i], vo[i], acc);
      }
      if (dst != nullptr) {
#pragma unroll
        for (int i = 0; i < 8; ++i) vy[i] *= g;
        store8(dst + c, vy);
      }
    }
  }
  if (d_w == nullptr) return;
  acc = warp_sum(acc);
  if constexpr (W > 1) {
    if (lane == 0) part[warp] = acc;
    __syncthreads();
    if (slice == 0) {
      acc = 0.f;
#pragma unroll
      for (int i = 0; i < W; ++i) acc += part[warp + i];
    }
  }
  if (slice == 0 && lane == 0 && a < rows) d_w[a] = acc;
}

template <typename TA>
cudaError_t launch_combine_grad(const TA* dy, const float* o, const int32_t* inv, const float* w,
                                TA* d_o, float* d_w, int T, int H, int K, int num_sms,
                                cudaStream_t s) {
  const int rows = T * K;
  // enough warps to keep every SM's load queue full: about 16 per SM
  const long long want = 16ll * num_sms;
  const int W = rows >= want ? 1 : 2ll * rows >= want ? 2 : 4ll * rows >= want ? 4 : 8;
  const dim3 grid(static_cast<unsigned>((static_cast<long long>(rows) * W + kWarps - 1) / kWarps));
  const dim3 block(32 * kWarps);
  auto kernel = W == 1   ? combine_grad_kernel<TA, 1>
                : W == 2 ? combine_grad_kernel<TA, 2>
                : W == 4 ? combine_grad_kernel<TA, 4>
                         : combine_grad_kernel<TA, 8>;
  return launch_pdl(kernel, grid, block, 0, s, dy, o, inv, w, d_o, d_w, rows, H, K);
}

inline bool misaligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

}  // namespace
}  // namespace moe

extern "C" moe_status_t moe_combine_backward(const moe_config_t* cfg, const void* dy,
                                             const float* out_perm, const int32_t* inv,
                                             const float* topk_w, void* d_out_perm,
                                             float* d_topk_w, moe_stream_t stream) {
  using namespace moe;
  moe_status_t st = fault_point("moe_combine_backward");
  if (st != MOE_OK) return st;
  size_t ignored = 0;
  st = moe_workspace_size(cfg, &ignored);  // validates cfg on the host
  if (st != MOE_OK) return st;
  if (cfg->T == 0) return MOE_OK;
  if (dy == nullptr || inv == nullptr || (d_out_perm == nullptr && d_topk_w == nullptr) ||
      (d_topk_w != nullptr && out_perm == nullptr) || (d_out_perm != nullptr && topk_w == nullptr))
    return MOE_ERR_INVALID_ARG;
  for (const void* q : {dy, static_cast<const void*>(out_perm), static_cast<const void*>(inv),
                        static_cast<const void*>(topk_w), static_cast<const void*>(d_out_perm),
                        static_cast<const void*>(d_topk_w)})
    if (misaligned16(q)) return MOE_ERR_MISALIGNED;
  st = check_current_device();
  if (st != MOE_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int sms = device_num_sms();
  const cudaError_t e =
      cfg->dtype == MOE_BF16
          ? launch_combine_grad(static_cast<const __nv_bfloat16*>(dy), out_perm, inv, topk_w,
                                static_cast<__nv_bfloat16*>(d_out_perm), d_topk_w, cfg->T, cfg->H,
                                cfg->K, sms, s)
          : launch_combine_grad(static_cast<const float*>(dy), out_perm, inv, topk_w,
                                static_cast<float*>(d_out_perm), d_topk_w, cfg->T, cfg->H, cfg->K,
                                sms, s);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
