// What the tensor-core products over strided operands share (linear_gemm.cu, grouped_gemm.cu):
// matrix descriptors of both operand layouts, the end of a TMA pipeline, and the host's tensor
// map encoder and shared-memory limit.
#pragma once

#include <atomic>
#include <mutex>

#include <cudaTypedefs.h>

#include "common.cuh"

namespace moe {

// Descriptor of a 128-byte-swizzled operand tile, k-contiguous (64 k x R rows per box) or
// row-contiguous (mn: boxes of 64 rows x 64 k, 8 KB each): k-contiguous tiles have 1024 bytes between 8-row atoms (the other offset is not used), row-contiguous ones
// 1024 bytes between atoms of 8 k and 8192 between chunks of 64 rows.
__device__ __forceinline__ uint64_t operand_desc(uint32_t saddr, int mn) {
  uint64_t d = smem_desc_sw128(saddr);
  if (mn) d = (d & ~(0x3FFFull << 16)) | (static_cast<uint64_t>(8192u >> 4) << 16);
  return d;
}

// The producer warp's last act: no load or commit may still be in flight when the CTA gives up
// its shared memory.  The commits of the last min(issued, S) stages arrive after their loads and
// MMAs; each lane waits for one of them (one after the other they cost 0.1 us each).  If the
// pipeline gave up, the loads alone are waited for, where they complete on this CTA's barriers.
// stage, phase, issued: the issuing lane's (`leader`) state after its last load.
template <int S, typename Empty, typename Full>
__device__ __forceinline__ void drain_stages(bool leader, int lane, int stage, uint32_t phase,
                                             int issued, Empty empty_bar, Full full_bar,
                                             bool own_loads, volatile int* abort_flag,
                                             unsigned* err) {
  const int src = __ffs(__ballot_sync(0xffffffffu, leader)) - 1;
  stage = __shfl_sync(0xffffffffu, stage, src);
  phase = __shfl_sync(0xffffffffu, phase, src);
  const int n = min(__shfl_sync(0xffffffffu, issued, src), S);
  static_assert(S <= 32, "one lane per stage");
  if (lane < n) {
    int s = stage - n + lane;
    if (s < 0) {
      s += S;
      phase ^= 1u;
    }
    volatile int no_abort = 0;
    if (!mbar_wait(empty_bar(s), phase, abort_flag, err) && own_loads)
      mbar_wait(full_bar(s), phase, &no_abort, err);
  }
  __syncwarp();
}

inline PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  });
  return fn;
}

// Raises a kernel's dynamic shared memory limit, once per device (`done` belongs to the kernel).
template <typename K>
cudaError_t allow_smem(K kernel, int bytes, std::atomic<unsigned long long>* done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (dev < 64 && (done->load(std::memory_order_acquire) & bit)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done->fetch_or(bit, std::memory_order_release);
  return e;
}

}  // namespace moe
