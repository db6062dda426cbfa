// What the operators over strided arrays share: eight values of either type at a time on the device, and
// the host's checks of pointers and strides.
#pragma once

#include "common.cuh"
#include "kernels.h"

namespace moe {

// bf16's largest value.
constexpr float kMaxBf16 = 0x1.fep127f;

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }

__device__ __forceinline__ void unpack8(const uint4& u, float (&v)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
// Eight values at p (16-byte aligned).
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
  unpack8(*reinterpret_cast<const uint4*>(p), v);
}
// n of eight values at p, zeros after them; 16-byte loads when `vec` and all eight are there.
template <typename T>
__device__ __forceinline__ void load_n(const T* p, int n, bool vec, float (&v)[8]) {
  if (vec && n >= 8) {
    load8(p, v);
    return;
  }
#pragma unroll
  for (int q = 0; q < 8; ++q) v[q] = q < n ? to_f(p[q]) : 0.f;
}

inline bool odd_stride(long long stride, int dtype) {
  return stride * static_cast<long long>(act_bytes(dtype)) % 16 != 0;
}
inline long long pad8(long long n) { return (n + 7) / 8 * 8; }
inline bool unaligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }
inline bool vec_ok(const void* p, long long ld, int dtype) {
  return !unaligned(p, 16) && !odd_stride(ld, dtype);
}
// An operand's pointer: the alignment of an element, and a 16-byte boundary when its stride says
// that it is read in place.
inline bool bad_operand(const void* p, long long ld, int dtype) {
  return unaligned(p, odd_stride(ld, dtype) ? act_bytes(dtype) : 16);
}
inline moe_status_t status_of(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

}  // namespace moe
