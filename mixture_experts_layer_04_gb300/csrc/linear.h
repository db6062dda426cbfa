// The tensor-core product behind the linear layers (linear.cu, linear_gemm.cu).
#pragma once

#include "kernels.h"

namespace moe {

// C[i, j] = epilogue(sum_k A(i, k) B(j, k)) for i < rows, j < cols, with A and B in bf16.
// An operand lies either k-contiguous ([rows][depth], mn = 0) or row-contiguous ([depth][rows],
// mn = 1); its base and row stride are multiples of 16 bytes.  planes = 3: every operand is
// three bf16 matrices, `plane` elements apart, whose sum is the float32 value; the six
// products above 2^-24 are taken.  Epilogue: v += bias[j]; z[i, j] = v; v = act(v) + res[i, j];
// C and z, res are float or bf16 as given; strides in elements.
struct LinearGemm {
  int rows, cols, depth, planes;
  const void* a;
  long long lda, a_plane;
  int a_mn;
  const void* b;
  long long ldb, b_plane;
  int b_mn;
  void* c;
  int c_f32;
  long long ldc;
  const float* bias;
  int act;
  int act_f32;  // type of res and z
  const void* res;
  long long ldr;
  void* z;
  long long ldz;
};

cudaError_t launch_linear_gemm(const LinearGemm& g, unsigned* err, int num_sms, cudaStream_t s);

}  // namespace moe
