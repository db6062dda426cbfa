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
  // tile kernel only: column sums of an earlier pass to finish along the way, or null:
  // sum_out[i] = sum over s of sum_parts[s][i], i < rows
  const float* sum_parts;
  float* sum_out;
  int sum_slices;
};

// Whether the product runs on CTA pairs (and not in the tile kernel).
bool linear_gemm_on_pairs(const LinearGemm& g, int num_sms);

// One product, or two with operands and results of the same types and no dependence on each
// other (in one launch where both suit the tile kernel and one tile suits both).
cudaError_t launch_linear_gemms(const LinearGemm* jobs, int n, unsigned* err, int num_sms,
                                cudaStream_t s);

}  // namespace moe
