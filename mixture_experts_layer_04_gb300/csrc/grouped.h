// The tensor-core product behind the products grouped by expert (grouped.cu, grouped_gemm.cu).
#pragma once

#include "kernels.h"

namespace moe {

enum class GroupedKind : int {
  kForward = 0,       // C rows r of group g = A_r . B_g^T            (B_g [features][depth])
  kInputGrad = 1,     // C rows r of group g = A_r . B_g              (B_g [depth][features])
  kWeightGrad = 2,    // C_g [rows][features] = A_g^T . B_g           (A_g, B_g: the group's rows)
};

// What the kernels need to know about the groups, in device memory: made by grouped_plan.cuh.
struct GroupPlan {
  int* bounds;    // [groups + 1], the offsets clamped to ascend within 0..rows
  int4* tiles;    // per tile of rows: {group, first row of its chunk, first tile of its chunk,
                  //                    tiles in its chunk | rows of each << 4}
  int* count;     // tiles of rows
  void* maps;     // tensor maps of every group's rows, [groups][2], or null
  const int32_t* offsets;  // not null: no plan was made, the product's kernel reads the offsets
};

// One grouped product.  Operands are bf16, in parts whose sum is the value (1; 3 each for float32
// values; for a bf16 SwiGLU layer's gradients with a float32 dx 3 of A for dx and 2 for dw), with
// rows at 16-byte boundaries.  A: activations [total rows][a_inner]; B: weights
// [groups][w_rows][w_inner], or for the weight gradient activations [total rows][b_inner].
struct GroupedProduct {
  GroupedKind kind;
  int groups, total_rows;
  int a_parts, b_parts;
  int depth;           // reduction (forward, input gradient); unused by the weight gradient
  int rows;            // weight gradient: rows of C_g
  int features;        // columns of C
  int swiglu;          // forward: features of each half; C = silu(gate) * up, z takes both
  const void* a;
  long long lda, a_plane;
  const void* b;
  long long ldb, b_plane;
  void* c;
  int c_f32;
  long long ldc, c_group;  // c_group: elements between the groups of a weight gradient
  void* z;                 // forward with swiglu: [total rows][2 features] or null
  int z_f32;
  long long ldz;
};

// Rows that a tile of the forward or input-gradient product takes, by the rule in grouped_gemm.cu.
int grouped_tile_rows(int total_rows, int groups, bool f32);
// Whether the forward and input-gradient kernels for these tiles can do without a plan.
bool grouped_plans_itself(int tile_rows, bool f32);
size_t grouped_max_tiles(int total_rows, int groups, int tile_rows);

// n products (1 or 2) one after the other; those of float32 operands in one launch.
cudaError_t launch_grouped_products(const GroupedProduct* g, int n, const GroupPlan& plan,
                                    unsigned* err, int num_sms, cudaStream_t s);

}  // namespace moe
