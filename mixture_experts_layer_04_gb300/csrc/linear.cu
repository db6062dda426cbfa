// moe_linear and moe_linear_backward: argument checks, the workspace, the passes around the
// tensor-core product (linear_gemm.cu) and the product for a few rows.
//
//  - linear_rows_kernel (a few rows): every weight is used `rows` times only, so the call is
//    bound by reading the weights once.  A block takes two or four output features, its eight
//    warps split the input features, so each weight row is in flight as a whole; fp32 FMAs,
//    partial sums joined in shared memory in warp order.  Any alignment and either type.  One
//    row through 4096 x 4096 bf16 weights: 7.5 us with every weight from HBM, 4.5 TB/s (6.4 us
//    with three copies in turn, which L2 holds in part; 5.1 us with one).
//  - pack_kernel: an operand the tensor cores cannot read in place.  Float32 values become
//    three bf16 parts (p0 = bf16(v), p1 = bf16(v - p0), p2 = bf16(v - p0 - p1): 24 bits), and
//    rows whose stride is not a multiple of 16 bytes are copied to one that is.
//  - dz_kernel: dz = dy * act'(z) in the product's operand form (rounded to bf16, or three
//    parts) and, in the same pass, the column sums of the unrounded dz over a slice of rows;
//    the dw product adds the slices in order along the way (column_sum_kernel where there is
//    none, or where it runs on CTA pairs).  Bound by reading dy and z and writing dz: 54 us for
//    8192 x 7168 with GELU (352 MB, 52 us at the copy rate).
#include "common.cuh"
#include "kernels.h"
#include "linear.h"
#include "linear_act.cuh"
#include "operand_io.cuh"
#include "topk.cuh"

namespace moe {
namespace {

// Whether moe_linear runs on the CUDA cores.  One FMA per weight and row: with two rows through
// 4096 x 4096 bf16 weights the tensor cores are ahead (9.2 us against 10.3; one row 7.5 here),
// with few weights, where the launch is what counts, the CUDA cores (4 rows through 2048 x 256:
// 2.8 us against 4.2; through 512 x 2048: 4.7 against 4.2).  Operands that would have to be
// packed first, all of float32, gain more from being read once (float32 4096 x 4096, 8 rows: 28
// and 45 us).
constexpr int kMaxFewRows = 8;
bool few_rows(const moe_linear_config_t* c, bool packed) {
  if (c->rows == 1 || (packed && c->rows <= kMaxFewRows)) return true;
  return c->rows <= 4 &&
         static_cast<long long>(c->rows) * c->in_features * c->out_features <= 1ll << 21;
}

__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Eight values in PL bf16 parts at dst, dst + plane, ...  A value that is not finite goes
// whole into the first part.  A finite one that rounding would take past bf16's largest (above
// 3.39e38) has that for its first part: what is left fits the others.
template <int PL>
__device__ __forceinline__ void store_parts(__nv_bfloat16* dst, long long plane, float (&v)[8]) {
#pragma unroll
  for (int pl = 0; pl < PL; ++pl) {
    uint4 u = pack8(v);
    if (PL > 1 && pl == 0) {
      float most = 0.f;
#pragma unroll
      for (int q = 0; q < 8; ++q) most = fmaxf(most, fabsf(v[q]));
      if (most > kMaxBf16) {
        float t[8];
#pragma unroll
        for (int q = 0; q < 8; ++q)
          t[q] = fabsf(v[q]) < INFINITY ? fminf(fmaxf(v[q], -kMaxBf16), kMaxBf16) : v[q];
        u = pack8(t);
      }
    }
    *reinterpret_cast<uint4*>(dst + pl * plane) = u;
    if (pl + 1 < PL) {
      float r[8];
      unpack8(u, r);
#pragma unroll
      for (int q = 0; q < 8; ++q) v[q] = fabsf(r[q]) < INFINITY ? v[q] - r[q] : 0.f;
    }
  }
}

// ------------------------------------------------------------------ packing ----

struct PackTask {
  const void* src;
  long long ld;
  __nv_bfloat16* dst;
  long long dst_ld, plane;
  int rows, cols, vec;
  int blocks;  // of 256 threads, 0: nothing to pack
};

// One task by `blocks` blocks, of which this is number `block`.
template <typename T, int PL>
__device__ __forceinline__ void pack_task(const PackTask& t, int block) {
  const int per_row = static_cast<int>(t.dst_ld / 8);
  const long long items = static_cast<long long>(t.rows) * per_row;
  for (long long i = block * 256ll + threadIdx.x; i < items; i += t.blocks * 256ll) {
    const long long r = i / per_row;
    const int c = static_cast<int>(i - r * per_row) * 8;
    float v[8];
    load_n(static_cast<const T*>(t.src) + r * t.ld + c, t.cols - c, t.vec != 0, v);
    store_parts<PL>(t.dst + r * t.dst_ld + c, t.plane, v);
  }
}

template <typename T, int PL>
__global__ void __launch_bounds__(256)
    pack_kernel(const __grid_constant__ PackTask x, const __grid_constant__ PackTask w) {
  grid_dep_wait();
  grid_dep_trigger();
  const int b = static_cast<int>(blockIdx.x);
  if (b < x.blocks) pack_task<T, PL>(x, b);
  else pack_task<T, PL>(w, b - x.blocks);
}

// ----------------------------------------------------------------------- dz ----

struct DzParams {
  const void* dy;
  const void* z;  // null without an activation
  long long ldy, ldz;
  __nv_bfloat16* dz;  // null: only the column sums
  long long dz_ld, plane;
  float* sums;  // [slices][cols], or null
  int rows, cols, rows_per_slice;
  int act;
  int vec_y, vec_z;  // 16-byte loads allowed
  int col_blocks, blocks;  // blocks of dz: col_blocks x slices; then x's and w's packing
  PackTask x, w;
};

// Eight values as they lie in memory, to be on their way before any is used.
template <typename T>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
  uint4 u;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    u = *reinterpret_cast<const uint4*>(p);
  }
  __device__ __forceinline__ void get(float (&v)[8]) const { unpack8(u, v); }
};
template <>
struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
};

// A block takes 256 columns of a slice of rows, a warp every eighth row of it.
template <typename TY, typename TA, int PL, int ACT>
__global__ void __launch_bounds__(256, PL == 1 ? 4 : 2)
    dz_kernel(const __grid_constant__ DzParams p) {
  constexpr int U = PL == 1 ? 4 : 2;  // rows a thread has in flight
  __shared__ float s_sum[8][256];
  grid_dep_wait();
  grid_dep_trigger();
  const int block = static_cast<int>(blockIdx.x) - p.blocks;
  if (block >= 0) {
    if (block < p.x.blocks) pack_task<TA, PL>(p.x, block);
    else pack_task<TA, PL>(p.w, block - p.x.blocks);
    return;
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int slice = static_cast<int>(blockIdx.x) / p.col_blocks;
  const int col_block = static_cast<int>(blockIdx.x) - slice * p.col_blocks;
  const int c = col_block * 256 + lane * 8;
  const int r0 = slice * p.rows_per_slice;
  const int r1 = min(p.rows, r0 + p.rows_per_slice);
  const TY* dy = static_cast<const TY*>(p.dy);
  const TA* z = static_cast<const TA*>(p.z);
  float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  auto take = [&](int r, float (&v)[8], float (&zv)[8]) {
    if constexpr (ACT != MOE_ACT_NONE) {
#pragma unroll
      for (int q = 0; q < 8; ++q) v[q] *= act_slope<sizeof(TA) == 2>(ACT, zv[q]);
    }
#pragma unroll
    for (int q = 0; q < 8; ++q) sum[q] += v[q];
    if (p.dz != nullptr)
      store_parts<PL>(p.dz + static_cast<size_t>(r) * p.dz_ld + c, p.plane, v);
  };
  if (c + 8 <= p.cols && p.vec_y && (ACT == MOE_ACT_NONE || p.vec_z)) {
    for (int rb = r0 + warp; rb < r1; rb += 8 * U) {
      Raw8<TY> ry[U];
      Raw8<TA> rz[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int r = min(rb + 8 * u, r1 - 1);
        ry[u].load(dy + static_cast<size_t>(r) * p.ldy + c);
        if constexpr (ACT != MOE_ACT_NONE) rz[u].load(z + static_cast<size_t>(r) * p.ldz + c);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (rb + 8 * u < r1) {
          float v[8], zv[8];
          ry[u].get(v);
          if constexpr (ACT != MOE_ACT_NONE) rz[u].get(zv);
          take(rb + 8 * u, v, zv);
        }
      }
    }
  } else if (c < p.cols) {
    for (int r = r0 + warp; r < r1; r += 8) {
      float v[8], zv[8];
      load_n(dy + static_cast<size_t>(r) * p.ldy + c, p.cols - c, p.vec_y != 0, v);
      if constexpr (ACT != MOE_ACT_NONE)
        load_n(z + static_cast<size_t>(r) * p.ldz + c, p.cols - c, p.vec_z != 0, zv);
      take(r, v, zv);
    }
  }
  if (p.sums == nullptr) return;
#pragma unroll
  for (int q = 0; q < 8; ++q) s_sum[warp][q * 32 + lane] = sum[q];
  __syncthreads();
  // column 8 l + q of the block sits at [q * 32 + l]
  const int at = (threadIdx.x & 7) * 32 + (threadIdx.x >> 3);
  float total = 0.f;
#pragma unroll
  for (int w = 0; w < 8; ++w) total += s_sum[w][at];
  const int col = col_block * 256 + threadIdx.x;
  if (col < p.cols) p.sums[static_cast<size_t>(slice) * p.cols + col] = total;
}

// The slices' column sums: 32 columns per block, each warp adds every eighth slice, then the
// eight partial sums in warp order.
__global__ void __launch_bounds__(256)
    column_sum_kernel(const float* __restrict__ parts, int slices, int cols,
                      float* __restrict__ out) {
  __shared__ float s_sum[8][32];
  grid_dep_wait();
  grid_dep_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float total = 0.f;
  if (c < cols) {
#pragma unroll 8
    for (int s = warp; s < slices; s += 8) total += parts[static_cast<size_t>(s) * cols + c];
  }
  s_sum[warp][lane] = total;
  __syncthreads();
  if (warp != 0 || c >= cols) return;
  total = 0.f;
#pragma unroll
  for (int w = 0; w < 8; ++w) total += s_sum[w][lane];
  out[c] = total;
}

template <typename TY, typename TA, int PL>
cudaError_t launch_dz(const DzParams& p, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>(p.blocks) + static_cast<unsigned>(p.x.blocks) +
                  static_cast<unsigned>(p.w.blocks));
  switch (p.act) {
    case MOE_ACT_RELU:
      return launch_pdl(dz_kernel<TY, TA, PL, MOE_ACT_RELU>, grid, dim3(256), 0, s, p);
    case MOE_ACT_GELU:
      return launch_pdl(dz_kernel<TY, TA, PL, MOE_ACT_GELU>, grid, dim3(256), 0, s, p);
    case MOE_ACT_GELU_TANH:
      return launch_pdl(dz_kernel<TY, TA, PL, MOE_ACT_GELU_TANH>, grid, dim3(256), 0, s, p);
    case MOE_ACT_SILU:
      return launch_pdl(dz_kernel<TY, TA, PL, MOE_ACT_SILU>, grid, dim3(256), 0, s, p);
    default:
      return launch_pdl(dz_kernel<TY, TA, PL, MOE_ACT_NONE>, grid, dim3(256), 0, s, p);
  }
}

// ----------------------------------------------------------------- few rows ----

struct RowsParams {
  const void* x;
  const void* w;
  const float* bias;
  const void* res;
  void* y;
  void* z;
  long long ldx, ldw, ldr, ldy, ldz;
  int rows, in, out, act, y_f32, vec;
};

// Output features per block, and blocks per SM to compile for: with one row two features in all
// the blocks that an SM can hold keep the most bytes in flight (4096 x 4096 bf16, weights from
// HBM: 7.5 us, four features 9.4 us, eight 10.8 us).
constexpr int rows_features(int mt) { return mt <= 2 ? 2 : 4; }
constexpr int rows_blocks(int mt) { return mt == 1 ? 8 : 1; }

template <typename TA, int MT>
__global__ void __launch_bounds__(256, rows_blocks(MT)) linear_rows_kernel(const __grid_constant__ RowsParams p) {
  constexpr int kFeatures = rows_features(MT);
  __shared__ float part[8][kFeatures * MT];
  grid_dep_wait();
  grid_dep_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int n0 = blockIdx.x * kFeatures;
  const TA* x = static_cast<const TA*>(p.x);
  const TA* w[kFeatures];
#pragma unroll
  for (int f = 0; f < kFeatures; ++f)  // rows past the end repeat the last one, unused
    w[f] = static_cast<const TA*>(p.w) + static_cast<size_t>(min(n0 + f, p.out - 1)) * p.ldw;
  float acc[kFeatures][MT];
#pragma unroll
  for (int f = 0; f < kFeatures; ++f)
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[f][m] = 0.f;
  int done = 0;
  if (p.vec) {
    const int vecs = p.in / 8;
    done = vecs * 8;
#pragma unroll 1
    for (int i = threadIdx.x; i < vecs; i += 256) {
      float wv[kFeatures][8];
#pragma unroll
      for (int f = 0; f < kFeatures; ++f) load8(w[f] + i * 8, wv[f]);
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        if (m < p.rows) {
          float xv[8];
          load8(x + m * p.ldx + i * 8, xv);
#pragma unroll
          for (int f = 0; f < kFeatures; ++f)
#pragma unroll
            for (int q = 0; q < 8; ++q) acc[f][m] = fmaf(wv[f][q], xv[q], acc[f][m]);
        }
      }
    }
  }
#pragma unroll 4
  for (int i = done + threadIdx.x; i < p.in; i += 256) {
    float wv[kFeatures];
#pragma unroll
    for (int f = 0; f < kFeatures; ++f) wv[f] = to_f(w[f][i]);
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      if (m < p.rows) {
        const float xv = to_f(x[m * p.ldx + i]);
#pragma unroll
        for (int f = 0; f < kFeatures; ++f) acc[f][m] = fmaf(wv[f], xv, acc[f][m]);
      }
    }
  }
#pragma unroll
  for (int f = 0; f < kFeatures; ++f)
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const float v = warp_sum(acc[f][m]);
      if (lane == 0) part[warp][f * MT + m] = v;
    }
  __syncthreads();
  const int f = threadIdx.x / MT, m = threadIdx.x - f * MT, n = n0 + f;
  if (f >= kFeatures || m >= p.rows || n >= p.out) return;
  float v = 0.f;
#pragma unroll
  for (int k = 0; k < 8; ++k) v += part[k][f * MT + m];
  if (p.bias != nullptr) v += p.bias[n];
  if (p.z != nullptr) {
    if constexpr (sizeof(TA) == 4) static_cast<float*>(p.z)[m * p.ldz + n] = v;
    else static_cast<__nv_bfloat16*>(p.z)[m * p.ldz + n] = __float2bfloat16_rn(v);
  }
  v = act_value<sizeof(TA) == 2>(p.act, v);
  if (p.res != nullptr) v += to_f(static_cast<const TA*>(p.res)[m * p.ldr + n]);
  if (p.y_f32) static_cast<float*>(p.y)[m * p.ldy + n] = v;
  else static_cast<__nv_bfloat16*>(p.y)[m * p.ldy + n] = __float2bfloat16_rn(v);
}

template <typename TA>
cudaError_t launch_rows(const RowsParams& p, cudaStream_t s) {
  const int features = rows_features(p.rows);
  const dim3 grid((static_cast<unsigned>(p.out) + features - 1) / features), block(256);
  if (p.rows == 1) return launch_pdl(linear_rows_kernel<TA, 1>, grid, block, 0, s, p);
  if (p.rows == 2) return launch_pdl(linear_rows_kernel<TA, 2>, grid, block, 0, s, p);
  if (p.rows <= 4) return launch_pdl(linear_rows_kernel<TA, 4>, grid, block, 0, s, p);
  return launch_pdl(linear_rows_kernel<TA, 8>, grid, block, 0, s, p);
}

// --------------------------------------------------------------------- host ----

moe_status_t check_linear_config(const moe_linear_config_t* c) {
  if (c == nullptr) return MOE_ERR_INVALID_ARG;
  if (c->rows < 0 || c->rows > (1 << 30)) return MOE_ERR_INVALID_ARG;
  if (c->in_features <= 0 || c->in_features > (1 << 20)) return MOE_ERR_INVALID_ARG;
  if (c->out_features <= 0 || c->out_features > (1 << 20)) return MOE_ERR_INVALID_ARG;
  if (c->dtype != MOE_F32 && c->dtype != MOE_BF16) return MOE_ERR_INVALID_ARG;
  if (c->out_dtype != c->dtype && c->out_dtype != MOE_F32) return MOE_ERR_INVALID_ARG;
  if (c->activation < MOE_ACT_NONE || c->activation > MOE_ACT_SILU) return MOE_ERR_INVALID_ARG;
  const long long in = c->in_features, out = c->out_features, most = 1ll << 31;
  const struct {
    long long stride, least;
  } s[] = {{c->x_stride, in},  {c->w_stride, in},  {c->residual_stride, out}, {c->y_stride, out},
           {c->z_stride, out}, {c->dx_stride, in}, {c->dw_stride, in}};
  for (const auto& q : s)
    if (q.stride != 0 && (q.stride < q.least || q.stride > most)) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

struct Strides {
  long long x, w, r, y, z, dx, dw;
  explicit Strides(const moe_linear_config_t* c)
      : x(pick(c->x_stride, c->in_features)), w(pick(c->w_stride, c->in_features)),
        r(pick(c->residual_stride, c->out_features)), y(pick(c->y_stride, c->out_features)),
        z(pick(c->z_stride, c->out_features)), dx(pick(c->dx_stride, c->in_features)),
        dw(pick(c->dw_stride, c->in_features)) {}
  static long long pick(long long s, int n) { return s != 0 ? s : n; }
};

inline size_t up256(size_t v) { return (v + 255) & ~static_cast<size_t>(255); }

// Slices of rows whose column sums are taken separately: enough blocks for the GPU, at least
// 8 rows (one per warp) each.
int dz_slices(int rows, int out) {
  const int col_blocks = (out + 255) / 256;
  const int want = (1216 + col_blocks - 1) / col_blocks;
  const int most = (rows + 7) / 8;
  const int n = want < most ? want : most;
  return n < 1 ? 1 : n;
}

// Workspace: packed x and w, dz in operand form, column sums.
struct LinearPlan {
  bool pack_x, pack_w, make_dz;
  size_t x, w, dz, sums, total;
};

LinearPlan make_linear_plan(const moe_linear_config_t* c) {
  const Strides st(c);
  const bool f32 = c->dtype == MOE_F32;
  const size_t parts = f32 ? 3 : 1;
  LinearPlan p;
  p.pack_x = f32 || odd_stride(st.x, c->dtype);
  p.pack_w = f32 || odd_stride(st.w, c->dtype);
  p.make_dz = f32 || c->out_dtype != c->dtype || c->activation != MOE_ACT_NONE ||
              odd_stride(st.y, c->out_dtype);
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o += up256(bytes);
    return at;
  };
  const size_t rows = c->rows, in = pad8(c->in_features), out = pad8(c->out_features);
  p.x = take(p.pack_x ? parts * rows * in * 2 : 0);
  p.w = take(p.pack_w ? parts * c->out_features * in * 2 : 0);
  p.dz = take(p.make_dz ? parts * rows * out * 2 : 0);
  p.sums = take(static_cast<size_t>(dz_slices(c->rows, c->out_features)) * c->out_features * 4);
  p.total = o;
  return p;
}

// An operand of the product as it lies in memory: [outer rows][inner] with a row stride.
struct Operand {
  const void* p;
  long long ld, plane;
};

// The operand in place, or packed into `dst` by the task it fills in.
Operand operand(const void* src, long long ld, int rows, int cols, int dtype, bool pack, void* dst,
                int num_sms, PackTask* task) {
  if (!pack) return Operand{src, ld, 0};
  PackTask t;
  t.src = src;
  t.ld = ld;
  t.dst = static_cast<__nv_bfloat16*>(dst);
  t.dst_ld = pad8(cols);
  t.plane = t.dst_ld * rows;
  t.rows = rows;
  t.cols = cols;
  t.vec = vec_ok(src, ld, dtype) ? 1 : 0;
  const long long blocks = (t.plane / 8 + 255) / 256, most = 16ll * num_sms;
  t.blocks = static_cast<int>(blocks < most ? blocks : most);
  *task = t;
  return Operand{dst, t.dst_ld, t.plane};
}

template <typename T>
T* at(void* ws, size_t off) {
  return reinterpret_cast<T*>(static_cast<char*>(ws) + off);
}

}  // namespace
}  // namespace moe

extern "C" moe_status_t moe_linear_workspace_size(const moe_linear_config_t* cfg, size_t* bytes) {
  using namespace moe;
  moe_status_t st = fault_point("moe_linear_workspace_size");
  if (st != MOE_OK) return st;
  st = check_linear_config(cfg);
  if (st != MOE_OK) return st;
  if (bytes == nullptr) return MOE_ERR_INVALID_ARG;
  *bytes = make_linear_plan(cfg).total;
  return MOE_OK;
}

extern "C" moe_status_t moe_linear(const moe_linear_config_t* cfg, const void* x, const void* w,
                                   const float* bias, const void* residual, void* y, void* z,
                                   void* ws, size_t ws_bytes, moe_stream_t stream) {
  using namespace moe;
  moe_status_t st = fault_point("moe_linear");
  if (st != MOE_OK) return st;
  st = check_linear_config(cfg);
  if (st != MOE_OK) return st;
  if (cfg->rows == 0) return MOE_OK;
  if (x == nullptr || w == nullptr || y == nullptr) return MOE_ERR_INVALID_ARG;
  const Strides ld(cfg);
  const size_t ab = act_bytes(cfg->dtype);
  if (bad_operand(x, ld.x, cfg->dtype) || bad_operand(w, ld.w, cfg->dtype) ||
      unaligned(bias, 4) || unaligned(residual, ab) || unaligned(z, ab) ||
      unaligned(y, act_bytes(cfg->out_dtype)))
    return MOE_ERR_MISALIGNED;
  const LinearPlan plan = make_linear_plan(cfg);
  const bool few = few_rows(cfg, plan.pack_x || plan.pack_w);  // needs no workspace
  if (!few && (ws == nullptr || ws_bytes < plan.total)) return MOE_ERR_WORKSPACE;
  if (!few && unaligned(ws, 16)) return MOE_ERR_MISALIGNED;
  st = check_current_device();
  if (st != MOE_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);

  if (few) {
    RowsParams p{};
    p.x = x;
    p.w = w;
    p.bias = bias;
    p.res = residual;
    p.y = y;
    p.z = z;
    p.ldx = ld.x;
    p.ldw = ld.w;
    p.ldr = ld.r;
    p.ldy = ld.y;
    p.ldz = ld.z;
    p.rows = cfg->rows;
    p.in = cfg->in_features;
    p.out = cfg->out_features;
    p.act = cfg->activation;
    p.y_f32 = cfg->out_dtype == MOE_F32;
    p.vec = vec_ok(x, ld.x, cfg->dtype) && vec_ok(w, ld.w, cfg->dtype);
    return status_of(cfg->dtype == MOE_BF16 ? launch_rows<__nv_bfloat16>(p, s)
                                            : launch_rows<float>(p, s));
  }

  const int sms = device_num_sms();
  PackTask tx{}, tw{};
  const Operand ox = operand(x, ld.x, cfg->rows, cfg->in_features, cfg->dtype, plan.pack_x,
                             at<void>(ws, plan.x), sms, &tx);
  const Operand ow = operand(w, ld.w, cfg->out_features, cfg->in_features, cfg->dtype,
                             plan.pack_w, at<void>(ws, plan.w), sms, &tw);
  if (tx.blocks + tw.blocks > 0) {
    const dim3 grid(static_cast<unsigned>(tx.blocks + tw.blocks));
    const cudaError_t e =
        cfg->dtype == MOE_F32
            ? launch_pdl(pack_kernel<float, 3>, grid, dim3(256), 0, s, tx, tw)
            : launch_pdl(pack_kernel<__nv_bfloat16, 1>, grid, dim3(256), 0, s, tx, tw);
    if (e != cudaSuccess) return MOE_ERR_CUDA;
  }
  LinearGemm g{};
  g.rows = cfg->rows;
  g.cols = cfg->out_features;
  g.depth = cfg->in_features;
  g.planes = cfg->dtype == MOE_F32 ? 3 : 1;
  g.a = ox.p;
  g.lda = ox.ld;
  g.a_plane = ox.plane;
  g.b = ow.p;
  g.ldb = ow.ld;
  g.b_plane = ow.plane;
  g.c = y;
  g.c_f32 = cfg->out_dtype == MOE_F32;
  g.ldc = ld.y;
  g.bias = bias;
  g.act = cfg->activation;
  g.act_f32 = cfg->dtype == MOE_F32;
  g.res = residual;
  g.ldr = ld.r;
  g.z = z;
  g.ldz = ld.z;
  return status_of(launch_linear_gemms(&g, 1, device_error_word(), sms, s));
}

extern "C" moe_status_t moe_linear_backward(const moe_linear_config_t* cfg, const void* dy,
                                            const void* x, const void* w, const void* z, void* dx,
                                            void* dw, float* dbias, void* ws, size_t ws_bytes,
                                            moe_stream_t stream) {
  using namespace moe;
  moe_status_t st = fault_point("moe_linear_backward");
  if (st != MOE_OK) return st;
  st = check_linear_config(cfg);
  if (st != MOE_OK) return st;
  const Strides ld(cfg);
  const size_t ab = act_bytes(cfg->dtype);
  const bool has_act = cfg->activation != MOE_ACT_NONE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (unaligned(dx, ab) || unaligned(dw, ab) || unaligned(dbias, 4)) return MOE_ERR_MISALIGNED;
  if (cfg->rows == 0) {
    if (dw == nullptr && dbias == nullptr) return MOE_OK;
    st = check_current_device();
    if (st != MOE_OK) return st;
    if (dw != nullptr &&
        cudaMemset2DAsync(dw, ld.dw * ab, 0, cfg->in_features * ab, cfg->out_features, s) !=
            cudaSuccess)
      return MOE_ERR_CUDA;
    if (dbias != nullptr &&
        cudaMemsetAsync(dbias, 0, static_cast<size_t>(cfg->out_features) * 4, s) != cudaSuccess)
      return MOE_ERR_CUDA;
    return MOE_OK;
  }
  if (dy == nullptr || (dx == nullptr && dw == nullptr && dbias == nullptr) ||
      (dx != nullptr && w == nullptr) || (dw != nullptr && x == nullptr) ||
      (has_act && z == nullptr))
    return MOE_ERR_INVALID_ARG;
  if (bad_operand(dy, ld.y, cfg->out_dtype) ||
      (dw != nullptr && bad_operand(x, ld.x, cfg->dtype)) ||
      (dx != nullptr && bad_operand(w, ld.w, cfg->dtype)) || (has_act && unaligned(z, ab)))
    return MOE_ERR_MISALIGNED;
  const LinearPlan plan = make_linear_plan(cfg);
  if (ws == nullptr || ws_bytes < plan.total) return MOE_ERR_WORKSPACE;
  if (unaligned(ws, 16)) return MOE_ERR_MISALIGNED;
  st = check_current_device();
  if (st != MOE_OK) return st;
  const int sms = device_num_sms();
  const bool f32 = cfg->dtype == MOE_F32;
  const int rows = cfg->rows, in = cfg->in_features, out = cfg->out_features;

  // One pass: dz, the slices of the column sums, and x and w where they have to be packed.
  DzParams p{};
  Operand odz{dy, ld.y, 0}, ox{}, ow{};
  const bool products = dx != nullptr || dw != nullptr;
  if (dx != nullptr)
    ow = operand(w, ld.w, out, in, cfg->dtype, plan.pack_w, at<void>(ws, plan.w), sms, &p.w);
  if (dw != nullptr)
    ox = operand(x, ld.x, rows, in, cfg->dtype, plan.pack_x, at<void>(ws, plan.x), sms, &p.x);
  int slices = 0;
  if ((plan.make_dz && products) || dbias != nullptr) {
    p.dy = dy;
    p.ldy = ld.y;
    p.z = has_act ? z : nullptr;
    p.ldz = ld.z;
    p.rows = rows;
    p.cols = out;
    p.act = cfg->activation;
    p.vec_y = vec_ok(dy, ld.y, cfg->out_dtype);
    p.vec_z = vec_ok(z, ld.z, cfg->dtype);
    if (plan.make_dz && products) {
      p.dz = at<__nv_bfloat16>(ws, plan.dz);
      p.dz_ld = pad8(out);
      p.plane = p.dz_ld * rows;
      odz = Operand{p.dz, p.dz_ld, p.plane};
    }
    const int want = dz_slices(rows, out);
    p.rows_per_slice = ((rows + want - 1) / want + 7) / 8 * 8;
    slices = (rows + p.rows_per_slice - 1) / p.rows_per_slice;
    if (dbias != nullptr) p.sums = slices == 1 ? dbias : at<float>(ws, plan.sums);
    p.col_blocks = (out + 255) / 256;
    p.blocks = p.col_blocks * slices;
  }
  if (p.blocks + p.x.blocks + p.w.blocks > 0) {
    const cudaError_t e = f32 ? launch_dz<float, float, 3>(p, s)
                          : cfg->out_dtype == MOE_F32
                              ? launch_dz<float, __nv_bfloat16, 1>(p, s)
                              : launch_dz<__nv_bfloat16, __nv_bfloat16, 1>(p, s);
    if (e != cudaSuccess) return MOE_ERR_CUDA;
  }
  LinearGemm g{};
  g.planes = f32 ? 3 : 1;
  g.c_f32 = f32;
  g.act_f32 = f32;
  g.a = odz.p;
  g.lda = odz.ld;
  g.a_plane = odz.plane;
  g.cols = in;
  g.b_mn = 1;
  LinearGemm jobs[2];
  int n = 0;
  bool sums_left = dbias != nullptr && slices > 1;
  if (dx != nullptr) {
    LinearGemm& q = jobs[n++] = g;
    q.rows = rows;
    q.depth = out;
    q.b = ow.p;
    q.ldb = ow.ld;
    q.b_plane = ow.plane;
    q.c = dx;
    q.ldc = ld.dx;
  }
  if (dw != nullptr) {
    LinearGemm& q = jobs[n++] = g;
    q.rows = out;
    q.depth = rows;
    q.a_mn = 1;
    q.b = ox.p;
    q.ldb = ox.ld;
    q.b_plane = ox.plane;
    q.c = dw;
    q.ldc = ld.dw;
    if (sums_left && !linear_gemm_on_pairs(q, sms)) {
      q.sum_parts = p.sums;
      q.sum_out = dbias;
      q.sum_slices = slices;
      sums_left = false;
    }
  }
  if (sums_left) {
    const cudaError_t e =
        launch_pdl(column_sum_kernel, dim3((static_cast<unsigned>(out) + 31) / 32), dim3(256), 0,
                   s, static_cast<const float*>(p.sums), slices, out, dbias);
    if (e != cudaSuccess) return MOE_ERR_CUDA;
  }
  if (n == 0) return MOE_OK;
  return status_of(launch_linear_gemms(jobs, n, device_error_word(), sms, s));
}
