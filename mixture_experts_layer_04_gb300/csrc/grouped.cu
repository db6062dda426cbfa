// moe_grouped_linear and moe_grouped_linear_backward: argument checks, the workspace and the
// passes around the grouped tensor-core product (grouped_gemm.cu).
//
//  - prepare_kernel: the plan of the groups (grouped_plan.cuh); operands the tensor cores cannot
//    read in place (float32 values become three bf16 parts, rows whose stride is not a multiple of
//    16 bytes are copied to one that is); and the gradient of SwiGLU, dz = (dy u silu'(g),
//    dy silu(g)), in one bf16 part or three.  Rows that belong to no group and weights of empty
//    groups are passed over.  Bound by reading dy and z and writing dz: 63011 rows of 768 with three
//    parts, 871 MB: 152 us (130 at a copy's rate).
#include "common.cuh"
#include "grouped.h"
#include "grouped_plan.cuh"
#include "kernels.h"
#include "linear_act.cuh"
#include "operand_io.cuh"

namespace moe {
namespace {

// The next bf16 part of v, and what it leaves.  A value that is not finite goes whole into the
// first part; a finite one that rounding would take past bf16's largest has that for its first
// part.
template <int PL>
__device__ __forceinline__ __nv_bfloat16 take_part(float* v, bool first) {
  float t = *v;
  if (PL > 1 && first && fabsf(t) < INFINITY) t = fminf(fmaxf(t, -kMaxBf16), kMaxBf16);
  const __nv_bfloat16 h = __float2bfloat16_rn(t);
  const float r = __bfloat162float(h);
  *v = fabsf(r) < INFINITY ? *v - r : 0.f;
  return h;
}

// n <= 8 values in PL bf16 parts at dst, dst + plane, ...; 16-byte stores when `vec`.
template <int PL>
__device__ __forceinline__ void store_parts(__nv_bfloat16* dst, long long plane, int n, bool vec,
                                            float (&v)[8]) {
#pragma unroll
  for (int pl = 0; pl < PL; ++pl) {
    __nv_bfloat16 h[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) h[q] = take_part<PL>(&v[q], pl == 0);
    __nv_bfloat16* d = dst + pl * plane;
    if (vec && n == 8) {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[i] = static_cast<uint32_t>(__bfloat16_as_ushort(h[2 * i])) |
               (static_cast<uint32_t>(__bfloat16_as_ushort(h[2 * i + 1])) << 16);
      *reinterpret_cast<uint4*>(d) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (q < n) d[q] = h[q];
    }
  }
}

// A matrix to copy in parts: rows of `cols` values.  Activations (group_rows == 0): the rows below
// the last bound; weights: the groups that have rows.
struct PackTask {
  const void* src;
  long long ld;
  __nv_bfloat16* dst;
  long long dst_ld, plane;
  long long rows;
  int cols, vec, group_rows;
  int blocks;  // of 256 threads, 0: nothing to pack
};

struct DzTask {
  const void* dy;
  const void* z;
  long long ldy, ldz;
  __nv_bfloat16* dz;
  long long dz_ld, plane;
  int cols;              // of dy; dz has twice as many
  int parts;
  int vec_y, vec_z, vec_dz;
  int blocks;
};

struct PrepareParams {
  const int32_t* offsets;
  int rows, groups;
  PlanTask plan;
  DzTask dz;
  PackTask dy, x, w;
};

// Calls f(row, eight of columns) for the items that are this thread's; 32-bit divisions where they
// do (64-bit ones cost more than the rest of an item).
template <typename F>
__device__ __forceinline__ void each_item(long long rows, int per_row, int block, int blocks, F f) {
  const long long items = rows * per_row;
  const long long step = blocks * 256ll;
  if (items + step <= 0xffffffffll) {
    for (uint32_t i = block * 256u + threadIdx.x; i < static_cast<uint32_t>(items);
         i += static_cast<uint32_t>(step)) {
      const uint32_t r = i / static_cast<uint32_t>(per_row);
      f(static_cast<long long>(r), static_cast<int>(i - r * static_cast<uint32_t>(per_row)));
    }
    return;
  }
  for (long long i = block * 256ll + threadIdx.x; i < items; i += step) {
    const long long r = i / per_row;
    f(r, static_cast<int>(i - r * per_row));
  }
}

template <typename T, int PL>
__device__ __forceinline__ void pack_task(const PackTask& t, const PrepareParams& p, int used,
                                          int block) {
  each_item(t.group_rows == 0 ? used : t.rows, static_cast<int>(t.dst_ld / 8), block, t.blocks,
            [&](long long r, int piece) {
              const int c = piece * 8;
              if (t.group_rows != 0) {
                const int g = static_cast<int>(static_cast<uint32_t>(r) /
                                               static_cast<uint32_t>(t.group_rows));
                // (where offsets are held, a group with rows still has an offset above the last)
                if (p.offsets[g + 1] <= p.offsets[g]) return;
              }
              float v[8];
              load_n(static_cast<const T*>(t.src) + r * t.ld + c, t.cols - c, t.vec != 0, v);
              store_parts<PL>(t.dst + r * t.dst_ld + c, t.plane, 8, true, v);
            });
}

template <int PL>
__device__ __forceinline__ void store_dz(__nv_bfloat16* dst, const DzTask& t, int n,
                                         float (&v)[8]) {
  if (PL == 3 || t.parts == 1) store_parts<PL>(dst, t.plane, n, t.vec_dz != 0, v);
  else store_parts<3>(dst, t.plane, n, t.vec_dz != 0, v);
}

// silu(z) = z p and its slope, with p the logistic function of z, for bf16 z: one exponential and one
// reciprocal for both.
__device__ __forceinline__ void silu_both(float z, float* value, float* slope) {
  const float t = __expf(-fabsf(z)), r = rcp_ftz(1.0f + t), tr = t * r;
  const float p = z > 0.f ? r : tr, q = z > 0.f ? tr : r;
  *value = z * p;
  *slope = silu_slope<true>(z, p, q);
}

template <typename T, int PL>
__device__ __forceinline__ void dz_task(const DzTask& t, int used, int block) {
  each_item(used, (t.cols + 7) / 8, block, t.blocks, [&](long long r, int piece) {
    const int c = piece * 8, n = min(8, t.cols - c);
    float dy[8], gate[8], up[8];
    load_n(static_cast<const T*>(t.dy) + r * t.ldy + c, n, t.vec_y != 0, dy);
    const T* z = static_cast<const T*>(t.z) + r * t.ldz + c;
    load_n(z, n, t.vec_z != 0, gate);
    load_n(z + t.cols, n, t.vec_z != 0, up);
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      float value, slope;
      if constexpr (PL == 1) {
        silu_both(gate[q], &value, &slope);
      } else {
        value = act_value<false>(MOE_ACT_SILU, gate[q]);
        slope = act_slope<false>(MOE_ACT_SILU, gate[q]);
      }
      gate[q] = dy[q] * up[q] * slope;
      up[q] = dy[q] * value;
    }
    __nv_bfloat16* dst = t.dz + r * t.dz_ld + c;
    store_dz<PL>(dst, t, n, gate);
    store_dz<PL>(dst + t.cols, t, n, up);
  });
}

// The plan's blocks first: they are the longest where little is packed.  (One launch for both: a
// packing that followed the plan's launch took 2 to 5 us more.)
template <typename T, int PL>
__global__ void __launch_bounds__(256) prepare_kernel(const __grid_constant__ PrepareParams p) {
  __shared__ int s_used;
  grid_dep_wait();
  grid_dep_trigger();
  int b = static_cast<int>(blockIdx.x);
  if (b < p.plan.blocks) {
    plan_block(p.plan, b);
    return;
  }
  b -= p.plan.blocks;
  if (threadIdx.x == 0) s_used = 0;
  __syncthreads();
  // the end of the last group: the largest offset, held to the rows
  int used = 0;
  for (int i = threadIdx.x; i <= p.groups; i += 256) used = max(used, p.offsets[i]);
  used = __reduce_max_sync(0xffffffffu, used);
  if ((threadIdx.x & 31) == 0) atomicMax(&s_used, used);
  __syncthreads();
  used = min(s_used, p.rows);
  if (b < p.dz.blocks) {
    dz_task<T, PL>(p.dz, used, b);
    return;
  }
  b -= p.dz.blocks;
  if (b < p.dy.blocks) {
    pack_task<T, PL>(p.dy, p, used, b);
    return;
  }
  b -= p.dy.blocks;
  if (b < p.x.blocks) pack_task<T, PL>(p.x, p, used, b);
  else pack_task<T, PL>(p.w, p, used, b - p.x.blocks);
}

cudaError_t launch_prepare(const PrepareParams& p, bool f32, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>(p.plan.blocks + p.dz.blocks + p.dy.blocks + p.x.blocks +
                                        p.w.blocks));
  return f32 ? launch_pdl(prepare_kernel<float, 3>, grid, dim3(256), 0, s, p)
             : launch_pdl(prepare_kernel<__nv_bfloat16, 1>, grid, dim3(256), 0, s, p);
}

// --------------------------------------------------------------------- host ----

struct Shape {
  long long x, w, y, z, dx, dw;  // row strides
  int w_rows;                    // rows of a group's weights, columns of z
  bool swiglu, f32;
};

Shape shape_of(const moe_grouped_config_t* c) {
  auto pick = [](long long s, long long n) { return s != 0 ? s : n; };
  Shape s;
  s.swiglu = c->activation == MOE_ACT_SWIGLU;
  s.f32 = c->dtype == MOE_F32;
  s.w_rows = c->out_features * (s.swiglu ? 2 : 1);
  s.x = pick(c->x_stride, c->in_features);
  s.w = pick(c->w_stride, c->in_features);
  s.y = pick(c->y_stride, c->out_features);
  s.z = pick(c->z_stride, s.w_rows);
  s.dx = pick(c->dx_stride, c->in_features);
  s.dw = pick(c->dw_stride, c->in_features);
  return s;
}

moe_status_t check_grouped_config(const moe_grouped_config_t* c) {
  if (c == nullptr) return MOE_ERR_INVALID_ARG;
  if (c->rows < 0 || c->rows > (1 << 30)) return MOE_ERR_INVALID_ARG;
  if (c->groups < 1 || c->groups > 1024) return MOE_ERR_INVALID_ARG;
  if (c->in_features < 1 || c->in_features > (1 << 18)) return MOE_ERR_INVALID_ARG;
  if (c->out_features < 1 || c->out_features > (1 << 18)) return MOE_ERR_INVALID_ARG;
  if (c->dtype != MOE_F32 && c->dtype != MOE_BF16) return MOE_ERR_INVALID_ARG;
  if (c->out_dtype != c->dtype && c->out_dtype != MOE_F32) return MOE_ERR_INVALID_ARG;
  if (c->dx_dtype != c->dtype && c->dx_dtype != MOE_F32) return MOE_ERR_INVALID_ARG;
  if (c->activation != MOE_ACT_NONE && c->activation != MOE_ACT_SWIGLU)
    return c->activation < 0 || c->activation > MOE_ACT_SWIGLU ? MOE_ERR_INVALID_ARG
                                                               : MOE_ERR_UNSUPPORTED;
  const Shape s = shape_of(c);
  const long long most = 1ll << 31;
  const struct {
    long long stride, least;
  } q[] = {{c->x_stride, c->in_features},  {c->w_stride, c->in_features},
           {c->y_stride, c->out_features}, {c->z_stride, s.w_rows},
           {c->dx_stride, c->in_features}, {c->dw_stride, c->in_features}};
  for (const auto& v : q)
    if (v.stride != 0 && (v.stride < v.least || v.stride > most)) return MOE_ERR_INVALID_ARG;
  // tiles of a product are numbered in 31 bits (the smallest tile: 32 rows, 64 features, but for
  // tiles that go round the SMs once)
  const long long rows = c->rows / 32 + c->groups;
  const long long widest = c->in_features > c->out_features ? c->in_features : c->out_features;
  const long long wg = (s.w_rows + 127ll) / 128 * ((c->in_features + 127ll) / 128) * c->groups;
  if (rows * (widest / 64 + 1) >= (1ll << 30) || wg >= (1ll << 30)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// Workspace: the plan (bounds, tiles of rows, tensor maps), packed x and w, dz in operand form.
struct Layout {
  bool pack_x, pack_w, make_dz;
  int parts;     // bf16 parts of an operand's value
  int dz_parts;  // and of dz
  int tile_rows;
  size_t bounds, count, tiles, maps, x, w, dz, total;
};

Layout layout_of(const moe_grouped_config_t* c) {
  const Shape s = shape_of(c);
  Layout l;
  l.parts = s.f32 ? 3 : 1;
  // The caller's choice, by dx_dtype.  MOE_BF16: dz rounded to bf16, as a program that keeps it in bf16
  // has it (dw 2.3e-3 off in relative L2, of which 1.7e-3 are dw's own rounding).  MOE_F32: its 24
  // bits for dx, in three parts, and two of these for dw (1.7e-3).  63011 rows of 128 groups, 2048 ->
  // 768: 745 us and 1,500; two parts for both left a float32 dx 2.7e-6 off instead of 8e-7 (1,210 us).
  l.dz_parts = s.f32 || (s.swiglu && c->dx_dtype == MOE_F32) ? 3 : 1;
  l.tile_rows = grouped_tile_rows(c->rows, c->groups, s.f32);
  l.pack_x = s.f32 || odd_stride(s.x, c->dtype);
  l.pack_w = s.f32 || odd_stride(s.w, c->dtype);
  l.make_dz = s.f32 || s.swiglu || odd_stride(s.y, c->dtype);
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o += (bytes + 255) & ~static_cast<size_t>(255);
    return at;
  };
  const size_t rows = c->rows, groups = c->groups, parts = l.parts;
  l.bounds = take((groups + 1) * 4);
  l.count = take(4);
  l.tiles = take(grouped_max_tiles(c->rows, c->groups, l.tile_rows) * 16);
  l.maps = take(groups * 2 * 128);
  l.x = take(l.pack_x ? parts * rows * pad8(c->in_features) * 2 : 0);
  l.w = take(l.pack_w ? parts * groups * s.w_rows * pad8(c->in_features) * 2 : 0);
  l.dz = take(l.make_dz ? l.dz_parts * rows * pad8(s.w_rows) * 2 : 0);
  l.total = o + 256;  // the start is moved up to a multiple of 256
  return l;
}

struct Workspace {
  char* base;
  explicit Workspace(void* ws)
      : base(reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(ws) + 255) &
                                     ~static_cast<uintptr_t>(255))) {}
  template <typename T>
  T* at(size_t off) const {
    return reinterpret_cast<T*>(base + off);
  }
  GroupPlan plan(const Layout& l) const {
    return GroupPlan{at<int>(l.bounds), at<int4>(l.tiles), at<int>(l.count), at<void>(l.maps),
                     nullptr};
  }
};

int blocks_for(long long items, int num_sms) {
  const long long blocks = (items + 255) / 256, most = 16ll * num_sms;
  return static_cast<int>(blocks < most ? blocks : most);
}

struct Operand {
  const void* p;
  long long ld, plane;
};

// The matrix in place, or packed into `dst` by the task it fills in.
Operand operand(const void* src, long long ld, long long rows, int cols, int group_rows, int dtype,
                bool pack, void* dst, int num_sms, PackTask* t) {
  if (!pack) return Operand{src, ld, 0};
  t->src = src;
  t->ld = ld;
  t->dst = static_cast<__nv_bfloat16*>(dst);
  t->dst_ld = pad8(cols);
  t->plane = t->dst_ld * rows;
  t->rows = rows;
  t->cols = cols;
  t->vec = vec_ok(src, ld, dtype);
  t->group_rows = group_rows;
  t->blocks = blocks_for(t->plane / 8, num_sms);
  return Operand{dst, t->dst_ld, t->plane};
}

}  // namespace
}  // namespace moe

extern "C" moe_status_t moe_grouped_linear_workspace_size(const moe_grouped_config_t* cfg,
                                                          size_t* bytes) {
  using namespace moe;
  moe_status_t st = fault_point("moe_grouped_linear_workspace_size");
  if (st != MOE_OK) return st;
  st = check_grouped_config(cfg);
  if (st != MOE_OK) return st;
  if (bytes == nullptr) return MOE_ERR_INVALID_ARG;
  *bytes = layout_of(cfg).total;
  return MOE_OK;
}

extern "C" moe_status_t moe_grouped_linear(const moe_grouped_config_t* cfg, const void* x,
                                           const int32_t* offsets, const void* w, void* y, void* z,
                                           void* ws, size_t ws_bytes, moe_stream_t stream) {
  using namespace moe;
  moe_status_t st = fault_point("moe_grouped_linear");
  if (st != MOE_OK) return st;
  st = check_grouped_config(cfg);
  if (st != MOE_OK) return st;
  if (cfg->rows == 0) return MOE_OK;
  const Shape sh = shape_of(cfg);
  if (x == nullptr || offsets == nullptr || w == nullptr || y == nullptr ||
      (z != nullptr && !sh.swiglu))
    return MOE_ERR_INVALID_ARG;
  if (bad_operand(x, sh.x, cfg->dtype) || bad_operand(w, sh.w, cfg->dtype) ||
      unaligned(offsets, 4) || unaligned(y, act_bytes(cfg->out_dtype)) ||
      unaligned(z, act_bytes(cfg->dtype)))
    return MOE_ERR_MISALIGNED;
  const Layout l = layout_of(cfg);
  if (ws == nullptr || ws_bytes < l.total) return MOE_ERR_WORKSPACE;
  if (unaligned(ws, 16)) return MOE_ERR_MISALIGNED;
  st = check_current_device();
  if (st != MOE_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int sms = device_num_sms();
  const Workspace at(ws);
  GroupPlan plan = at.plan(l);
  unsigned* err = device_error_word();
  PrepareParams pp{};
  pp.offsets = offsets;
  pp.rows = cfg->rows;
  pp.groups = cfg->groups;
  const Operand ox = operand(x, sh.x, cfg->rows, cfg->in_features, 0, cfg->dtype, l.pack_x,
                             at.at<void>(l.x), sms, &pp.x);
  const Operand ow = operand(w, sh.w, static_cast<long long>(cfg->groups) * sh.w_rows,
                             cfg->in_features, sh.w_rows, cfg->dtype, l.pack_w, at.at<void>(l.w),
                             sms, &pp.w);
  if (pp.x.blocks + pp.w.blocks == 0 && grouped_plans_itself(l.tile_rows, sh.f32)) {
    plan.offsets = offsets;
  } else if (!group_plan_task(offsets, cfg->rows, cfg->groups, l.tile_rows, plan, nullptr, err,
                              &pp.plan) ||
             launch_prepare(pp, sh.f32, s) != cudaSuccess) {
    return MOE_ERR_CUDA;
  }
  GroupedProduct g{};
  g.kind = GroupedKind::kForward;
  g.groups = cfg->groups;
  g.total_rows = cfg->rows;
  g.a_parts = g.b_parts = l.parts;
  g.depth = cfg->in_features;
  g.features = cfg->out_features;
  g.swiglu = sh.swiglu;
  g.a = ox.p;
  g.lda = ox.ld;
  g.a_plane = ox.plane;
  g.b = ow.p;
  g.ldb = ow.ld;
  g.b_plane = ow.plane;
  g.c = y;
  g.c_f32 = cfg->out_dtype == MOE_F32;
  g.ldc = sh.y;
  g.z = z;
  g.z_f32 = sh.f32;
  g.ldz = sh.z;
  return status_of(launch_grouped_products(&g, 1, plan, err, sms, s));
}

extern "C" moe_status_t moe_grouped_linear_backward(const moe_grouped_config_t* cfg, const void* dy,
                                                    const void* x, const int32_t* offsets,
                                                    const void* w, const void* z, void* dx,
                                                    void* dw, void* ws, size_t ws_bytes,
                                                    moe_stream_t stream) {
  using namespace moe;
  moe_status_t st = fault_point("moe_grouped_linear_backward");
  if (st != MOE_OK) return st;
  st = check_grouped_config(cfg);
  if (st != MOE_OK) return st;
  const Shape sh = shape_of(cfg);
  const size_t ab = act_bytes(cfg->dtype);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (unaligned(dx, act_bytes(cfg->dx_dtype)) || unaligned(dw, ab)) return MOE_ERR_MISALIGNED;
  if (cfg->rows == 0) {
    if (dw == nullptr) return MOE_OK;
    st = check_current_device();
    if (st != MOE_OK) return st;
    return status_of(cudaMemset2DAsync(dw, sh.dw * ab, 0, cfg->in_features * ab,
                                       static_cast<size_t>(cfg->groups) * sh.w_rows, s));
  }
  if (dy == nullptr || offsets == nullptr || (dx == nullptr && dw == nullptr) ||
      (dx != nullptr && w == nullptr) || (dw != nullptr && x == nullptr) ||
      (sh.swiglu && z == nullptr))
    return MOE_ERR_INVALID_ARG;
  if (bad_operand(dy, sh.y, cfg->dtype) || (dw != nullptr && bad_operand(x, sh.x, cfg->dtype)) ||
      (dx != nullptr && bad_operand(w, sh.w, cfg->dtype)) || unaligned(offsets, 4) ||
      (sh.swiglu && unaligned(z, ab)))
    return MOE_ERR_MISALIGNED;
  const Layout l = layout_of(cfg);
  if (ws == nullptr || ws_bytes < l.total) return MOE_ERR_WORKSPACE;
  if (unaligned(ws, 16)) return MOE_ERR_MISALIGNED;
  st = check_current_device();
  if (st != MOE_OK) return st;
  const int sms = device_num_sms();
  const Workspace at(ws);
  GroupPlan plan = at.plan(l);
  unsigned* err = device_error_word();

  PrepareParams pp{};
  pp.offsets = offsets;
  pp.rows = cfg->rows;
  pp.groups = cfg->groups;
  Operand ox{}, ow{}, odz{dy, sh.y, 0};
  if (dw != nullptr)
    ox = operand(x, sh.x, cfg->rows, cfg->in_features, 0, cfg->dtype, l.pack_x, at.at<void>(l.x),
                 sms, &pp.x);
  if (dx != nullptr)
    ow = operand(w, sh.w, static_cast<long long>(cfg->groups) * sh.w_rows, cfg->in_features,
                 sh.w_rows, cfg->dtype, l.pack_w, at.at<void>(l.w), sms, &pp.w);
  if (l.make_dz && !sh.swiglu) {
    odz = operand(dy, sh.y, cfg->rows, cfg->out_features, 0, cfg->dtype, true, at.at<void>(l.dz),
                  sms, &pp.dy);
  } else if (l.make_dz) {
    DzTask& t = pp.dz;
    t.dy = dy;
    t.z = z;
    t.ldy = sh.y;
    t.ldz = sh.z;
    t.dz = at.at<__nv_bfloat16>(l.dz);
    t.dz_ld = pad8(sh.w_rows);
    t.plane = t.dz_ld * cfg->rows;
    t.cols = cfg->out_features;
    t.parts = l.dz_parts;
    const bool eights = cfg->out_features % 8 == 0;
    t.vec_y = vec_ok(dy, sh.y, cfg->dtype);
    t.vec_z = eights && vec_ok(z, sh.z, cfg->dtype);
    t.vec_dz = eights;
    t.blocks = blocks_for(static_cast<long long>(cfg->rows) * ((t.cols + 7) / 8), sms);
    odz = Operand{t.dz, t.dz_ld, t.plane};
  }

  GroupedProduct q{};
  q.groups = cfg->groups;
  q.total_rows = cfg->rows;
  q.a_parts = l.dz_parts;
  q.b_parts = l.parts;
  q.a = odz.p;
  q.lda = odz.ld;
  q.a_plane = odz.plane;
  q.features = cfg->in_features;
  GroupedProduct gx = q, gw = q;
  gx.kind = GroupedKind::kInputGrad;
  gx.depth = sh.w_rows;
  gx.b = ow.p;
  gx.ldb = ow.ld;
  gx.b_plane = ow.plane;
  gx.c = dx;
  gx.c_f32 = cfg->dx_dtype == MOE_F32;
  gx.ldc = sh.dx;
  gw.kind = GroupedKind::kWeightGrad;
  if (!sh.f32 && gw.a_parts == 3) gw.a_parts = 2;  // (16 bits of dz, for a bf16 result)
  gw.rows = sh.w_rows;
  gw.b = ox.p;
  gw.ldb = ox.ld;
  gw.b_plane = ox.plane;
  gw.c = dw;
  gw.c_f32 = sh.f32;
  gw.ldc = sh.dw;
  gw.c_group = sh.dw * sh.w_rows;

  const bool pack = pp.dz.blocks + pp.dy.blocks + pp.x.blocks + pp.w.blocks > 0;
  if (dw == nullptr && !pack && grouped_plans_itself(l.tile_rows, sh.f32)) {
    plan.offsets = offsets;
  } else if (!group_plan_task(offsets, cfg->rows, cfg->groups, l.tile_rows, plan,
                              dw != nullptr ? &gw : nullptr, err, &pp.plan) ||
             launch_prepare(pp, sh.f32, s) != cudaSuccess) {
    return MOE_ERR_CUDA;
  }
  GroupedProduct both[2];
  int n = 0;
  if (dx != nullptr) both[n++] = gx;
  if (dw != nullptr) both[n++] = gw;
  return status_of(launch_grouped_products(both, n, plan, err, sms, s));
}
