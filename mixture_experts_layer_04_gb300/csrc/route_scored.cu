// Routing from scores and its gradient (moe_route_scored, moe_route_scored_backward).
//
// One warp per token.  Lane i holds the NJ consecutive experts i*NJ .. i*NJ+NJ-1, so that
// among equal keys the lowest lane (and in it the lowest register) is the lowest expert, and
// a group whose size is a multiple of NJ never straddles lanes.
//
// The choice.  It is defined on 64-bit keys s[e] + bias[e], and 64-bit arithmetic is slow on
// this GPU (16 clocks per warp instruction), so it is taken in float first and certified
// with a bound on the error of every float score.  The bound is the one of the largest score
// there can be, not those of the two experts compared: an expert further down in the order may
// have a larger score (and a lower bias) than they, and its key may be off by more than theirs.
// Where two neighbouring choices (the K-th and the first one left out among them) are closer
// than two such bounds, the K+1 best are put in order by their 64-bit keys, one per lane; groups
// whose sums cannot be told apart at the border between kept and dropped are compared by 64-bit
// sums; and only if in such a case the first two experts left out are close to each other too
// is the whole token chosen again.  Without a bias the keys are ordered as the logits are, so
// the logits themselves are compared.  Two experts of equal logit and equal bias tie in any
// precision, so they need no certificate; but where the K-th and the first one left out tie,
// it is the experts after them that must be clear of both.
//
// The K+1 best come from each lane's own four best, kept in order in registers as integers:
// the float's bits made monotone, the last log2(NJ) of them replaced by the register's number
// (the bounds count that rounding).  Keeping them in order is then minima and maxima alone,
// and a step is one warp-wide maximum, a ballot and a shuffle.
//
// What bounds it: the row of logits is read once (T*E elements) and K ids and weights are
// written, but the instructions come first: 924 per token at 256 experts in 8 groups and K = 8,
// most of them on the half-rate integer and compare pipe (60% busy).  16384 such tokens take
// 18 to 21 us (2.6 us of memory traffic), one token 4.3 us, which is its launch.
#include <cfloat>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "topk.cuh"

namespace moe {
namespace {

constexpr int kWarps = 8;

struct RouteParams {
  const void* logits;
  const float* bias;  // or null
  int32_t* ids;
  float* w;
  const int32_t* ids_in;  // backward
  const float* d_w;
  void* d_logits;
  long long stride;  // elements between rows
  int T, E, K, groups, per, top_groups, rank;
  int renorm;
  int vec;  // rows allow whole-lane vector loads (and, backward, 16-byte stores)
  int vec_bias;  // whole-lane vector loads of the bias
  int group_lanes;  // lanes per group where groups do not share lanes, else 0
  int lane_shift;   // their logarithm where that is whole, else -1
  float scale;
};

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_float(float v);
template <>
__device__ __forceinline__ float from_float<float>(float v) {
  return v;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

// A logit as the definition reads it: NaN counts as -inf (masked), +inf as the largest float.
__device__ __forceinline__ float clean_logit(float l) {
  return l > -INFINITY ? fminf(l, FLT_MAX) : -INFINITY;
}

// The warp's largest value (no NaN among them).
__device__ __forceinline__ float warp_max(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

// This lane's NJ logits of one row as they are in memory (those past E as -inf).
template <int NJ, typename TL>
__device__ __forceinline__ void load_raw(const TL* row, int E, int lane, int vec, float (&l)[NJ]) {
  const int e0 = lane * NJ;
  constexpr int kBytes = NJ * static_cast<int>(sizeof(TL));
  if constexpr (kBytes >= 4) {
    if (vec) {
      constexpr int kVec = kBytes >= 16 ? 16 : kBytes;  // bytes per load
      constexpr int kPer = kVec / static_cast<int>(sizeof(TL));
      if (e0 < E) {
#pragma unroll
        for (int i = 0; i < NJ / kPer; ++i) {
          alignas(16) TL v[kPer];
          if constexpr (kVec == 16)
            *reinterpret_cast<uint4*>(v) = reinterpret_cast<const uint4*>(row + e0)[i];
          else if constexpr (kVec == 8)
            *reinterpret_cast<uint2*>(v) = reinterpret_cast<const uint2*>(row + e0)[i];
          else
            *reinterpret_cast<uint32_t*>(v) = reinterpret_cast<const uint32_t*>(row + e0)[i];
#pragma unroll
          for (int q = 0; q < kPer; ++q) l[i * kPer + q] = to_float(v[q]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < NJ; ++j) l[j] = -INFINITY;
      }
      return;
    }
  }
#pragma unroll
  for (int j = 0; j < NJ; ++j) l[j] = e0 + j < E ? to_float(row[e0 + j]) : -INFINITY;
}

// The same as the definition reads them (clean_logit).  A sum finds out whether any needs it:
// it is NaN if one of them is (or if +inf meets -inf), +inf if one of them is.
template <int NJ, typename TL>
__device__ __forceinline__ void load_row(const TL* row, int E, int lane, int vec, float (&l)[NJ]) {
  load_raw<NJ, TL>(row, E, lane, vec, l);
  float sum = l[0];
#pragma unroll
  for (int j = 1; j < NJ; ++j) sum += l[j];
  if (!(sum < INFINITY)) {
#pragma unroll
    for (int j = 0; j < NJ; ++j) l[j] = clean_logit(l[j]);
  }
}

// This lane's NJ biases (those past E as 0).
template <int NJ>
__device__ __forceinline__ void load_bias(const RouteParams& p, int lane, float (&b)[NJ]) {
  const int e0 = lane * NJ;
  if constexpr (NJ >= 4) {
    if (p.vec_bias) {
      if (e0 < p.E) {
#pragma unroll
        for (int i = 0; i < NJ; i += 4) {
          const float4 v = __ldg(reinterpret_cast<const float4*>(p.bias + e0 + i));
          b[i] = v.x, b[i + 1] = v.y, b[i + 2] = v.z, b[i + 3] = v.w;
        }
      } else {
#pragma unroll
        for (int j = 0; j < NJ; ++j) b[j] = 0.f;
      }
      return;
    }
  }
#pragma unroll
  for (int j = 0; j < NJ; ++j) b[j] = e0 + j < p.E ? __ldg(p.bias + e0 + j) : 0.f;
}

// The 64-bit score of a logit, and what it needs of its row: the softmax's sum.
template <bool kSig>
__device__ __forceinline__ double score64(float l, float m, double sum) {
  if (!(l > -INFINITY)) return 0.0;
  return kSig ? 1.0 / (1.0 + exp(-static_cast<double>(l)))
              : exp(static_cast<double>(l) - static_cast<double>(m)) / sum;
}
template <int NJ, typename TL>
__device__ __forceinline__ double softmax_sum64(const TL* row, int E, float m, int lane) {
  double sum = 0.0;
#pragma unroll 4
  for (int j = 0; j < NJ; ++j) {
    const int e = lane * NJ + j;
    const float l = e < E ? clean_logit(to_float(row[e])) : -INFINITY;
    if (l > -INFINITY) sum += exp(static_cast<double>(l) - static_cast<double>(m));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  return sum;
}

// The largest key of a warp's candidates (kNone: no candidate) with its expert, ties to the
// lower expert, -1 if there is none.
__device__ __forceinline__ int warp_best64(double* key, int e) {
  double k = *key;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const double ko = __shfl_xor_sync(0xffffffffu, k, o);
    const int eo = __shfl_xor_sync(0xffffffffu, e, o);
    if (eo >= 0 && (e < 0 || ko > k || (ko == k && eo < e))) {
      k = ko;
      e = eo;
    }
  }
  *key = k;
  return e;
}

template <bool kSig, typename TL>
__device__ __forceinline__ double key64(const RouteParams& p, const TL* row, int e, float m,
                                        double sum) {
  const float l = e < p.E ? clean_logit(to_float(row[e])) : -INFINITY;
  const float b = e < p.E && p.bias != nullptr ? p.bias[e] : 0.f;
  if (!(l > -INFINITY && b > -INFINITY)) return -INFINITY;
  return score64<kSig>(l, m, sum) + static_cast<double>(b);
}

// The sums of the groups in `contested` by 64-bit keys, lane g returns group g's.
template <int NJ, typename TL, bool kSig>
__device__ __noinline__ double group_sums64(const RouteParams& p, const TL* row, float m, int lane,
                                            uint32_t contested) {
  const double sum = kSig ? 0.0 : softmax_sum64<NJ, TL>(row, p.E, m, lane);
  double mine = -INFINITY;
  while (contested != 0u) {
    const int g = __ffs(contested) - 1;
    contested &= contested - 1u;
    // this lane's two best of the group, then the warp's
    double v1 = -INFINITY, v2 = -INFINITY;
    int e1 = -1;
#pragma unroll 1
    for (int i = lane; i < p.per; i += 32) {
      const double k = key64<kSig>(p, row, g * p.per + i, m, sum);
      if (k > v1) {
        v2 = v1;
        v1 = k;
        e1 = g * p.per + i;
      } else if (k > v2) {
        v2 = k;
      }
    }
    double best = v1;
    const int e = warp_best64(&best, e1);
    double total = best;
    if (p.rank > 1) {
      double second = e1 == e ? v2 : v1;
      warp_best64(&second, second > -INFINITY ? lane : -1);
      if (second > -INFINITY) total += second;
    }
    if (lane == g) mine = total;
  }
  return mine;
}

// The choice from 64-bit keys throughout, among the groups in `live`; lane k < K returns the
// k-th expert or -1.  m: the row's largest logit (softmax).
template <int NJ, typename TL, bool kSig>
__device__ __noinline__ int choose64(const RouteParams& p, const TL* row, float m, int lane,
                                     uint32_t live) {
  double key[NJ];
  const int e0 = lane * NJ;
  const double sum = kSig ? 0.0 : softmax_sum64<NJ, TL>(row, p.E, m, lane);
#pragma unroll 1
  for (int j = 0; j < NJ; ++j) {
    const bool in = e0 + j < p.E && ((live >> ((e0 + j) / p.per)) & 1u);
    key[j] = in ? key64<kSig>(p, row, e0 + j, m, sum) : -INFINITY;
  }
  int chosen = -1;
#pragma unroll 1
  for (int k = 0; k < p.K; ++k) {
    double v = -INFINITY;
    int mine = -1;
#pragma unroll 1
    for (int j = 0; j < NJ; ++j)
      if (key[j] > v) {
        v = key[j];
        mine = e0 + j;
      }
    const int e = warp_best64(&v, mine);
    if (e < 0) break;
    if (lane == k) chosen = e;
    if (e >= e0 && e < e0 + NJ) key[e - e0] = -INFINITY;
  }
  return chosen;
}

// Puts the experts in lanes 0..K (-1 from the first empty lane on) in the order of their
// 64-bit keys, or of their logits where those decide, ties to the lower expert.
template <int NJ, typename TL, bool kSig>
__device__ __noinline__ int order64(const RouteParams& p, const TL* row, float m, int lane,
                                    int mine, float l, float b, bool by_logit) {
  double key = l;
  if (!by_logit) {
    const double sum = kSig ? 0.0 : softmax_sum64<NJ, TL>(row, p.E, m, lane);
    key = score64<kSig>(l, m, sum) + static_cast<double>(b);
  }
  const int n = __popc(__ballot_sync(0xffffffffu, mine >= 0));
  int rank = 0;
#pragma unroll 1
  for (int j = 0; j < n; ++j) {
    const double kj = __shfl_sync(0xffffffffu, key, j);
    const int ej = __shfl_sync(0xffffffffu, mine, j);
    rank += (kj > key || (kj == key && ej < mine)) ? 1 : 0;
  }
  int out = -1;
#pragma unroll 1
  for (int j = 0; j < n; ++j) {
    const int rj = __shfl_sync(0xffffffffu, rank, j);
    const int ej = __shfl_sync(0xffffffffu, mine, j);
    if (lane == rj) out = ej;
  }
  return out;
}

__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// A float score.  Its absolute error, in units of 2^-23 of the score: the hardware exponential
// is off by at most 2 + 1.17 |x| of them.  Logistic function: for l > 0 that is damped by 1 - s
// to 1.1, the sum and the reciprocal add under 3: 5 + 1.2 max(-l, 0).  Softmax: the sum adds its
// terms' mean error (|x| averages at most ln 1024) and its additions' roundings, 17 in all, the
// products 2: 21 + 1.2 (m - l).  The scores fall faster than these grow, so no score of a row is
// off by more than the largest there can be: 5 units of 1, 21 units of inv_sum.  Scores under
// 2^-126 may come out as 0, which the bounds' floor covers.
template <bool kSig>
__device__ __forceinline__ float score_of(float l, float m, float inv_sum) {
  if (kSig) return rcp_approx(1.0f + __expf(-l));
  return __expf(l - m) * inv_sum;
}
template <bool kSig>
__device__ __forceinline__ float score_error(float inv_sum) {
  return kSig ? 5.0f * 0x1p-23f : 21.0f * 0x1p-23f * inv_sum;
}
constexpr float kErrFloor = 1e-34f;

// One chosen (or next best) expert as a lane holds it.
struct Pick {
  float l, b, key;
};

// Without a bias the order of the scores is the order of the logits, but scores a few 2^-53 of
// their size apart may round together in 64 bits.  a.l >= b.l here.
template <bool kSig>
__device__ __forceinline__ bool scores_merge(const Pick& a, const Pick& b, float m) {
  const float gap = a.l - b.l;
  if (kSig) return a.l > 80.f || b.l < -600.f || !(__fdividef(gap, 1.0f + __expf(a.l)) > 1e-14f);
  return !(gap > 1e-14f) || b.l - m < -600.f;
}

// Whether a and b, a before b, are too close to rely on a being before b and everything after b
// in the order of the keys (rounded to `unit`, each with an error of up to `err`).
template <bool kSig>
__device__ __forceinline__ bool close(const Pick& a, const Pick& b, bool has_bias, float m,
                                      float err, float unit) {
  if (has_bias)
    return !(a.key - b.key >
             2.0f * (err + kErrFloor) + unit * (fabsf(a.key) + fabsf(b.key)));
  return !(a.l - b.l > unit * (fabsf(a.l) + fabsf(b.l)) + 1e-30f) || scores_merge<kSig>(a, b, m);
}

// Whether an expert in play other than those that tie with `a` is too close to it.  Needed where
// three or more tie at the border: 16384 tokens of 256 equal logits take 24 us, without it 14.
template <int NJ, typename TL, bool kSig>
__device__ __noinline__ bool others_close(const RouteParams& p, const TL* row, const Pick& a,
                                          float m, float inv_sum, int lane, uint32_t live,
                                          float err, float unit) {
  float l[NJ];
  load_row<NJ, TL>(row, p.E, lane, p.vec, l);
  const bool has_bias = p.bias != nullptr;
  bool near = false;
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const int e = lane * NJ + j;
    if (!(l[j] > -INFINITY) || !((live >> (e / p.per)) & 1u)) continue;
    Pick q{l[j], has_bias ? __ldg(p.bias + e) : 0.f, 0.f};
    if (!(q.b > -INFINITY) || (q.l == a.l && q.b == a.b)) continue;
    q.key = score_of<kSig>(q.l, m, inv_sum) + q.b;
    const bool above = has_bias ? q.key > a.key : q.l > a.l;
    near |= above ? close<kSig>(q, a, has_bias, m, err, unit)
                  : close<kSig>(a, q, has_bias, m, err, unit);
  }
  return __any_sync(0xffffffffu, near);
}

// A chosen expert's score over one factor common to the token's chosen (of largest logit `top`),
// which renormalisation takes out again: the logistic function is e^min(l,0) / (1 + e^-|l|), so
// that nothing overflows and small scores keep their ratio.
template <bool kSig>
__device__ __forceinline__ float relative_score(float l, float top) {
  if (!kSig) return expf(l - top);
  return __fdividef(expf(fminf(l, 0.f) - fminf(top, 0.f)), 1.0f + expf(-fabsf(l)));
}

// Descending order of two, and of four.
__device__ __forceinline__ void order2(uint32_t& a, uint32_t& b) {
  const uint32_t hi = max(a, b);
  b = min(a, b);
  a = hi;
}
__device__ __forceinline__ void order4(uint32_t& a, uint32_t& b, uint32_t& c, uint32_t& d) {
  order2(a, b);
  order2(c, d);
  order2(a, c);
  order2(b, d);
  order2(b, c);
}

// The four largest of v[0..NJ-1] (zeros after them), descending.
template <int NJ>
__device__ __forceinline__ void four_best(const uint32_t (&v)[NJ], uint32_t (&o)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = i < NJ ? v[i < NJ ? i : 0] : 0u;
  if constexpr (NJ == 2) order2(o[0], o[1]);
  if constexpr (NJ >= 4) order4(o[0], o[1], o[2], o[3]);
#pragma unroll
  for (int j = 4; j < NJ; j += 4) {
    uint32_t q0 = v[j], q1 = v[j + 1], q2 = v[j + 2], q3 = v[j + 3];
    order4(q0, q1, q2, q3);
    // the larger of opposite ends: the four best of the eight, as a bitonic sequence
    o[0] = max(o[0], q3);
    o[1] = max(o[1], q2);
    o[2] = max(o[2], q1);
    o[3] = max(o[3], q0);
    order2(o[0], o[2]);
    order2(o[1], o[3]);
    order2(o[0], o[1]);
    order2(o[2], o[3]);
  }
}

template <int NJ, typename TL, bool kSig>
__global__ void __launch_bounds__(32 * kWarps)
    route_scored_kernel(const __grid_constant__ RouteParams p) {
  __shared__ float s_key[kWarps][NJ * 32];
  grid_dep_wait();
  grid_dep_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = blockIdx.x * kWarps + warp;
  if (t >= p.T) return;
  const TL* row = static_cast<const TL*>(p.logits) + static_cast<size_t>(t) * p.stride;
  const int e0 = lane * NJ;
  float l[NJ];
  load_row<NJ, TL>(row, p.E, lane, p.vec, l);
  const bool has_bias = p.bias != nullptr;

  float m = 0.f, inv_sum = 0.f;
  if (!kSig) {
    m = l[0];
#pragma unroll
    for (int j = 1; j < NJ; ++j) m = fmaxf(m, l[j]);
    m = warp_max(m);
    if (m == -INFINITY) m = 0.f;  // every expert is masked
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < NJ; ++j) sum += __expf(l[j] - m);
    inv_sum = 1.0f / warp_sum(sum);
  }

  const float err = score_error<kSig>(inv_sum);

  // `ord` orders the experts by their keys; those at kNone or below are not available
  constexpr uint32_t kLow = NJ - 1, kNone = 0x007fffffu;  // kNone: -inf's
  auto order_key = [](float v, int j) {
    const uint32_t u = __float_as_uint(v + 0.0f);  // -0 counts as +0
    const uint32_t mono = u ^ (static_cast<uint32_t>(static_cast<int>(u) >> 31) | 0x80000000u);
    return (mono & ~kLow) | (kLow - static_cast<uint32_t>(j));
  };
  const bool grouped = p.top_groups < p.groups;
  uint32_t ord[NJ], best[4];  // all keys; the lane's four best still in play, descending
  uint32_t live = 0xffffffffu;  // groups in play
  auto value_of = [](uint32_t o) {  // the float of an ordered key, its low bits cleared
    const uint32_t u = o & ~kLow;
    return __uint_as_float((u & 0x80000000u) ? u ^ 0x80000000u : ~u);
  };
  if (has_bias) {
    float b[NJ];
    load_bias<NJ>(p, lane, b);
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      // a masked logit makes this NaN (0 * -inf), as a NaN bias does, and the maximum -inf
      const float k = fmaf(0.0f, l[j], score_of<kSig>(l[j], m, inv_sum) + b[j]);
      ord[j] = order_key(fmaxf(k, -INFINITY), j);
    }
  } else {
#pragma unroll
    for (int j = 0; j < NJ; ++j) ord[j] = order_key(l[j], j);
  }
  four_best<NJ>(ord, best);

  if (grouped) {
    // The sum of a group's best one or two keys, for group g in lane g.  Keys come from the
    // ordered integers (without a bias those hold logits).
    auto key_of = [&](uint32_t o) {
      if (o <= (kNone | kLow)) return -INFINITY;
      const float v = value_of(o);
      return has_bias ? v : score_of<kSig>(v, m, inv_sum);
    };
    float v1 = -INFINITY, v2 = -INFINITY;
    if (p.lane_shift >= 0) {
      // a power of two of lanes per group: this lane's best two, then those of its neighbours
      v1 = key_of(best[0]);
      v2 = NJ > 1 ? key_of(best[1]) : -INFINITY;
      for (int o = 1; o < p.group_lanes; o <<= 1) {
        const float x1 = __shfl_xor_sync(0xffffffffu, v1, o);
        const float x2 = __shfl_xor_sync(0xffffffffu, v2, o);
        v2 = fmaxf(fmaxf(v2, x2), fminf(v1, x1));
        v1 = fmaxf(v1, x1);
      }
      v1 = __shfl_sync(0xffffffffu, v1, (lane << p.lane_shift) & 31);
      v2 = __shfl_sync(0xffffffffu, v2, (lane << p.lane_shift) & 31);
    } else {
#pragma unroll
      for (int j = 0; j < NJ; ++j) s_key[warp][e0 + j] = key_of(ord[j]);
      __syncwarp();
      if (lane < p.groups) {
        for (int i = 0; i < p.per; ++i) {
          const float k = s_key[warp][lane * p.per + i];
          v2 = fmaxf(v2, fminf(v1, k));
          v1 = fmaxf(v1, k);
        }
      }
    }
    const bool two = p.rank > 1 && v2 > -INFINITY;
    const bool there = lane < p.groups && v1 > -INFINITY;
    const float gs = there ? (two ? v1 + v2 : v1) : -INFINITY;
    // the top_groups best sums, ties to the lower group; the last one in and the first one out
    uint32_t left = there ? float_key(gs) : 0u, last = 0u;
    live = 0u;
    for (int r = 0; r < p.top_groups; ++r) {
      last = __reduce_max_sync(0xffffffffu, left);
      if (last == 0u) break;  // the groups left have nothing available
      const uint32_t who = __ballot_sync(0xffffffffu, left == last);
      const uint32_t first = who & (~who + 1u);
      live |= first;
      left = (first >> lane) & 1u ? 0u : left;
    }
    const uint32_t out = __reduce_max_sync(0xffffffffu, left);
    if (last != 0u && out != 0u) {
      auto sum_of = [](uint32_t k) {
        return __uint_as_float((k & 0x80000000u) ? k ^ 0x80000000u : ~k);
      };
      const float lowest_in = sum_of(last), best_out = sum_of(out);
      // A sum is off by its keys' errors, a score's being largest at the largest score (1 for
      // the logistic function, inv_sum for the softmax), by two additions, and by the rounding
      // of the ordered values: of the keys, or without a bias of the logits, which moves a
      // logistic score by |l| s (1 - s) < 0.3 and a softmax score by |l| s <= |m| s + |x| s with
      // |x| s < 0.4 inv_sum.
      const float mag = warp_max(there ? fabsf(v1) + (two ? fabsf(v2) : 0.f) : 0.f);
      const float top = kSig ? 1.0f : inv_sum;
      const float unit = NJ * 0x1p-23f;
      float rounding = mag * unit;
      if (!has_bias) rounding = unit * (kSig ? 0.6f : mag * fabsf(m) + 0.8f * top);
      const float slack = 2.0f * (2.0f * err + 2.0f * kErrFloor + mag * 0x1p-22f + rounding);
      if (!(lowest_in - best_out > slack)) {
        // the groups at the border, by 64-bit sums, for the places that the clear ones leave
        const bool in = (live >> lane) & 1u;
        const bool clear_in = in && gs > best_out + slack;
        const bool contested = there && !clear_in && !(gs < lowest_in - slack);
        const uint32_t open = __ballot_sync(0xffffffffu, contested);
        const uint32_t sure = __ballot_sync(0xffffffffu, clear_in);
        const double g64 = group_sums64<NJ, TL, kSig>(p, row, m, lane, open);
        int before = 0;
        for (int h = 0; h < p.groups; ++h) {
          const double v = __shfl_sync(0xffffffffu, g64, h);
          before += ((open >> h) & 1u) && (v > g64 || (v == g64 && h < lane)) ? 1 : 0;
        }
        live = sure | __ballot_sync(0xffffffffu, contested && before < p.top_groups - __popc(sure));
      }
    }
    if (p.group_lanes > 0) {  // a lane's experts are of one group
      const int g = p.lane_shift >= 0 ? lane >> p.lane_shift : lane / p.group_lanes;
      if (!((live >> (g & 31)) & 1u)) best[0] = best[1] = best[2] = best[3] = 0u;
    } else {
      int g = e0 / p.per, r = e0 - g * p.per;
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        if (!((live >> (g & 31)) & 1u)) ord[j] = 0u;
        if (++r == p.per) {
          r = 0;
          ++g;
        }
      }
      four_best<NJ>(ord, best);
    }
  }

  // Takes the best expert still in play: its lane and ordered key (uniform over the warp), or
  // lane -1.  The register numbers do not count between lanes: among equal keys the lower lane.
  int held = 4;
  auto take_best = [&](int k, uint32_t* taken) {
    const uint32_t first = best[0] & ~kLow;
    const uint32_t top = __reduce_max_sync(0xffffffffu, first);
    if (top <= kNone) return -1;
    const int win = __ffs(__ballot_sync(0xffffffffu, first == top)) - 1;
    *taken = __shfl_sync(0xffffffffu, best[0], win);
    const bool mine = lane == win;
    best[0] = mine ? best[1] : best[0];
    best[1] = mine ? best[2] : best[1];
    best[2] = mine ? best[3] : best[2];
    best[3] = mine ? 0u : best[3];
    if constexpr (NJ > 4) {
      held -= mine ? 1 : 0;
      if (k >= 3 && __any_sync(0xffffffffu, held == 0)) {  // the lane's next four
        uint32_t left[NJ], four[4];
#pragma unroll
        for (int j = 0; j < NJ; ++j) left[j] = ord[j] < *taken ? ord[j] : 0u;
        four_best<NJ>(left, four);
        if (held == 0) {
          held = 4;
#pragma unroll
          for (int i = 0; i < 4; ++i) best[i] = four[i];
        }
      }
    }
    return win;
  };
  auto expert_of = [&](int win, uint32_t taken) {
    return win * NJ + static_cast<int>(kLow - (taken & kLow));
  };
  auto pick_of = [&](int e) {
    Pick q{-INFINITY, 0.f, 0.f};
    if (e >= 0) {
      q.l = clean_logit(to_float(row[e]));
      q.b = has_bias ? __ldg(p.bias + e) : 0.f;
      q.key = score_of<kSig>(q.l, m, inv_sum) + q.b;
    }
    return q;
  };

  // the K best and the one after them; lane k keeps the k-th
  int my_win = -1;
  uint32_t my_key = 0u;
  for (int k = 0; k <= p.K; ++k) {
    uint32_t taken;
    const int win = take_best(k, &taken);
    if (win < 0) break;
    my_win = lane == k ? win : my_win;
    my_key = lane == k ? taken : my_key;
  }
  int mine = my_win < 0 ? -1 : expert_of(my_win, my_key);

  // certify the order of neighbours
  const Pick me = pick_of(mine);
  const Pick next{__shfl_down_sync(0xffffffffu, me.l, 1), __shfl_down_sync(0xffffffffu, me.b, 1),
                  __shfl_down_sync(0xffffffffu, me.key, 1)};
  const int next_e = __shfl_down_sync(0xffffffffu, mine, 1);
  // (bf16 logits keep all their bits in the order)
  const bool by_bf16 = sizeof(TL) == 2 && !has_bias;
  const float unit = by_bf16 ? 0.f : (1 + NJ) * 0x1p-23f;
  const bool tie = me.l == next.l && me.b == next.b;  // in any precision
  const bool doubt = __any_sync(0xffffffffu, lane < p.K && next_e >= 0 && !tie &&
                                                 close<kSig>(me, next, has_bias, m, err, unit));
  bool open = lane == p.K - 1 && next_e >= 0 && tie;
  if (by_bf16)  // what follows is at least a step lower
    open = open && scores_merge<kSig>(me, Pick{me.l - 0x1p-9f * fabsf(me.l), 0.f, 0.f}, m);
  const bool border = __any_sync(0xffffffffu, open);
  if (doubt || border) {
    // what comes after the first one left out must be clear of it, or tie with it where only
    // the border is at stake
    uint32_t taken = 0u;
    const int win = take_best(p.K + 1, &taken);
    const int second = win < 0 ? -1 : expert_of(win, taken);
    const Pick q = pick_of(second);
    bool whole = __shfl_sync(
        0xffffffffu, second >= 0 && close<kSig>(me, q, has_bias, m, err, unit), p.K);
    if (whole && !doubt) {
      const Pick last{__shfl_sync(0xffffffffu, me.l, p.K), __shfl_sync(0xffffffffu, me.b, p.K),
                      __shfl_sync(0xffffffffu, me.key, p.K)};
      whole = others_close<NJ, TL, kSig>(p, row, last, m, inv_sum, lane, live, err, unit);
    }
    if (whole) {
      mine = choose64<NJ, TL, kSig>(p, row, m, lane, live);
    } else if (doubt) {
      // the logits decide unless some neighbours' scores may round together
      Pick hi = me, lo = next;
      if (me.l < next.l) hi = next, lo = me;
      const bool merge = lane < p.K && next_e >= 0 && !tie && scores_merge<kSig>(hi, lo, m);
      const bool by_logit = !has_bias && !__any_sync(0xffffffffu, merge);
      mine = order64<NJ, TL, kSig>(p, row, m, lane, mine, me.l, me.b, by_logit);
    }
  }
  if (lane >= p.K) mine = -1;

  // weights from the unbiased scores
  float kl = mine >= 0 ? me.l : -INFINITY;
  if ((doubt || border) && mine >= 0) kl = clean_logit(to_float(row[mine]));
  float s = 0.f;
  if (p.renorm) {
    const float top = warp_max(kl);
    if (mine >= 0) s = relative_score<kSig>(kl, top);
    const float total = warp_sum(s);
    s = mine >= 0 ? __fdividef(s, total) : 0.f;
  } else if (mine >= 0) {
    s = kSig ? 1.0f / (1.0f + expf(-kl)) : expf(kl - m) * inv_sum;
  }
  if (lane < p.K) {
    const size_t at = static_cast<size_t>(t) * p.K + lane;
    p.ids[at] = mine;
    p.w[at] = s * p.scale;
  }
}

// The gradient, one warp per token.  Only a softmax without renormalisation reaches every
// expert; in the other cases the gradient is zero off the K chosen experts (with
// renormalisation the softmax's own sum cancels), so K logits are gathered, the row is put
// together in shared memory and written once.  Bound by the write of T*E elements: 16384 tokens
// of 256 experts take 6.7 us, 2.7 us of them at the copy rate.
template <int NJ, typename TL, bool kSig>
__global__ void __launch_bounds__(32 * kWarps)
    route_scored_grad_kernel(const __grid_constant__ RouteParams p) {
  __shared__ __align__(16) float s_row[kWarps][NJ * 32];
  grid_dep_wait();
  grid_dep_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = blockIdx.x * kWarps + warp;
  if (t >= p.T) return;
  const TL* row = static_cast<const TL*>(p.logits) + static_cast<size_t>(t) * p.stride;
  TL* out = static_cast<TL*>(p.d_logits) + static_cast<size_t>(t) * p.stride;
  float* sr = s_row[warp];

  int id = -1;
  float dw = 0.f, kl = -INFINITY;
  if (lane < p.K) {
    const size_t at = static_cast<size_t>(t) * p.K + lane;
    id = p.ids_in[at];
    if (id < 0 || id >= p.E) id = -1;
    if (id >= 0) kl = clean_logit(to_float(row[id]));
    if (kl == -INFINITY) id = -1;
    if (id >= 0) dw = p.scale * p.d_w[at];
  }
  if (!kSig && !p.renorm) {
    const int e0 = lane * NJ;
    float l[NJ];
    load_row<NJ, TL>(row, p.E, lane, p.vec, l);
    float m = l[0];
#pragma unroll
    for (int j = 1; j < NJ; ++j) m = fmaxf(m, l[j]);
    m = warp_max(m);
    if (m == -INFINITY) m = 0.f;
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      l[j] = expf(l[j] - m);
      sum += l[j];
    }
    sum = warp_sum(sum);
    const float inv = sum > 0.f ? 1.0f / sum : 0.f;
    const float sk = id >= 0 ? expf(kl - m) * inv : 0.f;
    const float dot = warp_sum(dw * sk);
#pragma unroll
    for (int j = 0; j < NJ; ++j) sr[e0 + j] = -l[j] * inv * dot;
    __syncwarp();
    if (id >= 0) sr[id] = sk * (dw - dot);
  } else {
    float d = 0.f;
    if (p.renorm) {
      const float top = warp_max(kl);
      float s = 0.f;
      if (id >= 0) s = relative_score<kSig>(kl, top);
      const float total = warp_sum(s);
      const float rho = id >= 0 ? s / total : 0.f;
      const float dot = warp_sum(dw * rho);
      d = (dw - dot) * rho;
    } else if (id >= 0) {
      d = dw / (1.0f + expf(-kl));
    }
    if (kSig) d /= 1.0f + expf(kl);  // 1 - s
#pragma unroll
    for (int j = 0; j < NJ; ++j) sr[lane + 32 * j] = 0.f;
    __syncwarp();
    if (id >= 0) sr[id] = d;
  }
  __syncwarp();
  if (p.vec) {
    constexpr int kPer = 16 / static_cast<int>(sizeof(TL));
    for (int c = lane * kPer; c < p.E; c += 32 * kPer) {
      alignas(16) TL v[kPer];
#pragma unroll
      for (int q = 0; q < kPer; q += 4) {
        const float4 f = *reinterpret_cast<const float4*>(sr + c + q);
        v[q] = from_float<TL>(f.x);
        v[q + 1] = from_float<TL>(f.y);
        v[q + 2] = from_float<TL>(f.z);
        v[q + 3] = from_float<TL>(f.w);
      }
      *reinterpret_cast<uint4*>(out + c) = *reinterpret_cast<const uint4*>(v);
    }
  } else {
    for (int c = lane; c < p.E; c += 32) out[c] = from_float<TL>(sr[c]);
  }
}

template <int NJ, typename TL, bool kGrad>
cudaError_t launch_typed(bool sigmoid, const RouteParams& p, cudaStream_t s) {
  const dim3 grid((static_cast<unsigned>(p.T) + kWarps - 1) / kWarps), block(32 * kWarps);
  if constexpr (kGrad)
    return sigmoid ? launch_pdl(route_scored_grad_kernel<NJ, TL, true>, grid, block, 0, s, p)
                   : launch_pdl(route_scored_grad_kernel<NJ, TL, false>, grid, block, 0, s, p);
  else
    return sigmoid ? launch_pdl(route_scored_kernel<NJ, TL, true>, grid, block, 0, s, p)
                   : launch_pdl(route_scored_kernel<NJ, TL, false>, grid, block, 0, s, p);
}

template <bool kGrad>
cudaError_t launch_route(const moe_route_config_t& c, RouteParams p, cudaStream_t s) {
  const int nj = (c.E + 31) / 32;
  const int NJ = nj <= 1 ? 1 : nj <= 2 ? 2 : nj <= 4 ? 4 : nj <= 8 ? 8 : nj <= 16 ? 16 : 32;
  // whole-lane vector loads (and the gradient's 16-byte stores): rows on 16-byte boundaries,
  // no lane or vector half inside the row
  const int eb = static_cast<int>(act_bytes(c.dtype));
  const int q = kGrad && 16 / eb > NJ ? 16 / eb : NJ;
  p.vec = c.E % q == 0 && (p.stride * eb) % 16 == 0 &&
          (reinterpret_cast<uintptr_t>(p.logits) & 15u) == 0 &&
          (reinterpret_cast<uintptr_t>(p.d_logits) & 15u) == 0;
  p.group_lanes = p.per % NJ == 0 ? p.per / NJ : 0;
  p.lane_shift = -1;
  for (int i = 0; i <= 5; ++i)
    if (p.group_lanes == 1 << i) p.lane_shift = i;
  p.vec_bias = c.E % NJ == 0 && (reinterpret_cast<uintptr_t>(p.bias) & 15u) == 0;
  const bool sig = c.score == MOE_SCORE_SIGMOID;
  auto go = [&](auto nj_c) {
    constexpr int N = decltype(nj_c)::value;
    return c.dtype == MOE_BF16 ? launch_typed<N, __nv_bfloat16, kGrad>(sig, p, s)
                               : launch_typed<N, float, kGrad>(sig, p, s);
  };
  switch (NJ) {
    case 1: return go(std::integral_constant<int, 1>{});
    case 2: return go(std::integral_constant<int, 2>{});
    case 4: return go(std::integral_constant<int, 4>{});
    case 8: return go(std::integral_constant<int, 8>{});
    case 16: return go(std::integral_constant<int, 16>{});
    default: return go(std::integral_constant<int, 32>{});
  }
}

moe_status_t check_route_config(const moe_route_config_t* c) {
  if (c == nullptr) return MOE_ERR_INVALID_ARG;
  if (c->dtype != MOE_F32 && c->dtype != MOE_BF16) return MOE_ERR_INVALID_ARG;
  if (c->score != MOE_SCORE_SOFTMAX && c->score != MOE_SCORE_SIGMOID) return MOE_ERR_INVALID_ARG;
  if (c->renormalise != 0 && c->renormalise != 1) return MOE_ERR_INVALID_ARG;
  if (c->T < 0 || c->E <= 0 || c->E > 1024 || c->K <= 0 || c->K > 16) return MOE_ERR_INVALID_ARG;
  if (c->groups <= 0 || c->groups > 32 || c->E % c->groups != 0) return MOE_ERR_INVALID_ARG;
  if (c->top_groups <= 0 || c->top_groups > c->groups) return MOE_ERR_INVALID_ARG;
  if (c->group_rank != 1 && c->group_rank != 2) return MOE_ERR_INVALID_ARG;
  if (c->K > c->top_groups * (c->E / c->groups)) return MOE_ERR_INVALID_ARG;
  if (!(c->scale > 0.0f && c->scale <= FLT_MAX)) return MOE_ERR_INVALID_ARG;
  if (c->logits_stride != 0 && (c->logits_stride < c->E || c->logits_stride > (1ll << 31)))
    return MOE_ERR_INVALID_ARG;
  if (static_cast<long long>(c->T) * c->K >= (1ll << 31)) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

inline bool unaligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }

RouteParams base_params(const moe_route_config_t* c, const void* logits) {
  RouteParams p{};
  p.logits = logits;
  p.stride = c->logits_stride != 0 ? c->logits_stride : c->E;
  p.T = c->T;
  p.E = c->E;
  p.K = c->K;
  p.groups = c->groups;
  p.per = c->E / c->groups;
  p.top_groups = c->top_groups;
  p.rank = c->group_rank;
  p.renorm = c->renormalise;
  p.scale = c->scale;
  return p;
}

}  // namespace
}  // namespace moe

extern "C" moe_status_t moe_route_scored(const moe_route_config_t* cfg, const void* logits,
                                         const float* expert_bias, int32_t* topk_ids,
                                         float* topk_w, moe_stream_t stream) {
  using namespace moe;
  moe_status_t st = fault_point("moe_route_scored");
  if (st != MOE_OK) return st;
  st = check_route_config(cfg);
  if (st != MOE_OK) return st;
  if (cfg->T == 0) return MOE_OK;
  if (logits == nullptr || topk_ids == nullptr || topk_w == nullptr) return MOE_ERR_INVALID_ARG;
  if (unaligned(logits, act_bytes(cfg->dtype)) || unaligned(expert_bias, 4) ||
      unaligned(topk_ids, 4) || unaligned(topk_w, 4))
    return MOE_ERR_MISALIGNED;
  st = check_current_device();
  if (st != MOE_OK) return st;
  RouteParams p = base_params(cfg, logits);
  p.bias = expert_bias;
  p.ids = topk_ids;
  p.w = topk_w;
  const cudaError_t e = launch_route<false>(*cfg, p, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

extern "C" moe_status_t moe_route_scored_backward(const moe_route_config_t* cfg,
                                                  const void* logits, const int32_t* topk_ids,
                                                  const float* d_topk_w, void* d_logits,
                                                  moe_stream_t stream) {
  using namespace moe;
  moe_status_t st = fault_point("moe_route_scored_backward");
  if (st != MOE_OK) return st;
  st = check_route_config(cfg);
  if (st != MOE_OK) return st;
  if (cfg->T == 0) return MOE_OK;
  if (logits == nullptr || topk_ids == nullptr || d_topk_w == nullptr || d_logits == nullptr)
    return MOE_ERR_INVALID_ARG;
  if (unaligned(logits, act_bytes(cfg->dtype)) || unaligned(topk_ids, 4) ||
      unaligned(d_topk_w, 4) || unaligned(d_logits, act_bytes(cfg->dtype)))
    return MOE_ERR_MISALIGNED;
  st = check_current_device();
  if (st != MOE_OK) return st;
  RouteParams p = base_params(cfg, logits);
  p.ids_in = topk_ids;
  p.d_w = d_topk_w;
  p.d_logits = d_logits;
  const cudaError_t e = launch_route<true>(*cfg, p, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
