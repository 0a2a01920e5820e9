// fs_route.cuh -- routing tokens to experts: softmax or sigmoid scores of a row of logits, a
// bias that only the choice sees, the choice within the best groups of experts, the top k,
// and their weights; the weights' gradient for the logits.
//
// With s_j = softmax(z)_j or 1 / (1 + e^(-z_j)) and c_j = s_j + b_j: the kept groups are the
// top_groups with the largest sums of their two largest c; the choice is the k largest c in
// them, equal c by the lower index; w_a = scale s_a / sum_b s_b (renormalised) or scale s_a.
//
// Which experts are picked is decided at borders, and a border that two implementations
// round differently sends a token elsewhere. So the choice is the one of c in 64 bits: the
// fast path works in fp32 with a bound on its error, and a row in which two neighbours of
// the order (the last pick and the first that is left included) lie within their bounds is
// done over in 64 bits by the same warp. Experts of equal logit and bias are equal in any
// precision and need no second look. About one row in 500 is done over on normal logits of
// 256 experts.
//
// One warp takes a row: lane l holds experts l, l + 32, ... as whole-number keys that order
// like c, and each pick is two warp reductions (the largest key, the lowest index holding
// it).
#pragma once

#include "fs_rowload.cuh"

namespace fs {

constexpr int kRouteWarps = 8;
constexpr int kRouteMaxExperts = 1024;
constexpr int kRouteMaxK = 31;       // lane k holds the first expert left out
constexpr int kRouteMaxGroups = 32;  // one bit each in a mask

enum RouteScore : int { kScoreSoftmax = 0, kScoreSigmoid = 1 };

struct RouteParams {
  const void* z;
  int64_t ld;
  int64_t rows;
  int32_t experts;
  int32_t k;
  int32_t groups, per_group, top_groups;
  int32_t score;
  int32_t renorm;
  float scale;
  const float* bias;
  float* weights;
  int32_t* ids;
  int32_t* load;  // zeroed before the launch, or NULL
};

__device__ __forceinline__ float warp_maxf(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ float warp_sumf(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Score of one logit in fp32; m and inv are the row's maximum and 1 / sum (softmax).
__device__ __forceinline__ float route_score(float z, int kind, float m, float inv) {
  return kind == kScoreSigmoid ? __fdividef(1.0f, 1.0f + ex2(-z * kLog2e)) : ex2((z - m) * kLog2e) * inv;
}
__device__ __forceinline__ double route_score64(double z, int kind, double m, double sum) {
  return kind == kScoreSigmoid ? 1.0 / (1.0 + exp(-z)) : exp(z - m) / sum;
}

// Bound on the error of c = s + b in fp32. exp's argument x carries 2^-24 |x| twice (the
// difference or product, and its rounding), ex2 2^-22, the sum and the quotient a few 2^-24;
// s inherits them as relative errors, c one more rounding, and a score below 2^-126 is
// flushed. Doubled against what was left out.
__device__ __forceinline__ float route_err(float z, float s, float c, int kind, float m) {
  const float x = kind == kScoreSigmoid ? fabsf(z) : m - z;
  return s * (x + 8.0f) * 0x1p-21f + fabsf(c) * 0x1p-23f + 0x1p-124f;
}

// A row whose maximum or sum shows NaN (a NaN logit or bias, +inf under softmax) has no
// order: ids -1 and weights NaN.
__device__ __forceinline__ void route_write(const RouteParams& P, int64_t row, int lane, int id,
                                            float w) {
  if (lane < P.k) {
    P.ids[row * P.k + lane] = id;
    P.weights[row * P.k + lane] = w;
  }
}

// The row in 64 bits, with c in shared memory. Called by a whole warp.
template <typename T>
__device__ __noinline__ void route_row64(const RouteParams& P, const T* z, int64_t row,
                                         double* c, int* hist, int lane) {
  const double inf = __longlong_as_double(0x7FF0000000000000ll);
  const int E = P.experts;
  double m = 0.0, sum = 1.0;
  if (P.score == kScoreSoftmax) {
    m = -inf;
    for (int j = lane; j < E; j += 32) m = fmax(m, static_cast<double>(Elem<T>::to_f(z[j])));
    m = warp_max(m);
    sum = 0.0;
    for (int j = lane; j < E; j += 32) sum += exp(static_cast<double>(Elem<T>::to_f(z[j])) - m);
    sum = warp_sum(sum);
  }
  for (int j = lane; j < E; j += 32) {
    const float zj = Elem<T>::to_f(z[j]);
    c[j] = zj == -INFINITY ? -inf
                           : route_score64(zj, P.score, m, sum) +
                                 (P.bias ? static_cast<double>(P.bias[j]) : 0.0);
  }
  __syncwarp();
  if (P.groups > 1) {
    double gs = -inf;
    if (lane < P.groups) {
      double a = -inf, b = -inf;
      for (int j = 0; j < P.per_group; ++j) {
        const double v = c[lane * P.per_group + j];
        if (v > a) {
          b = a;
          a = v;
        } else {
          b = fmax(b, v);
        }
      }
      gs = b == -inf ? a : a + b;
    }
    int ahead = 0;
    for (int g = 0; g < P.groups; ++g) {
      const double o = __shfl_sync(0xffffffffu, gs, g);
      ahead += o > gs || (o == gs && g < lane);
    }
    if (lane < P.groups && ahead >= P.top_groups)
      for (int j = 0; j < P.per_group; ++j) c[lane * P.per_group + j] = -inf;
    __syncwarp();
  }
  int mine = -1;
  for (int r = 0; r < P.k; ++r) {
    double best = -inf;
    int at = 0x7FFFFFFF;
    for (int j = lane; j < E; j += 32)
      if (c[j] > best) {  // ascending j: the lowest index of equal values stays
        best = c[j];
        at = j;
      }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const double ov = __shfl_xor_sync(0xffffffffu, best, o);
      const int oi = __shfl_xor_sync(0xffffffffu, at, o);
      if (ov > best || (ov == best && oi < at)) {
        best = ov;
        at = oi;
      }
    }
    if (at == 0x7FFFFFFF) break;
    if (lane == r) mine = at;
    if (lane == 0) c[at] = -inf;
    __syncwarp();
  }
  double s = 0.0;
  if (lane < P.k && mine >= 0) s = route_score64(Elem<T>::to_f(z[mine]), P.score, m, sum);
  const double tot = P.renorm ? warp_sum(s) : 1.0;
  if (hist && lane < P.k && mine >= 0) atomicAdd(&hist[mine], 1);
  route_write(P, row, lane, mine, tot > 0.0 ? static_cast<float>(P.scale * (s / tot)) : 0.0f);
}

// NL: experts per lane. Dynamic shared memory: experts doubles per warp, then the CTA's load.
template <typename T, int NL>
__global__ void __launch_bounds__(kRouteWarps * 32) route_kernel(const RouteParams P) {
  extern __shared__ __align__(16) unsigned char route_smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int E = P.experts;
  double* c64 = reinterpret_cast<double*>(route_smem) + warp * E;
  float* c32 = reinterpret_cast<float*>(c64);
  int* hist = nullptr;
  if (P.load) {
    hist = reinterpret_cast<int*>(reinterpret_cast<double*>(route_smem) + kRouteWarps * E);
    for (int j = threadIdx.x; j < E; j += blockDim.x) hist[j] = 0;
    __syncthreads();
  }
  const bool sig = P.score == kScoreSigmoid;
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * kRouteWarps + warp; row < P.rows;
       row += static_cast<int64_t>(gridDim.x) * kRouteWarps) {
    const T* z = static_cast<const T*>(P.z) + row * P.ld;
    float v[NL];
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const int j = lane + 32 * i;
      v[i] = j < E ? Elem<T>::to_f(z[j]) : -INFINITY;
    }
    float m = 0.0f, inv = 1.0f;
    if (!sig) {
      m = v[0];
#pragma unroll
      for (int i = 1; i < NL; ++i) m = fmaxf(m, v[i]);
      m = warp_maxf(m);
      float sum = 0.0f;
      const float mm = m == -INFINITY ? 0.0f : m;
#pragma unroll
      for (int i = 0; i < NL; ++i) sum += ex2((v[i] - mm) * kLog2e);
      inv = 1.0f / warp_sumf(sum);
    }
    uint32_t key[NL];
    bool bad = false;
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const int j = lane + 32 * i;
      float c = route_score(v[i], P.score, m, inv);
      if (P.bias && j < E) c += P.bias[j];
      // closed: a logit or a bias of -inf
      const bool open = v[i] != -INFINITY && c != -INFINITY;
      bad |= open && c != c;
      key[i] = open ? order_key(c) : 0u;
    }
    if (__any_sync(0xffffffffu, bad)) {
      route_write(P, row, lane, -1, __int_as_float(0x7FC00000));
      continue;
    }
    bool again = false;  // a border too close for fp32
    if (P.groups > 1) {
#pragma unroll
      for (int i = 0; i < NL; ++i)
        if (lane + 32 * i < E) c32[lane + 32 * i] = key[i] ? order_unkey(key[i]) : -INFINITY;
      __syncwarp();
      // the two largest of each group: `lanes` neighbouring lanes scan one group
      int lanes = 32;
      while (lanes * P.groups > 32) lanes >>= 1;
      const int g = lane / lanes;
      float a = -INFINITY, b = -INFINITY;
      if (g < P.groups)
        for (int j = lane % lanes; j < P.per_group; j += lanes) {
          const float x = c32[g * P.per_group + j];
          b = fmaxf(b, fminf(a, x));
          a = fmaxf(a, x);
        }
      for (int o = 1; o < lanes; o <<= 1) {
        const float oa = __shfl_xor_sync(0xffffffffu, a, o);
        const float ob = __shfl_xor_sync(0xffffffffu, b, o);
        b = fmaxf(fmaxf(b, ob), fminf(a, oa));
        a = fmaxf(a, oa);
      }
      const float gs = g >= P.groups || a == -INFINITY ? -INFINITY : (b == -INFINITY ? a : a + b);
      int ahead = 0;
      for (int q = 0; q < P.groups; ++q) {
        const float o = __shfl_sync(0xffffffffu, gs, q * lanes);
        ahead += o > gs || (o == gs && q < g);
      }
      const bool kept = g < P.groups && ahead < P.top_groups;
      // the border between kept and dropped groups; each score is off by at most 20 * 2^-21
      const float lo = -warp_maxf(kept ? -gs : -INFINITY);
      const float hi = warp_maxf(g < P.groups && !kept ? gs : -INFINITY);
      again = hi != -INFINITY &&
              !(lo - hi > 80.0f * 0x1p-21f + (fabsf(lo) + fabsf(hi)) * 0x1p-22f);
      if (g < P.groups && !kept)
        for (int j = lane % lanes; j < P.per_group; j += lanes) c32[g * P.per_group + j] = -INFINITY;
      __syncwarp();
#pragma unroll
      for (int i = 0; i < NL; ++i)
        if (lane + 32 * i < E && c32[lane + 32 * i] == -INFINITY) key[i] = 0u;
      __syncwarp();
    }
    // k picks and the first expert left out
    uint32_t lk = key[0];
    int li = lane;
#pragma unroll
    for (int i = 1; i < NL; ++i)
      if (key[i] > lk) {
        lk = key[i];
        li = lane + 32 * i;
      }
    int mine = -1;
    uint32_t mine_key = 0u;
    for (int r = 0; r <= P.k; ++r) {
      const uint32_t top = __reduce_max_sync(0xffffffffu, lk);
      if (top == 0u) break;
      const int at = static_cast<int>(
          __reduce_min_sync(0xffffffffu, lk == top ? static_cast<unsigned>(li) : 0x7FFFFFFFu));
      if (lane == r) {
        mine = at;
        mine_key = top;
      }
      if ((at & 31) == lane) {
#pragma unroll
        for (int i = 0; i < NL; ++i)
          if (lane + 32 * i == at) key[i] = 0u;
        lk = key[0];
        li = lane;
#pragma unroll
        for (int i = 1; i < NL; ++i)
          if (key[i] > lk) {
            lk = key[i];
            li = lane + 32 * i;
          }
      }
    }
    float zr = 0.0f, s = 0.0f, br = 0.0f, c = 0.0f, err = 0.0f;
    if (mine >= 0) {
      zr = Elem<T>::to_f(z[mine]);
      s = route_score(zr, P.score, m, inv);
      br = P.bias ? P.bias[mine] : 0.0f;
      c = order_unkey(mine_key);
      err = route_err(zr, s, c, P.score, m);
    }
    const int nmine = __shfl_down_sync(0xffffffffu, mine, 1);
    const float nz = __shfl_down_sync(0xffffffffu, zr, 1);
    const float nb = __shfl_down_sync(0xffffffffu, br, 1);
    const float nc = __shfl_down_sync(0xffffffffu, c, 1);
    const float ne = __shfl_down_sync(0xffffffffu, err, 1);
    again |= lane < P.k && mine >= 0 && nmine >= 0 && !(c - nc > err + ne) &&
             !(zr == nz && br == nb);
    // a score that fp32 flushes also loses its weight
    again |= lane < P.k && mine >= 0 && s < 0x1p-100f;
    if (__any_sync(0xffffffffu, again)) {
      route_row64(P, z, row, c64, hist, lane);
      __syncwarp();
      continue;
    }
    if (lane >= P.k) {
      mine = -1;
      s = 0.0f;
    }
    const float tot = P.renorm ? warp_sumf(s) : 1.0f;
    if (hist && mine >= 0) atomicAdd(&hist[mine], 1);
    route_write(P, row, lane, mine, tot > 0.0f ? P.scale * (s / tot) : 0.0f);
  }
  if (P.load) {
    // whole numbers: the order of the atomics changes nothing
    __syncthreads();
    for (int j = threadIdx.x; j < E; j += blockDim.x)
      if (hist[j]) atomicAdd(&P.load[j], hist[j]);
  }
}

// ---- gradient -------------------------------------------------------------------------------
//
// With r_a = w_a / scale and G = sum_a gw_a r_a (renormalised), the gradient is nonzero at the
// picked experts only, except for softmax weights taken as they are:
//   softmax, renormalised:  dz_a = scale r_a (gw_a - G)            (from w alone)
//   sigmoid, renormalised:  dz_a = scale r_a (gw_a - G) (1 - s_a)
//   sigmoid as it is:       dz_a = scale gw_a s_a (1 - s_a)
//   softmax as it is:       dz_j = scale s_j (gw_j [j picked] - sum_a gw_a s_a)
struct RouteGradParams {
  const void* z;
  int64_t ld;
  int64_t rows;
  int32_t experts;
  int32_t k;
  int32_t score;
  int32_t renorm;
  float scale;
  const float* weights;
  const int32_t* ids;
  const float* g_weights;
  void* grad;  // (rows, experts), contiguous
};

// One warp per row: the row's zeros (or the dense part) in coalesced stores, then lane a
// rewrites its picked expert.
template <typename T, int NL>
__global__ void __launch_bounds__(kRouteWarps * 32) route_grad_kernel(const RouteGradParams P) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int E = P.experts;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kRouteWarps + warp;
  if (row >= P.rows) return;
  const T* z = static_cast<const T*>(P.z) + row * P.ld;
  T* out = static_cast<T*>(P.grad) + row * E;
  int id = -1;
  float gw = 0.0f, w = 0.0f;
  if (lane < P.k) {
    id = P.ids[row * P.k + lane];
    if (id >= E) id = -1;
    gw = P.g_weights[row * P.k + lane];
    w = P.weights[row * P.k + lane];
  }
  const bool nan = __any_sync(0xffffffffu, w != w);  // a row without an order
  float r = id >= 0 && P.scale != 0.0f ? w / P.scale : 0.0f;
  if (id < 0) gw = 0.0f;
  const float G = warp_sumf(gw * r);
  float d = 0.0f;
  const bool dense = P.score == kScoreSoftmax && !P.renorm;
  if (nan) {
    for (int j = lane; j < E; j += 32) out[j] = Elem<T>::from_f(__int_as_float(0x7FC00000));
    return;
  }
  if (dense) {
    float v[NL];
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const int j = lane + 32 * i;
      v[i] = j < E ? Elem<T>::to_f(z[j]) : -INFINITY;
    }
    float m = v[0];
#pragma unroll
    for (int i = 1; i < NL; ++i) m = fmaxf(m, v[i]);
    m = warp_maxf(m);
    const float mm = m == -INFINITY ? 0.0f : m;
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      v[i] = ex2((v[i] - mm) * kLog2e);
      sum += v[i];
    }
    sum = warp_sumf(sum);
    const float f = sum > 0.0f ? -P.scale * G / sum : 0.0f;
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const int j = lane + 32 * i;
      if (j < E) out[j] = Elem<T>::from_f(v[i] * f);
    }
    d = P.scale * r * (gw - G);
  } else {
    constexpr int V = Elem<T>::kVec;
    if ((E % V) == 0 && (reinterpret_cast<uintptr_t>(out) & 15u) == 0) {
      for (int j = lane * V; j < E; j += 32 * V)
        *reinterpret_cast<uint4*>(out + j) = make_uint4(0u, 0u, 0u, 0u);
    } else {
      for (int j = lane; j < E; j += 32) out[j] = Elem<T>::from_f(0.0f);
    }
    if (id >= 0) {
      if (P.score == kScoreSoftmax) {
        d = P.scale * r * (gw - G);
      } else {
        // 1 - s = 1 / (1 + e^z) keeps its digits where s is near 1
        const float zi = Elem<T>::to_f(z[id]);
        const float rest = 1.0f / (1.0f + ex2(zi * kLog2e));
        d = P.renorm ? P.scale * r * (gw - G) * rest : P.scale * gw * r * rest;
      }
    }
  }
  __syncwarp();  // orders the zeros before the picked experts' values
  if (id >= 0) out[id] = Elem<T>::from_f(d);
}

}  // namespace fs
