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
// fast path works in fp32 with a bound on its error, and a row in which two neighbours among the
// picks, or the last pick and any expert that is left, lie within their bounds is done over in 64
// bits by the same warp. (Any: bounds differ, and an expert behind the first one left, with a
// larger bound or behind a tie, may be the better one.) Experts of equal logit and bias are equal
// in any precision and need no second look. About one row in 1000 is done over on normal logits
// of 256 experts.
//
// One warp takes a row, each lane a few neighbouring experts. What bounds it is instructions: 895
// a row at 256 experts, 8 of them picked out of 4 of 8 groups (32768 rows: 50 us, the read of the
// logits alone 5), 513 at 64 experts (80 and 53 of them compare what is left with the last pick).
#pragma once

#include <cfloat>

#include "fs_rowload.cuh"

namespace fs {

constexpr int kRouteWarps = 8;
constexpr int kRouteMaxExperts = 1024;
constexpr int kRouteMaxK = 31;       // lane k holds the first expert left out
constexpr int kRouteMaxGroups = 32;  // one bit each in a mask

// Doubles of a warp's scratch: one per expert, at least 32 candidates of 16 bytes, and whole
// 16-byte units, so that every warp's candidates are aligned.
__host__ __device__ constexpr int route_room(int experts) {
  return experts < 64 ? 64 : (experts + 1) / 2 * 2;
}

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
// Score of one logit in fp32; m and inv are the row's maximum and 1 / sum (softmax).
__device__ __forceinline__ float route_score(float z, int kind, float m, float inv) {
  return kind == kScoreSigmoid ? __fdividef(1.0f, 1.0f + ex2(-z * kLog2e)) : ex2((z - m) * kLog2e) * inv;
}
__device__ __forceinline__ double route_score64(double z, int kind, double m, double sum) {
  return kind == kScoreSigmoid ? 1.0 / (1.0 + exp(-z)) : exp(z - m) / sum;
}

// Bounds on the error of c = s + b in fp32, u = 2^-24.
// Sigmoid: e = ex2(-z log2 e) is off by 2 |z| u (product, constant) + 4 u (ex2); s = 1 / (1 + e)
// takes (1 - s) of that, u for the sum and 4 u for the quotient: s ((1 - s) (2 |z| + 4) u + 5 u).
// Softmax, d = m - z: e is off by 3 d u + 4 u, the sum by the e-weighted mean of the same, at
// most 3 ln(1024) u + 4 u, and 12 u of additions, inverse and product by 4 u:
// s (3 d + 45) u. c rounds once more, |c| u; scores below 2^-126 are flushed. All times 1.5.
__device__ __forceinline__ float route_err(float z, float s, float c, bool sig, float m) {
  constexpr float u = 1.5f * 0x1p-24f;
  const float e = sig ? s * ((1.0f - s) * (2.0f * fabsf(z) + 4.0f) + 5.0f) : s * (3.0f * (m - z) + 45.0f);
  return e * u + fabsf(c) * u + 0x1p-124f;
}
// The same for every expert whose c is not above this one's. c + |c| u grows with c. Without a
// bias s is not above this one's either, and the bounds grow with s: softmax's for all s <= inv,
// sigmoid's s (2 |z| + 9) for z <= 0; none is above 6.5 for sigmoid, 48 inv for softmax.
__device__ __forceinline__ float route_left_err(float z, float s, float c, bool sig, float m,
                                                float inv, bool biased) {
  constexpr float u = 1.5f * 0x1p-24f;
  const float e = sig ? (biased || z > 0.0f ? 6.5f : s * (2.0f * fabsf(z) + 9.0f))
                      : (biased ? 48.0f * inv : s * (3.0f * (m - z) + 45.0f));
  return e * u + fabsf(c) * u + 0x1p-124f;
}
// The same for the sum of a group's two best, a and b (or a alone, b = -inf), whichever they are:
// s (1 - s) (2 |z| + 4) <= 1.5 for sigmoid; s <= inv, the largest score, and s d <= inv for softmax.
// Each has been rounded at its own size, and the sum at its.
__device__ __forceinline__ float route_group_err(float a, float b, float sum, bool sig, float inv) {
  constexpr float u = 1.5f * 0x1p-24f;
  const float terms = fabsf(a) + (b == -INFINITY ? 0.0f : fabsf(b));
  return (2.0f * (sig ? 6.5f : 48.0f * inv) + terms + fabsf(sum) + 4.0f) * u;
}

__device__ __forceinline__ float redux_max(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
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

// The k + 1 best c of the warp in order, the r-th in lane r (-inf stands for a closed expert;
// lane l holds experts l * NL + i; c is used up). Pick by pick: the largest c by one warp
// reduction, the lowest lane and in it the lowest index that holds it.
template <int NL>
__device__ __forceinline__ void route_pick_each(float* c, int k, int lane, int& mine,
                                                float& mine_c) {
  float lc = c[0];
  int li = 0;
#pragma unroll
  for (int i = 1; i < NL; ++i)
    if (c[i] > lc) {
      lc = c[i];
      li = i;
    }
  for (int r = 0; r <= k; ++r) {
    const float top = redux_max(lc);
    if (top == -INFINITY) break;
    const int src = __ffs(__ballot_sync(0xffffffffu, lc == top)) - 1;
    const int at = __shfl_sync(0xffffffffu, lane * NL + li, src);
    if (lane == r) {
      mine = at;
      mine_c = top;
    }
    if (lane == src) {
#pragma unroll
      for (int i = 0; i < NL; ++i)
        if (i == li) c[i] = -INFINITY;
      lc = c[0];
      li = 0;
#pragma unroll
      for (int i = 1; i < NL; ++i)
        if (c[i] > lc) {
          lc = c[i];
          li = i;
        }
    }
  }
}

// The same by way of candidates, for few picks of many experts: the (k + 1)-th largest value
// among the lanes' maxima is a bar that at least k + 1 scores reach and about
// -32 ln(1 - (k + 1) / 32) do (10 for k = 8). They are set aside, each lane takes one and counts
// those ahead of it. False (nothing picked) where more than 32 reach the bar.
template <int NL>
__device__ __forceinline__ bool route_pick_few(const float* c, const float* z, int k, int lane,
                                               float4* buffer, int& mine, float& mine_c,
                                               float& mine_z) {
  float lc = c[0];
#pragma unroll
  for (int i = 1; i < NL; ++i) lc = fmaxf(lc, c[i]);
  float bar = -INFINITY;
  for (int r = 0; r <= k; ++r) {
    bar = redux_max(lc);  // (equal maxima count once: the bar only gets lower)
    if (lc == bar) lc = -INFINITY;
  }
  // fewer lanes than that have an open expert: every open one counts
  if (bar == -INFINITY) bar = -FLT_MAX;
  int count = 0;
#pragma unroll
  for (int i = 0; i < NL; ++i) count += c[i] >= bar;
  int before = count;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int q = __shfl_up_sync(0xffffffffu, before, o);
    if (lane >= o) before += q;
  }
  const int total = __shfl_sync(0xffffffffu, before, 31);
  if (total > 32) return false;
  if (count) {
    int at = before - count;
#pragma unroll
    for (int i = 0; i < NL; ++i)
      if (c[i] >= bar) buffer[at++] = make_float4(c[i], __int_as_float(lane * NL + i), z[i], 0.0f);
  }
  __syncwarp();
  const float4 my = buffer[lane];
  int ahead = 0;
#pragma unroll 4
  for (int t = 0; t < total; ++t) {
    // (set aside by ascending expert: of equal scores the earlier ones are ahead)
    const float o = buffer[t].x;
    ahead += o > my.x || (o == my.x && t < lane);
  }
  __syncwarp();
  if (lane < total) buffer[ahead] = my;
  __syncwarp();
  if (lane <= k && lane < total) {
    const float4 o = buffer[lane];
    mine = __float_as_int(o.y);
    mine_c = o.x;
    mine_z = o.z;
  }
  __syncwarp();
  return true;
}

// Picks of at most this many go by way of candidates where a lane holds several experts: at 256
// experts 8 picks take 34 us that way and 42 one by one, 12 take 39 and 54; beyond, too many
// experts reach the bar (32768 rows; 1 or 2 picks take nearly the same time either way).
constexpr int kRouteFew = 12;

// NL: experts per lane, lane l holding l * NL .. + NL - 1. Dynamic shared memory: route_room
// doubles per warp, then the CTA's load.
template <typename T, int NL, bool SIG>
__global__ void __launch_bounds__(kRouteWarps * 32, NL <= 8 ? 5 : 1) route_kernel(const __grid_constant__ RouteParams P) {
  extern __shared__ __align__(16) unsigned char route_smem[];
  constexpr int kind = SIG ? kScoreSigmoid : kScoreSoftmax;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int E = P.experts;
  const int room = route_room(E);
  double* c64 = reinterpret_cast<double*>(route_smem) + warp * room;
  float* c32 = reinterpret_cast<float*>(c64);
  int* hist = nullptr;
  if (P.load) {
    hist = reinterpret_cast<int*>(reinterpret_cast<double*>(route_smem) + kRouteWarps * room);
    for (int j = threadIdx.x; j < E; j += blockDim.x) hist[j] = 0;
    __syncthreads();
  }
  const int j0 = lane * NL;
  // whole lanes of a power of two of them make up a group: its two best meet by shuffles
  const int group_lanes = P.per_group / NL;
  const bool by_lanes = P.per_group % NL == 0 && (group_lanes & (group_lanes - 1)) == 0;
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * kRouteWarps + warp; row < P.rows;
       row += static_cast<int64_t>(gridDim.x) * kRouteWarps) {
    const T* z = static_cast<const T*>(P.z) + row * P.ld;
    float v[NL];
    constexpr int V = Elem<T>::kVec;
    if (NL % V == 0 && E == 32 * NL && (reinterpret_cast<uintptr_t>(z) & 15u) == 0) {
#pragma unroll
      for (int i = 0; i < NL / V; ++i)
        Elem<T>::unpack(ld_stream(z + j0 + i * V), v + i * V);
    } else {
#pragma unroll
      for (int i = 0; i < NL; ++i) v[i] = j0 + i < E ? Elem<T>::to_f(z[j0 + i]) : -INFINITY;
    }
    float m = 0.0f, inv = 1.0f;
    if (!SIG) {
      m = v[0];
#pragma unroll
      for (int i = 1; i < NL; ++i) m = fmaxf(m, v[i]);
      m = redux_max(m);
      float sum = 0.0f;
      const float mm = m == -INFINITY ? 0.0f : m;
#pragma unroll
      for (int i = 0; i < NL; ++i) sum += ex2((v[i] - mm) * kLog2e);
      inv = 1.0f / warp_sumf(sum);
    }
    float c[NL];
    bool bad = false;
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      c[i] = route_score(v[i], kind, m, inv);
      if (P.bias && j0 + i < E) c[i] += P.bias[j0 + i];
      if (v[i] == -INFINITY) c[i] = -INFINITY;  // closed
      bad |= c[i] != c[i];
    }
    if (__any_sync(0xffffffffu, bad)) {
      route_write(P, row, lane, -1, __int_as_float(0x7FC00000));
      continue;
    }
    bool again = false;  // a border too close for fp32
    if (P.groups > 1) {
      float a = -INFINITY, b = -INFINITY;
      int g, lanes;  // this lane's group, and how many lanes share it
      if (by_lanes) {
        g = lane / group_lanes;
        lanes = group_lanes;
#pragma unroll
        for (int i = 0; i < NL; ++i) {
          b = fmaxf(b, fminf(a, c[i]));
          a = fmaxf(a, c[i]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < NL; ++i)
          if (j0 + i < E) c32[j0 + i] = c[i];
        __syncwarp();
        lanes = 32;
        while (lanes * P.groups > 32) lanes >>= 1;
        g = lane / lanes;
        if (g < P.groups)
          for (int j = lane % lanes; j < P.per_group; j += lanes) {
            const float x = c32[g * P.per_group + j];
            b = fmaxf(b, fminf(a, x));
            a = fmaxf(a, x);
          }
      }
      for (int o = 1; o < lanes; o <<= 1) {
        const float oa = __shfl_xor_sync(0xffffffffu, a, o);
        const float ob = __shfl_xor_sync(0xffffffffu, b, o);
        b = fmaxf(fmaxf(b, ob), fminf(a, oa));
        a = fmaxf(a, oa);
      }
      const float gs = g >= P.groups ? -INFINITY : (b == -INFINITY ? a : a + b);
      // kept: the groups down to the top_groups-th largest sum; where equal sums make it more,
      // or one that is kept and one that is not are within their bounds, 64 bits decide
      float left = gs, lo = -INFINITY;
      for (int r = 0; r < P.top_groups; ++r) {
        const float t = redux_max(left);
        if (t != -INFINITY) lo = t;
        if (left == t) left = -INFINITY;
      }
      const bool kept = gs >= lo && gs != -INFINITY;
      const bool open = gs != -INFINITY;
      const float ge = open ? route_group_err(a, b, gs, SIG, inv) : 0.0f;
      const float hi = redux_max(open && !kept ? gs + ge : -INFINITY);
      const float least = -redux_max(kept ? ge - gs : -INFINITY);
      again = (hi != -INFINITY && !(least > hi)) ||
              __popc(__ballot_sync(0xffffffffu, kept && lane % lanes == 0)) > P.top_groups;
      if (by_lanes) {
        if (!kept) {
#pragma unroll
          for (int i = 0; i < NL; ++i) c[i] = -INFINITY;
        }
      } else {
        if (g < P.groups && !kept)
          for (int j = lane % lanes; j < P.per_group; j += lanes)
            c32[g * P.per_group + j] = -INFINITY;
        __syncwarp();
#pragma unroll
        for (int i = 0; i < NL; ++i)
          if (j0 + i < E) c[i] = c32[j0 + i];
        __syncwarp();
      }
    }
    int mine = -1;
    float cr = -INFINITY;
    float zr = 0.0f, s = 0.0f, br = 0.0f, err = 0.0f;
    // what c still holds of the order: everything, or what is behind the first expert left out
    const bool few = NL > 1 && P.k <= kRouteFew &&
                     route_pick_few<NL>(c, v, P.k, lane, reinterpret_cast<float4*>(c64), mine, cr, zr);
    if (!few) {
      route_pick_each<NL>(c, P.k, lane, mine, cr);
      if (mine >= 0) zr = Elem<T>::to_f(z[mine]);
    }
    if (mine >= 0) {
      s = route_score(zr, kind, m, inv);
      br = P.bias ? P.bias[mine] : 0.0f;
      err = route_err(zr, s, cr, SIG, m);
    }
    const float nz = __shfl_down_sync(0xffffffffu, zr, 1);
    const float nb = __shfl_down_sync(0xffffffffu, br, 1);
    const float nc = __shfl_down_sync(0xffffffffu, cr, 1);
    const float ne = __shfl_down_sync(0xffffffffu, err, 1);
    if (lane < P.k && mine >= 0) {
      again |= lane < P.k - 1 && nc != -INFINITY && !(cr - nc > err + ne) && !(zr == nz && br == nb);
      // a score that fp32 flushes also loses its weight
      again |= s < 0x1p-100f;
    }
    // experts that are left, with c so near the last pick's that they may belong before it
    const float near = __shfl_sync(
        0xffffffffu,
        mine >= 0 ? cr - err - route_left_err(zr, s, cr, SIG, m, inv, P.bias != nullptr) : INFINITY,
        P.k - 1);
    int found = !few && lane == P.k && mine >= 0 && cr >= near ? 1 : 0;
#pragma unroll
    for (int i = 0; i < NL; ++i) found += c[i] >= near ? 1 : 0;
    again |= near != near;
    if (__reduce_add_sync(0xffffffffu, found) > (few ? P.k : 0)) {
      // all but those that equal it in any precision
      const float lz = __shfl_sync(0xffffffffu, zr, P.k - 1);
      const float lb = __shfl_sync(0xffffffffu, br, P.k - 1);
      const float lc = __shfl_sync(0xffffffffu, cr, P.k - 1);
      again |= !few && lane == P.k && mine >= 0 && cr >= near && !(zr == lz && br == lb);
#pragma unroll
      for (int i = 0; i < NL; ++i)
        if (c[i] >= near && c[i] <= lc)
          again |= !(v[i] == lz && (!P.bias || (j0 + i < E && P.bias[j0 + i] == lb)));
    }
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
    route_write(P, row, lane, mine, tot > 0.0f ? P.scale * __fdividef(s, tot) : 0.0f);
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
