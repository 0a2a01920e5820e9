// fs_tokens.cuh -- log probabilities of given tokens from a matrix of scores, with each
// row's entropy and its best alternatives, and the gradient of all of them.
//
// With u = z / eps, for each row: lse = log sum_j e^(u_j), logp = u_id - lse,
// H = lse - sum_j p_j u_j, p_j = e^(u_j - lse). One pass reads the row once and keeps, per
// thread, the running maximum m of z, l = sum e^(u_j - m/eps) and a = sum e^(u_j - m/eps)
// (u_j - m/eps); then lse = m/eps + log l and H = log l - a/l. Differences z - m are taken
// before scaling, so a row of the type's lowest value (a mask) is a uniform row and not an
// overflow. The pass is bound by the read of the matrix: 1 exponential and about 6 other
// instructions per score stay below it (4096 x 65536 bf16, forward: see kTokenThreads).
//
// Order of alternatives: larger z first, equal z by the lower index. Each warp keeps its best
// (value, index) pairs as sorted whole numbers across its lanes, and the CTA the largest of the
// warps' last kept pairs: a round of vectors is looked at one by one only where its maximum
// reaches that bar, which after the first round happens about top * ln(n / n0) times a row.
//
// A row is read by one CTA, or by a cluster of up to 8 when there are few rows (a decoding
// step), whose partial results meet in the first CTA through distributed shared memory: one
// launch either way, no workspace, and the same order of additions on every call.
#pragma once

#include <cooperative_groups.h>

#include "fs_rowload.cuh"

namespace fs {

constexpr int kTokenThreads = 256;
constexpr int kTokenWarps = kTokenThreads / 32;
constexpr int kTokenUnroll = 4;  // 16-byte vectors in flight per thread
constexpr int kTokenMaxTop = 32;
constexpr int kTokenMaxCluster = 8;

struct TokenParams {
  const void* z;
  int64_t ld;
  const void* ids;
  int64_t rows;
  int32_t cols;
  int32_t ids_wide;
  int32_t top;
  float inv_eps;
  float* logp;
  float* entropy;
  float* lse;
  float2* stats;  // (max z, log sum) per row for the gradient
  float* top_logp;
  int32_t* top_ids;
};

// Running maximum, sum and entropy sum of some of a row's scores.
struct TokenSum {
  float m, l, a;
};

// Both parts' sums about the common maximum. A part that has seen no score above -inf has
// l = a = 0 (or NaN, which stays): its factor is 2^-inf = 0, and the clamp keeps 0 * inf out
// of the entropy sum. k2 = log2(e) / eps.
__device__ __forceinline__ TokenSum token_merge(TokenSum x, TokenSum y, float k2) {
  const float m = fmaxf(x.m, y.m);
  const float mm = m == -INFINITY ? 0.0f : m;
  const float dx = (x.m - mm) * k2, dy = (y.m - mm) * k2;
  const float cx = fmaxf(dx, -1.0e30f), cy = fmaxf(dy, -1.0e30f);
  const float sx = ex2(dx), sy = ex2(dy);
  return {m, x.l * sx + y.l * sy, sx * (x.a + x.l * cx) + sy * (y.a + y.l * cy)};
}

// Adds N scores to the running sums.
template <int N>
__device__ __forceinline__ void token_add(TokenSum& s, const float* z, float zmax, float k2) {
  if (zmax > s.m) {
    const float d = (s.m - zmax) * k2;
    const float sc = ex2(d);
    s.a = s.m == -INFINITY ? s.a : sc * (s.a + s.l * fmaxf(d, -1.0e30f));
    s.l *= sc;
    s.m = zmax;
  }
  const float mm = s.m == -INFINITY ? 0.0f : s.m;
  if constexpr (N % 2 == 0) {
    const u64 m2 = pk(mm, mm), kk = pk(k2, k2);
    u64 l2 = pk(0.0f, 0.0f), a2 = pk(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const u64 d = mul2(sub2(pk(z[i], z[i + 1]), m2), kk);
      float d0, d1;
      upk(d, d0, d1);
      const u64 e = pk(ex2(d0), ex2(d1));
      l2 = add2(l2, e);
      // a masked score has d = -inf and e = 0; below -200 e is 0 already
      a2 = fma2(e, pk(fmaxf(d0, -200.0f), fmaxf(d1, -200.0f)), a2);
    }
    float x, y;
    upk(l2, x, y);
    s.l += x + y;
    upk(a2, x, y);
    s.a += x + y;
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float d = (z[i] - mm) * k2;
      const float e = ex2(d);
      s.l += e;
      s.a += e * fmaxf(d, -200.0f);
    }
  }
}

// A score and its column as one whole number: larger score first, then the lower column. 0 is
// below all of them and stands for none.
__device__ __forceinline__ u64 token_key(float v, int i) {
  return (static_cast<u64>(order_key(v)) << 32) | (0xFFFFFFFFu - static_cast<uint32_t>(i));
}
__device__ __forceinline__ float token_key_value(u64 k) {
  return order_unkey(static_cast<uint32_t>(k >> 32));
}
__device__ __forceinline__ int token_key_index(u64 k) {
  return static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(k));
}
__device__ __forceinline__ u64 max_u64(u64 a, u64 b) { return a > b ? a : b; }
__device__ __forceinline__ u64 min_u64(u64 a, u64 b) { return a < b ? a : b; }

// The warp's keys, one per lane, sorted: the largest in lane 0 (bitonic, 15 exchanges).
__device__ __forceinline__ u64 token_sort(u64 k, int lane) {
#pragma unroll
  for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
    for (int o = size >> 1; o > 0; o >>= 1) {
      const u64 p = __shfl_xor_sync(0xffffffffu, k, o);
      k = ((lane & o) == 0) == ((lane & size) == 0) ? max_u64(k, p) : min_u64(k, p);
    }
  return k;
}

// The 32 largest of two sorted lists, sorted: each lane keeps the larger of a's i-th and b's
// i-th last, which leaves a bitonic sequence, and five exchanges sort it.
__device__ __forceinline__ u64 token_join(u64 a, u64 b, int lane) {
  a = max_u64(a, __shfl_sync(0xffffffffu, b, 31 - lane));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const u64 p = __shfl_xor_sync(0xffffffffu, a, o);
    a = (lane & o) == 0 ? max_u64(a, p) : min_u64(a, p);
  }
  return a;
}

// Inserts key (the same in every lane) into the sorted list.
__device__ __forceinline__ u64 token_insert(u64 list, u64 key, int lane) {
  const int pos = __popc(__ballot_sync(0xffffffffu, list > key));
  const u64 up = __shfl_up_sync(0xffffffffu, list, 1);
  return lane > pos ? up : lane == pos ? key : list;
}

// Inserts the lanes' keys (0: none) that are above the list's last kept one.
__device__ __forceinline__ u64 token_offer(u64 list, u64 key, int top, int lane) {
  unsigned c = __ballot_sync(0xffffffffu, key > __shfl_sync(0xffffffffu, list, top - 1));
  while (c) {
    const int src = __ffs(c) - 1;
    c &= c - 1;
    list = token_insert(list, __shfl_sync(0xffffffffu, key, src), lane);
  }
  return list;
}

// Candidates that a warp gathers from one round of vectors before it sorts them.
constexpr int kTokenBuffer = 128;

struct TokenShared {
  TokenSum sum[kTokenWarps];
  u64 best[kTokenWarps][32];
  u64 buffer[kTokenWarps][kTokenBuffer];
  // the largest of the warps' last kept keys: nothing below it is among the row's best
  u64 bar;
  // the CTA's result, read by the cluster's first CTA
  TokenSum total;
  u64 total_best[32];
};

// Adds one round's vectors (f: U x V scores of this lane, the first of vector u at column
// first + u * stride, n of them valid) to the warp's list. Gathers the scores above the bar in
// shared memory, then inserts a few one by one or sorts and joins many at once. In the first
// round the bar is raised beforehand: `top` lanes' maxima are at or above the top-th largest
// of them, so whatever lies below that one is not among the row's best.
template <typename T, int U>
__device__ __forceinline__ u64 token_gather(u64 list, u64& bar, const float* f, const float* vmax,
                                            float bm, int n, int first, int stride, int top,
                                            const T* z, u64* buffer, u64* shared_bar, int lane) {
  constexpr int V = Elem<T>::kVec;
  float bar_v = token_key_value(bar);
  int bar_i = token_key_index(bar);
  if (bar == 0) {
    bar_v = -INFINITY;
    bar_i = 0x7FFFFFFF;
    uint32_t mine = n > 0 && bm == bm ? order_key(bm) : 0u, t = 0u;
    for (int r = 0; r < top; ++r) {
      t = __reduce_max_sync(0xffffffffu, mine);
      if (t == 0u) break;
      // (equal maxima count one by one)
      const unsigned at = __ballot_sync(0xffffffffu, mine == t);
      if (lane == __ffs(at) - 1) mine = 0u;
    }
    if (t != 0u) bar_v = order_unkey(t);
  }
  int count = 0;
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (u < n && vmax[u] >= bar_v) {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float v = f[u * V + e];
        count += v > bar_v || (v == bar_v && first + u * stride + e < bar_i);
      }
    }
  int before = count;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int q = __shfl_up_sync(0xffffffffu, before, o);
    if (lane >= o) before += q;
  }
  const int total = __shfl_sync(0xffffffffu, before, 31);
  if (total == 0) return list;
  if (total <= kTokenBuffer) {
    int at = before - count;
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (u < n && vmax[u] >= bar_v) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float v = f[u * V + e];
          const int i = first + u * stride + e;
          if (v > bar_v || (v == bar_v && i < bar_i)) buffer[at++] = token_key(v, i);
        }
      }
    __syncwarp();
    if (total <= 6) {
      for (int c = 0; c < total; ++c) list = token_insert(list, buffer[c], lane);
    } else {
      for (int c = 0; c < total; c += 32)
        list = token_join(list, token_sort(c + lane < total ? buffer[c + lane] : 0ull, lane), lane);
    }
    __syncwarp();
  } else {
    // more than the buffer holds (many equal scores, or many alternatives): one by one
#pragma unroll 1
    for (int u = 0; u < U; ++u)
#pragma unroll 1
      for (int e = 0; e < V; ++e) {
        const int i = first + u * stride + e;
        const float v = u < n ? Elem<T>::to_f(z[i]) : __int_as_float(0x7FC00000);
        list = token_offer(list, v >= bar_v ? token_key(v, i) : 0ull, top, lane);
      }
  }
  const u64 last = __shfl_sync(0xffffffffu, list, top - 1);
  if (last > bar) {
    bar = last;
    if (lane == 0) atomicMax(shared_bar, last);
  }
  return list;
}

template <typename T, bool TOP>
__global__ void __launch_bounds__(kTokenThreads)
    token_logprobs_kernel(const TokenParams P, const int cluster) {
  namespace cg = cooperative_groups;
  constexpr int V = Elem<T>::kVec, U = kTokenUnroll;
  __shared__ TokenShared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t row = blockIdx.x / cluster;
  const int rank = static_cast<int>(blockIdx.x % cluster);
  const T* z = static_cast<const T*>(P.z) + row * P.ld;
  const float k2 = P.inv_eps * kLog2e;
  const int64_t id = ld_id(P.ids, row, P.ids_wide != 0);
  if (id < 0) {  // nobody asks about this row (the same in all CTAs of its cluster)
    if (rank == 0) {
      if (tid == 0) {
        P.logp[row] = 0.0f;
        P.entropy[row] = 0.0f;
        if (P.lse) P.lse[row] = 0.0f;
        if (P.stats) P.stats[row] = make_float2(0.0f, 0.0f);
      }
      if (TOP && tid < P.top) {
        P.top_logp[row * P.top + tid] = -INFINITY;
        P.top_ids[row * P.top + tid] = -1;
      }
    }
    return;
  }
  if (TOP) {
    if (tid == 0) sh.bar = 0;
    __syncthreads();
  }

  int head, nvec;
  row_split(z, P.cols, head, nvec);
  const int v0 = static_cast<int>(static_cast<int64_t>(nvec) * rank / cluster);
  const int v1 = static_cast<int>(static_cast<int64_t>(nvec) * (rank + 1) / cluster);
  TokenSum s = {-INFINITY, 0.0f, 0.0f};
  u64 list = 0, bar = 0;

  for (int b = v0; b < v1; b += kTokenThreads * U) {
    uint4 r[U];
    float f[U * V];
    float vmax[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int v = b + u * kTokenThreads + tid;
      if (v < v1) r[u] = ld_stream(z + head + static_cast<int64_t>(v) * V);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int v = b + u * kTokenThreads + tid;
      if (v < v1) {
        Elem<T>::unpack(r[u], f + u * V);
      } else {
#pragma unroll
        for (int e = 0; e < V; ++e) f[u * V + e] = -INFINITY;
      }
      float mx = fmaxf(f[u * V], f[u * V + 1]);
#pragma unroll
      for (int e = 2; e < V; e += 2) mx = max3(mx, f[u * V + e], f[u * V + e + 1]);
      vmax[u] = mx;
    }
    float bm = vmax[0];
#pragma unroll
    for (int u = 1; u < U; ++u) bm = fmaxf(bm, vmax[u]);
    if constexpr (TOP) {
      bar = max_u64(bar, *static_cast<volatile u64*>(&sh.bar));
      // (a lane's read of the shared bar may be older than another's: the warp takes lane 0's)
      bar = __shfl_sync(0xffffffffu, bar, 0);
      if (bar == 0 || __any_sync(0xffffffffu, bm >= token_key_value(bar))) {
        const int v = b + tid;
        const int n = v < v1 ? min(U, (v1 - v + kTokenThreads - 1) / kTokenThreads) : 0;
        list = token_gather<T, U>(list, bar, f, vmax, bm, n, head + v * V, kTokenThreads * V, P.top,
                                  z, sh.buffer[warp], &sh.bar, lane);
      }
    }
    token_add<U * V>(s, f, bm, k2);
  }
  if (warp == 0) {  // the unaligned ends: at most 7 scores each
    const int tail = head + nvec * V;
    const bool hd = rank == 0 && lane < head;
    const bool tl = rank == cluster - 1 && lane < P.cols - tail;
    const float zh = hd ? Elem<T>::to_f(z[lane]) : -INFINITY;
    const float zt = tl ? Elem<T>::to_f(z[tail + lane]) : -INFINITY;
    const float f[2] = {zh, zt};
    token_add<2>(s, f, fmaxf(zh, zt), k2);
    if constexpr (TOP) {
      list = token_offer(list, hd && zh == zh ? token_key(zh, lane) : 0ull, P.top, lane);
      list = token_offer(list, tl && zt == zt ? token_key(zt, tail + lane) : 0ull, P.top, lane);
    }
  }

#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    TokenSum q;
    q.m = __shfl_xor_sync(0xffffffffu, s.m, o);
    q.l = __shfl_xor_sync(0xffffffffu, s.l, o);
    q.a = __shfl_xor_sync(0xffffffffu, s.a, o);
    // the lower lane's part first, so both lanes add in one order
    s = (lane & o) ? token_merge(q, s, k2) : token_merge(s, q, k2);
  }
  if (lane == 0) sh.sum[warp] = s;
  if (TOP) sh.best[warp][lane] = list;
  __syncthreads();
  if constexpr (TOP) {
    // pairs of warps join their lists, then pairs of pairs
#pragma unroll
    for (int half = kTokenWarps / 2; half > 0; half >>= 1) {
      if (warp < half) {
        const u64 other = sh.best[warp + half][lane];
        // (lists mostly end below the bar of another warp)
        if (__any_sync(0xffffffffu, other > __shfl_sync(0xffffffffu, list, P.top - 1))) {
          list = token_join(list, other, lane);
          sh.best[warp][lane] = list;
        }
      }
      __syncthreads();
    }
  }
  if (warp == 0) {
    s = sh.sum[lane % kTokenWarps];  // (every eight lanes arrive at the same sum)
#pragma unroll
    for (int o = kTokenWarps / 2; o > 0; o >>= 1) {
      TokenSum q;
      q.m = __shfl_xor_sync(0xffffffffu, s.m, o);
      q.l = __shfl_xor_sync(0xffffffffu, s.l, o);
      q.a = __shfl_xor_sync(0xffffffffu, s.a, o);
      s = (lane & o) ? token_merge(q, s, k2) : token_merge(s, q, k2);
    }
  }
  if (cluster > 1) {
    cg::cluster_group cl = cg::this_cluster();
    if (warp == 0) {
      if (lane == 0) sh.total = s;
      sh.total_best[lane] = list;
    }
    cl.sync();
    if (rank == 0 && warp == 0) {
      TokenSum t[kTokenMaxCluster];
      u64 o[kTokenMaxCluster];
#pragma unroll
      for (int q = 1; q < kTokenMaxCluster; ++q)
        if (q < cluster) {
          const TokenShared* other = cl.map_shared_rank(&sh, q);
          t[q] = other->total;
          if (TOP) o[q] = other->total_best[lane];
        }
#pragma unroll
      for (int q = 1; q < kTokenMaxCluster; ++q)
        if (q < cluster) {
          s = token_merge(s, t[q], k2);
          if (TOP) list = token_join(list, o[q], lane);
        }
    }
    cl.sync();  // no CTA ends while its shared memory is read
    if (rank != 0) return;
  }
  if (warp != 0) return;
  const bool empty = s.m == -INFINITY && s.l == 0.0f;  // every score is -inf
  const float log_l = logf(s.l);
  if (lane == 0) {
    const float zi = id < P.cols ? Elem<T>::to_f(z[id]) : __int_as_float(0x7FC00000);
    P.logp[row] = empty ? (id < P.cols ? -INFINITY : zi) : (zi - s.m) * P.inv_eps - log_l;
    P.entropy[row] = empty ? 0.0f : log_l - s.a / s.l * kLn2;
    if (P.lse) P.lse[row] = empty ? -INFINITY : s.m * P.inv_eps + log_l;
    if (P.stats) P.stats[row] = make_float2(s.m, empty ? 0.0f : log_l);
  }
  if (TOP && lane < P.top) {
    const bool have = list != 0;
    P.top_logp[row * P.top + lane] =
        empty ? -INFINITY : (have ? (token_key_value(list) - s.m) * P.inv_eps - log_l
                                  : __int_as_float(0x7FC00000));
    P.top_ids[row * P.top + lane] = have ? token_key_index(list) : -1;
  }
}

// ---- gradient -------------------------------------------------------------------------------

struct TokenGradParams {
  const void* z;
  int64_t ld;
  const void* ids;
  int64_t rows;
  int32_t cols;
  int32_t ids_wide;
  int32_t top;
  int32_t chunks;  // CTAs per row
  float inv_eps;
  const float2* stats;
  const float* entropy;
  const int32_t* top_ids;
  const float* g_logp;
  const float* g_entropy;
  const float* g_lse;
  const float* g_top;
  void* grad;
  int64_t ld_grad;
};

// What the gradient of a row needs besides its scores:
//   dz_j = (1/eps) [ p_j (c - ge (log p_j + H)) + hot_j ],  c = g_lse - g_logp - sum_k g_top_k,
// hot_j = g_logp at the given token plus g_top_k at each alternative.
struct TokenRow {
  float m, log2_l;  // p_j = 2^((z_j - m) k2 - log2_l)
  float c, ge;      // already divided by eps
};

__device__ __forceinline__ float token_dscore(const TokenRow& r, float z, float k2, float H) {
  const float t = (z - r.m) * k2 - r.log2_l;
  // p = 0 where t = -inf; the clamp keeps 0 * inf out
  return ex2(t) * (r.c - r.ge * (fmaxf(t, -1.0e30f) * kLn2 + H));
}

// One CTA writes kTokenThreads * kTokenUnroll vectors of a row: one read, one exponential and
// one write per score. The given token and the alternatives are rewritten afterwards from the
// scores, their terms added in fp32 before the one rounding to the output's type.
template <typename T>
__global__ void __launch_bounds__(kTokenThreads)
    token_logprobs_grad_kernel(const TokenGradParams P) {
  constexpr int V = Elem<T>::kVec, U = kTokenUnroll;
  constexpr int64_t kChunk = static_cast<int64_t>(kTokenThreads) * U * V;
  const int tid = threadIdx.x;
  const int64_t row = blockIdx.x / P.chunks;
  const int chunk = static_cast<int>(blockIdx.x % P.chunks);
  const T* z = static_cast<const T*>(P.z) + row * P.ld;
  T* out = static_cast<T*>(P.grad) + row * P.ld_grad;
  const int64_t id = ld_id(P.ids, row, P.ids_wide != 0);
  const float2 st = P.stats[row];
  // a row not asked about, or an empty one (max -inf, log sum 0; NaN scores leave log sum NaN)
  const bool zero = id < 0 || (st.x == -INFINITY && st.y == 0.0f);
  const float k2 = P.inv_eps * kLog2e;
  // a token outside the matrix has no log probability: the row's gradient is NaN with it
  float gl = P.g_logp ? P.g_logp[row] : 0.0f;
  if (id >= P.cols) gl = __int_as_float(0x7FC00000);
  TokenRow r;
  r.m = st.x;
  r.log2_l = st.y * kLog2e;
  r.ge = P.g_entropy ? P.g_entropy[row] * P.inv_eps : 0.0f;
  r.c = (P.g_lse ? P.g_lse[row] : 0.0f) - gl;
  if (P.g_top)
    for (int k = 0; k < P.top; ++k) r.c -= P.g_top[row * P.top + k];
  r.c *= P.inv_eps;
  const float H = P.entropy[row];

  // vectors by the output's alignment; the scores' are read as vectors where theirs agrees
  int head, nvec;
  row_split(out, P.cols, head, nvec);
  const bool same = ((reinterpret_cast<uintptr_t>(z) ^ reinterpret_cast<uintptr_t>(out)) & 15u) == 0;
  const int64_t b = static_cast<int64_t>(chunk) * (kTokenThreads * U);
  uint4 q[U];
  if (same && !zero) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t v = b + u * kTokenThreads + tid;
      if (v < nvec) q[u] = ld_stream(z + head + v * V);
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t v = b + u * kTokenThreads + tid;
    if (v >= nvec) break;
    float f[V];
    if (zero) {
#pragma unroll
      for (int e = 0; e < V; ++e) f[e] = 0.0f;
    } else {
      if (same) {
        Elem<T>::unpack(q[u], f);
      } else {
#pragma unroll
        for (int e = 0; e < V; ++e) f[e] = Elem<T>::to_f(z[head + v * V + e]);
      }
#pragma unroll
      for (int e = 0; e < V; ++e) f[e] = token_dscore(r, f[e], k2, H);
    }
    __stcs(reinterpret_cast<uint4*>(out + head + v * V), Elem<T>::pack(f));
  }
  if (chunk == 0 && tid < 32) {
    const int tail = head + nvec * V;
    if (tid < head) out[tid] = Elem<T>::from_f(zero ? 0.0f : token_dscore(r, Elem<T>::to_f(z[tid]), k2, H));
    if (tid < P.cols - tail)
      out[tail + tid] =
          Elem<T>::from_f(zero ? 0.0f : token_dscore(r, Elem<T>::to_f(z[tail + tid]), k2, H));
  }
  if (zero) return;
  // the CTA that wrote an element also adds its hot terms
  const int n_hot = 1 + (P.g_top ? P.top : 0);
  __syncthreads();
  if (tid < n_hot) {
    const int64_t at = tid == 0 ? id : P.top_ids[row * P.top + tid - 1];
    const int64_t rel = at - head;
    const bool in_vec = rel >= 0 && rel < static_cast<int64_t>(nvec) * V;
    const int owner = in_vec ? static_cast<int>(rel / kChunk) : 0;
    if (at >= 0 && at < P.cols && owner == chunk) {
      float hot = 0.0f;
      bool first = true;
      for (int k = 0; k < n_hot; ++k) {
        const int64_t o = k == 0 ? id : P.top_ids[row * P.top + k - 1];
        if (o != at) continue;
        if (k < tid) first = false;
        hot += k == 0 ? gl : P.g_top[row * P.top + k - 1];
      }
      if (first)
        out[at] = Elem<T>::from_f(token_dscore(r, Elem<T>::to_f(z[at]), k2, H) + hot * P.inv_eps);
    }
  }
}

}  // namespace fs
