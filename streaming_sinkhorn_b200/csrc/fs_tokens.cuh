// fs_tokens.cuh -- log probabilities of given tokens from a matrix of scores, with each
// row's entropy and its best alternatives, and the gradient of all of them.
//
// With u = z / eps, for each row: lse = log sum_j e^(u_j), logp = u_id - lse,
// H = lse - sum_j p_j u_j, p_j = e^(u_j - lse). One pass reads the row once and keeps, per
// thread, the running maximum m of z, l = sum e^(u_j - m/eps) and a = sum e^(u_j - m/eps)
// (u_j - m/eps); then lse = m/eps + log l and H = log l - a/l. Differences z - m are taken
// before scaling, so a row of the type's lowest value (a mask) is a uniform row and not an
// overflow. What bounds it: the read of the matrix at 4 bytes a score (2048 x 65536: 6.0 TB/s),
// at 2 bytes the read together with one exponential and 7 other instructions a score (4096 x
// 65536: 102 us, 5.3 TB/s; exponentials alone would take 60 us, the read 82). The gradient reads
// and writes the matrix once (158 us, 6.8 TB/s).
//
// Order of alternatives: larger z first, equal z by the lower index. The first round of a row
// gives a bar that at least `top` scores reach; a warp sets the few vectors that reach it aside,
// and at the row's end all scores that do are (value, index) pairs, as whole numbers, in shared
// memory, where each counts those above it. A warp that has set aside too many looks at them
// meanwhile and keeps its best pairs sorted across its lanes.
//
// A row is read by one CTA, or by a cluster of up to 8 when there are few rows (a decoding
// step), whose partial results meet in the first CTA through distributed shared memory: one
// launch either way, no workspace, and the same order of additions on every call.
#pragma once

#include <cooperative_groups.h>

#include <type_traits>

#include "fs_rowload.cuh"
#include "fs_tcgen05.cuh"

namespace fs {

constexpr int kTokenUnroll = 4;  // 16-byte vectors of a thread in one round
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

// Moves the running sums to a new maximum.
__device__ __forceinline__ void token_raise(TokenSum& s, float zmax, float k2) {
  if (zmax > s.m) {
    const float d = (s.m - zmax) * k2;
    const float sc = ex2(d);
    s.a = s.m == -INFINITY ? s.a : sc * (s.a + s.l * fmaxf(d, -1.0e30f));
    s.l *= sc;
    s.m = zmax;
  }
}

// Adds N (even) scores to the running sums. A masked score has d = -inf and e = 0, and 0 * inf
// must stay out of the entropy sum: d is clamped at -200, where e is 0 already.
template <int N>
__device__ __forceinline__ void token_add(TokenSum& s, const float* z, float zmax, float k2) {
  token_raise(s, zmax, k2);
  const float mm = s.m == -INFINITY ? 0.0f : s.m;
  const u64 m2 = pk(-mm, -mm), kk = pk(k2, k2);
  u64 l2 = pk(0.0f, 0.0f), a2 = pk(0.0f, 0.0f);
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    const u64 d = mul2(add2(pk(z[i], z[i + 1]), m2), kk);
    float d0, d1;
    upk(d, d0, d1);
    const u64 e = pk(ex2(d0), ex2(d1));
    l2 = add2(l2, e);
    a2 = fma2(e, pk(fmaxf(d0, -200.0f), fmaxf(d1, -200.0f)), a2);
  }
  float x, y;
  upk(l2, x, y);
  s.l += x + y;
  upk(a2, x, y);
  s.a += x + y;
}

// The sum of the parts of LANES neighbouring lanes, in every one of them: each part is brought
// to the common maximum once, then both sums are added up.
template <int LANES>
__device__ __forceinline__ TokenSum token_reduce(TokenSum s, float k2) {
  float m = s.m;
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  const float d = (s.m - (m == -INFINITY ? 0.0f : m)) * k2;
  const float sc = ex2(d);
  float l = s.l * sc, a = sc * (s.a + s.l * fmaxf(d, -1.0e30f));
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) {
    l += __shfl_xor_sync(0xffffffffu, l, o);
    a += __shfl_xor_sync(0xffffffffu, a, o);
  }
  return {m, l, a};
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
  // (rolled up, as is the join: the pass's loop should stay in the instruction cache)
#pragma unroll 1
  for (int size = 2; size <= 32; size <<= 1)
#pragma unroll 1
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
#pragma unroll 1
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

constexpr int kTokenFew = 6;  // alternatives whose bar is merged one by one

// Vectors that reach the bar, kept by a warp until it looks at their scores.
constexpr int kTokenKept = 64;

template <int NW>
struct TokenShape {
  static constexpr int kThreads = NW * 32;  // computing threads; one more warp copies
  static constexpr int kRound = kThreads * kTokenUnroll;  // vectors of a stage
  static constexpr uint32_t kStageBytes = kRound * 16u;
  static constexpr int kStages = NW == 8 ? 3 : 4;
  static constexpr int kRing = kStages * static_cast<int>(kStageBytes);
};

template <int NW>
struct TokenShared {
  uint64_t full[TokenShape<NW>::kStages], empty[TokenShape<NW>::kStages];
  int abort;  // a wait has expired: the rest of the CTA's rows are NaN
  TokenSum sum[2][NW];  // by row parity: warps run ahead of the one that reads
  TokenSum total;       // the CTA's result, read by the cluster's first CTA
};
template <int NW>
struct TokenTop {  // alternatives
  uint4 kept[NW][kTokenKept];
  int kept_at[NW][kTokenKept];  // a vector's first column
  uint32_t maxima[64];
  u64 best[NW][32];  // a warp's pairs, in no order
  int count[NW];
  u64 total_best[32];  // the CTA's, sorted
};
struct TokenNoTop {};

// Meeting point of the computing warps (the copying warp goes its own way).
template <int NW>
__device__ __forceinline__ void token_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(NW * 32) : "memory");
}

// The bar of a row after its first round of `vectors`, a score that at least `top` of its scores
// reach: the top-th largest of the warps' m largest thread maxima (bm; have: this thread has read
// a vector). A few are merged one by one; for more, two from each warp beyond its share, whose
// top-th largest hardly ever lies below that of all, and each counts those above it (1 x 128000
// bf16, 20 alternatives: 11.1 us, 12.7 one by one; with 5 the same, and 1531 x 50257 72 against
// 75 by counting). Called by all computing warps.
template <int NW>
__device__ __noinline__ float token_bar(float bm, int vectors, bool have, int top,
                                        TokenTop<NW>& sh, int warp, int lane) {
  const int warps = min(NW, (vectors + 31) / 32);  // those that have read any
  const bool few = top <= kTokenFew;
  const int m = few ? top : min(top, (top + warps - 1) / warps + 2);
  uint32_t mine = have && bm == bm ? order_key(bm) : 0u, t = 0u;
  for (int r = 0; r < m; ++r) {
    t = __reduce_max_sync(0xffffffffu, mine);
    if (warp < warps && lane == 0) sh.maxima[warp * m + r] = t;
    // (equal maxima count one by one)
    if (lane == __ffs(__ballot_sync(0xffffffffu, mine == t)) - 1) mine = 0u;
  }
  const int n = warps * m;  // top .. 60
  if (warp == 0 && lane < 4) sh.maxima[n + lane] = 0u;  // (read by fours)
  token_sync<NW>();
  if (few) {
    int next = lane * m;
    uint32_t head = lane < warps ? sh.maxima[next] : 0u;
    for (int r = 0; r < top; ++r) {
      t = __reduce_max_sync(0xffffffffu, head);
      if (t == 0u) break;
      if (lane == __ffs(__ballot_sync(0xffffffffu, head == t)) - 1) {
        ++next;
        head = next < (lane + 1) * m ? sh.maxima[next] : 0u;
      }
    }
  } else {
    const uint32_t x = lane < n ? sh.maxima[lane] : 0u;
    const uint32_t y = lane + 32 < n ? sh.maxima[lane + 32] : 0u;
    int px = 0, py = 0;  // places: equal ones in their order
#pragma unroll 1
    for (int i = 0; i < n; i += 4) {
      const uint4 o = *reinterpret_cast<const uint4*>(sh.maxima + i);
      const uint32_t v[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        px += v[e] > x || (v[e] == x && i + e < lane) ? 1 : 0;
        py += v[e] > y || (v[e] == y && i + e < lane + 32) ? 1 : 0;
      }
    }
    const uint32_t hit = lane < n && px == top - 1 ? x : lane + 32 < n && py == top - 1 ? y : 0u;
    t = __reduce_max_sync(0xffffffffu, hit);
  }
  // with fewer maxima everything counts, -inf included
  return t != 0u ? order_unkey(t) : -INFINITY;
}

// Looks at the scores of the warp's `n` kept vectors: those not below the bar go into the
// sorted list, a few one by one, many sorted and joined. Raises the bar to the list's last
// kept score.
template <typename T>
__device__ __noinline__ u64 token_look(u64 list, float& bar, const uint4* kept, const int* kept_at,
                                       int n, int top, int lane) {
  constexpr int V = Elem<T>::kVec;
  __syncwarp();
  for (int c = 0; c < n; c += 32) {
    const bool have = c + lane < n;
    const T* x = reinterpret_cast<const T*>(kept + (have ? c + lane : 0));
    const int at = have ? kept_at[c + lane] : 0;
#pragma unroll 1
    for (int e = 0; e < V; ++e) {
      const float v = Elem<T>::to_f(x[e]);
      const u64 key = have && v >= bar ? token_key(v, at + e) : 0ull;
      const u64 last = __shfl_sync(0xffffffffu, list, top - 1);
      const unsigned above = __ballot_sync(0xffffffffu, key > last);
      if (__popc(above) > 6)
        list = token_join(list, token_sort(key, lane), lane);
      else if (above)
        list = token_offer(list, key, top, lane);
    }
  }
  __syncwarp();
  const u64 last = __shfl_sync(0xffffffffu, list, top - 1);
  if (last) bar = fmaxf(bar, token_key_value(last));
  return list;
}

// The scores of the warp's `n` (up to 32) kept vectors that reach the bar, as pairs in no order:
// their number, the first 32 of them in `out`.
template <typename T>
__device__ __forceinline__ int token_give(float bar, const uint4* kept, const int* kept_at, int n,
                                       u64* out, int lane) {
  constexpr int V = Elem<T>::kVec;
  const unsigned below = (1u << lane) - 1u;
  __syncwarp();
  float f[V];
  Elem<T>::unpack(kept[lane < n ? lane : 0], f);
  const int at = kept_at[lane < n ? lane : 0];
  int count = 0;
#pragma unroll
  for (int e = 0; e < V; ++e) {
    const bool reach = lane < n && f[e] >= bar;
    const unsigned who = __ballot_sync(0xffffffffu, reach);
    const int to = count + __popc(who & below);
    if (reach && to < 32) out[to] = token_key(f[e], at + e);
    count += __popc(who);
  }
  return count;
}

// The end of a row for a warp: its scores that reach the bar (of warp 0 the unaligned ends too)
// become its pairs in shared memory, in no order; if there are more than 32, its best ones.
template <typename T, int NW>
__device__ __noinline__ void token_finish(u64 list, float bar, int kept, TokenTop<NW>& best,
                                          bool hd, float zh, bool tl, float zt, int tail, int top,
                                          int warp, int lane) {
  int n = 0;
  const bool looked = __any_sync(0xffffffffu, list != 0);
  if (!looked) {
    if (kept > 0)
      n = token_give<T>(bar, best.kept[warp], best.kept_at[warp], kept, best.best[warp], lane);
    if (warp == 0) {
      const bool rh = hd && zh >= bar, rt = tl && zt >= bar;
      const unsigned wh = __ballot_sync(0xffffffffu, rh), wt = __ballot_sync(0xffffffffu, rt);
      const unsigned below = (1u << lane) - 1u;
      const int th = n + __popc(wh & below), tt = n + __popc(wh) + __popc(wt & below);
      if (rh && th < 32) best.best[0][th] = token_key(zh, lane);
      if (rt && tt < 32) best.best[0][tt] = token_key(zt, tail + lane);
      n += __popc(wh) + __popc(wt);
    }
  }
  if (looked || n > 32) {
    list = token_look<T>(list, bar, best.kept[warp], best.kept_at[warp], kept, top, lane);
    if (warp == 0) {
      list = token_offer(list, hd && zh == zh ? token_key(zh, lane) : 0ull, top, lane);
      list = token_offer(list, tl && zt == zt ? token_key(zt, tail + lane) : 0ull, top, lane);
    }
    n = __popc(__ballot_sync(0xffffffffu, lane < top && list != 0));
    best.best[warp][lane] = list;
  }
  __syncwarp();
  if (lane >= n && lane < max(4, n + (n & 1))) best.best[warp][lane] = 0;  // (read in pairs)
  if (lane == 0) best.count[warp] = n;
  if (warp == 0) best.total_best[lane] = 0;
}

// How many of all warps' pairs are above `key`. Every warp's list ends with a 0 or at 32, and has
// 4 entries at least.
template <int NW>
__device__ __noinline__ int token_place(u64 key, const u64 (*best)[32], const int* count) {
  int place = 0;
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    const ulonglong2 a = *reinterpret_cast<const ulonglong2*>(&best[w][0]);
    const ulonglong2 b = *reinterpret_cast<const ulonglong2*>(&best[w][2]);
    place += (a.x > key ? 1 : 0) + (a.y > key ? 1 : 0) + (b.x > key ? 1 : 0) + (b.y > key ? 1 : 0);
  }
#pragma unroll 1
  for (int w = 0; w < NW; ++w)
    for (int i = 4; i < count[w]; i += 2) {
      const ulonglong2 o = *reinterpret_cast<const ulonglong2*>(&best[w][i]);
      place += (o.x > key ? 1 : 0) + (o.y > key ? 1 : 0);
    }
  return place;
}

// The part of a row that a CTA reads: `nvec` vectors from element `head` on are shared by the
// cluster in order, vectors [v0, v1) are this CTA's.
struct TokenPart {
  int head, nvec, v0, v1;
};
template <typename T>
__device__ __forceinline__ TokenPart token_part(const T* z, int cols, int rank, int cluster) {
  TokenPart p;
  row_split(z, cols, p.head, p.nvec);
  p.v0 = static_cast<int>(static_cast<int64_t>(p.nvec) * rank / cluster);
  p.v1 = static_cast<int>(static_cast<int64_t>(p.nvec) * (rank + 1) / cluster);
  return p;
}

// CTAs stay and take rows blockIdx.x, + gridDim.x, ... (a cluster takes one row). The last warp
// copies the CTA's parts of its rows, one after the other, into a ring in shared memory (bulk
// copies), so the next row is on its way while the last one is summed up; NW warps compute.
template <typename T, bool TOP, int NW>
__global__ void __launch_bounds__(NW * 32 + 32, NW == 8 ? (TOP ? 3 : 4) : (TOP ? 5 : 6))
    token_logprobs_kernel(const TokenParams P, const int cluster) {
  namespace cg = cooperative_groups;
  using H = TokenShape<NW>;
  constexpr int V = Elem<T>::kVec, U = kTokenUnroll, S = H::kStages, NT = H::kThreads;
  extern __shared__ __align__(128) unsigned char token_ring[];
  __shared__ TokenShared<NW> sh;
  __shared__ std::conditional_t<TOP, TokenTop<NW>, TokenNoTop> best;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = static_cast<int>(blockIdx.x % cluster);
  const int64_t row0 = blockIdx.x / cluster, row_step = gridDim.x / cluster;
  const float k2 = P.inv_eps * kLog2e;
  volatile int* abort = &sh.abort;
  if (tid == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], NW);
    }
    sh.abort = 0;
    fence_mbar_init();
  }
  __syncthreads();

  if (warp == NW) {
    if (lane != 0) return;
    int64_t q = 0;
    bool ok = true;
    for (int64_t row = row0; ok && row < P.rows; row += row_step) {
      if (ld_id(P.ids, row, P.ids_wide != 0) < 0) continue;
      const T* z = static_cast<const T*>(P.z) + row * P.ld;
      const TokenPart p = token_part(z, P.cols, rank, cluster);
      for (int b = p.v0; b < p.v1; b += H::kRound, ++q) {
        const int i = static_cast<int>(q % S);
        const uint32_t round = static_cast<uint32_t>(q / S);
        if (round > 0 && !tc_wait(&sh.empty[i], (round - 1) & 1u, abort)) {
          ok = false;
          break;
        }
        const uint32_t bytes = static_cast<uint32_t>(min(H::kRound, p.v1 - b)) * 16u;
        mbar_expect_tx(&sh.full[i], bytes);
        bulk_g2s(token_ring + i * H::kStageBytes, z + p.head + static_cast<int64_t>(b) * V, bytes,
                 &sh.full[i]);
      }
    }
    if (*abort)  // the copies in flight land before the CTA's shared memory goes
      for (int64_t v = q > S ? q - S : 0; v < q; ++v)
        (void)mbar_wait_bounded(&sh.full[v % S], static_cast<uint32_t>(v / S) & 1u);
    return;
  }

  // A wait that expires raises abort; every warp then goes on (each wait gives up soon), so that
  // all still meet at the same barriers, and the rows come out as NaN.
  int i = 0;           // stage
  uint32_t phase = 0;  // of its barrier
  int parity = 0;
  // (each row's id and the given token's score are asked for before they are needed)
  int64_t next_id = row0 < P.rows ? ld_id(P.ids, row0, P.ids_wide != 0) : 0;
  for (int64_t row = row0; row < P.rows; row += row_step) {
    const T* z = static_cast<const T*>(P.z) + row * P.ld;
    const int64_t id = next_id;
    if (row + row_step < P.rows) next_id = ld_id(P.ids, row + row_step, P.ids_wide != 0);
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
      continue;
    }
    const TokenPart p = token_part(z, P.cols, rank, cluster);
    float zi = __int_as_float(0x7FC00000);
    if (tid == 0 && rank == 0 && id < P.cols) zi = Elem<T>::to_f(z[id]);
    TokenSum s = {-INFINITY, 0.0f, 0.0f};
    u64 list = 0;
    float bar = -INFINITY;
    int kept = 0;
    for (int b = p.v0; b < p.v1; b += H::kRound) {
      (void)tc_wait(&sh.full[i], phase, abort);
      const uint4* stage = reinterpret_cast<const uint4*>(token_ring + i * H::kStageBytes) + tid;
      const int left = p.v1 - b - tid;  // vectors from this lane's first on
      uint4 r[U];
      if (p.v1 - b >= H::kRound) {
#pragma unroll
        for (int u = 0; u < U; ++u) r[u] = stage[u * NT];
      } else {
#pragma unroll
        for (int u = 0; u < U; ++u) r[u] = u * NT < left ? stage[u * NT] : Elem<T>::masked();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.empty[i]);
      if (++i == S) {
        i = 0;
        phase ^= 1u;
      }
      float f[U * V];
      float vmax[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        Elem<T>::unpack(r[u], f + u * V);
        float mx = fmaxf(f[u * V], f[u * V + 1]);
#pragma unroll
        for (int e = 2; e < V; e += 2) mx = max3(mx, f[u * V + e], f[u * V + e + 1]);
        vmax[u] = mx;
      }
      float bm = vmax[0];
#pragma unroll
      for (int u = 1; u < U; ++u) bm = fmaxf(bm, vmax[u]);
      token_add<U * V>(s, f, bm, k2);
      if constexpr (TOP) {
        if (b == p.v0) bar = token_bar<NW>(bm, p.v1 - b, left > 0, P.top, best, warp, lane);
        if (__any_sync(0xffffffffu, bm >= bar)) {
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const bool reach = u * NT < left && vmax[u] >= bar;
            const unsigned who = __ballot_sync(0xffffffffu, reach);
            if (who) {
              if (reach) {
                const int at = kept + __popc(who & ((1u << lane) - 1u));
                best.kept[warp][at] = r[u];
                best.kept_at[warp][at] = p.head + (b + u * NT + tid) * V;
              }
              kept += __popc(who);
              if (kept > kTokenKept - 32) {
                list = token_look<T>(list, bar, best.kept[warp], best.kept_at[warp], kept, P.top,
                                     lane);
                kept = 0;
              }
            }
          }
        }
      }
    }
    float zh = -INFINITY, zt = -INFINITY;  // the unaligned ends: at most 7 scores each
    const int tail = p.head + p.nvec * V;
    const bool hd = warp == 0 && rank == 0 && lane < p.head;
    const bool tl = warp == 0 && rank == cluster - 1 && lane < P.cols - tail;
    if (warp == 0) {
      if (hd) zh = Elem<T>::to_f(z[lane]);
      if (tl) zt = Elem<T>::to_f(z[tail + lane]);
      const float f[2] = {zh, zt};
      token_add<2>(s, f, fmaxf(zh, zt), k2);
    }
    if constexpr (TOP)
      token_finish<T, NW>(list, bar, kept, best, hd, zh, tl, zt, tail, P.top, warp, lane);

    s = token_reduce<32>(s, k2);
    parity ^= 1;
    if (lane == 0) sh.sum[parity][warp] = s;
    token_sync<NW>();
    if constexpr (TOP) {
      // every pair's place among all warps' (no two are equal)
      const int n = best.count[warp];
      if (n > 0) {
        const u64 key = lane < n ? best.best[warp][lane] : 0ull;
        const int place = token_place<NW>(key, best.best, best.count);
        if (key != 0 && place < P.top) best.total_best[place] = key;
      }
      token_sync<NW>();
      if (warp == 0) list = best.total_best[lane];
    }
    if (warp == 0) {
      s = token_reduce<NW>(sh.sum[parity][lane % NW], k2);
      if (*abort) s.l = __int_as_float(0x7FC00000);
    }
    if (cluster > 1) {
      cg::cluster_group cl = cg::this_cluster();
      if (warp == 0) {
        if (lane == 0) sh.total = s;
      }
      cl.sync();  // (the copying warps leave by themselves)
      if (rank == 0) {
        if constexpr (TOP) {
          // the CTAs' lists by pairs, a warp each
          static_assert(NW >= kTokenMaxCluster / 2, "a warp for each pair of lists");
          if (2 * warp < cluster) {
            list = token_join(cl.map_shared_rank(&best, 2 * warp)->total_best[lane],
                              cl.map_shared_rank(&best, 2 * warp + 1)->total_best[lane], lane);
            best.best[warp][lane] = list;
          }
          token_sync<NW>();
#pragma unroll 1
          for (int half = cluster / 4; half > 0; half >>= 1) {
            if (warp < half) {
              list = token_join(list, best.best[warp + half][lane], lane);
              best.best[warp][lane] = list;
            }
            token_sync<NW>();
          }
        }
        if (warp == 0) {
          // lane c takes CTA c's sum
          const int c0 = lane % kTokenMaxCluster;
          s = token_reduce<kTokenMaxCluster>(c0 < cluster ? cl.map_shared_rank(&sh, c0)->total
                                                          : TokenSum{-INFINITY, 0.0f, 0.0f},
                                             k2);
        }
      }
      cl.sync();  // no CTA ends while its shared memory is read
    }
    if (warp == 0 && rank == 0) {
      const bool empty = s.m == -INFINITY && s.l == 0.0f;  // every score is -inf
      const float log_l = logf(s.l);
      if (lane == 0) {
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
  }
}

// ---- gradient -------------------------------------------------------------------------------

constexpr int kTokenGradThreads = 256;

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

// One CTA writes kTokenGradThreads * kTokenUnroll vectors of a row: one read, one exponential and
// one write per score. The given token and the alternatives are rewritten afterwards from the
// scores, their terms added in fp32 before the one rounding to the output's type.
template <typename T>
__global__ void __launch_bounds__(kTokenGradThreads)
    token_logprobs_grad_kernel(const TokenGradParams P) {
  constexpr int V = Elem<T>::kVec, U = kTokenUnroll;
  constexpr int64_t kChunk = static_cast<int64_t>(kTokenGradThreads) * U * V;
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
  const int64_t b = static_cast<int64_t>(chunk) * (kTokenGradThreads * U);
  uint4 q[U];
  if (same && !zero) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t v = b + u * kTokenGradThreads + tid;
      if (v < nvec) q[u] = ld_stream(z + head + v * V);
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t v = b + u * kTokenGradThreads + tid;
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
