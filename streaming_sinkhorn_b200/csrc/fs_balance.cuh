// fs_balance.cuh -- Sinkhorn potentials of a given score matrix: the bias that spreads rows
// (tokens) over columns (experts) by a given load.
//
// The alternating updates of the point-cloud solve with C = -s, s the router's scores:
//   f_i = -eps log mean_j beta_j e^((s_ij + g_j)/eps),   g_j = -eps log mean_i e^((s_ij + f_i)/eps),
// beta_j = load_j / mean(load). In base 2, with u = s log2(e)/eps and
// gamma_j = g_j log2(e)/eps + log2 beta_j, both updates come from one exponential per score:
//   e_ij = 2^(u_ij + gamma_j - m_i),  S_i = sum_j e_ij,  phi_i = -(m_i + log2(S_i / E)),
//   c_j = mean_i e_ij E / S_i,        gamma_j <- gamma_j - log2 c_j + log2 beta_j,
// since 2^(u_ij + phi_i) = e_ij (E / S_i) 2^-gamma_j. Means and not sums with the logarithm of
// a weight: those would cancel. A column whose c_j comes out below 2^-40 (its terms may have
// been flushed) is done over with its own maximum.
//
// One launch does all iterations. Every CTA keeps its rows' u in fp32, in shared memory and, when
// that is full, in the SM's tensor memory, which has no products to serve here (the rest, if
// they do not all fit, in the workspace, read through L2 one step ahead). A group of lanes takes
// a row, two rows at a time, each lane holding the column sums of its columns in registers. All
// rows of a CTA share one offset in place of m_i (none at all while the largest u of the CTA plus
// the largest gamma is in range of ex2), so a row needs one reduction; a row whose sum comes out
// below 2^-60 is done over with its own maximum. Per iteration the CTAs exchange one row of column
// sums each: small problems through distributed shared memory in a cluster of up to 16 CTAs, else
// by integer atomics and a grid barrier. That launch is cooperative, so all CTAs run at once, and
// its waits are bounded: when one expires the call's outputs are NaN.
//
// 65536 x 256 fp32, 20 iterations: 220 us, 9.2 an iteration, of which 5 are the exponentials and
// their instructions (3.7 at the rate of ex2 alone) and 4 the exchange; 37 go into the scores.
#pragma once

#include "fs_rowload.cuh"
#include "fs_route.cuh"
#include "fs_tcgen05.cuh"

namespace fs {

constexpr int kBalClusterWarps = 16;
constexpr int kBalGridWarps = 32;
constexpr int kBalMaxCluster = 16;
constexpr float kBalLowSum = 0x1p-60f;   // a row's sum that may have lost terms
constexpr float kBalFlushed = 0x1p-40f;  // a column's mean that may have lost terms

// Words of one iteration's column sums across the grid: copies of high and low parts, a flag, the
// open rows. A CTA adds to one of the copies, so that fewer atomics meet at an address, and all
// read every copy (65536 x 256, an iteration: 9.6 us with 1 copy, 9.2 with 4, 9.4 with 8, 10.1
// with 16; reading each CTA's sums one by one 11.7).
constexpr int kBalCopies = 4;
__host__ __device__ constexpr int bal_sums(int cols) { return kBalCopies * 2 * cols + 2; }

struct BalanceParams {
  const void* z;
  int64_t ld;
  int64_t rows;
  int32_t experts;
  int32_t cols;      // experts padded to NL x (lanes of a row)
  int32_t score;
  int32_t n_iters;
  int32_t per_cta;   // rows of a CTA
  int32_t resident;  // of them, rows kept in shared memory; the next ones are in tensor memory
  float eps;
  const float* load;    // or NULL: uniform
  const float* g_init;  // or NULL: 0
  float* f;
  float* g;
  unsigned* sync;   // [0] arrivals, [1] nonzero once a wait has expired; zeroed before the launch
  u64* sums;        // grid: [3][bal_sums] column sums in whole numbers, by iteration; zeroed, too
  float2* redo;     // [gridDim][cols] (max, sum) of columns done over
  float* spill;     // u of the rows beyond `resident`, (gridDim, per_cta - resident, cols)
};

// All CTAs arrive; false once a wait anywhere has expired.
__device__ __forceinline__ bool grid_barrier(unsigned* sync, unsigned target, int* ok_sh) {
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    atomicAdd(&sync[0], 1u);
    const unsigned long long t0 = global_ns();
    int ok = 1;
    for (unsigned k = 1;; ++k) {
      unsigned now;
      asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(now) : "l"(&sync[0]) : "memory");
      if (now >= target) break;
      if ((k & 63u) == 0u) {
        if (*static_cast<volatile unsigned*>(&sync[1]) || global_ns() - t0 > kWaitLimitNs) {
          atomicExch(&sync[1], 1u);
          ok = 0;
          break;
        }
      }
    }
    *ok_sh = ok;
  }
  __syncthreads();
  return *ok_sh != 0;
}

// Lane l of the LPT lanes of a row holds columns 4 (LPT q + l) .. + 3 for q = 0 .. NL / 4 - 1:
// 16-byte accesses of neighbouring lanes are neighbours in memory.
template <int NL, int LPT, int NW>
struct BalShape {
  static constexpr int kThreads = NW * 32;
  static constexpr int kQuads = NL * LPT / 4;
  static constexpr int kCols = NL * LPT;
  static constexpr int kGroups = 32 / LPT;               // rows a warp takes at once
  static constexpr int kRowStep = kGroups * NW;          // rows a CTA takes at once
  // Steps whose rows tensor memory holds: the NW / 4 warps of a lane quarter share its 512
  // columns, a lane's NL columns of a row lie in as many of its own TMEM lane.
  static constexpr int kTmemWarp = 512 / (NW / 4);
  static constexpr int kTmemSteps = kTmemWarp / NL;
  static __host__ __device__ constexpr int column(int l, int i) {
    return 4 * (LPT * (i / 4) + l) + i % 4;
  }
};

template <int LPT>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
  for (int o = LPT / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
template <int LPT>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = LPT / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The exponentials e_i = 2^(u_i + g_i) of H rows over this lane's columns and their sums over
// the rows; g holds gamma less the offset. A sum too low for comfort is taken again about the
// row's own maximum, which `extra` returns (0 otherwise). Called by whole warps.
template <int NL, int LPT, int H>
__device__ __forceinline__ void bal_rows(const float4 (*u)[NL / 4], const float* g, float (*e)[NL],
                                         float* sum, float* extra) {
#pragma unroll
  for (int h = 0; h < H; ++h) {
    u64 acc = pk(0.0f, 0.0f);
#pragma unroll
    for (int q = 0; q < NL / 4; ++q) {
      const float4 x = u[h][q];
      float t0, t1, t2, t3;
      upk(add2(pk(x.x, x.y), pk(g[4 * q], g[4 * q + 1])), t0, t1);
      upk(add2(pk(x.z, x.w), pk(g[4 * q + 2], g[4 * q + 3])), t2, t3);
      e[h][4 * q] = ex2(t0);
      e[h][4 * q + 1] = ex2(t1);
      e[h][4 * q + 2] = ex2(t2);
      e[h][4 * q + 3] = ex2(t3);
      acc = add2(acc, add2(pk(e[h][4 * q], e[h][4 * q + 1]), pk(e[h][4 * q + 2], e[h][4 * q + 3])));
    }
    float x, y;
    upk(acc, x, y);
    sum[h] = x + y;
    extra[h] = 0.0f;
  }
#pragma unroll
  for (int h = 0; h < H; ++h) sum[h] = group_sum<LPT>(sum[h]);
  bool any = sum[0] < kBalLowSum;
  if (H == 2) any |= sum[H - 1] < kBalLowSum;
  if (LPT < 32) any = __any_sync(0xffffffffu, any);  // (whole warps have one row: one sum)
  if (any) {
#pragma unroll
    for (int h = 0; h < H; ++h) {
      float m = -INFINITY;
#pragma unroll
      for (int q = 0; q < NL / 4; ++q) {
        m = fmaxf(m, fmaxf(u[h][q].x + g[4 * q], u[h][q].y + g[4 * q + 1]));
        m = fmaxf(m, fmaxf(u[h][q].z + g[4 * q + 2], u[h][q].w + g[4 * q + 3]));
      }
      m = group_max<LPT>(m);
      const bool low = sum[h] < kBalLowSum && m != -INFINITY;  // (no open column: 0)
      float s = 0.0f;
#pragma unroll
      for (int q = 0; q < NL / 4; ++q) {
        const float t[4] = {u[h][q].x + g[4 * q], u[h][q].y + g[4 * q + 1], u[h][q].z + g[4 * q + 2],
                            u[h][q].w + g[4 * q + 3]};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (low) e[h][4 * q + i] = ex2(t[i] - m);
          s += e[h][4 * q + i];
        }
      }
      s = group_sum<LPT>(s);
      if (low) {
        sum[h] = s;
        extra[h] = m;
      }
    }
  }
}

// Four neighbouring logits of a row, -inf beyond the last.
template <typename T>
__device__ __forceinline__ float4 bal_load(const T* z, int j, int E, bool vec) {
  if (vec && j < E) {
    if constexpr (sizeof(T) == 4) {
      return *reinterpret_cast<const float4*>(z + j);
    } else {
      const uint2 r = *reinterpret_cast<const uint2*>(z + j);
      float f[8];
      Elem<T>::unpack(make_uint4(r.x, r.y, 0u, 0u), f);
      return make_float4(f[0], f[1], f[2], f[3]);
    }
  }
  return make_float4(j < E ? Elem<T>::to_f(z[j]) : -INFINITY,
                     j + 1 < E ? Elem<T>::to_f(z[j + 1]) : -INFINITY,
                     j + 2 < E ? Elem<T>::to_f(z[j + 2]) : -INFINITY,
                     j + 3 < E ? Elem<T>::to_f(z[j + 3]) : -INFINITY);
}

// log2 of a positive float about two offsets, the whole numbers added up in 64 bits.
__device__ __forceinline__ double bal_log2(float v, float off, float extra) {
  int k;
  const float f = frexpf(v, &k);
  return (static_cast<double>(off) + extra + k) + log2f(f);
}

// Column sums across the grid are added up by atomics on whole numbers, whose order does not
// change the result: c in units of 2^-20 (c <= rows x experts < 2^41) and what that leaves in
// units of 2^-60. Each CTA's part is off by less than 2^-60: of the smallest mean that counts
// (2^-40) a part in 2^20 times the number of rows. NaN sets a flag.
template <int C>  // padded columns; sums: [kBalCopies][2][C], then the flag
__device__ __forceinline__ void bal_add(u64* sums, int j, float c) {
  if (!(c < 0x1p42f)) {
    sums[kBalCopies * 2 * C] = 1;  // (every CTA that writes it writes the same)
    return;
  }
  const float hi = truncf(c * 0x1p20f);
  sums += (blockIdx.x % kBalCopies) * 2 * C + j;
  atomicAdd(sums, static_cast<u64>(hi));
  atomicAdd(sums + C, static_cast<u64>(fmaf(hi, -0x1p-20f, c) * 0x1p60f));
}
template <int C>
__device__ __forceinline__ double bal_sum(const u64* sums, int j) {
  u64 hi = 0, lo = 0;
#pragma unroll
  for (int i = 0; i < kBalCopies; ++i) {
    hi += __ldcg(sums + i * 2 * C + j);
    lo += __ldcg(sums + i * 2 * C + C + j);
  }
  if (__ldcg(sums + kBalCopies * 2 * C) != 0) return __longlong_as_double(0x7FF8000000000000ll);
  return static_cast<double>(hi) * 0x1p-20 + static_cast<double>(lo) * 0x1p-60;
}

// Joins two parts of a sum of exponentials, each about its own maximum (in every order the same
// but for rounding). A part without terms is (-inf, 0); NaN stays.
__device__ __forceinline__ void bal_join(float& m, float& l, float om, float ol) {
  const float mm = fmaxf(m, om);
  if (mm == -INFINITY) {
    l += ol;
    return;
  }
  l = l * ex2(m - mm) + ol * ex2(om - mm);
  m = mm;
}

// Columns done over in their own range: maximum and sum over the CTA's rows of 2^(u_ij + phi_i), for
// all columns, into out. Groups of lanes take rows as the iterations do, phi_i once for each, from
// the gammas that the iteration's rows have seen; a lane keeps its columns' parts, then the groups
// and the warps join theirs in order. csum has the columns' means, and afterwards 1 where a column
// is to be done over and 0 elsewhere. (65536 x 256, 20 iterations, at eps = 0.003, where nearly all
// columns are done over in each: 375 us against 220 without; 8191 x 64, 10 iterations: 74 and 47. A
// column closed to every row costs one look: 249 and 61.)
template <int NL, int LPT, int NW>
__device__ __noinline__ void bal_redo(const float* u_res, const float* u_spill, int n, int resident,
                                      int E, const double* gam, const float* lb, float* csum,
                                      float2* out) {
  using S = BalShape<NL, LPT, NW>;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int l = lane % LPT, grp = lane / LPT;
  float g[NL], m[NL], s[NL];
#pragma unroll
  for (int i = 0; i < NL; ++i) {
    const int j = S::column(l, i);
    const float c = j < E ? csum[j] : 0.0f;
    // (a column that has been updated already: without what that added)
    g[i] = static_cast<float>(lb[j] == -INFINITY || c < kBalFlushed ? gam[j]
                                                                    : gam[j] + log2f(c) - lb[j]);
    m[i] = -INFINITY;
    s[i] = 0.0f;
  }
  // (which of them, before csum serves as scratch: each thread its own, as in the update)
  uint32_t again = 0u;
  for (int j = threadIdx.x, q = 0; j < E; j += S::kThreads, ++q)
    if (lb[j] != -INFINITY && csum[j] < kBalFlushed) again |= 1u << q;
  __syncthreads();
  for (int b = warp * S::kGroups; b < n; b += S::kRowStep) {
    const int r = b + grp;
    const float4* src = reinterpret_cast<const float4*>(
        r < resident ? u_res + static_cast<int64_t>(r) * S::kCols
                     : u_spill + static_cast<int64_t>(r - resident) * S::kCols);
    float u[NL];
#pragma unroll
    for (int q = 0; q < NL / 4; ++q) {
      const float4 x = r < n ? src[LPT * q + l]
                             : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      u[4 * q] = x.x;
      u[4 * q + 1] = x.y;
      u[4 * q + 2] = x.z;
      u[4 * q + 3] = x.w;
    }
    float top = -INFINITY, sum = 0.0f;
#pragma unroll
    for (int i = 0; i < NL; ++i) top = fmaxf(top, u[i] + g[i]);
    top = group_max<LPT>(top);
    const float mm = top == -INFINITY ? 0.0f : top;
#pragma unroll
    for (int i = 0; i < NL; ++i) sum += ex2(u[i] + g[i] - mm);
    sum = group_sum<LPT>(sum);
    if (r >= n || sum == 0.0f) continue;  // (no open column: the row takes no part)
    const float phi = -(mm + log2f(sum / static_cast<float>(E)));
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const float x = u[i] + phi;
      if (x > m[i]) {
        s[i] = s[i] * ex2(m[i] - x) + 1.0f;
        m[i] = x;
      } else if (x != -INFINITY) {
        s[i] += ex2(x - m[i]);
      }
    }
  }
  __syncwarp();
#pragma unroll
  for (int i = 0; i < NL; ++i)
#pragma unroll
    for (int o = LPT; o < 32; o <<= 1) {
      const float om = __shfl_xor_sync(0xffffffffu, m[i], o);
      const float os = __shfl_xor_sync(0xffffffffu, s[i], o);
      bal_join(m[i], s[i], om, os);
    }
  float2* parts = reinterpret_cast<float2*>(csum);  // NW / 2 rows of pairs
#pragma unroll 1
  for (int half = NW / 2; half > 0; half >>= 1) {
    if (warp >= half && warp < 2 * half && grp == 0) {
#pragma unroll
      for (int i = 0; i < NL; ++i)
        parts[(warp - half) * S::kCols + S::column(l, i)] = make_float2(m[i], s[i]);
    }
    __syncthreads();
    if (warp < half && grp == 0) {
#pragma unroll
      for (int i = 0; i < NL; ++i) {
        const float2 o = parts[warp * S::kCols + S::column(l, i)];
        bal_join(m[i], s[i], o.x, o.y);
      }
    }
    __syncthreads();
  }
  if (warp == 0 && grp == 0) {
#pragma unroll
    for (int i = 0; i < NL; ++i) out[S::column(l, i)] = make_float2(m[i], s[i]);
  }
  for (int j = threadIdx.x, q = 0; j < E; j += S::kThreads, ++q)
    csum[j] = again >> q & 1u ? 1.0f : 0.0f;
}

// All CTAs' parts of the columns done over, a warp each: their gammas.
template <int NW>
__device__ __noinline__ void bal_redo_join(const float2* redo, int cols, int G, int E,
                                           const float* csum, float* lb, double inv_open,
                                           double* gam) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int j = warp; j < E; j += NW) {  // (csum: which columns those are)
    if (csum[j] == 0.0f) continue;
    float cm = -INFINITY, cl = 0.0f;
    for (int q = lane; q < G; q += 32) {
      const float2 o = __ldcg(&redo[static_cast<int64_t>(q) * cols + j]);
      bal_join(cm, cl, o.x, o.y);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float om = __shfl_xor_sync(0xffffffffu, cm, o);
      const float ol = __shfl_xor_sync(0xffffffffu, cl, o);
      bal_join(cm, cl, om, ol);
    }
    if (lane == 0) {
      // a column closed to every row is like one of no load from here on
      if (cm == -INFINITY && cl == 0.0f) lb[j] = -INFINITY;
      gam[j] = -(cm + log2f(static_cast<float>(cl * inv_open))) + lb[j];
      if (lb[j] == -INFINITY) gam[j] = -INFINITY;
    }
  }
}

template <typename T, int NL, int LPT, int NW, bool CLUSTER>
__global__ void __launch_bounds__(NW * 32, 1) balance_kernel(const BalanceParams P) {
  using S = BalShape<NL, LPT, NW>;
  constexpr int kPartCols = S::kCols + 4;  // column sums, then the open rows
  constexpr int kSums = bal_sums(S::kCols);
  extern __shared__ __align__(16) double bal_smem[];
  __shared__ int ok_sh;
  __shared__ float warp_sh[2][NW];
  __shared__ uint64_t part_bar[2];  // CLUSTER: all CTAs' sums have arrived (by parity)
  __shared__ int redo_sh;
  __shared__ uint32_t tmem_sh;
  // gamma is carried in 64 bits: it is a sum over the iterations, and next to 20 (eps = 0.05) a
  // float's rounding would show in g
  double* gam = bal_smem;                                  // [cols]
  float* lb = reinterpret_cast<float*>(gam + S::kCols);    // [cols] log2 beta
  float* csum = lb + S::kCols;        // [NW][cols] partial sums
  float* parts = csum + NW * S::kCols;  // CLUSTER: [2][16][kPartCols]
  float* u_res = parts + (CLUSTER ? 2 * kBalMaxCluster * kPartCols : 0);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int l = lane % LPT, grp = lane / LPT;
  const int E = P.experts;
  const float ke = kLog2e / P.eps, inv_e = 1.0f / static_cast<float>(E);
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * P.per_cta;
  const int n = static_cast<int>(
      P.rows - row0 < P.per_cta ? (P.rows > row0 ? P.rows - row0 : 0) : P.per_cta);
  float* u_spill = P.spill + static_cast<int64_t>(blockIdx.x) * (P.per_cta - P.resident) * S::kCols;
  const int G = gridDim.x;
  unsigned arrivals = 0;
  // (generic addressing: resident rows lie in shared memory, the rest in the workspace)
  auto row_of = [&](int r) -> float* {
    return r < P.resident ? u_res + static_cast<int64_t>(r) * S::kCols
                          : u_spill + static_cast<int64_t>(r - P.resident) * S::kCols;
  };

  // Rows that tensor memory holds (the workspace has them too, for columns done over). The CTA
  // takes all of it and never waits for it: its registers fill the SM, so no other is on it.
  const int n_tm = CLUSTER || n <= P.resident
                       ? 0
                       : (n - P.resident < S::kTmemSteps * S::kRowStep
                              ? n - P.resident
                              : S::kTmemSteps * S::kRowStep);
  uint32_t tmem = 0;
  if constexpr (!CLUSTER) {
    if (n_tm > 0) {
      if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
            smem_u32(&tmem_sh)));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
      }
      tc_fence_before();
      __syncthreads();
      tc_fence_after();
      // this warp's lanes and columns
      tmem = tmem_sh + (static_cast<uint32_t>(warp & 3) << 21) +
             static_cast<uint32_t>((warp >> 2) * S::kTmemWarp);
    }
  }

  // log2 beta, gamma of the start
  if (warp == 0) {
    double tot = 0.0;
    bool bad = false;
    if (P.load)
      for (int j = lane; j < E; j += 32) {
        tot += P.load[j];
        bad |= !(P.load[j] >= 0.0f && P.load[j] < INFINITY);
      }
    // (a sum of 0 makes every share NaN; so does a bad entry, those of an expert of load 0 too)
    tot = __any_sync(0xffffffffu, bad) ? __longlong_as_double(0x7FF8000000000000ll) : warp_sum(tot);
    for (int j = lane; j < S::kCols; j += 32) {
      float b = 0.0f;
      if (j >= E)
        b = -INFINITY;
      else if (P.load)
        b = static_cast<float>(log2(static_cast<double>(P.load[j]) * E / tot));
      lb[j] = b;
      gam[j] = j < E ? (P.g_init ? static_cast<double>(P.g_init[j]) * ke : 0.0) + b : -INFINITY;
    }
  }

  // u of the CTA's rows and the largest of them; rows without an open column are counted out
  int open = 0;
  float umax = -INFINITY;
  const T* z0 = static_cast<const T*>(P.z) + row0 * P.ld;
  const bool vec = E % 4 == 0 && P.ld % 4 == 0 &&
                   (reinterpret_cast<uintptr_t>(P.z) & (4 * sizeof(T) - 1)) == 0;
  float4 ahead[NL / 4];
  auto read = [&](int b) {
    const int r = b + grp < n ? b + grp : n - 1;
#pragma unroll
    for (int q = 0; q < NL / 4; ++q)
      ahead[q] = bal_load(z0 + static_cast<int64_t>(r) * P.ld, S::column(l, 4 * q), E, vec);
  };
  if (warp * S::kGroups < n) read(warp * S::kGroups);
  for (int b = warp * S::kGroups; b < n; b += S::kRowStep) {
    const int r = b + grp;
    const bool have = r < n;
    float v[NL];
    float m = -INFINITY;
#pragma unroll
    for (int q = 0; q < NL / 4; ++q) {
      v[4 * q] = have ? ahead[q].x : -INFINITY;
      v[4 * q + 1] = have ? ahead[q].y : -INFINITY;
      v[4 * q + 2] = have ? ahead[q].z : -INFINITY;
      v[4 * q + 3] = have ? ahead[q].w : -INFINITY;
    }
    if (b + S::kRowStep < n) read(b + S::kRowStep);
#pragma unroll
    for (int i = 0; i < NL; ++i) m = fmaxf(m, v[i]);
    if (P.score == kScoreSoftmax) {
      m = group_max<LPT>(m);
      const float mm = m == -INFINITY ? 0.0f : m;
      float e[NL];
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < NL; ++i) {
        e[i] = ex2((v[i] - mm) * kLog2e);
        sum += e[i];
      }
      const float inv = ke / group_sum<LPT>(sum);
#pragma unroll
      for (int i = 0; i < NL; ++i) v[i] = v[i] == -INFINITY ? -INFINITY : e[i] * inv;
    } else {
#pragma unroll
      for (int i = 0; i < NL; ++i)
        v[i] = v[i] == -INFINITY ? -INFINITY : route_score(v[i], kScoreSigmoid, 0.0f, 0.0f) * ke;
      m = group_max<LPT>(m);
    }
#pragma unroll
    for (int i = 0; i < NL; ++i) umax = fmaxf(umax, v[i]);
    // (a row of NaN is open: its NaN reaches every output)
    if (have && l == 0 && m != -INFINITY) ++open;
    if (have) {
      float4* dst = reinterpret_cast<float4*>(row_of(r));
#pragma unroll
      for (int q = 0; q < NL / 4; ++q)
        dst[LPT * q + l] = make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
    }
  }
  open = __reduce_add_sync(0xffffffffu, open);
  umax = warp_maxf(umax);
  if (lane == 0) {
    warp_sh[0][warp] = static_cast<float>(open);
    warp_sh[1][warp] = umax;
  }
  __syncthreads();
  if constexpr (!CLUSTER) {
    for (int b = warp * S::kGroups, q0 = 0; b < n_tm; b += S::kRowStep, q0 += NL) {
      const int r = b + grp;  // (written by any warp, before the barrier)
      const float4* src = reinterpret_cast<const float4*>(u_spill) + r * S::kQuads + l;
      float v[NL];
#pragma unroll
      for (int q = 0; q < NL / 4; ++q) {
        const float4 x = r < n_tm ? src[LPT * q]
                                  : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
        v[4 * q] = x.x;
        v[4 * q + 1] = x.y;
        v[4 * q + 2] = x.z;
        v[4 * q + 3] = x.w;
      }
      __syncwarp();
#pragma unroll
      for (int q = 0; q < NL; q += 8) tc_st8(tmem + q0 + q, v + q);
    }
    tc_wait_st();
  }
  umax = warp_maxf(lane < NW ? warp_sh[1][lane] : -INFINITY);
  if (umax == -INFINITY) umax = 0.0f;

  if (CLUSTER && G > 1) {
    if (tid == 0) {
      mbar_init(&part_bar[0], 1);
      mbar_init(&part_bar[1], 1);
      fence_mbar_init();
    }
    cluster_barrier();  // no CTA writes into another's shared memory before that one is ready
  }

  double inv_open = 0.0;  // 1 / rows that take part
  bool alive = true;
  for (int it = 0; it < P.n_iters && alive; ++it) {
    const bool last = it == P.n_iters - 1;
    float gm[NL], acc[NL];
    float off = -INFINITY;
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      gm[i] = static_cast<float>(gam[S::column(l, i)]);
      off = fmaxf(off, gm[i]);
      acc[i] = 0.0f;
    }
    off = group_max<LPT>(off);
    off = (off == -INFINITY ? 0.0f : off) + umax;
    // No u + gamma lies above off. 2^100 and sums of 1024 such terms are within range, so up to
    // there no offset is taken at all: gamma less a large offset would lose digits of every
    // column's gamma in every iteration (1e-6 of g at eps = 2 / experts).
    off = off > 100.0f ? off - 100.0f : off < -20.0f ? off : 0.0f;
#pragma unroll
    for (int i = 0; i < NL; ++i) gm[i] = static_cast<float>(gam[S::column(l, i)] - off);
    // With 16 warps two rows a step (b + grp and the next group's); more than 256 columns leave
    // no registers for that.
    constexpr int kH = NL == 8 && NW == 16 ? 2 : 1;
    constexpr int kStep = kH * S::kRowStep;
    const int b0 = warp * kH * S::kGroups;
    // u: the step's rows, r0 the first of them, n0 the end of the rows it is taken from
    auto step = [&](const float4 (*u)[NL / 4], int r0, int n0) {
      float e[kH][NL], sum[kH], extra[kH];
      bal_rows<NL, LPT, kH>(u, gm, e, sum, extra);
#pragma unroll
      for (int h = 0; h < kH; ++h) {
        // One correction of the quick quotient: its error has a sign, and one that all rows share
        // would move every gamma the same way in every iteration.
        float w = __fdividef(static_cast<float>(E), sum[h]);
        w = fmaf(w * inv_e, fmaf(-w, sum[h], static_cast<float>(E)), w);
        if (sum[h] == 0.0f) w = 0.0f;
        const u64 w2 = pk(w, w);
#pragma unroll
        for (int i = 0; i < NL; i += 2) {
          const u64 a = fma2(pk(e[h][i], e[h][i + 1]), w2, pk(acc[i], acc[i + 1]));
          upk(a, acc[i], acc[i + 1]);
        }
        if (last) {
          const int r = r0 + h * S::kGroups + grp;
          if (l == 0 && r < n0)
            P.f[row0 + r] = sum[h] == 0.0f
                                ? 0.0f
                                : static_cast<float>(-bal_log2(sum[h] * inv_e, off, extra[h]) / ke);
        }
      }
    };
    const float4 closed = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
    const int n_res = n < P.resident ? n : P.resident;
    {
      const float4* src = reinterpret_cast<const float4*>(u_res) + (b0 + grp) * S::kQuads + l;
      for (int b = b0; b < n_res; b += kStep, src += kStep * S::kQuads) {
        float4 u[kH][NL / 4];
#pragma unroll
        for (int h = 0; h < kH; ++h)
#pragma unroll
          for (int q = 0; q < NL / 4; ++q)
            u[h][q] = S::kGroups * kH == 1 || b + h * S::kGroups + grp < n_res
                          ? src[h * S::kGroups * S::kQuads + LPT * q]
                          : closed;
        step(u, b, n_res);
      }
    }
    if constexpr (!CLUSTER) {
      static_assert(kH == 1, "a step of tensor memory is one row of each group");
      for (int b = b0, q0 = 0; b < n_tm; b += kStep, q0 += NL) {
        float v[NL];
        __syncwarp();
#pragma unroll
        for (int q = 0; q < NL; q += 8) tc_ld8(tmem + q0 + q, v + q);
        float4 u[kH][NL / 4];
#pragma unroll
        for (int q = 0; q < NL / 4; ++q)
          u[0][q] = make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
        step(u, n_res + b, n);
      }
      // the rows in the workspace, read one step ahead
      const int n_sp = n - n_res - n_tm;
      const float4* src =
          reinterpret_cast<const float4*>(u_spill) + (n_tm + b0 + grp) * S::kQuads + l;
      float4 nx[kH][NL / 4];
      auto fetch = [&](int b) {
#pragma unroll
        for (int h = 0; h < kH; ++h)
#pragma unroll
          for (int q = 0; q < NL / 4; ++q)
            nx[h][q] = S::kGroups * kH == 1 || b + h * S::kGroups + grp < n_sp
                           ? __ldcg(src + h * S::kGroups * S::kQuads + LPT * q)
                           : closed;
      };
      if (b0 < n_sp) fetch(b0);
      for (int b = b0; b < n_sp; b += kStep) {
        float4 u[kH][NL / 4];
#pragma unroll
        for (int h = 0; h < kH; ++h)
#pragma unroll
          for (int q = 0; q < NL / 4; ++q) u[h][q] = nx[h][q];
        src += kStep * S::kQuads;
        if (b + kStep < n_sp) fetch(b + kStep);
        step(u, n_res + n_tm + b, n);
      }
    }
    // the CTA's column sums: the rows of a warp (in each exchange a lane keeps half of its
    // columns and its partner the other half, until one is left), then the warps in their order
    int first = 0, kept = NL;  // the columns that this lane still holds: acc[0 .. kept - 1]
    bool writes = true;
#pragma unroll
    for (int o = LPT; o < 32; o <<= 1) {
      if (kept > 1) {
        const bool up = (lane & o) != 0;
        kept /= 2;
#pragma unroll
        for (int i = 0; i < NL / 2; ++i)
          if (i < kept) {
            const float send = up ? acc[i] : acc[i + kept];
            acc[i] = (up ? acc[i + kept] : acc[i]) + __shfl_xor_sync(0xffffffffu, send, o);
          }
        if (up) first += kept;
      } else {
        acc[0] += __shfl_xor_sync(0xffffffffu, acc[0], o);
        writes = writes && (lane & o) == 0;
      }
    }
#pragma unroll
    for (int i = 0; i < NL; ++i)
      if (i < kept && writes) csum[warp * S::kCols + S::column(l, first + i)] = acc[i];
    if (tid == 0) redo_sh = 0;
    __syncthreads();
    if constexpr (CLUSTER) {
      // every column's sum to every CTA, counted on its barrier of this parity. (A CTA two
      // iterations ahead cannot be: it waits for this one's sums in between.)
      float* part = parts + (it & 1) * kBalMaxCluster * kPartCols;
      uint64_t* bar = &part_bar[it & 1];
      constexpr int kAtOnce = S::kThreads / S::kCols;  // CTAs written to at a time
      const int j = tid % S::kCols;
      float c = 0.0f;
#pragma unroll
      for (int w = 0; w < NW; ++w) c += csum[w * S::kCols + j];
      float o = 0.0f;
      if (it == 0 && tid < G)
        for (int w = 0; w < NW; ++w) o += warp_sh[0][w];
      if (G == 1) {  // (a launch without a cluster: nothing to exchange)
        if (tid < S::kCols) part[j] = c;
        if (it == 0 && tid == 0) part[S::kCols] = o;
        __syncthreads();
      } else {
        if (tid == 0)
          mbar_expect_tx(bar, static_cast<uint32_t>(G) * (S::kCols + (it == 0 ? 1 : 0)) * 4u);
        for (int q = tid / S::kCols; q < G; q += kAtOnce)
          st_async_cluster(part + blockIdx.x * kPartCols + j, q, c, bar);
        if (it == 0 && tid < G)
          st_async_cluster(part + blockIdx.x * kPartCols + S::kCols, tid, o, bar);
        const bool ok = mbar_wait_cluster_bounded(bar, static_cast<uint32_t>(it >> 1) & 1u);
        if (__syncthreads_or(!ok)) {
          alive = false;
          break;
        }
      }
      if (it == 0) {
        double o2 = 0.0;
        for (int q = 0; q < G; ++q) o2 += part[q * kPartCols + S::kCols];
        inv_open = 1.0 / fmax(o2, 1.0);  // (no open row at all: f = g = 0)
      }
    } else {
      u64* sums = P.sums + (it % 3) * kSums;
      for (int j = tid; j <= S::kCols; j += S::kThreads) {
        float c = 0.0f;
#pragma unroll
        for (int w = 0; w < NW; ++w) c += j < S::kCols ? csum[w * S::kCols + j] : warp_sh[0][w];
        if (j < E)
          bal_add<S::kCols>(sums, j, c);
        else if (j == S::kCols && it == 0)
          atomicAdd(sums + kSums - 1, static_cast<u64>(c));
      }
      arrivals += G;
      alive = grid_barrier(P.sync, arrivals, &ok_sh);
      if (!alive) break;
      // all CTAs have read the sums of the iteration before, and none adds to their place before
      // the next barrier
      if (blockIdx.x == 0)
        for (int j = tid; j < kSums; j += S::kThreads) P.sums[(it + 2) % 3 * kSums + j] = 0;
      if (it == 0)
        inv_open = 1.0 / fmax(static_cast<double>(__ldcg(sums + kSums - 1)), 1.0);
    }
    for (int j = tid; j < E; j += S::kThreads) {
      float c = 0.0f;
      if constexpr (CLUSTER) {
        const float* part = parts + (it & 1) * kBalMaxCluster * kPartCols + j;
        for (int q = 0; q < G; ++q) c += part[q * kPartCols];
        c = static_cast<float>(c * inv_open);
      } else {
        c = static_cast<float>(bal_sum<S::kCols>(P.sums + (it % 3) * kSums, j) * inv_open);
      }
      csum[j] = c;  // (all sums over the warps have been read)
      if (lb[j] == -INFINITY) {
        gam[j] = -INFINITY;  // nothing is wanted of this column, or it is closed
      } else if (c < kBalFlushed) {
        redo_sh = 1;
      } else {
        // the gamma that the rows have seen is the rounded one less the offset
        gam[j] = (static_cast<double>(static_cast<float>(gam[j] - off)) + off) - log2f(c) + lb[j];
      }
    }
    __syncthreads();
    if (redo_sh) {  // the same in every CTA: all have the same sums
      bal_redo<NL, LPT, NW>(u_res, u_spill, n, P.resident, E, gam, lb, csum,
                            P.redo + static_cast<int64_t>(blockIdx.x) * S::kCols);
      if constexpr (CLUSTER) {
        __threadfence();
        if (G > 1) cluster_barrier();
        __syncthreads();
      } else {
        arrivals += G;
        alive = grid_barrier(P.sync, arrivals, &ok_sh);
        if (!alive) break;
      }
      bal_redo_join<NW>(P.redo, S::kCols, G, E, csum, lb, inv_open, gam);
      __syncthreads();
    }
  }
  if (CLUSTER && G > 1) cluster_barrier();  // no CTA leaves while sums are on their way to it
  if constexpr (!CLUSTER) {
    if (n_tm > 0) {
      tc_fence_before();
      __syncthreads();
      tc_fence_after();
      if (warp == 0)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem_sh));
    }
  }
  if (!alive) {
    for (int r = tid; r < n; r += S::kThreads) P.f[row0 + r] = __int_as_float(0x7FC00000);
    if (blockIdx.x == 0)
      for (int j = tid; j < E; j += S::kThreads) P.g[j] = __int_as_float(0x7FC00000);
    return;
  }
  if (blockIdx.x == 0)
    for (int j = tid; j < E; j += S::kThreads)
      // (without beta a column has no load, -inf, or was closed to every row, 0)
      P.g[j] = lb[j] != -INFINITY ? static_cast<float>((gam[j] - lb[j]) / ke)
               : P.load && P.load[j] == 0.0f ? -INFINITY
                                             : 0.0f;
}

}  // namespace fs
