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
// a weight: those would cancel. A column whose c_j comes out below 2^-100 (its terms may have
// been flushed) is done over with its own maximum.
//
// One launch does all iterations. Every CTA keeps its rows' u in shared memory in fp32 (the
// rest, if they do not all fit, in the workspace, read through L2), a group of lanes takes a
// row, each lane holding the column sums of its columns in registers; per iteration the CTAs
// exchange one row of column sums each and meet at a grid barrier. The launch is cooperative,
// so all CTAs run at once, and every wait is bounded: when one expires the call's outputs are
// NaN.
#pragma once

#include "fs_rowload.cuh"
#include "fs_route.cuh"

namespace fs {

constexpr int kBalThreads = 512;
constexpr int kBalWarps = kBalThreads / 32;
constexpr float kBalFlushed = 0x1p-100f;

struct BalanceParams {
  const void* z;
  int64_t ld;
  int64_t rows;
  int32_t experts;
  int32_t cols;      // experts padded to NL x (lanes of a row)
  int32_t score;
  int32_t n_iters;
  int32_t per_cta;   // rows of a CTA
  int32_t resident;  // of them, rows kept in shared memory
  float eps;
  const float* load;    // or NULL: uniform
  const float* g_init;  // or NULL: 0
  float* f;
  float* g;
  unsigned* sync;   // [0] arrivals, [1] nonzero once a wait has expired; zeroed before the launch
  float* part;      // [2][gridDim][cols + 1] column sums (and open rows) by iteration parity
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
template <int NL, int LPT>
struct BalShape {
  static constexpr int kCols = NL * LPT;
  static constexpr int kGroups = 32 / LPT;               // rows a warp takes at once
  static constexpr int kRowStep = kGroups * kBalWarps;   // rows a CTA takes at once
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

template <typename T, int NL, int LPT>
__global__ void __launch_bounds__(kBalThreads, 1) balance_kernel(const BalanceParams P) {
  using S = BalShape<NL, LPT>;
  extern __shared__ __align__(16) float bal_smem[];
  __shared__ int ok_sh;
  __shared__ float open_sh[kBalWarps];
  __shared__ int redo_sh;
  float* gam = bal_smem;              // [cols] gamma
  float* lb = gam + S::kCols;         // [cols] log2 beta
  float* csum = lb + S::kCols;        // [max(kBalWarps, threads / cols)][cols] partial sums
  float* u_res = csum + kBalWarps * S::kCols;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int l = lane % LPT, grp = lane / LPT;
  const int E = P.experts;
  const float ke = kLog2e / P.eps;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * P.per_cta;
  const int n = static_cast<int>(
      P.rows - row0 < P.per_cta ? (P.rows > row0 ? P.rows - row0 : 0) : P.per_cta);
  float* u_spill = P.spill + static_cast<int64_t>(blockIdx.x) * (P.per_cta - P.resident) * S::kCols;
  const int G = gridDim.x;
  unsigned arrivals = 0;

  // log2 beta, gamma of the start
  if (warp == 0) {
    double tot = 0.0;
    if (P.load)
      for (int j = lane; j < E; j += 32) tot += P.load[j];
    tot = warp_sum(tot);
    for (int j = lane; j < S::kCols; j += 32) {
      float b = 0.0f;
      if (j >= E)
        b = -INFINITY;
      else if (P.load)
        b = static_cast<float>(log2(static_cast<double>(P.load[j]) * E / tot));
      lb[j] = b;
      gam[j] = j < E ? (P.g_init ? P.g_init[j] * ke : 0.0f) + b : -INFINITY;
    }
  }

  // u of the CTA's rows; rows without an open column are counted out
  int open = 0;
  for (int b = warp * S::kGroups; b < n; b += S::kRowStep) {
    const int r = b + grp;
    const bool have = r < n;
    const T* z = static_cast<const T*>(P.z) + (row0 + (have ? r : 0)) * P.ld;
    float v[NL];
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const int j = S::column(l, i);
      v[i] = have && j < E ? Elem<T>::to_f(z[j]) : -INFINITY;
      m = fmaxf(m, v[i]);
    }
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
    // (a row of NaN is open: its NaN reaches every output)
    if (have && l == 0 && m != -INFINITY) ++open;
    if (have) {
      float* dst = r < P.resident ? u_res + static_cast<int64_t>(r) * S::kCols
                                  : u_spill + static_cast<int64_t>(r - P.resident) * S::kCols;
#pragma unroll
      for (int q = 0; q < NL / 4; ++q)
        reinterpret_cast<float4*>(dst)[LPT * q + l] =
            make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
    }
  }
  open = __reduce_add_sync(0xffffffffu, open);
  if (lane == 0) open_sh[warp] = static_cast<float>(open);
  __syncthreads();

  double open_rows = 0.0;
  bool alive = true;
  for (int it = 0; it < P.n_iters && alive; ++it) {
    const bool last = it == P.n_iters - 1;
    float gm[NL], acc[NL];
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      gm[i] = gam[S::column(l, i)];
      acc[i] = 0.0f;
    }
    for (int b = warp * S::kGroups; b < n; b += S::kRowStep) {
      const int r = b + grp;
      const bool have = r < n;
      const int rr = have ? r : b;
      const float* src = rr < P.resident ? u_res + static_cast<int64_t>(rr) * S::kCols
                                         : u_spill + static_cast<int64_t>(rr - P.resident) * S::kCols;
      float t[NL];
      float m = -INFINITY;
#pragma unroll
      for (int q = 0; q < NL / 4; ++q) {
        const float4 x = reinterpret_cast<const float4*>(src)[LPT * q + l];
        t[4 * q] = x.x + gm[4 * q];
        t[4 * q + 1] = x.y + gm[4 * q + 1];
        t[4 * q + 2] = x.z + gm[4 * q + 2];
        t[4 * q + 3] = x.w + gm[4 * q + 3];
        m = max3(m, t[4 * q], t[4 * q + 1]);
        m = max3(m, t[4 * q + 2], t[4 * q + 3]);
      }
      m = group_max<LPT>(m);
      const bool empty = m == -INFINITY;  // no open column (or only NaN, which the sum keeps)
      const float mm = empty ? 0.0f : m;
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < NL; ++i) {
        t[i] = ex2(t[i] - mm);
        sum += t[i];
      }
      sum = group_sum<LPT>(sum);
      const float w = !have || sum == 0.0f ? 0.0f : static_cast<float>(E) / sum;
#pragma unroll
      for (int i = 0; i < NL; ++i) acc[i] = fmaf(t[i], w, acc[i]);
      if (last && have && l == 0)
        P.f[row0 + r] = sum == 0.0f ? 0.0f : -(mm + log2f(sum / static_cast<float>(E))) / ke;
    }
    // the CTA's column sums: rows of a warp, then the warps in their order
#pragma unroll
    for (int i = 0; i < NL; ++i) {
#pragma unroll
      for (int o = LPT; o < 32; o <<= 1) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
      if (grp == 0) csum[warp * S::kCols + S::column(l, i)] = acc[i];
    }
    __syncthreads();
    float* part = P.part + static_cast<int64_t>(it & 1) * G * (S::kCols + 1);
    for (int j = tid; j < S::kCols; j += kBalThreads) {
      float c = 0.0f;
#pragma unroll
      for (int w = 0; w < kBalWarps; ++w) c += csum[w * S::kCols + j];
      part[static_cast<int64_t>(blockIdx.x) * (S::kCols + 1) + j] = c;
    }
    if (tid == 0) {
      float c = 0.0f;
      for (int w = 0; w < kBalWarps; ++w) c += open_sh[w];
      part[static_cast<int64_t>(blockIdx.x) * (S::kCols + 1) + S::kCols] = c;
      redo_sh = 0;
    }
    arrivals += G;
    alive = grid_barrier(P.sync, arrivals, &ok_sh);
    if (!alive) break;
    if (it == 0) {
      for (int q = 0; q < G; ++q)
        open_rows += __ldcg(part + static_cast<int64_t>(q) * (S::kCols + 1) + S::kCols);
      open_rows = fmax(open_rows, 1.0);  // (no open row at all: f = g = 0)
    }
    // every CTA adds all CTAs' sums in the same order
    constexpr int kParts = S::kCols >= kBalThreads ? 1 : (kBalThreads / S::kCols < kBalWarps
                                                              ? kBalThreads / S::kCols
                                                              : kBalWarps);
    for (int w = tid; w < kParts * S::kCols; w += kBalThreads) {
      const int j = w % S::kCols, pt = w / S::kCols;
      float c = 0.0f;
#pragma unroll 8
      for (int q = pt; q < G; q += kParts)
        c += __ldcg(part + static_cast<int64_t>(q) * (S::kCols + 1) + j);
      csum[w] = c;
    }
    __syncthreads();
    for (int j = tid; j < E; j += kBalThreads) {
      float c = 0.0f;
#pragma unroll
      for (int pt = 0; pt < kParts; ++pt) c += csum[pt * S::kCols + j];
      c = static_cast<float>(c / open_rows);
      csum[j] = c;  // (each thread rewrites only what it alone has read: part 0 of its column)
      if (lb[j] == -INFINITY) {
        gam[j] = -INFINITY;  // nothing is wanted of this column
      } else if (c < kBalFlushed) {
        redo_sh = 1;
      } else {
        gam[j] = gam[j] - log2f(c) + lb[j];
      }
    }
    __syncthreads();
    if (redo_sh) {  // the same in every CTA: all have the same sums
      // columns done over in their own range: max and sum of u_ij + phi_i over the rows
      for (int j = tid; j < E; j += kBalThreads) {
        if (lb[j] == -INFINITY || !(csum[j] < kBalFlushed)) continue;
        float cm = -INFINITY, cl = 0.0f;
        for (int r = 0; r < n; ++r) {
          const float* src = r < P.resident ? u_res + static_cast<int64_t>(r) * S::kCols
                                            : u_spill + static_cast<int64_t>(r - P.resident) * S::kCols;
          // phi_i again, from the gammas the rows have seen: gamma + what this update added
          float m = -INFINITY;
          for (int k = 0; k < E; ++k) {
            const float ck = csum[k];
            const float gk = lb[k] == -INFINITY || ck < kBalFlushed ? gam[k] : gam[k] + log2f(ck) - lb[k];
            m = fmaxf(m, src[k] + gk);
          }
          if (m == -INFINITY) continue;
          float sum = 0.0f;
          for (int k = 0; k < E; ++k) {
            const float ck = csum[k];
            const float gk = lb[k] == -INFINITY || ck < kBalFlushed ? gam[k] : gam[k] + log2f(ck) - lb[k];
            sum += ex2(src[k] + gk - m);
          }
          const float x = src[j] - (m + log2f(sum / static_cast<float>(E)));
          if (x > cm) {
            cl = cl * ex2(cm - x) + 1.0f;
            cm = x;
          } else if (x != -INFINITY) {
            cl += ex2(x - cm);
          }
        }
        P.redo[static_cast<int64_t>(blockIdx.x) * S::kCols + j] = make_float2(cm, cl);
      }
      arrivals += G;
      alive = grid_barrier(P.sync, arrivals, &ok_sh);
      if (!alive) break;
      for (int j = tid; j < E; j += kBalThreads) {
        if (lb[j] == -INFINITY || !(csum[j] < kBalFlushed)) continue;
        float cm = -INFINITY, cl = 0.0f;
        for (int q = 0; q < G; ++q) {
          const float2 o = __ldcg(&P.redo[static_cast<int64_t>(q) * S::kCols + j]);
          if (o.x == -INFINITY) continue;
          const float mm = fmaxf(cm, o.x);
          cl = cl * ex2(cm - mm) + o.y * ex2(o.x - mm);
          cm = mm;
        }
        // a column closed to every row keeps g = 0
        gam[j] = cm == -INFINITY ? lb[j]
                                 : -(cm + log2f(static_cast<float>(cl / open_rows))) + lb[j];
      }
      __syncthreads();
    }
  }
  if (!alive) {
    for (int r = tid; r < n; r += kBalThreads) P.f[row0 + r] = __int_as_float(0x7FC00000);
    if (blockIdx.x == 0)
      for (int j = tid; j < E; j += kBalThreads) P.g[j] = __int_as_float(0x7FC00000);
    return;
  }
  if (blockIdx.x == 0)
    for (int j = tid; j < E; j += kBalThreads)
      P.g[j] = lb[j] == -INFINITY ? -INFINITY : (gam[j] - lb[j]) / ke;
}

}  // namespace fs
