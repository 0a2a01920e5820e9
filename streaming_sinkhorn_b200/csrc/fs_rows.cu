// fs_rows.cu -- C ABI of the row-softmax operators on a given score matrix (include/fs.h):
// argument checks, launch plans and launches. Nothing here waits for the device.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "fs_balance.cuh"
#include "fs_host.h"
#include "fs_route.cuh"
#include "fs_tokens.cuh"

namespace fs {
namespace {

constexpr int64_t kMaxInt = 0x7FFFFFFF;
constexpr int32_t kMaxIters = 1000000;  // two arrivals a CTA and iteration stay below 2^32

fs_status check_matrix(const fs_matrix* z) {
  if (!z) return FS_ERR_NULL;
  if (z->dtype < FS_F32 || z->dtype > FS_BF16) return FS_ERR_DTYPE;
  if (z->rows < 0 || z->rows > kMaxInt || z->cols < 1 || z->cols > kMaxInt || z->ld < z->cols ||
      z->ld > (INT64_MAX >> 3) / std::max<int64_t>(z->rows, 1))
    return FS_ERR_SHAPE;
  if (z->rows > 0 && !z->data) return FS_ERR_NULL;
  if (!aligned(z->data, z->dtype == FS_F32 ? 4 : 2)) return FS_ERR_ALIGNMENT;
  return FS_OK;
}

// Calls f with a null pointer of the matrix's element type.
template <typename F>
fs_status by_type(int32_t dtype, F&& f) {
  switch (dtype) {
    case FS_F32: return f(static_cast<float*>(nullptr));
    case FS_F16: return f(static_cast<__half*>(nullptr));
    default: return f(static_cast<__nv_bfloat16*>(nullptr));
  }
}

// CTAs per row of the forward pass. Up to half as many rows as SMs, a row is shared by a cluster,
// which shortens the way through it (128000 bf16: one row 12.7 -> 5.3 us, 16 rows 13.1 -> 6.2),
// while each CTA keeps at least a round of vectors; from there on the rows alone fill the SMs,
// and joining parts costs more than it gains (64 x 50257 fp32, 5 alternatives: 16.8 us with one
// CTA a row, 22.0 with eight).
int token_cluster(int64_t rows, int64_t cols, int vec) {
  const int64_t sms = current_sms();
  int c = 1;
  while (c < kTokenMaxCluster && rows * c * 2 <= sms &&
         cols >= 2ll * c * TokenShape<8>::kRound / kTokenUnroll * vec)
    c *= 2;
  return c;
}

template <typename T, bool TOP, int NW>
fs_status launch_tokens(const TokenParams& P, int cluster, cudaStream_t st) {
  constexpr auto fn = token_logprobs_kernel<T, TOP, NW>;
  static PerDeviceOnce once;
  const fs_status s = once.run("cudaFuncSetAttribute", [&] {
    return cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                TokenShape<NW>::kRing);
  });
  if (s != FS_OK) return s;
  static PerDeviceOccupancy occupancy;
  const int per_sm = occupancy.get(reinterpret_cast<const void*>(fn), NW * 32 + 32,
                                   TokenShape<NW>::kRing);
  const int64_t ctas =
      cluster > 1 ? P.rows * cluster : std::min<int64_t>(P.rows, int64_t(per_sm) * current_sms());
  return launch("fs_token_logprobs", fn, dim3(static_cast<unsigned>(ctas)), NW * 32 + 32,
                TokenShape<NW>::kRing, st, cluster, P, cluster);
}

fs_status token_logprobs(const fs_matrix* z, float eps, const void* ids, int32_t ids_64,
                         int32_t top, float* logp, float* entropy, float* lse, float* stats,
                         float* top_logp, int32_t* top_ids, cudaStream_t st) {
  fs_status s = check_matrix(z);
  if (s != FS_OK) return s;
  if ((s = check_eps(eps)) != FS_OK) return s;
  if (top < 0 || top > FS_MAX_TOP || top > z->cols || (ids_64 != 0 && ids_64 != 1))
    return FS_ERR_OPTION;
  if (z->rows == 0) return FS_OK;
  if (!ids || !logp || !entropy || (top > 0 && (!top_logp || !top_ids))) return FS_ERR_NULL;
  if (!aligned(ids, ids_64 ? 8 : 4) || !aligned(logp, 4) || !aligned(entropy, 4) ||
      !aligned(lse, 4) || !aligned(stats, 8) || !aligned(top_logp, 4) || !aligned(top_ids, 4))
    return FS_ERR_ALIGNMENT;
  TokenParams P{};
  P.z = z->data;
  P.ld = z->ld;
  P.ids = ids;
  P.rows = z->rows;
  P.cols = static_cast<int32_t>(z->cols);
  P.ids_wide = ids_64;
  P.top = top;
  P.inv_eps = 1.0f / eps;
  P.logp = logp;
  P.entropy = entropy;
  P.lse = lse;
  P.stats = reinterpret_cast<float2*>(stats);
  P.top_logp = top_logp;
  P.top_ids = top_ids;
  return by_type(z->dtype, [&](auto* t) -> fs_status {
    using T = std::remove_pointer_t<decltype(t)>;
    const int c = token_cluster(z->rows, z->cols, Elem<T>::kVec);
    // Eight warps on a row; four, which pay a row's fixed costs with twice as many CTAs, where
    // there are many rows (4096 x 65536 bf16 100 us against 105; with 5 alternatives 16384 x 1000
    // bf16 149 against 249). Alternatives have each warp wait for the others more often and want
    // the shorter way up to more rows (1531 x 50257 fp32, 5 of them: 72 us against 86).
    const int64_t many = (top > 0 ? 16ll : 4ll) * current_sms();
    if (top > 0)
      return P.rows * c < many ? launch_tokens<T, true, 8>(P, c, st)
                               : launch_tokens<T, true, 4>(P, c, st);
    return P.rows * c < many ? launch_tokens<T, false, 8>(P, c, st)
                             : launch_tokens<T, false, 4>(P, c, st);
  });
}

fs_status token_logprobs_grad(const fs_matrix* z, float eps, const void* ids, int32_t ids_64,
                              int32_t top, const int32_t* top_ids, const float* stats,
                              const float* entropy, const float* g_logp, const float* g_entropy,
                              const float* g_lse, const float* g_top, void* grad, int64_t ld_grad,
                              cudaStream_t st) {
  fs_status s = check_matrix(z);
  if (s != FS_OK) return s;
  if ((s = check_eps(eps)) != FS_OK) return s;
  if (top < 0 || top > FS_MAX_TOP || top > z->cols || (ids_64 != 0 && ids_64 != 1))
    return FS_ERR_OPTION;
  if (ld_grad < z->cols || ld_grad > (INT64_MAX >> 3) / std::max<int64_t>(z->rows, 1))
    return FS_ERR_SHAPE;
  if (z->rows == 0) return FS_OK;
  if (!ids || !stats || !entropy || !grad || (top > 0 && g_top && !top_ids)) return FS_ERR_NULL;
  if (!aligned(ids, ids_64 ? 8 : 4) || !aligned(stats, 8) || !aligned(entropy, 4) ||
      !aligned(g_logp, 4) || !aligned(g_entropy, 4) || !aligned(g_lse, 4) || !aligned(g_top, 4) ||
      !aligned(top_ids, 4) || !aligned(grad, z->dtype == FS_F32 ? 4 : 2))
    return FS_ERR_ALIGNMENT;
  TokenGradParams P{};
  P.z = z->data;
  P.ld = z->ld;
  P.ids = ids;
  P.rows = z->rows;
  P.cols = static_cast<int32_t>(z->cols);
  P.ids_wide = ids_64;
  P.top = top;
  P.inv_eps = 1.0f / eps;
  P.stats = reinterpret_cast<const float2*>(stats);
  P.entropy = entropy;
  P.top_ids = top_ids;
  P.g_logp = g_logp;
  P.g_entropy = g_entropy;
  P.g_lse = g_lse;
  P.g_top = top > 0 ? g_top : nullptr;
  P.grad = grad;
  P.ld_grad = ld_grad;
  return by_type(z->dtype, [&](auto* t) -> fs_status {
    using T = std::remove_pointer_t<decltype(t)>;
    const int64_t per = static_cast<int64_t>(kTokenGradThreads) * kTokenUnroll * Elem<T>::kVec;
    const int64_t chunks = (z->cols + per - 1) / per;
    if (chunks * z->rows > kMaxInt) return FS_ERR_SHAPE;
    P.chunks = static_cast<int32_t>(chunks);
    return launch("fs_token_logprobs_grad", token_logprobs_grad_kernel<T>,
                  dim3(static_cast<unsigned>(chunks * z->rows)), kTokenGradThreads, 0, st, 1, P);
  });
}

// ---- routing --------------------------------------------------------------------------------

fs_status check_route(const fs_matrix* z, const fs_route_options* o) {
  const fs_status s = check_matrix(z);
  if (s != FS_OK) return s;
  if (!o) return FS_ERR_NULL;
  if (z->cols > FS_MAX_EXPERTS) return FS_ERR_SHAPE;
  if ((o->score != FS_SCORE_SOFTMAX && o->score != FS_SCORE_SIGMOID) || o->groups < 1 ||
      o->groups > kRouteMaxGroups || z->cols % o->groups != 0 || o->top_groups < 1 ||
      o->top_groups > o->groups || o->k < 1 || o->k > FS_MAX_ROUTE_K ||
      o->k > o->top_groups * (z->cols / o->groups) ||
      (o->renormalize != 0 && o->renormalize != 1) || !std::isfinite(o->scale))
    return FS_ERR_OPTION;
  if (!aligned(o->bias, 4)) return FS_ERR_ALIGNMENT;
  return FS_OK;
}

// Experts per lane of a warp, rounded up to one of these.
template <typename F>
fs_status by_width(int64_t experts, F&& f) {
  if (experts <= 32) return f(std::integral_constant<int, 1>());
  if (experts <= 64) return f(std::integral_constant<int, 2>());
  if (experts <= 128) return f(std::integral_constant<int, 4>());
  if (experts <= 160) return f(std::integral_constant<int, 5>());
  if (experts <= 256) return f(std::integral_constant<int, 8>());
  if (experts <= 384) return f(std::integral_constant<int, 12>());
  if (experts <= 512) return f(std::integral_constant<int, 16>());
  return f(std::integral_constant<int, 32>());
}

template <typename T, int NL, bool SIG>
fs_status launch_route(const RouteParams& P, int64_t ctas, size_t smem, cudaStream_t st) {
  constexpr auto fn = route_kernel<T, NL, SIG>;
  static PerDeviceOnce once;
  const fs_status s = once.run("cudaFuncSetAttribute", [&] {
    return cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                FS_MAX_EXPERTS * (kRouteWarps * 8 + 4));
  });
  if (s != FS_OK) return s;
  // with a load to count, CTAs stay and take several rows each, so that few histograms are
  // added up
  if (P.load) {
    static PerDeviceOccupancy occupancy;
    ctas = std::min<int64_t>(
        ctas, int64_t(current_sms()) *
                  occupancy.get(reinterpret_cast<const void*>(fn), kRouteWarps * 32, smem));
  }
  return launch("fs_route", fn, dim3(static_cast<unsigned>(ctas)), kRouteWarps * 32, smem, st, 1,
                P);
}

fs_status route(const fs_matrix* z, const fs_route_options* o, float* weights, int32_t* ids,
                int32_t* load, cudaStream_t st) {
  fs_status s = check_route(z, o);
  if (s != FS_OK) return s;
  if (!aligned(weights, 4) || !aligned(ids, 4) || !aligned(load, 4)) return FS_ERR_ALIGNMENT;
  if (z->rows > 0 && (!weights || !ids)) return FS_ERR_NULL;
  if (load) {
    s = cuda_status(cudaMemsetAsync(load, 0, z->cols * sizeof(int32_t), st), "cudaMemsetAsync");
    if (s != FS_OK) return s;
  }
  if (z->rows == 0) return FS_OK;
  RouteParams P{};
  P.z = z->data;
  P.ld = z->ld;
  P.rows = z->rows;
  P.experts = static_cast<int32_t>(z->cols);
  P.k = o->k;
  P.groups = o->top_groups == o->groups ? 1 : o->groups;  // all groups kept: no groups
  P.per_group = P.experts / P.groups;
  P.top_groups = o->top_groups;
  P.score = o->score;
  P.renorm = o->renormalize;
  P.scale = o->scale;
  P.bias = o->bias;
  P.weights = weights;
  P.ids = ids;
  P.load = load;
  const int64_t ctas = (z->rows + kRouteWarps - 1) / kRouteWarps;  // one warp per row
  const size_t smem = static_cast<size_t>(route_room(P.experts)) * kRouteWarps * sizeof(double) +
                      P.experts * sizeof(int);
  return by_type(z->dtype, [&](auto* t) -> fs_status {
    using T = std::remove_pointer_t<decltype(t)>;
    return by_width(z->cols, [&](auto nl) -> fs_status {
      constexpr int NL = decltype(nl)::value;
      return o->score == FS_SCORE_SIGMOID ? launch_route<T, NL, true>(P, ctas, smem, st)
                                          : launch_route<T, NL, false>(P, ctas, smem, st);
    });
  });
}

fs_status route_grad(const fs_matrix* z, const fs_route_options* o, const float* weights,
                     const int32_t* ids, const float* g_weights, void* grad, cudaStream_t st) {
  const fs_status s = check_route(z, o);
  if (s != FS_OK) return s;
  if (z->rows == 0) return FS_OK;
  if (!weights || !ids || !g_weights || !grad) return FS_ERR_NULL;
  if (!aligned(weights, 4) || !aligned(ids, 4) || !aligned(g_weights, 4) ||
      !aligned(grad, z->dtype == FS_F32 ? 4 : 2))
    return FS_ERR_ALIGNMENT;
  RouteGradParams P{};
  P.z = z->data;
  P.ld = z->ld;
  P.rows = z->rows;
  P.experts = static_cast<int32_t>(z->cols);
  P.k = o->k;
  P.score = o->score;
  P.renorm = o->renormalize;
  P.scale = o->scale;
  P.weights = weights;
  P.ids = ids;
  P.g_weights = g_weights;
  P.grad = grad;
  const int64_t ctas = (z->rows + kRouteWarps - 1) / kRouteWarps;
  return by_type(z->dtype, [&](auto* t) -> fs_status {
    using T = std::remove_pointer_t<decltype(t)>;
    return by_width(z->cols, [&](auto nl) -> fs_status {
      return launch("fs_route_grad", route_grad_kernel<T, decltype(nl)::value>,
                    dim3(static_cast<unsigned>(ctas)), kRouteWarps * 32, 0, st, 1, P);
    });
  });
}

// ---- balancing ------------------------------------------------------------------------------

// The launch of one problem: lanes per row, CTAs, and what fits in shared memory.
struct BalancePlan {
  int nl, lpt, nw, cols;
  bool cluster;  // one cluster, everything in shared memory
  int ctas, per_cta, resident;
  size_t smem;
  size_t off_redo, off_spill, total;  // workspace: sync word, column sums, redo, spill
};

constexpr size_t kBalSmemBudget = 224u * 1024u;  // of 227 KB; the static part is 300 bytes

// (balance_plan says why)
constexpr int64_t kBalClusterScores = 660 * 1000, kBalClusterRows = 680;

BalancePlan balance_plan(int64_t rows, int64_t experts, bool allow_cluster) {
  BalancePlan p{};
  p.nl = experts <= 256 ? 8 : experts <= 512 ? 16 : 32;
  p.lpt = 1;
  while (p.nl * p.lpt < experts) p.lpt *= 2;
  p.cols = p.nl * p.lpt;
  const size_t cluster_fixed =
      static_cast<size_t>(3 + kBalClusterWarps) * p.cols * 4 + 2ull * kBalMaxCluster * (p.cols + 4) * 4;
  const size_t row = static_cast<size_t>(p.cols) * 4;
  const int64_t step = (32 / p.lpt) * kBalClusterWarps;  // rows a CTA takes at once
  auto spread = [&](int64_t ctas) {
    const int64_t per = std::max<int64_t>(1, (rows + ctas - 1) / ctas);
    p.per_cta = static_cast<int>(per);
    p.ctas = static_cast<int>(std::max<int64_t>(1, (rows + per - 1) / per));
  };
  // A cluster exchanges its sums in less time than the grid's 4 us an iteration, but has only 16
  // SMs: it is taken, with fewer CTAs for fewer rows, while the exponentials of one iteration on
  // those take less than what it saves, and shared memory holds them. Wide rows reach that sooner
  // (10 iterations, us, cluster and grid: 512 x 16 23 and 48, 2048 x 64 30 and 51, 1000 x 256 43 and
  // 53, 1600 x 256 51 and 55, 2000 x 256 55 and 54, 4000 x 128 50 and 53, 5000 x 128 55 and 53,
  // 8191 x 64 47 and 51, 9000 x 64 52 and 53, 12000 x 64 59 and 53, 40000 x 16 50 and 52).
  p.cluster = false;
  if (allow_cluster && p.nl == 8 && (rows + kBalClusterRows) * p.cols <= kBalClusterScores) {
    for (int c = 1; c <= kBalMaxCluster && !p.cluster; c *= 2) {
      if (c < kBalMaxCluster && rows > 2 * step * c) continue;
      if ((rows + c - 1) / c * row + cluster_fixed > kBalSmemBudget) continue;
      p.cluster = true;
      // (a cluster launch wants all of its CTAs, empty ones too)
      p.per_cta = static_cast<int>(std::max<int64_t>(1, (rows + c - 1) / c));
      p.ctas = c;
    }
  }
  if (!p.cluster)
    spread(std::max<int64_t>(1, std::min<int64_t>((rows + 2 * step - 1) / (2 * step), current_sms())));
  // The grid's CTAs have many rows each and hide their latencies with more warps, where the
  // registers allow it.
  p.nw = p.cluster || p.nl > 8 ? kBalClusterWarps : kBalGridWarps;
  const size_t used = p.cluster ? cluster_fixed : static_cast<size_t>(3 + p.nw) * p.cols * 4;
  p.resident = static_cast<int>(std::min<int64_t>(p.per_cta, (kBalSmemBudget - used) / row));
  p.smem = used + p.resident * row;
  auto up = [](size_t v) { return (v + 255) & ~static_cast<size_t>(255); };
  p.off_redo = 256 + up(3 * static_cast<size_t>(bal_sums(p.cols)) * sizeof(u64));
  p.off_spill = p.off_redo + up(static_cast<size_t>(p.ctas) * p.cols * 8);
  p.total = p.off_spill + up(static_cast<size_t>(p.ctas) * (p.per_cta - p.resident) * row);
  return p;
}

fs_status check_balance(const fs_matrix* z) {
  const fs_status s = check_matrix(z);
  if (s != FS_OK) return s;
  return z->cols > FS_MAX_EXPERTS ? FS_ERR_SHAPE : FS_OK;
}

template <typename F>
fs_status by_shape(const BalancePlan& p, F&& f) {
  using std::integral_constant;
  if (p.nl == 16) return f(integral_constant<int, 16>(), integral_constant<int, 32>());
  if (p.nl == 32) return f(integral_constant<int, 32>(), integral_constant<int, 32>());
  switch (p.lpt) {
    case 1: return f(integral_constant<int, 8>(), integral_constant<int, 1>());
    case 2: return f(integral_constant<int, 8>(), integral_constant<int, 2>());
    case 4: return f(integral_constant<int, 8>(), integral_constant<int, 4>());
    case 8: return f(integral_constant<int, 8>(), integral_constant<int, 8>());
    case 16: return f(integral_constant<int, 8>(), integral_constant<int, 16>());
    default: return f(integral_constant<int, 8>(), integral_constant<int, 32>());
  }
}

// Whether the current device can run a cluster of 16 CTAs with all of the shared memory (asked
// once per device, of one of the kernels: all have the same block and budget).
bool cluster_runs() {
  static std::atomic<int> known[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) return false;
  int k = known[dev].load(std::memory_order_relaxed);
  if (k == 0) {
    constexpr auto fn = balance_kernel<float, 8, 8, kBalClusterWarps, true>;
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = kBalMaxCluster;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(kBalMaxCluster);
    cfg.blockDim = dim3(kBalClusterWarps * 32);
    cfg.dynamicSmemBytes = kBalSmemBudget;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    int n = 0;
    const bool ok =
        cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(kBalSmemBudget)) == cudaSuccess &&
        cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
        cudaOccupancyMaxActiveClusters(&n, fn, &cfg) == cudaSuccess && n > 0;
    cudaGetLastError();
    k = ok ? 1 : -1;
    known[dev].store(k, std::memory_order_relaxed);
  }
  return k > 0;
}

template <typename T, int NL, int LPT, int NW, bool CLUSTER>
fs_status launch_balance(const BalanceParams& P, const BalancePlan& p, cudaStream_t st) {
  constexpr auto fn = balance_kernel<T, NL, LPT, NW, CLUSTER>;
  static PerDeviceOnce once;
  const fs_status s = once.run("cudaFuncSetAttribute", [&] {
    const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(kBalSmemBudget));
    if (e != cudaSuccess || !CLUSTER) return e;
    return cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  });
  if (s != FS_OK) return s;
  return launch("fs_balance", fn, dim3(static_cast<unsigned>(p.ctas)), NW * 32, p.smem, st,
                CLUSTER ? p.ctas : kCooperative, P);
}

fs_status balance(const fs_matrix* z, int32_t score, float eps, int32_t n_iters, const float* load,
                  const float* g_init, float* f, float* g, void* ws, size_t ws_bytes,
                  cudaStream_t st) {
  fs_status s = check_balance(z);
  if (s != FS_OK) return s;
  if ((s = check_eps(eps)) != FS_OK) return s;
  if (score != FS_SCORE_SOFTMAX && score != FS_SCORE_SIGMOID) return FS_ERR_OPTION;
  if (n_iters < 1 || n_iters > kMaxIters) return FS_ERR_ITERS;
  if (z->rows == 0) return FS_OK;
  if (!f || !g) return FS_ERR_NULL;
  if (!aligned(load, 4) || !aligned(g_init, 4) || !aligned(f, 4) || !aligned(g, 4))
    return FS_ERR_ALIGNMENT;
  BalancePlan p = balance_plan(z->rows, z->cols, true);
  if (p.cluster && !cluster_runs()) p = balance_plan(z->rows, z->cols, false);
  if (!ws || !aligned(ws, 256) || ws_bytes < p.total) return FS_ERR_WORKSPACE;
  unsigned char* base = static_cast<unsigned char*>(ws);
  BalanceParams P{};
  P.z = z->data;
  P.ld = z->ld;
  P.rows = z->rows;
  P.experts = static_cast<int32_t>(z->cols);
  P.cols = p.cols;
  P.score = score;
  P.n_iters = n_iters;
  P.per_cta = p.per_cta;
  P.resident = p.resident;
  P.eps = eps;
  P.load = load;
  P.g_init = g_init;
  P.f = f;
  P.g = g;
  P.sync = reinterpret_cast<unsigned*>(base);
  P.sums = reinterpret_cast<u64*>(base + 256);
  P.redo = reinterpret_cast<float2*>(base + p.off_redo);
  P.spill = reinterpret_cast<float*>(base + p.off_spill);
  if (!p.cluster) {  // the grid barrier's word and the column sums
    s = cuda_status(cudaMemsetAsync(base, 0, p.off_redo, st), "cudaMemsetAsync");
    if (s != FS_OK) return s;
  }
  return by_type(z->dtype, [&](auto* t) -> fs_status {
    using T = std::remove_pointer_t<decltype(t)>;
    return by_shape(p, [&](auto nl, auto lpt) -> fs_status {
      constexpr int NL = decltype(nl)::value, LPT = decltype(lpt)::value;
      if constexpr (NL == 8)
        if (p.cluster) return launch_balance<T, NL, LPT, kBalClusterWarps, true>(P, p, st);
      return launch_balance<T, NL, LPT, NL == 8 ? kBalGridWarps : kBalClusterWarps, false>(P, p, st);
    });
  });
}

}  // namespace
}  // namespace fs

extern "C" {

fs_status fs_token_logprobs(const fs_matrix* z, float eps, const void* ids, int32_t ids_64,
                            int32_t top, float* logp, float* entropy, float* lse, float* stats,
                            float* top_logp, int32_t* top_ids, fs_stream_t stream) {
  return fs::token_logprobs(z, eps, ids, ids_64, top, logp, entropy, lse, stats, top_logp, top_ids,
                            reinterpret_cast<cudaStream_t>(stream));
}

fs_status fs_token_logprobs_grad(const fs_matrix* z, float eps, const void* ids, int32_t ids_64,
                                 int32_t top, const int32_t* top_ids, const float* stats,
                                 const float* entropy, const float* g_logp, const float* g_entropy,
                                 const float* g_lse, const float* g_top, void* grad,
                                 int64_t ld_grad, fs_stream_t stream) {
  return fs::token_logprobs_grad(z, eps, ids, ids_64, top, top_ids, stats, entropy, g_logp,
                                 g_entropy, g_lse, g_top, grad, ld_grad,
                                 reinterpret_cast<cudaStream_t>(stream));
}

fs_status fs_route(const fs_matrix* z, const fs_route_options* opt, float* weights, int32_t* ids,
                   int32_t* load, fs_stream_t stream) {
  return fs::route(z, opt, weights, ids, load, reinterpret_cast<cudaStream_t>(stream));
}

fs_status fs_route_grad(const fs_matrix* z, const fs_route_options* opt, const float* weights,
                        const int32_t* ids, const float* g_weights, void* grad,
                        fs_stream_t stream) {
  return fs::route_grad(z, opt, weights, ids, g_weights, grad,
                        reinterpret_cast<cudaStream_t>(stream));
}

size_t fs_balance_workspace_bytes(const fs_matrix* z) {
  if (!z || z->rows < 0 || z->rows > fs::kMaxInt || z->cols < 1 || z->cols > FS_MAX_EXPERTS)
    return 0;
  return std::max(fs::balance_plan(z->rows, z->cols, true).total,
                  fs::balance_plan(z->rows, z->cols, false).total);
}

fs_status fs_balance(const fs_matrix* z, int32_t score, float eps, int32_t n_iters,
                     const float* load, const float* g_init, float* f, float* g, void* ws,
                     size_t ws_bytes, fs_stream_t stream) {
  return fs::balance(z, score, eps, n_iters, load, g_init, f, g, ws, ws_bytes,
                     reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
