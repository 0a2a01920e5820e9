// fs_linear.cu -- C ABI of fs_linear_logprobs and its gradient (include/fs.h): argument checks,
// tensor maps, launch plans and launches. Nothing here waits for the device.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "fs_host.h"
#include "fs_linear.cuh"

namespace fs {
namespace {

constexpr int64_t kMaxInt = 0x7FFFFFFF;
constexpr size_t kHeader = 256;  // the error word
// Most bytes of G in the workspace; a larger one is made in chunks of columns.
constexpr int64_t kMaxG = int64_t(1) << 30;

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t round_up(int64_t a, int64_t b) { return ceil_div(a, b) * b; }

fs_status check_operand(const fs_matrix* m) {
  if (!m) return FS_ERR_NULL;
  // bf16 only: the gradient of a softmax falls below fp16's range, and fp32 operands have no
  // tensor-core product that keeps their bits
  if (m->dtype != FS_BF16) return FS_ERR_DTYPE;
  if (m->rows < 0 || m->rows > kMaxInt - 512 || m->cols < 1 || m->cols > (1 << 20) ||
      m->ld < m->cols || m->ld > (int64_t(1) << 36))
    return FS_ERR_SHAPE;
  if (m->rows > 0 && !m->data) return FS_ERR_NULL;
  // TMA: 16-byte aligned base and row stride
  if (!aligned(m->data, 16) || m->ld % 8 != 0) return FS_ERR_ALIGNMENT;
  return FS_OK;
}

fs_status check_pair(const fs_matrix* x, const fs_matrix* w, float eps) {
  fs_status s = check_operand(x);
  if (s != FS_OK) return s;
  if ((s = check_operand(w)) != FS_OK) return s;
  if (x->cols != w->cols || w->rows < 1) return FS_ERR_SHAPE;
  return check_eps(eps);
}

typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                             const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                             const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                             CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// cuTensorMapEncodeTiled by way of the runtime, so that the library needs no libcuda to load.
fs_status encode_fn(EncodeFn* out) {
  static std::atomic<void*> cached{nullptr};
  void* p = cached.load(std::memory_order_acquire);
  if (!p) {
    cudaDriverEntryPointQueryResult q;
    const fs_status s =
        cuda_status(cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000,
                                                     cudaEnableDefault, &q),
                    "cudaGetDriverEntryPointByVersion");
    if (s != FS_OK) return s;
    if (q != cudaDriverEntryPointSuccess || !p) {
      record_cuda_error("cuTensorMapEncodeTiled", cudaErrorSymbolNotFound);
      return FS_ERR_CUDA;
    }
    cached.store(p, std::memory_order_release);
  }
  *out = reinterpret_cast<EncodeFn>(p);
  return FS_OK;
}

// A (rows, cols) bf16 matrix read in boxes of 64 columns (128 bytes, swizzled) x box_rows rows;
// what lies outside reads as zero.
fs_status make_map(CUtensorMap* map, const void* data, int64_t rows, int64_t cols, int64_t ld,
                   int box_rows) {
  EncodeFn fn;
  const fs_status s = encode_fn(&fn);
  if (s != FS_OK) return s;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld) * 2};
  const cuuint32_t box[2] = {64, static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t step[2] = {1, 1};
  const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(data), dims,
                        strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) {
    record_cuda_error("cuTensorMapEncodeTiled", cudaErrorInvalidValue);
    return FS_ERR_CUDA;
  }
  return FS_OK;
}

// The two maps of a K-major A (its row blocks, and the last of them) and that block's rows.
fs_status make_rows_maps(CUtensorMap* map, CUtensorMap* tail, uint32_t* tail_rows,
                         const void* data, int64_t rows, int64_t cols, int64_t ld) {
  *tail_rows = static_cast<uint32_t>(rows - (ceil_div(rows, kLinM) - 1) * kLinM);
  const fs_status s = make_map(map, data, rows, cols, ld, kLinM);
  return s != FS_OK ? s : make_map(tail, data, rows, cols, ld, static_cast<int>(*tail_rows));
}

template <int BN, int CG, bool A_MN, bool B_MN, int EPI>
fs_status launch_linear(const char* what, const CUtensorMap& a, const CUtensorMap& tail,
                        const CUtensorMap& b, const LinParams& P, int sms, cudaStream_t st) {
  constexpr auto fn = linear_kernel<BN, CG, A_MN, B_MN, EPI>;
  static PerDeviceOnce once;
  const fs_status s = once.run("cudaFuncSetAttribute", [&] {
    return cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(LinShape<BN, CG>::SMEM));
  });
  if (s != FS_OK) return s;
  const int64_t grid = std::min<int64_t>(P.units, sms / CG) * CG;
  return launch(what, fn, dim3(static_cast<unsigned>(grid)), kLinThreads, LinShape<BN, CG>::SMEM,
                st, CG, a, tail, b, P);
}

// CTAs that share a tile of a product with this many rows: pairs once a pair has rows for both.
int pair_of(int64_t rows) { return rows > kLinM ? 2 : 1; }

// Width of a tile of scores. One row block reads w once and is bound by that read: narrow tiles
// spread it evenly over the SMs. More row blocks are bound by the products: wide tiles.
int tile_of(int cg) { return cg == 1 ? 128 : 256; }

// The factor that scores are multiplied by to put back what their accumulators' cuts take. Each cut
// (one for 16 products) is towards 0 and takes a share of the sum so far; where sums grow evenly
// along K that is half of the score on average, so a score of n cuts comes out too small by n times
// a constant of itself, 2^-23 / 8 as measured (1024 x 16000, dims 256 to 4096: mean error of the
// log-sum-exp over what this predicts 0.93 to 1.03). Relative error of the log-sum-exp and of the
// entropy at 4096: 8.2e-7 and 1.1e-6 without, 4.3e-8 and 7.5e-8 with it, as in fp32; with most of a
// score in 8 products at the beginning, the middle or the end of K the log-sum-exp's 2.7e-6, 1.5e-6,
// 3.5e-7 without and 1.3e-6, 1.2e-7, 1.1e-6 with it.
float uncut(int64_t dim, int cg) {
  const double accumulators = cg == 1 ? 2.0 : 1.0;
  const double cuts = static_cast<double>(ceil_div(dim, 16)) / accumulators;
  return static_cast<float>(1.0 + cuts * 0x1p-23 / 8);
}

// The forward pass: tile width, column tiles of a unit, and how many units share a row block.
struct ForwardPlan {
  int bn;
  int cg;  // CTAs of a tile
  int64_t m_blocks, n_blocks, per_unit, splits;
  int64_t m_pad;
  size_t off_given, total;
};

ForwardPlan forward_plan(int64_t rows, int64_t cols, int sms) {
  ForwardPlan p{};
  p.cg = pair_of(rows);
  p.m_blocks = ceil_div(rows, kLinM * p.cg);
  p.bn = tile_of(p.cg);
  p.n_blocks = ceil_div(cols, p.bn);
  // The split of the columns whose last wave is fullest, of those that fill 1 .. 16 waves; ties go
  // to fewer parts.
  const int workers = sms / p.cg;
  const double even = static_cast<double>(p.m_blocks * p.n_blocks) / workers;
  double best = 0.0;
  p.per_unit = p.n_blocks;
  for (int64_t wave = 1; wave <= 16; ++wave) {
    const int64_t splits = std::max<int64_t>(1, workers * wave / p.m_blocks);
    const int64_t per = ceil_div(p.n_blocks, std::min(splits, p.n_blocks));
    const int64_t units = p.m_blocks * ceil_div(p.n_blocks, per);
    // an even share, against the tiles that the busiest worker takes
    const double eff = even / static_cast<double>(ceil_div(units, workers) * per);
    if (eff > best + 1e-3) {
      best = eff;
      p.per_unit = per;
    }
    if (per == 1) break;
  }
  p.splits = ceil_div(p.n_blocks, p.per_unit);
  p.m_pad = p.m_blocks * kLinM * p.cg;
  p.off_given = kHeader + static_cast<size_t>(2 * p.splits * p.m_pad) * sizeof(float4);
  p.total = round_up(p.off_given + static_cast<size_t>(p.m_pad) * 4, 256);
  return p;
}

// The gradient: columns of a chunk of G, and the K splits of dx.
struct BackwardPlan {
  int64_t chunk, chunks, ld_g, splits;
  int64_t n_keys;  // of the sort: a power of two, at least the entries (2 a row)
  int64_t ld_x;    // of the states copied for dw
  size_t off_flags, off_x, off_keys, off_g, off_acc, total;
};

BackwardPlan backward_plan(int64_t rows, int64_t cols, int64_t dim, int sms) {
  BackwardPlan p{};
  const int64_t cap = std::max<int64_t>(256, kMaxG / (2 * rows) / 256 * 256);
  p.chunks = ceil_div(cols, cap);
  p.chunk = std::min(round_up(ceil_div(cols, p.chunks), 256), cap);
  p.chunks = ceil_div(cols, p.chunk);
  p.ld_g = round_up(std::min(p.chunk, cols), 256);
  // dx has few tiles and a long K: split K so that the last wave is full, counting the write
  // and read of each split's fp32 partial sums (about 1 K step per 2^16 floats and SM)
  const int cg = pair_of(rows);
  const int64_t tiles = ceil_div(rows, kLinM * cg) * ceil_div(dim, 256);
  const int workers = sms / cg;
  const int64_t k_steps = ceil_div(std::min(p.chunk, cols), kLinK);
  double best = 0.0;
  p.splits = 1;
  for (int64_t s = 1; s <= 64 && s <= std::max<int64_t>(1, k_steps / 8); ++s) {
    const double product =
        static_cast<double>(ceil_div(tiles * s, workers)) * static_cast<double>(ceil_div(k_steps, s));
    const double sums = s > 1 ? static_cast<double>(s) * rows * dim * 8.0 / 6.0e12 / 2.8e-7 : 0.0;
    const double cost = product + sums;
    if (s == 1 || cost < best) {
      best = cost;
      p.splits = s;
    }
  }
  p.n_keys = 32;
  while (p.n_keys < 2 * rows) p.n_keys *= 2;
  p.off_flags = kHeader + round_up(static_cast<size_t>(rows) * 2 * sizeof(LinRest), 256);
  p.ld_x = round_up(dim, 8);
  p.off_x = p.off_flags + round_up(std::min(p.chunk, cols), 256);
  p.off_keys = p.off_x + round_up(static_cast<size_t>(rows) * p.ld_x * 2, 256);
  p.off_g = p.off_keys + round_up(p.n_keys * sizeof(uint64_t), 256);
  p.off_acc = p.off_g + round_up(static_cast<size_t>(rows) * p.ld_g * 2, 256);
  const bool partial = p.splits > 1 || p.chunks > 1;
  p.total = round_up(p.off_acc + (partial ? static_cast<size_t>(p.splits) * rows * dim * 4 : 0), 256);
  return p;
}

// The entries of a chunk's columns that dw adds in fp32, in order, and their sums (fs_linear.cuh).
fs_status rests(const BackwardPlan& p, const LinRest* rest, int64_t rows, int64_t col0, int64_t n,
                const fs_matrix* x, uint64_t* keys, uint8_t* has_rest, __nv_bfloat16* gw, int sms,
                cudaStream_t st) {
  const char* what = "fs_linear_logprobs_grad (order)";
  const int64_t entries = 2 * rows;
  fs_status s;
  if (p.n_keys <= kSortSmem) {
    s = launch(what, linear_order_kernel, dim3(1), kSortBlock, 0, st, 1, rest, entries, col0, n,
               keys, static_cast<int>(p.n_keys));
  } else {
    const dim3 each(static_cast<unsigned>(ceil_div(p.n_keys, 256)));
    s = launch(what, linear_keys_kernel, each, 256, 0, st, 1, rest, entries, col0, n, keys, p.n_keys);
    const dim3 blocks(static_cast<unsigned>(p.n_keys / kSortSmem));
    const dim3 pairs(static_cast<unsigned>(p.n_keys / 2 / 256));
    if (s == FS_OK)
      s = launch(what, bitonic_smem_kernel, blocks, kSortBlock, 0, st, 1, keys, int64_t(0));
    for (int64_t k = 2 * kSortSmem; s == FS_OK && k <= p.n_keys; k <<= 1) {
      for (int64_t j = k / 2; s == FS_OK && j >= kSortSmem; j >>= 1)
        s = launch(what, bitonic_global_kernel, pairs, 256, 0, st, 1, keys, p.n_keys, k, j);
      if (s == FS_OK) s = launch(what, bitonic_smem_kernel, blocks, kSortBlock, 0, st, 1, keys, k);
    }
  }
  if (s != FS_OK) return s;
  const int64_t ctas = std::min<int64_t>(ceil_div(entries, 8), int64_t(8) * sms);
  return launch("fs_linear_logprobs_grad (rests)", linear_rests_kernel,
                dim3(static_cast<unsigned>(ctas), static_cast<unsigned>(ceil_div(x->cols, 256))), 256,
                0, st, 1, static_cast<const uint64_t*>(keys), p.n_keys, rest,
                static_cast<const __nv_bfloat16*>(x->data), x->ld, x->cols, gw, has_rest);
}

bool shape_ok(const fs_matrix* x, const fs_matrix* w) {
  return x && w && x->rows >= 0 && x->rows <= kMaxInt - 512 && w->rows >= 1 &&
         w->rows <= kMaxInt - 512 && x->cols == w->cols && x->cols >= 1 && x->cols <= (1 << 20);
}

fs_status forward(const fs_matrix* x, const fs_matrix* w, float eps, const void* ids,
                  int32_t ids_64, float* logp, float* entropy, float* lse, float* stats, void* ws,
                  size_t ws_bytes, cudaStream_t st) {
  fs_status s = check_pair(x, w, eps);
  if (s != FS_OK) return s;
  if (ids_64 != 0 && ids_64 != 1) return FS_ERR_OPTION;
  if (x->rows == 0) return FS_OK;
  if (!ids || !logp || !entropy) return FS_ERR_NULL;
  if (!aligned(ids, ids_64 ? 8 : 4) || !aligned(logp, 4) || !aligned(entropy, 4) ||
      !aligned(lse, 4) || !aligned(stats, 8))
    return FS_ERR_ALIGNMENT;
  const int sms = current_sms();
  const ForwardPlan p = forward_plan(x->rows, w->rows, sms);
  if (!ws || !aligned(ws, 256) || ws_bytes < p.total) return FS_ERR_WORKSPACE;
  unsigned char* base = static_cast<unsigned char*>(ws);
  unsigned* err = reinterpret_cast<unsigned*>(base);
  float4* part = reinterpret_cast<float4*>(base + kHeader);
  float* given = reinterpret_cast<float*>(base + p.off_given);
  const float inv_eps = 1.0f / eps;
  s = cuda_status(cudaMemsetAsync(base, 0, kHeader, st), "cudaMemsetAsync");
  if (s != FS_OK) return s;
  CUtensorMap ma, mt, mb;
  LinParams P{};
  s = make_rows_maps(&ma, &mt, &P.tail_rows, x->data, x->rows, x->cols, x->ld);
  if (s != FS_OK) return s;
  if ((s = make_map(&mb, w->data, w->rows, w->cols, w->ld, p.bn / p.cg)) != FS_OK) return s;
  P.m = x->rows;
  P.n = w->rows;
  P.k_steps = static_cast<int32_t>(ceil_div(x->cols, kLinK));
  P.m_blocks = static_cast<int32_t>(p.m_blocks);
  P.n_blocks = static_cast<int32_t>(p.n_blocks);
  P.n_per_unit = static_cast<int32_t>(p.per_unit);
  P.k_splits = 1;
  P.units = p.m_blocks * p.splits;
  P.err = err;
  P.inv_eps = inv_eps;
  P.uncut = uncut(x->cols, p.cg);
  P.ids = ids;
  P.ids_wide = ids_64;
  P.part = part;
  P.given = given;
  P.parts = 2 * p.splits;
  P.cols = w->rows;
  P.last_block = static_cast<int32_t>(ceil_div(x->rows, kLinM) - 1);
  s = p.cg == 1
          ? launch_linear<128, 1, false, false, kLinLse>("fs_linear_logprobs", ma, mt, mb, P, sms, st)
          : launch_linear<256, 2, false, false, kLinLse>("fs_linear_logprobs", ma, mt, mb, P, sms, st);
  if (s != FS_OK) return s;
  LinJoinParams J{};
  J.x = static_cast<const __nv_bfloat16*>(x->data);
  J.w = static_cast<const __nv_bfloat16*>(w->data);
  J.ld_x = x->ld;
  J.ld_w = w->ld;
  J.dim = x->cols;
  J.part = part;
  J.given = given;
  J.parts = P.parts;
  J.m = x->rows;
  J.cols = w->rows;
  J.ids = ids;
  J.ids_wide = ids_64;
  J.inv_eps = inv_eps;
  J.err = err;
  J.logp = logp;
  J.entropy = entropy;
  J.lse = lse;
  J.stats = reinterpret_cast<float2*>(stats);
  const char* what = "fs_linear_logprobs (join)";
  if (x->rows <= sms)  // a CTA each
    return launch(what, linear_join_kernel<8>, dim3(static_cast<unsigned>(x->rows)), 256, 0, st, 1,
                  J);
  return launch(what, linear_join_kernel<1>, dim3(static_cast<unsigned>(ceil_div(x->rows, 8))), 256,
                0, st, 1, J);
}

fs_status backward(const fs_matrix* x, const fs_matrix* w, float eps, const void* ids,
                   int32_t ids_64, const float* stats, const float* entropy, const float* g_logp,
                   const float* g_entropy, const float* g_lse, void* grad_x, void* grad_w, void* ws,
                   size_t ws_bytes, cudaStream_t st) {
  fs_status s = check_pair(x, w, eps);
  if (s != FS_OK) return s;
  if (ids_64 != 0 && ids_64 != 1) return FS_ERR_OPTION;
  if (!aligned(grad_x, 2) || !aligned(grad_w, 2)) return FS_ERR_ALIGNMENT;
  const int64_t rows = x->rows, cols = w->rows, dim = x->cols;
  if (rows == 0) {
    if (!grad_w) return FS_OK;
    return cuda_status(cudaMemsetAsync(grad_w, 0, static_cast<size_t>(cols) * dim * 2, st),
                       "cudaMemsetAsync");
  }
  if (!ids || !stats || !entropy) return FS_ERR_NULL;
  if (!aligned(ids, ids_64 ? 8 : 4) || !aligned(stats, 8) || !aligned(entropy, 4) ||
      !aligned(g_logp, 4) || !aligned(g_entropy, 4) || !aligned(g_lse, 4))
    return FS_ERR_ALIGNMENT;
  if (!grad_x && !grad_w) return FS_OK;
  const int sms = current_sms();
  const BackwardPlan p = backward_plan(rows, cols, dim, sms);
  if (!ws || !aligned(ws, 256) || ws_bytes < p.total) return FS_ERR_WORKSPACE;
  unsigned char* base = static_cast<unsigned char*>(ws);
  unsigned* err = reinterpret_cast<unsigned*>(base);
  LinRest* rest = reinterpret_cast<LinRest*>(base + kHeader);
  uint8_t* has_rest = base + p.off_flags;
  uint64_t* keys = reinterpret_cast<uint64_t*>(base + p.off_keys);
  __nv_bfloat16* G = reinterpret_cast<__nv_bfloat16*>(base + p.off_g);
  float* acc = reinterpret_cast<float*>(base + p.off_acc);
  const bool partial = p.splits > 1 || p.chunks > 1;
  __nv_bfloat16* gx = static_cast<__nv_bfloat16*>(grad_x);
  __nv_bfloat16* gw = static_cast<__nv_bfloat16*>(grad_w);
  // the error word, the rows' entries (none yet) and the tokens' flags
  s = cuda_status(cudaMemsetAsync(base, 0, p.off_x, st), "cudaMemsetAsync");
  if (s != FS_OK) return s;
  const __nv_bfloat16* wd = static_cast<const __nv_bfloat16*>(w->data);
  // dw's operand: the states of the rows that are asked about. (A row that is not has G = 0, but 0
  // times what a batch's padding may hold need not be 0.)
  __nv_bfloat16* xm = reinterpret_cast<__nv_bfloat16*>(base + p.off_x);
  if (gw) {
    const int64_t vecs = rows * (p.ld_x / 8);
    s = launch("fs_linear_logprobs_grad (states)", linear_asked_kernel,
               dim3(static_cast<unsigned>(std::min<int64_t>(ceil_div(vecs, 256), int64_t(16) * sms))),
               256, 0, st, 1, static_cast<const __nv_bfloat16*>(x->data), x->ld, rows, dim, ids,
               ids_64, xm, p.ld_x);
    if (s != FS_OK) return s;
  }
  const int cg = pair_of(rows);
  // the scores' tiles are the forward pass's, so that each score is cut in the same places and p
  // goes with the row's sums (states of 4096, a token with all but 5e-5 of the probability: 1 - p
  // was off by more than itself where a lone row block's scores were formed in wider tiles)
  const int bn = tile_of(cg);
  for (int64_t c = 0; c < p.chunks; ++c) {
    const int64_t col0 = c * p.chunk;
    const int64_t n = std::min(p.chunk, cols - col0);
    CUtensorMap ma, mt, mb;
    // G of the chunk: the scores again, and their gradient in the epilogue
    LinParams P{};
    s = make_rows_maps(&ma, &mt, &P.tail_rows, x->data, rows, dim, x->ld);
    if (s != FS_OK) return s;
    if ((s = make_map(&mb, wd + col0 * w->ld, n, dim, w->ld, bn / cg)) != FS_OK) return s;
    P.m = rows;
    P.n = n;
    P.k_steps = static_cast<int32_t>(ceil_div(dim, kLinK));
    P.m_blocks = static_cast<int32_t>(ceil_div(rows, kLinM * cg));
    P.last_block = static_cast<int32_t>(ceil_div(rows, kLinM) - 1);
    P.n_blocks = static_cast<int32_t>(ceil_div(n, bn));
    P.n_per_unit = 1;
    P.k_splits = 1;
    P.units = static_cast<int64_t>(P.m_blocks) * P.n_blocks;
    P.err = err;
    P.inv_eps = 1.0f / eps;
    P.uncut = uncut(dim, cg);
    P.ids = ids;
    P.ids_wide = ids_64;
    P.col0 = col0;
    P.cols = cols;
    P.stats = reinterpret_cast<const float2*>(stats);
    P.entropy = entropy;
    P.g_logp = g_logp;
    P.g_entropy = g_entropy;
    P.g_lse = g_lse;
    P.g_out = G;
    P.ld_g = p.ld_g;
    P.rest = rest;
    const char* what = "fs_linear_logprobs_grad (scores)";
    s = cg == 1 ? launch_linear<128, 1, false, false, kLinScoreGrad>(what, ma, mt, mb, P, sms, st)
                : launch_linear<256, 2, false, false, kLinScoreGrad>(what, ma, mt, mb, P, sms, st);
    if (s != FS_OK) return s;
    if (gx) {  // dx = G w: K runs along G's rows and down w's
      LinParams Q{};
      s = make_rows_maps(&ma, &mt, &Q.tail_rows, G, rows, n, p.ld_g);
      if (s != FS_OK) return s;
      if ((s = make_map(&mb, wd + col0 * w->ld, n, dim, w->ld, 64)) != FS_OK) return s;
      Q.m = rows;
      Q.n = dim;
      Q.k_steps = static_cast<int32_t>(ceil_div(n, kLinK));
      Q.m_blocks = P.m_blocks;
      Q.last_block = P.last_block;
      Q.n_blocks = static_cast<int32_t>(ceil_div(dim, 256));
      Q.k_splits = static_cast<int32_t>(p.splits);
      Q.units = static_cast<int64_t>(Q.m_blocks) * Q.n_blocks * p.splits;
      Q.err = err;
      Q.out = partial ? nullptr : gx;
      Q.acc = acc;
      Q.add = c > 0;
      Q.ld_out = dim;
      Q.ids = ids;
      Q.ids_wide = ids_64;
      Q.rest = rest;
      Q.w = wd;
      Q.ld_w = w->ld;
      what = "fs_linear_logprobs_grad (dx)";
      s = cg == 1 ? launch_linear<256, 1, false, true, kLinStore>(what, ma, mt, mb, Q, sms, st)
                  : launch_linear<256, 2, false, true, kLinStore>(what, ma, mt, mb, Q, sms, st);
      if (s != FS_OK) return s;
    }
    if (gw) {  // dw = G^T x: K runs down both
      if (c > 0) {
        s = cuda_status(cudaMemsetAsync(has_rest, 0, p.off_x - p.off_flags, st), "cudaMemsetAsync");
        if (s != FS_OK) return s;
      }
      s = rests(p, rest, rows, col0, n, x, keys, has_rest, gw + col0 * dim, sms, st);
      if (s != FS_OK) return s;
      LinParams Q{};
      if ((s = make_map(&ma, G, rows, n, p.ld_g, 64)) != FS_OK) return s;
      if ((s = make_map(&mb, xm, rows, dim, p.ld_x, 64)) != FS_OK) return s;
      Q.m = n;
      Q.n = dim;
      Q.k_steps = static_cast<int32_t>(ceil_div(rows, kLinK));
      const int cw = pair_of(n);
      Q.m_blocks = static_cast<int32_t>(ceil_div(n, kLinM * cw));
      Q.last_block = static_cast<int32_t>(ceil_div(n, kLinM) - 1);
      Q.n_blocks = static_cast<int32_t>(ceil_div(dim, 256));
      Q.k_splits = 1;
      Q.n_fast = 1;  // the tiles of one strip of G run together
      Q.units = static_cast<int64_t>(Q.m_blocks) * Q.n_blocks;
      Q.err = err;
      Q.out = gw + col0 * dim;
      Q.ld_out = dim;
      Q.has_rest = has_rest;
      what = "fs_linear_logprobs_grad (dw)";
      s = cw == 1 ? launch_linear<256, 1, true, true, kLinStore>(what, ma, ma, mb, Q, sms, st)
                  : launch_linear<256, 2, true, true, kLinStore>(what, ma, ma, mb, Q, sms, st);
      if (s != FS_OK) return s;
    }
  }
  if (gx && partial) {
    const int64_t count = rows * dim;
    s = launch("fs_linear_logprobs_grad (sum)", linear_reduce_kernel,
               dim3(static_cast<unsigned>(ceil_div(count, 1024))), 256, 0, st, 1,
               static_cast<const float*>(acc), static_cast<int>(p.splits), count, dim,
               ids, ids_64, static_cast<const LinRest*>(rest), wd, w->ld, gx);
    if (s != FS_OK) return s;
  }
  return launch("fs_linear_logprobs_grad (check)", linear_poison_kernel,
                dim3(static_cast<unsigned>(sms)), 256, 0, st, 1, static_cast<const unsigned*>(err),
                gx, gx ? rows * dim : int64_t(0), gw, gw ? cols * dim : int64_t(0));
}

}  // namespace
}  // namespace fs

extern "C" {

size_t fs_linear_logprobs_workspace_bytes(const fs_matrix* x, const fs_matrix* w) {
  if (!fs::shape_ok(x, w)) return 0;
  return fs::forward_plan(std::max<int64_t>(x->rows, 1), w->rows, fs::current_sms()).total;
}

size_t fs_linear_logprobs_grad_workspace_bytes(const fs_matrix* x, const fs_matrix* w) {
  if (!fs::shape_ok(x, w)) return 0;
  return fs::backward_plan(std::max<int64_t>(x->rows, 1), w->rows, x->cols, fs::current_sms()).total;
}

fs_status fs_linear_logprobs(const fs_matrix* x, const fs_matrix* w, float eps, const void* ids,
                             int32_t ids_64, float* logp, float* entropy, float* lse, float* stats,
                             void* ws, size_t ws_bytes, fs_stream_t stream) {
  return fs::forward(x, w, eps, ids, ids_64, logp, entropy, lse, stats, ws, ws_bytes,
                     reinterpret_cast<cudaStream_t>(stream));
}

fs_status fs_linear_logprobs_grad(const fs_matrix* x, const fs_matrix* w, float eps,
                                  const void* ids, int32_t ids_64, const float* stats,
                                  const float* entropy, const float* g_logp,
                                  const float* g_entropy, const float* g_lse, void* grad_x,
                                  void* grad_w, void* ws, size_t ws_bytes, fs_stream_t stream) {
  return fs::backward(x, w, eps, ids, ids_64, stats, entropy, g_logp, g_entropy, g_lse, grad_x,
                      grad_w, ws, ws_bytes, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
