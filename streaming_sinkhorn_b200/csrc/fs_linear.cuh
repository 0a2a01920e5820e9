// fs_linear.cuh -- log probabilities of given tokens straight from states x (T, D) and an
// embedding w (V, D), bf16, with z = x w^T never stored, and their gradients (sm_100a).
//
// Forward: one persistent pass forms 128-row score tiles on the tensor cores (products of
// bf16 are exact in the fp32 accumulators) and its epilogue folds each tile into the rows'
// running maximum, sum and entropy sum, as the pass over given scores does; a second kernel
// joins the partial rows. Gradient: the scores are formed again, the epilogue turns each tile
// into G_ij = dL/dz_ij in bf16 (at most 2^-8 relative in each term of the sums below: the
// operands of the tensor cores; bf16 and not fp16, whose range ends above a small probability
// over a batch's size), and two products finish it: dx = G w and dw = G^T x. G lives in the
// workspace, in chunks of columns when all of it would not fit the cap.
//
// Two entries of a row can make up most of it: the given token's and that of a token with more
// than half of the probability. Their rounding alone would be as large as that of the result (4096
// x 65536 x 2048: 2.3e-3 of the gradients' norm against 1.65e-3 for exact G). So what it left is
// kept in fp32 and added to the sums before they are rounded: r w[token] to dx, r x to dw[token],
// the rows of one token in their order.
//
// One kernel does all four: C = A B^T over 64-wide K steps, warp 0 streams both operands
// through a ring with TMA (128-byte swizzle), warp 1 issues the MMAs into one of two TMEM
// accumulators, eight warps run the epilogue of the other (lane quarter warp % 4, half of the
// columns each). An operand whose K runs along its rows' elements (x, w of the scores; G of dx)
// is K-major; one whose K runs down its rows (w of dx; G and x of dw) is read as it lies as an
// MN-major operand, so nothing is transposed in memory.
//
// With more than 128 rows a pair of CTAs works on 256 x 256 tiles: each brings its own 128 rows
// of A and half of B's 256, the first issues the MMAs of both, so B crosses from L2 once for 256
// rows: a single CTA's 128 x 256 tile wants 96 bytes a clock of L2 at the tensor cores' rate, a
// pair's 64 each (4096 x 65536 x 2048 with gradients takes 3.8 ms, with one CTA a tile 6 % more).
// That is still what bounds the products: 8.6 GB from L2 in 770 to 840 us (10 to 11 TB/s), tensor pipes
// 67 to 77 % active, 1.30 to 1.42 PFLOP/s. Up to 128 rows w is read once and bounds the pass: 4 x
// 128000 x 4096 takes 164 us, 6.4 TB/s.
//
// The last row block of a K-major A has a box of its own height: a 128-row box that ends outside
// the matrix loads slower than one that does not (4 states of 4096: 250 us against 183 for 16),
// and what stale rows of the stage add to the accumulator's other lanes is never looked at.
//
// Every wait is bounded; a CTA that gives up sets the call's error word, and the outputs are
// NaN.
#pragma once

#include <cuda.h>

#include "fs_bitonic.cuh"
#include "fs_tcgen05.cuh"
#include "fs_tokens.cuh"

namespace fs {

constexpr int kLinM = 128;       // rows of a tile (MMA M)
constexpr int kLinK = 64;        // K step: 128 bytes of bf16, one swizzle span
constexpr int kLinEpiWarps = 8;
constexpr int kLinThreads = (4 + kLinEpiWarps) * 32;  // producer, MMA, TMEM owner, idle; epilogue
constexpr uint32_t kLinRing = 192u * 1024u;           // bytes of the operand ring

enum LinEpi : int { kLinLse = 0, kLinScoreGrad = 1, kLinStore = 2 };

// CG: CTAs that share a tile (1 or 2).
template <int BN, int CG>
struct LinShape {
  static constexpr int BOX_N = BN / CG;  // rows of B that a CTA brings
  static constexpr uint32_t A_BYTES = kLinM * kLinK * 2;
  static constexpr uint32_t B_BYTES = BOX_N * kLinK * 2;
  // K steps of a stage. A lone row block is bound by the read of B: 256 neighbouring bytes of each
  // row asked for together come faster than 128.
  static constexpr int KS = CG == 1 && BN == 128 ? 2 : 1;
  static constexpr uint32_t STEP = A_BYTES + B_BYTES;
  static constexpr uint32_t STAGE = KS * STEP;
  static constexpr int STAGES = static_cast<int>(kLinRing / STAGE);
  static constexpr size_t SMEM = static_cast<size_t>(STAGES) * STAGE + 1024;
  // Two tiles' accumulators fill the tensor memory. Where a tile leaves room, the K steps of a
  // stage go to one each and meet in the epilogue: an accumulator's sum is cut to fp32 after every
  // 16 products, always towards 0, and half as many of smaller sums cost less than half (what is
  // left of the mean loss, the scores' factor puts back).
  static constexpr int ACCS = 512 / (2 * BN);
  static constexpr uint32_t TMEM = 512;
  static_assert(ACCS == 1 || ACCS == KS, "an accumulator for each K step of a stage");
};

// One of the two entries of a row of G that are not left rounded.
struct LinRest {
  int32_t token;  // the entry's column + 1; 0: none
  float rest;     // G - bf16(G)
};
// log2 of the probability above which a token's entry is kept (of one token at most, with room for
// the rounding of p).
constexpr float kLinLikely = -0.9714f;  // 0.51

struct LinParams {
  int64_t m, n;        // rows of C, columns of C that exist
  int32_t k_steps;     // of the whole product
  int32_t m_blocks, n_blocks;  // row blocks of a tile's height, column tiles
  int32_t last_block;          // the last 128-row block of the matrix
  int32_t n_per_unit;  // column tiles of a unit (kLinLse)
  int32_t k_splits;    // parts of the K range (kLinStore)
  int32_t n_fast;      // units go along n first
  uint32_t tail_rows;  // rows of the last row block (K-major A: its box is no higher)
  int64_t units;
  unsigned* err;
  float inv_eps;
  float uncut;  // factor of the scores: puts back what the accumulators' cuts take of them
  const void* ids;
  int32_t ids_wide;
  // kLinLse
  float4* part;    // (rows padded to whole blocks, parts): max, sum, entropy sum
  int64_t parts;   // of a row: two per unit
  float* given;    // (m) score of the given token
  // kLinScoreGrad
  int64_t col0;    // first column of the chunk
  int64_t cols;    // all columns (for the range of ids)
  const float2* stats;
  const float* entropy;
  const float* g_logp;
  const float* g_entropy;
  const float* g_lse;
  __nv_bfloat16* g_out;
  int64_t ld_g;
  LinRest* rest;  // (m, 2): the given token's, the likely token's; dx reads it
  // kLinStore
  __nv_bfloat16* out;  // bf16 output, or NULL: fp32 partial sums
  float* acc;          // (k_splits, m, n)
  int32_t add;         // add to acc (a later chunk)
  int64_t ld_out;
  const __nv_bfloat16* w;  // dx straight to bf16: the embedding that the rests go with, or NULL
  int64_t ld_w;
  const uint8_t* has_rest;  // dw: whether the output row holds a sum to be added, or NULL
};

// Adds to 32 sums of a row of dx, from column `col` of `n`, its two rests times their tokens' rows
// of w (16-byte aligned rows, col a multiple of 32).
__device__ __forceinline__ void lin_add_rests(float* v, const LinRest* rest, const __nv_bfloat16* w,
                                              int64_t ld_w, int64_t col, int64_t n) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const LinRest e = rest[h];
    if (e.token == 0 || e.rest == 0.0f) continue;
    const __nv_bfloat16* src = w + static_cast<int64_t>(e.token - 1) * ld_w + col;
    if (col + 32 <= n) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float f[8];
        Elem<__nv_bfloat16>::unpack(reinterpret_cast<const uint4*>(src)[j], f);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[8 * j + i] = fmaf(e.rest, f[i], v[8 * j + i]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (col + j < n) v[j] = fmaf(e.rest, __bfloat162float(src[j]), v[j]);
    }
  }
}

// Shared-memory matrix descriptor, 128-byte swizzle, sm_100 version field. K-major: lbo unused,
// sbo = 1024 (8 rows of 128 bytes). MN-major: a box is 64 K rows of 64 elements; lbo = its size
// (the next 64 elements along M or N), sbo = 1024 (the next 8 K rows).
__device__ __forceinline__ uint64_t lin_desc(uint32_t addr, uint32_t lbo) {
  return static_cast<uint64_t>((addr >> 4) & 0x3FFFu) |
         (static_cast<uint64_t>((lbo >> 4) & 0x3FFFu) << 16) |
         (static_cast<uint64_t>(1024u >> 4) << 32) | (1ull << 46) | (2ull << 61);
}

// kind::f16, bf16 operands, fp32 accumulators.
__host__ __device__ constexpr uint32_t lin_idesc(int M, int N, bool a_mn, bool b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) |
         (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// A box into this CTA's shared memory. With CG = 2 its bytes count on the barrier at this address
// in the pair's first CTA (the address bit that tells the two apart cleared).
template <int CG>
__device__ __forceinline__ void tma_load_2d(void* dst, const CUtensorMap* map, int x, int y,
                                            uint64_t* bar) {
  if constexpr (CG == 1) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, "
        "{%2, %3}], [%4];" ::"r"(smem_u32(dst)),
        "l"(map), "r"(x), "r"(y), "r"(smem_u32(bar))
        : "memory");
  } else {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3}], [%4];" ::"r"(smem_u32(dst)),
        "l"(map), "r"(x), "r"(y), "r"(smem_u32(bar) & 0xFEFFFFFFu)
        : "memory");
  }
}

// A commit that arrives in the issuing CTA alone.
template <int CG>
__device__ __forceinline__ void tc_commit_own(uint64_t* bar) {
  if constexpr (CG == 1)
    tc_commit(bar);
  else
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
            smem_u32(bar))
        : "memory");
}

// What a unit covers: row block, column tiles [n0, n1), K steps [k0, k1), split.
struct LinUnit {
  int mb, n0, n1, k0, k1, split;
};

template <int EPI>
__device__ __forceinline__ LinUnit lin_unit(const LinParams& P, int64_t u) {
  LinUnit r;
  if (EPI == kLinStore) {
    const int64_t tiles = static_cast<int64_t>(P.m_blocks) * P.n_blocks;
    r.split = static_cast<int>(u / tiles);
    const int64_t t = u % tiles;
    if (P.n_fast) {
      r.mb = static_cast<int>(t / P.n_blocks);
      r.n0 = static_cast<int>(t % P.n_blocks);
    } else {
      r.mb = static_cast<int>(t % P.m_blocks);
      r.n0 = static_cast<int>(t / P.m_blocks);
    }
    r.n1 = r.n0 + 1;
    r.k0 = static_cast<int>(static_cast<int64_t>(P.k_steps) * r.split / P.k_splits);
    r.k1 = static_cast<int>(static_cast<int64_t>(P.k_steps) * (r.split + 1) / P.k_splits);
  } else {
    // neighbouring CTAs take other rows of the same columns: w is read from L2 but once
    r.mb = static_cast<int>(u % P.m_blocks);
    r.split = static_cast<int>(u / P.m_blocks);
    r.n0 = r.split * P.n_per_unit;
    r.n1 = min(r.n0 + P.n_per_unit, P.n_blocks);
    r.k0 = 0;
    r.k1 = P.k_steps;
  }
  return r;
}

template <int BN, int CG, bool A_MN, bool B_MN, int EPI>
__global__ void __launch_bounds__(kLinThreads, 1)
    linear_kernel(const __grid_constant__ CUtensorMap map_a,
                  const __grid_constant__ CUtensorMap map_tail,
                  const __grid_constant__ CUtensorMap map_b, const LinParams P) {
  using S = LinShape<BN, CG>;
  extern __shared__ unsigned char lin_smem[];
  __shared__ uint64_t full_bar[S::STAGES], free_bar[S::STAGES];
  __shared__ uint64_t acc_bar[2], acc_free_bar[2];
  __shared__ uint64_t fin_bar;
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_sh;
  unsigned char* ring = lin_smem + ((1024u - (smem_u32(lin_smem) & 1023u)) & 1023u);
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int rank = CG == 2 ? static_cast<int>(blockIdx.x & 1u) : 0;  // in the pair
  const int64_t unit0 = blockIdx.x / CG, unit_step = gridDim.x / CG;
  volatile int* abort = &abort_sh;

  if (tid == 0) {
    for (int s = 0; s < S::STAGES; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&free_bar[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_bar[b], 1);
      mbar_init(&acc_free_bar[b], CG * kLinEpiWarps);
    }
    mbar_init(&fin_bar, 1);
    abort_sh = 0;
    fence_mbar_init();
  }
  if (warp == 2) {
    if constexpr (CG == 1) {
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                       smem_u32(&tmem_base_sh)),
                   "r"(S::TMEM));
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    } else {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                       smem_u32(&tmem_base_sh)),
                   "r"(S::TMEM));
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    }
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (CG == 2) cluster_barrier();  // both CTAs' barriers are ready
  tc_fence_after();
  const uint32_t tmem = tmem_base_sh;

  if (warp == 0) {
    if (lane == 0) {
      int64_t q = 0;
      bool ok = true;
      for (int64_t u = unit0; ok && u < P.units; u += unit_step) {
        const LinUnit w = lin_unit<EPI>(P, u);
        for (int nb = w.n0; ok && nb < w.n1; ++nb) {
          for (int k = w.k0; k < w.k1; k += S::KS, ++q) {
            const int s = static_cast<int>(q % S::STAGES);
            const uint32_t round = static_cast<uint32_t>(q / S::STAGES);
            if (round > 0 && !tc_wait(&free_bar[s], (round - 1) & 1u, abort)) {
              ok = false;
              break;
            }
            unsigned char* stage = ring + static_cast<uint32_t>(s) * S::STAGE;
            const int mb = w.mb * CG + rank;  // this CTA's 128 rows of A
            if (rank == 0) {
              // what all CTAs of the tile will bring (a block behind the last one: no rows)
              uint32_t bytes = CG * S::B_BYTES;
#pragma unroll
              for (int c = 0; c < CG; ++c)
                bytes += A_MN || mb + c < P.last_block ? S::A_BYTES
                         : mb + c == P.last_block      ? P.tail_rows * 128u
                                                       : 0u;
              mbar_expect_tx(&full_bar[s], S::KS * bytes);
            }
            // (a stage's steps behind the last one read as zero)
#pragma unroll
            for (int j = 0; j < S::KS; ++j) {
              const int x = (k + j) * kLinK;
              unsigned char* b = stage + j * S::STEP + S::A_BYTES;
              if constexpr (B_MN) {
#pragma unroll
                for (int i = 0; i < S::BOX_N / 64; ++i)
                  tma_load_2d<CG>(b + i * 8192, &map_b, nb * BN + rank * S::BOX_N + i * 64, x,
                                  &full_bar[s]);
              } else {
                tma_load_2d<CG>(b, &map_b, x, nb * BN + rank * S::BOX_N, &full_bar[s]);
              }
            }
#pragma unroll
            for (int j = 0; j < S::KS; ++j) {
              const int x = (k + j) * kLinK;
              unsigned char* a = stage + j * S::STEP;
              if constexpr (A_MN) {
#pragma unroll
                for (int i = 0; i < kLinM / 64; ++i)
                  tma_load_2d<CG>(a + i * 8192, &map_a, mb * kLinM + i * 64, x, &full_bar[s]);
              } else if (mb <= P.last_block) {
                tma_load_2d<CG>(a, mb == P.last_block ? &map_tail : &map_a, x, mb * kLinM,
                                &full_bar[s]);
              }
            }
          }
        }
      }
      if (*abort && rank == 0)  // the copies in flight land before the shared memory goes
        for (int64_t v = q > S::STAGES ? q - S::STAGES : 0; v < q; ++v)
          (void)mbar_wait_bounded(&full_bar[v % S::STAGES],
                                  static_cast<uint32_t>(v / S::STAGES) & 1u);
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      constexpr uint32_t idesc = lin_idesc(CG * kLinM, BN, A_MN, B_MN);
      int64_t q = 0;
      uint32_t t = 0;
      bool ok = true;
      for (int64_t u = unit0; ok && u < P.units; u += unit_step) {
        const LinUnit w = lin_unit<EPI>(P, u);
        for (int nb = w.n0; ok && nb < w.n1; ++nb, ++t) {
          const uint32_t b = t & 1u;
          if (t >= 2 && !tc_wait(&acc_free_bar[b], ((t >> 1) - 1) & 1u, abort)) {
            ok = false;
            break;
          }
          tc_fence_after();
          for (int k = w.k0; k < w.k1; k += S::KS, ++q) {
            const int s = static_cast<int>(q % S::STAGES);
            if (!tc_wait(&full_bar[s], static_cast<uint32_t>(q / S::STAGES) & 1u, abort)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t a0 = smem_u32(ring + static_cast<uint32_t>(s) * S::STAGE);
            const uint32_t b0 = a0 + S::A_BYTES;
#pragma unroll
            for (int ji = 0; ji < S::KS * kLinK / 16; ++ji) {
              const int i = ji % (kLinK / 16);
              const uint32_t o = ji / (kLinK / 16) * S::STEP;
              // 16 elements of K: 32 bytes along a K-major row, 16 rows of an MN-major box
              const uint64_t da = lin_desc(a0 + o + i * (A_MN ? 2048u : 32u), A_MN ? 8192u : 16u);
              const uint64_t db = lin_desc(b0 + o + i * (B_MN ? 2048u : 32u), B_MN ? 8192u : 16u);
              const int acc = S::ACCS == 1 ? 0 : ji / (kLinK / 16);
              const uint32_t d = tmem + (b * S::ACCS + acc) * BN;
              const uint32_t add = k > w.k0 || (S::ACCS == 1 ? ji : i) > 0 ? 1u : 0u;
              if constexpr (CG == 1)
                tc_mma_f16(d, da, db, idesc, add);
              else
                tc_mma_f16_pair(d, da, db, idesc, add);
            }
            if constexpr (CG == 1)
              tc_commit(&free_bar[s]);
            else
              tc_commit_pair(&free_bar[s]);
          }
          if (ok) {
            if constexpr (CG == 1)
              tc_commit(&acc_bar[b]);
            else
              tc_commit_pair(&acc_bar[b]);
          }
        }
      }
      // every MMA issued has completed once fin_bar fires: TMEM is never released under one
      tc_commit_own<CG>(&fin_bar);
      (void)mbar_wait_bounded(&fin_bar, 0);
    }
  } else if (warp >= 4) {
    const int quarter = warp & 3, grp = (warp - 4) >> 2;
    constexpr int GC = BN / 2;  // columns of this warp's half
    const int r = quarter * 32 + lane;
    const float k2 = P.inv_eps * kLog2e;
    uint32_t t = 0;
    bool ok = true;
    for (int64_t u = unit0; ok && u < P.units; u += unit_step) {
      const LinUnit w = lin_unit<EPI>(P, u);
      const int64_t row = (static_cast<int64_t>(w.mb) * CG + rank) * kLinM + r;
      const bool live = row < P.m;
      // per row of the unit
      TokenSum sum = {-INFINITY, 0.0f, 0.0f};
      int64_t id = -1;
      TokenRow tr = {0.0f, 0.0f, 0.0f, 0.0f};
      float H = 0.0f, hot = 0.0f;
      bool zero = true;
      if (EPI != kLinStore && live) id = ld_id(P.ids, row, P.ids_wide != 0);
      // (dx: 0 whatever w holds)
      const bool unasked =
          EPI == kLinStore && P.w && live && ld_id(P.ids, row, P.ids_wide != 0) < 0;
      if (EPI == kLinScoreGrad && live && id >= 0) {
        const float2 st = P.stats[row];
        float gl = P.g_logp ? P.g_logp[row] : 0.0f;
        if (id >= P.cols) gl = __int_as_float(0x7FC00000);
        zero = false;
        tr.m = st.x;
        tr.log2_l = st.y * kLog2e;
        tr.ge = P.g_entropy ? P.g_entropy[row] * P.inv_eps : 0.0f;
        tr.c = ((P.g_lse ? P.g_lse[row] : 0.0f) - gl) * P.inv_eps;
        hot = gl * P.inv_eps;
        H = P.entropy[row];
      }
      for (int nb = w.n0; nb < w.n1; ++nb, ++t) {
        const uint32_t b = t & 1u;
        if (!tc_wait(&acc_bar[b], (t >> 1) & 1u, abort)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t base = tmem + (static_cast<uint32_t>(quarter * 32) << 16) +
                              b * S::ACCS * BN + grp * GC;
        const int64_t c0 = static_cast<int64_t>(nb) * BN + grp * GC;
        // split 0 .. of a K range that is empty leaves no MMA: its sum is zero
        const bool none = EPI == kLinStore && w.k1 == w.k0;
#pragma unroll 1
        for (int c = 0; c < GC; c += 32) {
          float v[32];
          tc_ld32_nowait(base + c, v);
          tc_wait_ld();
          if constexpr (S::ACCS == 2) {
            float v1[32];
            tc_ld32_nowait(base + BN + c, v1);
            tc_wait_ld();
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] += v1[j];
          }
          if constexpr (EPI != kLinStore) {
            const u64 k = pk(P.uncut, P.uncut);
#pragma unroll
            for (int j = 0; j < 32; j += 2) upk(mul2(pk(v[j], v[j + 1]), k), v[j], v[j + 1]);
          }
          const int64_t col = c0 + c;
          if constexpr (EPI == kLinLse) {
            if (col + 32 > P.n) {
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (col + j >= P.n) v[j] = -INFINITY;
            }
            const int64_t at = id - col;
            if (__any_sync(0xffffffffu, at >= 0 && at < 32)) {
              float z = 0.0f;
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (at == j) z = v[j];
              if (at >= 0 && at < 32 && id < P.n) P.given[row] = z;
            }
            float mx = fmaxf(v[0], v[1]);
#pragma unroll
            for (int j = 2; j < 32; j += 2) mx = max3(mx, v[j], v[j + 1]);
            token_add<32>(sum, v, mx, k2);
          } else if constexpr (EPI == kLinScoreGrad) {
            const int64_t at = id - P.col0 - col;
            if (live && col < P.n) {
              const int64_t in = P.n - col;  // columns from here on
              int likely = -1;
              float mx = fmaxf(v[0], v[1]);
#pragma unroll
              for (int j = 2; j < 32; j += 2) mx = max3(mx, v[j], v[j + 1]);
              if (!zero && (mx - tr.m) * k2 - tr.log2_l > kLinLikely) {
#pragma unroll
                for (int j = 0; j < 32; ++j)
                  if (j < in && (v[j] - tr.m) * k2 - tr.log2_l > kLinLikely) likely = j;
              }
#pragma unroll
              for (int j = 0; j < 32; ++j) v[j] = zero ? 0.0f : token_dscore(tr, v[j], k2, H);
              const bool here = at >= 0 && at < 32 && at < in;
              if (here || likely >= 0) {
                float g = 0.0f, l = 0.0f;
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                  if (at == j) g = v[j] += hot;
                  if (likely == j) l = v[j];
                }
                const int32_t first = static_cast<int32_t>(P.col0 + col) + 1;
                if (here)
                  P.rest[2 * row] = {first + static_cast<int32_t>(at),
                                     g - __bfloat162float(__float2bfloat16_rn(g))};
                if (likely >= 0 && likely != at)
                  P.rest[2 * row + 1] = {first + likely,
                                         l - __bfloat162float(__float2bfloat16_rn(l))};
              }
              // (columns past the last one fall into the row's padding)
              uint4* o = reinterpret_cast<uint4*>(P.g_out + row * P.ld_g + col);
#pragma unroll
              for (int j = 0; j < 4; ++j) o[j] = Elem<__nv_bfloat16>::pack(v + 8 * j);
            }
          } else {
            if (live && col < P.n) {
              if (none) {
#pragma unroll
                for (int j = 0; j < 32; ++j) v[j] = 0.0f;
              }
              if (P.out) {
                __nv_bfloat16* o = P.out + row * P.ld_out + col;
                if (P.w) {
                  lin_add_rests(v, P.rest + 2 * row, P.w, P.ld_w, col, P.n);
                  if (unasked) {
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] = 0.0f;
                  }
                }
                if (P.has_rest && P.has_rest[row]) {
                  if (col + 32 <= P.n && (reinterpret_cast<uintptr_t>(o) & 15u) == 0) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                      float f[8];
                      Elem<__nv_bfloat16>::unpack(reinterpret_cast<const uint4*>(o)[j], f);
#pragma unroll
                      for (int i = 0; i < 8; ++i) v[8 * j + i] += f[i];
                    }
                  } else {
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                      if (col + j < P.n) v[j] += __bfloat162float(o[j]);
                  }
                }
                if (col + 32 <= P.n && (reinterpret_cast<uintptr_t>(o) & 15u) == 0) {
#pragma unroll
                  for (int j = 0; j < 4; ++j)
                    reinterpret_cast<uint4*>(o)[j] = Elem<__nv_bfloat16>::pack(v + 8 * j);
                } else {
#pragma unroll
                  for (int j = 0; j < 32; ++j)
                    if (col + j < P.n) o[j] = __float2bfloat16_rn(v[j]);
                }
              } else {
                float* o = P.acc + (static_cast<int64_t>(w.split) * P.m + row) * P.n + col;
                if (col + 32 <= P.n && (reinterpret_cast<uintptr_t>(o) & 15u) == 0) {
#pragma unroll
                  for (int j = 0; j < 8; ++j) {
                    float4* o4 = reinterpret_cast<float4*>(o) + j;
                    float4 x = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
                    if (P.add) {
                      const float4 y = *o4;
                      x = make_float4(y.x + x.x, y.y + x.y, y.z + x.z, y.w + x.w);
                    }
                    *o4 = x;
                  }
                } else {
#pragma unroll
                  for (int j = 0; j < 32; ++j)
                    if (col + j < P.n) o[j] = P.add ? o[j] + v[j] : v[j];
                }
              }
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if constexpr (CG == 1)
            mbar_arrive(&acc_free_bar[b]);
          else
            mbar_arrive_cluster(&acc_free_bar[b], 0);  // the first CTA issues for both
        }
      }
      if (EPI == kLinLse && ok)
        P.part[row * P.parts + w.split * 2 + grp] = make_float4(sum.m, sum.l, sum.a, 0.0f);
    }
  }

  tc_fence_before();
  __syncthreads();
  // neither CTA of a pair leaves while the other's MMAs, copies or arrivals may reach it
  if constexpr (CG == 2) cluster_barrier();
  tc_fence_after();
  if (abort_sh && tid == 0) atomicOr(P.err, kErrTimeout);
  if (warp == 2) {
    if constexpr (CG == 1)
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                   "r"(S::TMEM));
    else
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                   "r"(S::TMEM));
  }
}

// ---- joining the parts -------------------------------------------------------------------------

struct LinJoinParams {
  const __nv_bfloat16* x;
  const __nv_bfloat16* w;
  int64_t ld_x, ld_w, dim;
  const float4* part;
  const float* given;
  int64_t parts, m, cols;
  const void* ids;
  int32_t ids_wide;
  float inv_eps;
  const unsigned* err;
  float* logp;
  float* entropy;
  float* lse;
  float2* stats;
};

// A warp's share (of W warps) of x . w in fp32, the same in every lane: products of bf16 are exact,
// the sums rounded to nearest. Rows are 16-byte aligned.
template <int W>
__device__ __forceinline__ float lin_dot(const __nv_bfloat16* x, const __nv_bfloat16* w,
                                         int64_t dim, int share, int lane) {
  float s[8] = {};
  const int64_t vecs = dim / 8;
  for (int64_t v0 = share * 4 * 32 + lane; v0 < vecs; v0 += W * 4 * 32) {  // (eight reads at once)
    uint4 a[4], b[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int64_t v = v0 + 32 * u;
      a[u] = v < vecs ? *reinterpret_cast<const uint4*>(x + 8 * v) : make_uint4(0, 0, 0, 0);
      b[u] = v < vecs ? *reinterpret_cast<const uint4*>(w + 8 * v) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      float p[8], q[8];
      Elem<__nv_bfloat16>::unpack(a[u], p);
      Elem<__nv_bfloat16>::unpack(b[u], q);
#pragma unroll
      for (int e = 0; e < 8; ++e) s[e] = fmaf(p[e], q[e], s[e]);
    }
  }
  const int64_t last = 8 * vecs + lane;
  if (share == 0 && last < dim) s[0] = fmaf(__bfloat162float(x[last]), __bfloat162float(w[last]), s[0]);
  return warp_sumf(((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7])));
}

// W warps per row (8 where rows are few): the parts of all units, in the same order every time.
// The given token's score is formed again without the accumulators' cuts and takes its place in
// the sum, so that its log probability, the difference of the two, carries the error of the sum
// alone (4 x 128000 x 4096: 1.3e-6 -> 4e-7 relative at worst, with the second accumulator; 4e-8 with
// the scores' factor). The gradient's statistics stay those of the scores that it will form, in the
// same tiles.
template <int W>
__global__ void __launch_bounds__(256) linear_join_kernel(const LinJoinParams P) {
  static_assert(W == 1 || W == 8, "a warp or a CTA");
  __shared__ TokenSum sum_sh[8];
  __shared__ float dot_sh[8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int share = W == 8 ? warp : 0;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (8 / W) + (W == 8 ? 0 : warp);
  if (row >= P.m) return;
  const int64_t id = ld_id(P.ids, row, P.ids_wide != 0);
  const float k2 = P.inv_eps * kLog2e;
  TokenSum s = {-INFINITY, 0.0f, 0.0f};
  for (int64_t q = share * 4 * 32 + lane; q < P.parts; q += W * 4 * 32) {  // (four reads at once)
    float4 o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      o[i] = q + 32 * i < P.parts ? P.part[row * P.parts + q + 32 * i]
                                  : make_float4(-INFINITY, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < 4; ++i) s = token_merge(s, TokenSum{o[i].x, o[i].y, o[i].z}, k2);
  }
  s = token_reduce<32>(s, k2);
  const bool asked = id >= 0 && id < P.cols;
  float zi =
      asked ? lin_dot<W>(P.x + row * P.ld_x, P.w + id * P.ld_w, P.dim, share, lane) : 0.0f;
  if constexpr (W == 8) {
    if (lane == 0) {
      sum_sh[warp] = s;
      dot_sh[warp] = zi;
    }
    __syncthreads();
    if (warp != 0) return;
    s = token_reduce<8>(sum_sh[lane % 8], k2);
    zi = dot_sh[0];
    for (int i = 1; i < 8; ++i) zi += dot_sh[i];
  }
  if (lane != 0) return;
  const float nan = __int_as_float(0x7FC00000);
  const bool bad = *P.err != 0u;
  const float log_l = logf(s.l);
  if (id < 0 && !bad) {
    P.logp[row] = 0.0f;
    P.entropy[row] = 0.0f;
    if (P.lse) P.lse[row] = 0.0f;
    if (P.stats) P.stats[row] = make_float2(0.0f, 0.0f);
    return;
  }
  float l = s.l;
  if (asked) {
    const float rest = s.l - ex2((P.given[row] - s.m) * k2);
    l = (rest < 0.0f ? 0.0f : rest) + ex2((zi - s.m) * k2);
  }
  const float log_i = logf(l);
  P.logp[row] = bad || !asked ? nan : (zi - s.m) * P.inv_eps - log_i;
  P.entropy[row] = bad ? nan : log_l - s.a / s.l * kLn2;
  if (P.lse) P.lse[row] = bad ? nan : s.m * P.inv_eps + log_i;
  if (P.stats) P.stats[row] = bad ? make_float2(nan, nan) : make_float2(s.m, log_l);
}

// ---- the entries of G that are not left rounded --------------------------------------------------
//
// dx takes its two entries a row where its sums end (lin_add_rests). For dw the entries of a chunk
// of columns are put in order of their tokens, and of rows where those are equal, so that each
// token's are added up in the same order on every call: a sum of atomics would not repeat.

// The states with rows that nobody asks about, and the padding, as zeros: 16 bytes a thread and step.
__global__ void __launch_bounds__(256)
    linear_asked_kernel(const __nv_bfloat16* x, int64_t ld_x, int64_t rows, int64_t dim,
                        const void* ids, int ids_wide, __nv_bfloat16* out, int64_t ld_out) {
  const int64_t per = ld_out / 8, count = rows * per;
  for (int64_t v = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; v < count;
       v += static_cast<int64_t>(gridDim.x) * 256) {
    const int64_t row = v / per, d = (v - row * per) * 8;
    uint4 q = make_uint4(0u, 0u, 0u, 0u);
    if (ld_id(ids, row, ids_wide != 0) >= 0) {
      const __nv_bfloat16* src = x + row * ld_x + d;
      if (d + 8 <= dim) {
        q = *reinterpret_cast<const uint4*>(src);
      } else {
        uint32_t w[4] = {};
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (d + i < dim)
            w[i / 2] |= static_cast<uint32_t>(__bfloat16_as_ushort(src[i])) << (16 * (i & 1));
        q = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
    *reinterpret_cast<uint4*>(out + row * ld_out + d) = q;
  }
}

// The sort key of entry e (of 2 a row), or the largest one if it has no token in the chunk.
__device__ __forceinline__ uint64_t lin_rest_key(const LinRest* rest, int64_t e, int64_t entries,
                                                 int64_t col0, int64_t n) {
  if (e >= entries) return ~0ull;
  const LinRest r = rest[e];
  const int64_t col = static_cast<int64_t>(r.token) - 1 - col0;
  if (r.token == 0 || r.rest == 0.0f || col < 0 || col >= n) return ~0ull;
  return static_cast<uint64_t>(col) << 32 | static_cast<uint64_t>(e);
}

// All of them in order by one CTA: n_keys (a power of two, at most kSortSmem) >= entries.
__global__ void __launch_bounds__(kSortBlock)
    linear_order_kernel(const LinRest* rest, int64_t entries, int64_t col0, int64_t n,
                        uint64_t* keys, int n_keys) {
  __shared__ uint64_t s[kSortSmem];
  const int t = threadIdx.x;
  for (int e = t; e < n_keys; e += kSortBlock) s[e] = lin_rest_key(rest, e, entries, col0, n);
  __syncthreads();
  for (int k = 2; k <= n_keys; k <<= 1)
    for (int j = k / 2; j > 0; j >>= 1) {
      const int i = 2 * t - (t & (j - 1));
      if (i + j < n_keys) cmp_swap(s[i], s[i + j], (i & k) == 0);
      __syncthreads();
    }
  for (int e = t; e < n_keys; e += kSortBlock) keys[e] = s[e];
}

// More of them: the keys, which the bitonic kernels then sort.
__global__ void __launch_bounds__(256)
    linear_keys_kernel(const LinRest* rest, int64_t entries, int64_t col0, int64_t n,
                       uint64_t* keys, int64_t n_keys) {
  const int64_t e = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (e < n_keys) keys[e] = lin_rest_key(rest, e, entries, col0, n);
}

// Adds r x, from column d, of the entries whose keys are at [b, b + 32) and of token `col` to this
// lane's 8 sums; their number. Up to 8 rows of x are on their way at once. Called by a whole warp.
__device__ __forceinline__ int lin_rests_of(const uint64_t* keys, int64_t n_keys, int64_t b,
                                            uint32_t col, const LinRest* rest,
                                            const __nv_bfloat16* x, int64_t ld_x, int64_t d,
                                            int64_t dim, float* sum, int lane) {
  const uint64_t k = b + lane < n_keys ? keys[b + lane] : ~0ull;
  const bool mine = static_cast<uint32_t>(k >> 32) == col && k != ~0ull;
  const uint32_t e = mine ? static_cast<uint32_t>(k) : 0u;
  const float r = mine ? rest[e].rest : 0.0f;
  const int count = __popc(__ballot_sync(0xffffffffu, mine));  // (sorted: the first ones)
#pragma unroll 1
  for (int t0 = 0; t0 < count; t0 += 8) {
    uint4 q[8];
    float f[8];
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      const int at = min(t0 + t, count - 1);  // (the last one again, times 0)
      const float ft = __shfl_sync(0xffffffffu, r, at);
      const uint32_t row = __shfl_sync(0xffffffffu, e, at) >> 1;
      f[t] = t0 + t < count ? ft : 0.0f;
      const __nv_bfloat16* src = x + static_cast<int64_t>(row) * ld_x + d;
      if (d + 8 <= dim) {
        q[t] = *reinterpret_cast<const uint4*>(src);
      } else {
        uint32_t w[4] = {};
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (d + i < dim)
            w[i / 2] |= static_cast<uint32_t>(__bfloat16_as_ushort(src[i])) << (16 * (i & 1));
        q[t] = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      float v[8];
      Elem<__nv_bfloat16>::unpack(q[t], v);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[i] = fmaf(f[t], v[i], sum[i]);
    }
  }
  return count;
}

__device__ __forceinline__ void lin_rests_write(const float* sum, __nv_bfloat16* o, int64_t d,
                                                int64_t dim) {
  if (d + 8 <= dim && (reinterpret_cast<uintptr_t>(o) & 15u) == 0) {
    *reinterpret_cast<uint4*>(o) = Elem<__nv_bfloat16>::pack(sum);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (d + i < dim) o[i] = __float2bfloat16_rn(sum[i]);
  }
}

// The sums r x of each token of the chunk that has entries, rounded to bf16 (2^-8 of what is at
// most 2^-8 of the gradient) into its row of dw, where the product's epilogue adds them: no room of
// their own, which would be another matrix of the gradient's size. A warp takes a token's first key
// and 256 columns (grid y); a token with more than kLinMany entries is left to all warps of the
// CTA, 32 entries each in turn (4096 x 65536 x 2048: 28 us after 38 for the order, of 3.8 ms; 86
// with one token for all rows, 2041 by a warp).
constexpr int kLinMany = 64;
constexpr int kLinQueue = 64;

__global__ void __launch_bounds__(256)
    linear_rests_kernel(const uint64_t* keys, int64_t n_keys, const LinRest* rest,
                        const __nv_bfloat16* x, int64_t ld_x, int64_t dim, __nv_bfloat16* out,
                        uint8_t* has_rest) {
  __shared__ int64_t queue[kLinQueue];
  __shared__ int queued;
  __shared__ float part[8][32][9];  // (rows of 9: no two lanes of a quarter on a bank)
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * 8;
  const int64_t d = static_cast<int64_t>(blockIdx.y) * 256 + lane * 8;
  if (threadIdx.x == 0) queued = 0;
  __syncthreads();
  for (int64_t p = static_cast<int64_t>(blockIdx.x) * 8 + warp; p < n_keys; p += warps) {
    const uint64_t key = keys[p];
    if (key == ~0ull) break;  // (no entries from here on)
    const uint32_t col = static_cast<uint32_t>(key >> 32);
    if (p > 0 && static_cast<uint32_t>(keys[p - 1] >> 32) == col) continue;
    if (p + kLinMany < n_keys && keys[p + kLinMany] != ~0ull &&
        static_cast<uint32_t>(keys[p + kLinMany] >> 32) == col) {
      int at = 0;
      if (lane == 0) {
        at = atomicAdd(&queued, 1);
        if (at < kLinQueue) queue[at] = p;
      }
      if (__shfl_sync(0xffffffffu, at, 0) < kLinQueue) continue;
    }
    float sum[8] = {};
    for (int64_t b = p; b < n_keys; b += 32)
      if (lin_rests_of(keys, n_keys, b, col, rest, x, ld_x, d, dim, sum, lane) < 32) break;
    lin_rests_write(sum, out + static_cast<int64_t>(col) * dim + d, d, dim);
    if (blockIdx.y == 0 && lane == 0) has_rest[col] = 1;
  }
  __syncthreads();
  const int n = min(queued, kLinQueue);
  for (int q = 0; q < n; ++q) {
    const int64_t p = queue[q];
    const uint32_t col = static_cast<uint32_t>(keys[p] >> 32);
    float sum[8] = {};
    for (int64_t b = p + warp * 32; b < n_keys; b += 256)
      if (lin_rests_of(keys, n_keys, b, col, rest, x, ld_x, d, dim, sum, lane) < 32) break;
#pragma unroll
    for (int i = 0; i < 8; ++i) part[warp][lane][i] = sum[i];
    __syncthreads();
    if (warp == 0) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        for (int w = 1; w < 8; ++w) sum[i] += part[w][lane][i];
      lin_rests_write(sum, out + static_cast<int64_t>(col) * dim + d, d, dim);
      if (blockIdx.y == 0 && lane == 0) has_rest[col] = 1;
    }
    __syncthreads();
  }
}

// dx = bf16 of the sum of the splits' fp32 partial products, in their order, and of the row's two
// entries that were not left rounded; 0 for a row that nobody asks about.
__global__ void __launch_bounds__(256)
    linear_reduce_kernel(const float* acc, int splits, int64_t count, int64_t dim, const void* ids,
                         int ids_wide, const LinRest* rest, const __nv_bfloat16* w, int64_t ld_w,
                         __nv_bfloat16* out) {
  const int64_t i = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 4;
  if (i >= count) return;
  float v[4];
  const int left = count - i < 4 ? static_cast<int>(count - i) : 4;
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = 0.0f;
  for (int s = 0; s < splits; ++s) {
    const float* p = acc + s * count + i;
    if (left == 4 && (reinterpret_cast<uintptr_t>(p) & 15u) == 0) {
      const float4 x = *reinterpret_cast<const float4*>(p);
      v[0] += x.x;
      v[1] += x.y;
      v[2] += x.z;
      v[3] += x.w;
    } else {
      for (int j = 0; j < left; ++j) v[j] += p[j];
    }
  }
  int64_t row = i / dim, col = i - row * dim;
  for (int j = 0; j < left; ++j) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const LinRest e = rest[2 * row + h];
      if (e.token != 0 && e.rest != 0.0f)
        v[j] = fmaf(e.rest, __bfloat162float(w[static_cast<int64_t>(e.token - 1) * ld_w + col]), v[j]);
    }
    out[i + j] = __float2bfloat16_rn(ld_id(ids, row, ids_wide != 0) < 0 ? 0.0f : v[j]);
    if (++col == dim) {
      col = 0;
      ++row;
    }
  }
}

// After a wait that expired: NaN in place of the gradients.
__global__ void __launch_bounds__(256)
    linear_poison_kernel(const unsigned* err, __nv_bfloat16* a, int64_t na, __nv_bfloat16* b,
                         int64_t nb) {
  if (*err == 0u) return;
  const __nv_bfloat16 nan = __float2bfloat16_rn(__int_as_float(0x7FC00000));
  const int64_t step = static_cast<int64_t>(gridDim.x) * 256;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < na; i += step) a[i] = nan;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < nb; i += step) b[i] = nan;
}

}  // namespace fs
