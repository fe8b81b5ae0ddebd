// Tensor-core GEMM on the 5th-generation tensor cores: C (fp32) = alpha A B^T
// (+ C) with A [M x K] and B [N x K] in bf16, each stored either K-major
// (row-major [M][K], [N][K]) or MN-major (row-major [K][M], [K][N]: the
// transposed matrix), so products like G W or G^T H need no transposed copy.
//
// The dense products of the fused linear cross-entropy (logits, and the two
// gradient products) are real dense contractions, so they run here rather
// than on CUDA cores.  Pairs of CTAs (a cluster of two, one per SM of a
// TPC) walk the 256 x 256 tiles of C in a persistent grid, and each pair
// computes its tile with the pair form of the MMA (cta_group::2, M 256):
// every CTA holds 128 rows of A and 128 rows of B per K slab, the MMA reads
// both halves across the pair, and each CTA's TMEM receives its 128 rows of
// the 256 x 256 accumulator.  Per SM that is half the B tile in shared
// memory and half its shared-memory read traffic, compared with one CTA
// computing 128 x 256 alone, which leaves room for a 6-deep ring.  In each
// CTA:
//   warp 0       TMA producer: 64-wide K slabs of its A rows (128 x 64) and
//                B rows (128 x 64) into a 6-stage ring, 128-byte swizzled
//                (a K-major operand as one 128-row box, an MN-major one as
//                two boxes of 64 x 64); both CTAs' copies complete on the
//                first CTA's stage barrier;
//   warp 1       allocates 512 TMEM columns with its peer (two accumulators
//                of 256 fp32 columns); in the first CTA one elected thread
//                issues tcgen05.mma (M 256, N 256, K 16, bf16 in, fp32
//                accumulate), four per slab, into the accumulator both
//                epilogues have released; tcgen05.commit frees a stage in
//                both CTAs when its MMAs are done and, after a tile's last
//                slab, hands the accumulator to both epilogues;
//   warps 2..    epilogue: each reads its 32 TMEM lanes (rows) with
//                tcgen05.ld and writes (or reduce-adds into) C by tensor
//                stores from shared memory, while the next tile's MMAs run
//                into the other accumulator.
// The vocabulary-piece cross-entropy uses the same main loop with other
// epilogues (template argument EPI, below), M and K read on the device, and
// launches chained as programmatic dependents.  At 2048 x 32000 x 4096 (bf16,
// ncu): softmax statistics with kept exponentials 291-301 us, tensor pipe 80 %
// of elapsed cycles; bf16 C (dW) 255-260 us, 83 %; rows scattered (dH) 302-309 us,
// 76 % (128 tiles on 76 pairs).
// Every wait is bounded: a wait that runs out records an error for
// sf_sync_status, and the CTAs still release their TMEM before they exit.
// Sums over K run in slab order on the tensor cores; results are
// deterministic for a given shape.
#include <cuda_bf16.h>

#include <algorithm>
#include <map>
#include <mutex>

#include "tc_pair.cuh"

namespace sf {
namespace {

// Ring stages, epilogue warps, and staging boxes per warp.  The epilogues that
// write bf16 bound the tile after few K slabs (dW over few tokens, logits of
// short rows), so eight warps share the tile's columns there (cross-entropy of
// 262 x 112 x 89236 81 us, with four warps 84; 4463 x 112 x 33329 362 and 384;
// with 16 boxes and one stage less, long rows lose: 1003 x 2048 x 50001 448
// us against 429).
template <int EPI>
struct TcStages {
  static constexpr int kRing = 6;
  static constexpr int kWarps = EPI == kTcBf16 || EPI == kTcStats || EPI == kTcGrad ? 8 : 4;
  static constexpr int kBoxes = 8 / kWarps;
  static constexpr int kThreads = 64 + 32 * kWarps;
};
constexpr int kStageA = kBM * kBK * 2;         // 16 KB
constexpr int kStageB = kBRows * kBK * 2;      // 16 KB
constexpr int kStageBytes = kStageA + kStageB;
// the ring and the epilogue's boxes of 4 KB (32 rows x 128 bytes)
constexpr size_t kGemmSmem = (size_t)TcStages<kTcF32>::kRing * kStageBytes + 8 * 4096 + 1024 + 256;

struct TcGemmArgs {
  float* C;
  int64_t ldc;
  int32_t M, N, K;
  float alpha;
  int32_t accumulate;    // 1: C += alpha A B^T, 0: C = alpha A B^T
  int32_t tma;           // C written by tensor stores (reduce-add when accumulating) from shared memory
  int32_t n_fast;        // tile order: n fastest (A is the larger operand) or m fastest
  int32_t a_mn, b_mn;    // operand stored MN-major ([K][M], [K][N]) instead of K-major:
                         // 1 loaded as two 2D boxes, 2 as one 3D box (MN a multiple of 64)
  float2* row_stats;     // optional [M][n_tiles]: per row and column tile, (max, sum exp(c - max)) of C
  int32_t splits;        // parts of the sum over K, each a product of its own (kTcSplit: C is [splits][M][N])
  // softmax epilogues (kTcStats, kTcGrad)
  int32_t stats_ld;      // entries of a row of row_stats (kTcStats)
  int32_t col0;          // vocabulary id of column 0, a multiple of the tile width
  int32_t store;         // kTcStats: also write exp(c - tile maximum) to C
  const int32_t* labels; // [M]
  float* label_logit;    // [M]: receives C at each row's label (kTcStats)
  const float* lse;      // [M] (kTcGrad)
  const float* scale;    // kTcSplit, kTcBf16, kTcRows: one device value that multiplies alpha (may be null)
  const int32_t* m_dev;  // device-side M (<= M) and K (<= K) where not null
  const int32_t* k_dev;
  const int32_t* row_map;  // kTcRows: C's row of each product row
  int32_t out_fp32;        // kTcRows: C is fp32 (else bf16)
};

// Folds 32 values of a row into a running (max, sum of exp(x - max)):
// the chunk's maximum first, then one rescale of the running sum.
__device__ __forceinline__ void fold_row_stats(const float (&x)[32], int valid, float& m, float& s) {
  float cm = -INFINITY;
#pragma unroll
  for (int j = 0; j < 32; ++j)
    if (j < valid) cm = fmaxf(cm, x[j]);
  if (cm == -INFINITY) return;
  const float mn = fmaxf(m, cm);
  float acc = m == -INFINITY ? 0.0f : s * expf(m - mn);
#pragma unroll
  for (int j = 0; j < 32; ++j)
    if (j < valid) acc += expf(x[j] - mn);
  m = mn;
  s = acc;
}

__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, uint32_t src, int x, int y, int z) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(map),
               "r"(src), "r"(x), "r"(y), "r"(z)
               : "memory");
}
__device__ __forceinline__ void tma_reduce_add_3d(const CUtensorMap* map, uint32_t src, int x, int y, int z) {
  asm volatile("cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                   map),
               "r"(src), "r"(x), "r"(y), "r"(z)
               : "memory");
}

// The epilogue (template argument EPI) decides what becomes of a tile:
//   kTcF32    C (fp32) stored or added to, optional row statistics;
//   kTcSplit  fp32 partial products [splits][M][N], stored or added to;
//   kTcBf16   C rounded to bf16;
//   kTcRows   C in bf16 or fp32, row i of the product to row row_map[i];
//   kTcStats  per row and tile the maximum and sum of exponentials, the
//             label's logit, and optionally exp(c - maximum) in bf16: the
//             logits themselves never leave tensor memory;
//   kTcGrad   exp(c - lse), at the label expm1(c - lse), in bf16, 0 in rows past M.
template <int EPI>
__global__ void __launch_bounds__(TcStages<EPI>::kThreads, 1)
    k_tc_gemm(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
              const __grid_constant__ CUtensorMap map_c, const TcGemmArgs g) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  constexpr int kStages = TcStages<EPI>::kRing, kBoxes = TcStages<EPI>::kBoxes, kWarps = TcStages<EPI>::kWarps;
  // [ring: kStages x (A 16 KB + B 16 KB)] [epilogue staging: kWarps x kBoxes x 4 KB] [barriers]
  unsigned char* staging = smem + (size_t)kStages * kStageBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(staging + kWarps * kBoxes * 4096);   // used in the first CTA
  uint64_t* empty = full + kStages;
  uint64_t* tfull = empty + kStages;     // [2] accumulator buffer b holds a finished tile
  uint64_t* tempty = tfull + 2;          // [2] both CTAs have read buffer b out (first CTA)
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tempty + 2);
  const uint32_t smem_base = smem_u32(smem);
  const uint32_t empty_a = smem_u32(empty), tfull_a = smem_u32(tfull);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();              // 0: issues the MMAs, 1: its peer
  const int pair = blockIdx.x / kPair, n_pairs = gridDim.x / kPair;
  if (threadIdx.x == 0) {
    prefetch_tensormap(&map_a);
    prefetch_tensormap(&map_b);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);            // the first CTA's producer arrives, both CTAs' copies complete it
      mbar_init(&empty[s], 1);           // the MMA commit arrives in both CTAs
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], kWarps * kPair);  // one arrival per epilogue warp of the pair
    }
    fence_mbar_init_cluster();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), 2 * kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  cluster_sync();                        // barriers of both CTAs initialised, TMEM allocated
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // the plain product keeps its sizes in the launch arguments and is never
  // chained; the others read them from the device once what earlier launches
  // wrote is visible
  if constexpr (EPI != kTcF32) {
    griddep_launch_dependents();         // (a no-op unless the next launch asks for it)
    griddep_wait();
  }
  const int M = EPI != kTcF32 && g.m_dev ? *g.m_dev : g.M, K = EPI != kTcF32 && g.k_dev ? *g.k_dev : g.K;
  const int nk_all = (K + kBK - 1) / kBK;
  const int m_tiles = (M + kPair * kBM - 1) / (kPair * kBM);   // 256-row tiles
  const int n_tiles = (g.N + kBN - 1) / kBN;
  const int tiles = m_tiles * n_tiles;
  // work items: the tiles, once per part of K; part p takes the K slabs
  // [nk_all p / splits, nk_all (p + 1) / splits)
  const int splits = EPI == kTcSplit ? g.splits : 1;
  const int items = tiles * splits;
  auto slab0 = [&](int part) { return EPI == kTcSplit ? (int)((int64_t)nk_all * part / splits) : 0; };
  auto slab1 = [&](int part) { return EPI == kTcSplit ? (int)((int64_t)nk_all * (part + 1) / splits) : nk_all; };


  // tiles t = pair, + n_pairs, ...; the index runs fastest along the
  // dimension whose operand is the smaller one, so the pairs working at the
  // same time share the tile of the larger operand and it streams from
  // memory about once, while the smaller one is re-read from L2
  if (warp == 0) {
    if (lane == 0) {
      const uint32_t full_lead = cluster_addr(smem_u32(full), 0);
      const int a_mn = g.a_mn, b_mn = g.b_mn;
      int s = 0, issued = 0;
      uint32_t pass = 0;
      bool failed = false;
      for (int it = pair; it < items && !failed; it += n_pairs) {
        const int part = EPI == kTcSplit ? it / tiles : 0, t = EPI == kTcSplit ? it % tiles : it;
        const int mt = g.n_fast ? t / n_tiles : t % m_tiles, nt = g.n_fast ? t % n_tiles : t / m_tiles;
        const int m0 = mt * (kPair * kBM) + (int)rank * kBM;
        const int nb = nt * kBN + (int)rank * kBRows;
        const int k1 = slab1(part);
        for (int kb = slab0(part); kb < k1; ++kb) {
          if (issued >= kStages && !mbar_wait_cluster(&empty[s], pass ^ 1u)) {
            failed = true;
            break;
          }
          if (rank == 0) mbar_arrive_expect_tx(&full[s], (uint32_t)(kPair * kStageBytes));
          const uint32_t st = smem_base + (uint32_t)s * kStageBytes;
          const uint32_t bar = full_lead + 8u * (uint32_t)s;
          if (a_mn == 2) {
            tma_load_3d_pair(st, &map_a, bar, 0, kb * kBK, m0 >> 6);
          } else if (a_mn) {
            tma_load_2d_pair(st, &map_a, bar, m0, kb * kBK);
            tma_load_2d_pair(st + kMnBox, &map_a, bar, m0 + 64, kb * kBK);
          } else {
            tma_load_2d_pair(st, &map_a, bar, kb * kBK, m0);
          }
          if (b_mn == 2) {
            tma_load_3d_pair(st + kStageA, &map_b, bar, 0, kb * kBK, nb >> 6);
          } else if (b_mn) {
            tma_load_2d_pair(st + kStageA, &map_b, bar, nb, kb * kBK);
            tma_load_2d_pair(st + kStageA + kMnBox, &map_b, bar, nb + 64, kb * kBK);
          } else {
            tma_load_2d_pair(st + kStageA, &map_b, bar, kb * kBK, nb);
          }
          ++issued;
          if (++s == kStages) {
            s = 0;
            pass ^= 1u;
          }
        }
      }
      // the copies of the last stages (both CTAs') have landed before the
      // pair can exit: immediate when the MMA thread consumed them, bounded
      // otherwise
      if (rank == 0)
        for (int j = issued > kStages ? issued - kStages : 0; j < issued; ++j)
          mbar_wait_cluster(&full[j % kStages], (uint32_t)(j / kStages) & 1u);
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      // K-16 step in descriptor units (16 bytes): 32 bytes along a K-major
      // row, 16 rows of 128 bytes down an MN-major box
      const bool a_mn = g.a_mn != 0, b_mn = g.b_mn != 0;
      const uint32_t a_step = a_mn ? 128u : 2u, b_step = b_mn ? 128u : 2u;
      const uint32_t idesc = kIdesc | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16);
      int s = 0, j = 0;
      uint32_t pass = 0;
      bool failed = false;
      for (int it = pair; it < items && !failed; it += n_pairs, ++j) {
        const int part = EPI == kTcSplit ? it / tiles : 0, k0 = slab0(part), k1 = slab1(part);
        const int b = j & 1;
        const uint32_t use = (uint32_t)(j >> 1);
        // both epilogues have read this accumulator buffer out (its previous use)
        if (use > 0 && !mbar_wait_cluster(&tempty[b], (use - 1u) & 1u)) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem + (uint32_t)(b * kTmemCols);
        for (int kb = k0; kb < k1; ++kb) {
          if (!mbar_wait_cluster(&full[s], pass)) {
            failed = true;
            break;
          }
          tc_fence_after();
          const uint32_t a_addr = smem_base + (uint32_t)s * kStageBytes;
          const uint64_t adesc = a_mn ? umma_desc_mn_sw128(a_addr) : umma_desc_sw128(a_addr);
          const uint64_t bdesc = b_mn ? umma_desc_mn_sw128(a_addr + kStageA) : umma_desc_sw128(a_addr + kStageA);
#pragma unroll
          for (int k = 0; k < kBK / 16; ++k)
            tc_mma(d_tmem, adesc + a_step * (uint32_t)k, bdesc + b_step * (uint32_t)k, idesc, kb != k0 || k != 0 ? 1u : 0u);
          tc_commit_pair(empty_a + 8u * (uint32_t)s);
          if (++s == kStages) {
            s = 0;
            pass ^= 1u;
          }
        }
        tc_commit_pair(tfull_a + 8u * (uint32_t)b);
      }
    }
  } else {
    // epilogue: warp w reads TMEM lanes 32 (w % 4) .. + 31 = rows of this
    // CTA's half of the tile
    const int quarter = warp & 3;
    const uint32_t lane_off = (uint32_t)(32 * quarter) << 16;
    const uint32_t stg = smem_u32(staging) + (uint32_t)(warp - 2) * (kBoxes * 4096u);
    const uint32_t tempty_lead = cluster_addr(smem_u32(tempty), 0);
    int j = 0, boxes = 0;
    for (int it = pair; it < items; it += n_pairs, ++j) {
      const int part = EPI == kTcSplit ? it / tiles : 0, t = EPI == kTcSplit ? it % tiles : it;
      const int mt = g.n_fast ? t / n_tiles : t % m_tiles, nt = g.n_fast ? t % n_tiles : t / m_tiles;
      const int m0 = mt * (kPair * kBM) + (int)rank * kBM, n0 = nt * kBN;
      const int b = j & 1;
      if (!mbar_wait_cluster(&tfull[b], (uint32_t)(j >> 1) & 1u)) break;
      tc_fence_after();
      const uint32_t acc = tmem + (uint32_t)(b * kTmemCols) + lane_off;
      const int row = m0 + 32 * quarter + lane;
      const bool empty = slab0(part) >= slab1(part);     // nothing to sum: the accumulator was not written
      const float alpha = EPI != kTcF32 && g.scale ? g.alpha * *g.scale : g.alpha;
      if constexpr (EPI == kTcStats || EPI == kTcGrad || EPI == kTcBf16) {
        // 32 x 64 bf16 boxes through the warp's staging buffers; the columns go
        // by halves of a tile, one entry of the statistics each, shared out
        // over the warps of a row, as far as C has them
        static_assert(kBN == 2 * kTcStatCols, "two entries of the statistics a tile");
        const int row0 = m0 + 32 * quarter;
        const bool row_on = row < M;
        // a gradient's rows are also read as whole K slabs of 64: zeros past M
        const bool stored = row0 < (EPI == kTcGrad ? (M + 63) & ~63 : M) && (EPI != kTcStats || g.store);
        int label = -1;                    // the label's column within the tile, if it is one
        float ref = 0.0f;                  // what the exponents are taken relative to
        if constexpr (EPI != kTcBf16) {
          if (row_on) label = (int)((uint32_t)g.labels[row] - (uint32_t)(g.col0 + n0));
        }
        if constexpr (EPI == kTcGrad) ref = row_on ? g.lse[row] : 0.0f;
#pragma unroll 1
        for (int first = (warp - 2) / 4 * kTcStatCols; first < min(kBN, g.N - n0); first += kWarps / 4 * kTcStatCols) {
          const int end = min(first + kTcStatCols, g.N - n0);
          float m = -INFINITY;
          if constexpr (EPI == kTcStats) {
#pragma unroll 1
            for (int c0 = first; c0 < end; c0 += 64) {
              uint32_t r[64];
              __syncwarp();
              tmem_ld64(acc + (uint32_t)c0, r);
              if (c0 + 64 <= end) {
#pragma unroll
                for (int jj = 0; jj < 64; jj += 2) m = fmaxf(fmaxf(m, __uint_as_float(r[jj])), __uint_as_float(r[jj + 1]));
              } else {
#pragma unroll
                for (int jj = 0; jj < 64; ++jj)
                  if (jj < end - c0) m = fmaxf(m, __uint_as_float(r[jj]));
              }
              if ((unsigned)(label - c0) < 64u) {
#pragma unroll
                for (int jj = 0; jj < 64; ++jj)
                  if (label - c0 == jj) g.label_logit[row] = __uint_as_float(r[jj]);
              }
            }
            ref = m == -INFINITY ? 0.0f : m;
          }
          // exponentials of pairs: exp2((c - ref) log2 e); kTcBf16 multiplies by alpha
          const uint64_t minus_ref = pack_f2(-ref, -ref), factor = pack_f2(kLog2e, kLog2e), by = pack_f2(alpha, alpha);
          uint64_t sum[2] = {0, 0};
#pragma unroll 1
          for (int c0 = first; c0 < end; c0 += 64) {
            uint32_t r[64];
            __syncwarp();
            tmem_ld64(acc + (uint32_t)c0, r);
            const uint32_t buf = stg + (uint32_t)(boxes % kBoxes) * 4096u;
            if (stored && boxes >= kBoxes) {
              if (lane == 0) bulk_wait_read<kBoxes - 1>();
              __syncwarp();
            }
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              const int c1 = c0 + 32 * half;
              float x[32];
#pragma unroll
              for (int jj = 0; jj < 32; jj += 2) {
                const uint64_t v = pack_f2(__uint_as_float(r[32 * half + jj]), __uint_as_float(r[32 * half + jj + 1]));
                const float2 w = unpack_f2(EPI == kTcBf16 ? fmul2(v, by) : fmul2(fadd2(v, minus_ref), factor));
                x[jj] = EPI == kTcBf16 ? w.x : exp2_approx(w.x);
                x[jj + 1] = EPI == kTcBf16 ? w.y : exp2_approx(w.y);
              }
              if constexpr (EPI == kTcBf16) {
                if (empty) {
#pragma unroll
                  for (int jj = 0; jj < 32; ++jj) x[jj] = 0.0f;
                }
              } else if constexpr (EPI == kTcStats) {
                // short chains, then one addition of them
                const int valid = end - c1;
                uint64_t part[2] = {0, 0};
                if (valid >= 32) {
#pragma unroll
                  for (int jj = 0; jj < 32; jj += 2) part[jj >> 1 & 1] = fadd2(part[jj >> 1 & 1], pack_f2(x[jj], x[jj + 1]));
                } else {
#pragma unroll
                  for (int jj = 0; jj < 32; jj += 2)
                    part[jj >> 1 & 1] = fadd2(part[jj >> 1 & 1], pack_f2(jj < valid ? x[jj] : 0.0f, jj + 1 < valid ? x[jj + 1] : 0.0f));
                }
                sum[half] = fadd2(sum[half], fadd2(part[0], part[1]));
              } else {
                if ((unsigned)(label - c1) < 32u) {
                  // not the exponential - 1, which cancels where the model is sure
                  float z = 0.0f;
#pragma unroll
                  for (int jj = 0; jj < 32; ++jj)
                    if (label - c1 == jj) z = __uint_as_float(r[32 * half + jj]);
                  z = expm1f(z - ref);
#pragma unroll
                  for (int jj = 0; jj < 32; ++jj)
                    if (label - c1 == jj) x[jj] = z;
                }
                if (row0 + 32 > M) {
#pragma unroll
                  for (int jj = 0; jj < 32; ++jj) x[jj] = row_on ? x[jj] : 0.0f;
                }
              }
              if (stored) stage_bf16(buf, lane, half, x);
            }
            if (!stored) continue;
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              tma_store_2d(&map_c, buf, n0 + c0, row0);
              bulk_commit();
            }
            ++boxes;
            __syncwarp();
          }
          if constexpr (EPI == kTcStats) {
            const float2 both = unpack_f2(fadd2(sum[0], sum[1]));
            const float total = both.x + both.y;
            if (m == -INFINITY && total != 0.0f) m = 0.0f;      // nothing but NaN: it must not be left out
            if (row_on) g.row_stats[(int64_t)row * g.stats_ld + (g.col0 + n0 + first) / kTcStatCols] = make_float2(m, total);
          }
        }
      } else if constexpr (EPI == kTcSplit) {
        const int row0 = m0 + 32 * quarter;
#pragma unroll 1
        for (int ci = 0; ci < kBN / 32 && n0 + 32 * ci < g.N; ++ci, ++boxes) {
          uint32_t r[32];
          tmem_ld32(acc + (uint32_t)(32 * ci), r);
          tmem_ld_wait();
          if (empty) {
#pragma unroll
            for (int jj = 0; jj < 32; ++jj) r[jj] = 0;
          }
          const uint32_t buf = stg + (uint32_t)(boxes & 1) * 4096u;
          if (boxes >= 2) {
            if (lane == 0) bulk_wait_read_1();
            __syncwarp();
          }
#pragma unroll
          for (int q = 0; q < 8; ++q)
            sts_f4(buf + (uint32_t)lane * 128u + (uint32_t)((q ^ (lane & 7)) * 16), alpha * __uint_as_float(r[4 * q]),
                   alpha * __uint_as_float(r[4 * q + 1]), alpha * __uint_as_float(r[4 * q + 2]),
                   alpha * __uint_as_float(r[4 * q + 3]));
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            if (row0 < M) {
              if (g.accumulate) tma_reduce_add_3d(&map_c, buf, n0 + 32 * ci, row0, part);
              else tma_store_3d(&map_c, buf, n0 + 32 * ci, row0, part);
            }
            bulk_commit();
          }
          __syncwarp();
        }
      } else if constexpr (EPI == kTcRows) {
        // each lane writes its own row's 32 columns: 64 or 128 consecutive bytes
        const int32_t to = row < M ? g.row_map[row] : -1;
        const bool row_on = to >= 0 && to < g.M;      // a row map that is no map writes nothing
        if (row < M && !row_on) atomicOr(&g_device_error, kDevErrIndex);
        const int64_t dst = row_on ? (int64_t)to * g.ldc : 0;
#pragma unroll 1
        for (int c0 = 0; c0 < kBN && n0 + c0 < g.N; c0 += 32) {
          uint32_t r[32];
          __syncwarp();
          tmem_ld32(acc + (uint32_t)c0, r);
          tmem_ld_wait();
          const int col = n0 + c0, n = min(32, g.N - col);
          if (!row_on) continue;
#pragma unroll
          for (int jj = 0; jj < 32; ++jj) r[jj] = __float_as_uint(alpha * __uint_as_float(r[jj]));
          if (g.out_fp32) {
            float* p = g.C + dst + col;
#pragma unroll
            for (int q = 0; q < 8; ++q) {
              const float4 v = make_float4(__uint_as_float(r[4 * q]), __uint_as_float(r[4 * q + 1]),
                                           __uint_as_float(r[4 * q + 2]), __uint_as_float(r[4 * q + 3]));
              if (4 * q + 4 <= n) *reinterpret_cast<float4*>(p + 4 * q) = v;
            }
#pragma unroll
            for (int jj = 0; jj < 32; ++jj)
              if (jj >= (n & ~3) && jj < n) p[jj] = __uint_as_float(r[jj]);
          } else {
            __nv_bfloat16* p = reinterpret_cast<__nv_bfloat16*>(g.C) + dst + col;
            uint32_t w[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const __nv_bfloat162 h = __floats2bfloat162_rn(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
              w[i] = *reinterpret_cast<const uint32_t*>(&h);
            }
#pragma unroll
            for (int q = 0; q < 4; ++q)
              if (8 * q + 8 <= n) *reinterpret_cast<uint4*>(p + 8 * q) = make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
#pragma unroll
            for (int jj = 0; jj < 32; ++jj)
              if (jj >= (n & ~7) && jj < n) p[jj] = __float2bfloat16_rn(__uint_as_float(r[jj]));
          }
        }
      } else if (g.tma) {
        // 32 x 32 boxes through two 4 KB staging buffers per warp, 128-byte
        // swizzled to match the store's tensor map (conflict-free 16-byte
        // writes); one thread stores or reduce-adds each box, and a buffer
        // is rewritten only once its previous store has read it.  A tensor store
        // writes whole 16-byte units: of a C whose rows end inside one, the last
        // columns' box goes element by element, so that the padding stays as it
        // is (8192 x 8191 x 1024 in rows of 8192: 98 us, all of C that way 140, 8192 columns 99)
        const int row0 = m0 + 32 * quarter;
        const int whole = g.N & 3 ? g.N & ~31 : INT32_MAX;      // boxes from here on
        float rm = -INFINITY, rs = 0.0f;
#pragma unroll 1
        for (int ci = 0; ci < kBN / 32; ++ci) {
          uint32_t r[32];
          tmem_ld32(acc + (uint32_t)(32 * ci), r);
          tmem_ld_wait();
          if (g.row_stats) {
            float x[32];
#pragma unroll
            for (int jj = 0; jj < 32; ++jj) x[jj] = g.alpha * __uint_as_float(r[jj]);
            fold_row_stats(x, min(32, g.N - (n0 + 32 * ci)), rm, rs);
          }
          if (n0 + 32 * ci >= whole) {
            if (row < g.M) {
              float* p = g.C + (int64_t)row * g.ldc + n0 + 32 * ci;
#pragma unroll
              for (int jj = 0; jj < 32; ++jj)
                if (n0 + 32 * ci + jj < g.N) {
                  const float v = g.alpha * __uint_as_float(r[jj]);
                  p[jj] = g.accumulate ? p[jj] + v : v;
                }
            }
            __syncwarp();
            continue;
          }
          const uint32_t buf = stg + (uint32_t)(boxes & 1) * 4096u;
          if (boxes >= 2) {
            if (lane == 0) bulk_wait_read_1();
            __syncwarp();
          }
#pragma unroll
          for (int q = 0; q < 8; ++q)
            sts_f4(buf + (uint32_t)lane * 128u + (uint32_t)((q ^ (lane & 7)) * 16), g.alpha * __uint_as_float(r[4 * q]),
                   g.alpha * __uint_as_float(r[4 * q + 1]), g.alpha * __uint_as_float(r[4 * q + 2]),
                   g.alpha * __uint_as_float(r[4 * q + 3]));
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            if (row0 < g.M && n0 + 32 * ci < g.N) {
              if (g.accumulate) tma_reduce_add_2d(&map_c, buf, n0 + 32 * ci, row0);
              else tma_store_2d(&map_c, buf, n0 + 32 * ci, row0);
            }
            bulk_commit();
          }
          ++boxes;
          __syncwarp();
        }
        if (g.row_stats && row < g.M) g.row_stats[(int64_t)row * n_tiles + nt] = make_float2(rm, rs);
      } else {
        const bool row_on = row < g.M;
        float* crow = g.C + (int64_t)row * g.ldc;
        float rm = -INFINITY, rs = 0.0f;
#pragma unroll 1
        for (int c0 = 0; c0 < kBN; c0 += 32) {
          uint32_t r[32];
          tmem_ld32(acc + (uint32_t)c0, r);
          tmem_ld_wait();
          const int col0 = n0 + c0;
          if (g.row_stats) {
            float x[32];
#pragma unroll
            for (int jj = 0; jj < 32; ++jj) x[jj] = g.alpha * __uint_as_float(r[jj]);
            fold_row_stats(x, min(32, g.N - col0), rm, rs);
          }
          if (!row_on || col0 >= g.N) continue;
#pragma unroll
          for (int jj = 0; jj < 32; ++jj) {
            if (col0 + jj < g.N) {
              const float v = g.alpha * __uint_as_float(r[jj]);
              crow[col0 + jj] = g.accumulate ? crow[col0 + jj] + v : v;
            }
          }
        }
        if (g.row_stats && row_on) g.row_stats[(int64_t)row * n_tiles + nt] = make_float2(rm, rs);
      }
      // this warp is done with accumulator buffer b: tell the MMA thread
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (rank == 0) mbar_arrive_local(&tempty[b]);
        else mbar_arrive_remote_release(tempty_lead + 8u * (uint32_t)b);
      }
    }
    if (lane == 0) bulk_wait_all();
  }
  // both CTAs are done with the pair's TMEM (the peer's epilogue waited for
  // every MMA into it) before the pair releases it
  tc_fence_before();
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 2 * kTmemCols);
  }
}

// Map of the tensor stores of partial products [splits][M][N]: fp32, 3D boxes of 32 x 32 x 1.
sf_status make_map_split(CUtensorMap* map, float* C, int64_t M, int64_t N, int64_t ldc, int64_t splits) {
  cuuint64_t dims[3] = {(cuuint64_t)N, (cuuint64_t)M, (cuuint64_t)splits};
  cuuint64_t strides[2] = {(cuuint64_t)(ldc * 4), (cuuint64_t)(M * ldc * 4)};
  cuuint32_t box[3] = {32, 32, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = tensor_map_encoder()(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, C, dims, strides, box, estr,
                                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                                    CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(SF_ERR_CUDA, "cuTensorMapEncodeTiled (partial C) failed (%d)", (int)r);
  return SF_OK;
}

// Clusters of two GEMM CTAs that fit on the device at once (cached per
// device): the persistent grid's size.
sf_status resident_pairs(cudaLaunchConfig_t* cfg, int* out) {
  static std::mutex mu;
  static std::map<int, int> cache;
  int dev = 0;
  SF_CUDA_TRY(cudaGetDevice(&dev), "cudaGetDevice");
  std::lock_guard<std::mutex> lock(mu);
  auto it = cache.find(dev);
  if (it == cache.end()) {
    int n = 0;
    cudaLaunchConfig_t one = *cfg;       // the same for all epilogues: shared memory allows one CTA an SM
    cfg = &one;
    cfg->blockDim = dim3(TcStages<kTcF32>::kThreads);
    cfg->gridDim = dim3((unsigned)(kPair * std::max(1, sm_count() / kPair)));
    SF_TRY(allow_dynamic_smem(reinterpret_cast<const void*>(&k_tc_gemm<kTcF32>), kGemmSmem));
    SF_CUDA_TRY(cudaOccupancyMaxActiveClusters(&n, k_tc_gemm<kTcF32>, cfg), "cudaOccupancyMaxActiveClusters (k_tc_gemm)");
    if (n < 1) return fail(SF_ERR_UNSUPPORTED, "no cluster of two GEMM CTAs fits on this device");
    it = cache.emplace(dev, n).first;
  }
  *out = it->second;
  return SF_OK;
}

}  // namespace

// C = alpha A B^T (+ C); shared with the cross-entropy unit.
sf_status tc_gemm(const void* A, bool a_mn, const void* B, bool b_mn, float* C, int64_t M, int64_t N, int64_t K,
                  int64_t lda, int64_t ldb, int64_t ldc, float alpha, bool accumulate, cudaStream_t s,
                  float2* row_stats) {
  TcJob j;
  j.A = A;
  j.a_mn = a_mn;
  j.B = B;
  j.b_mn = b_mn;
  j.C = C;
  j.M = M;
  j.N = N;
  j.K = K;
  j.lda = lda;
  j.ldb = ldb;
  j.ldc = ldc;
  j.alpha = alpha;
  j.accumulate = accumulate;
  j.row_stats = row_stats;
  return tc_gemm(j, s);
}

sf_status tc_gemm(const TcJob& j, cudaStream_t s) {
  const bool writes = j.epi != kTcStats || j.store;      // whether C is written
  if (!j.A || !j.B || (writes && !j.C)) return fail(SF_ERR_INVALID, "A, B or C is NULL");
  if (j.M < 1 || j.N < 1 || j.K < 1) return fail(SF_ERR_INVALID, "M, N, K must be >= 1");
  if (j.M > INT32_MAX - 2 * kPair * kBM || j.N > INT32_MAX - kBN || j.K > INT32_MAX - kBK)
    return fail(SF_ERR_UNSUPPORTED, "M, N, K must be below 2^31");
  if (j.lda < (j.a_mn ? j.M : j.K) || j.ldb < (j.b_mn ? j.N : j.K) || (writes && j.ldc < j.N))
    return fail(SF_ERR_INVALID, "leading dimensions must be >= the stored rows' length (lda: K or M, ldb: K or N; "
                                "ldc: N)");
  if ((j.lda * 2) % 16 || (j.ldb * 2) % 16 || (reinterpret_cast<uintptr_t>(j.A) % 16) ||
      (reinterpret_cast<uintptr_t>(j.B) % 16))
    return fail(SF_ERR_UNSUPPORTED, "A and B need 16-byte aligned bases and rows (lda, ldb multiples of 8)");
  if (!tensor_map_encoder()) return fail(SF_ERR_UNSUPPORTED, "cuTensorMapEncodeTiled is not available");
  // the tensor maps below may only address this device's own memory
  if (!j.checked && (!on_current_device(j.A) || !on_current_device(j.B) || (writes && !on_current_device(j.C))))
    return fail(SF_ERR_INVALID, "A, B and C must be device memory of the current device");
  CUtensorMap ma, mb;
  int a_form = 0, b_form = 0;      // 0 K-major, 1 MN-major in 2D boxes, 2 MN-major in 3D boxes
  if (j.a_mn) {
    a_form = make_map_mn3d(&ma, j.A, j.M, j.K, j.lda) ? 2 : 1;
    if (a_form == 1) SF_TRY(make_map(&ma, j.A, j.M, j.K, j.lda, kBK));
  } else {
    SF_TRY(make_map(&ma, j.A, j.K, j.M, j.lda, kBM));
  }
  if (j.b_mn) {
    b_form = make_map_mn3d(&mb, j.B, j.N, j.K, j.ldb) ? 2 : 1;
    if (b_form == 1) SF_TRY(make_map(&mb, j.B, j.N, j.K, j.ldb, kBK));
  } else {
    SF_TRY(make_map(&mb, j.B, j.K, j.N, j.ldb, kBRows));
  }
  TcGemmArgs g{};
  g.C = static_cast<float*>(j.C);
  g.ldc = j.ldc;
  g.M = (int32_t)j.M;
  g.N = (int32_t)j.N;
  g.K = (int32_t)j.K;
  g.alpha = j.alpha;
  g.accumulate = j.accumulate ? 1 : 0;
  g.n_fast = j.M > j.N ? 1 : 0;
  g.a_mn = a_form;
  g.b_mn = b_form;
  g.row_stats = j.row_stats;
  g.splits = j.epi == kTcSplit ? j.splits : 1;
  g.stats_ld = j.stats_ld;
  g.col0 = j.col0;
  g.store = j.store ? 1 : 0;
  g.labels = j.labels;
  g.label_logit = j.label_logit;
  g.lse = j.lse;
  g.scale = j.scale;
  g.m_dev = j.m_dev;
  g.k_dev = j.k_dev;
  g.row_map = j.row_map;
  g.out_fp32 = j.out_fp32 ? 1 : 0;
  const bool c_aligned = reinterpret_cast<uintptr_t>(j.C) % 16 == 0;
  CUtensorMap mc = ma;       // unused unless C is written by tensor stores
  const void* kernel = nullptr;
  int threads = 0;
  auto take = [&](const void* k, int n) {
    kernel = k;
    threads = n;
  };
  switch (j.epi) {
    case kTcF32:
      g.tma = j.ldc % 4 == 0 && c_aligned ? 1 : 0;      // else element by element
      if (g.tma) SF_TRY(make_map_c(&mc, g.C, j.M, j.N, j.ldc));
      take(reinterpret_cast<const void*>(&k_tc_gemm<kTcF32>), TcStages<kTcF32>::kThreads);
      break;
    case kTcSplit:
      if (j.splits < 1 || j.splits > (j.K + kBK - 1) / kBK) return fail(SF_ERR_INVALID, "splits must lie in 1..slabs of K");
      if (j.ldc % 4 || !c_aligned) return fail(SF_ERR_UNSUPPORTED, "partial products need 16-byte aligned rows");
      SF_TRY(make_map_split(&mc, g.C, j.M, j.N, j.ldc, j.splits));
      take(reinterpret_cast<const void*>(&k_tc_gemm<kTcSplit>), TcStages<kTcSplit>::kThreads);
      break;
    case kTcRows:
      if (!c_aligned || j.ldc * (j.out_fp32 ? 4 : 2) % 16) return fail(SF_ERR_UNSUPPORTED, "C needs 16-byte aligned rows");
      take(reinterpret_cast<const void*>(&k_tc_gemm<kTcRows>), TcStages<kTcRows>::kThreads);
      break;
    case kTcBf16:
    case kTcGrad:
    case kTcStats:
      if (writes) {
        if (j.ldc % 8 || !c_aligned) return fail(SF_ERR_UNSUPPORTED, "a bf16 C needs 16-byte aligned rows");
        SF_TRY(make_map_c16(&mc, j.C, j.M, j.N, j.ldc));
      }
      if (j.epi == kTcBf16) take(reinterpret_cast<const void*>(&k_tc_gemm<kTcBf16>), TcStages<kTcBf16>::kThreads);
      else if (j.epi == kTcGrad) take(reinterpret_cast<const void*>(&k_tc_gemm<kTcGrad>), TcStages<kTcGrad>::kThreads);
      else take(reinterpret_cast<const void*>(&k_tc_gemm<kTcStats>), TcStages<kTcStats>::kThreads);
      break;
  }
  SF_TRY(allow_dynamic_smem(kernel, kGemmSmem));
  const int64_t items = ((j.M + kPair * kBM - 1) / (kPair * kBM)) * ((j.N + kBN - 1) / kBN) * g.splits;
  if (items > INT32_MAX) return fail(SF_ERR_UNSUPPORTED, "too many tiles");
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kPair;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = kGemmSmem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int pairs = 0;
  SF_TRY(resident_pairs(&cfg, &pairs));
  if (j.chained) cfg.numAttrs = 2;
  cfg.gridDim = dim3((unsigned)(kPair * std::min<int64_t>(items, pairs)));
  void* args[] = {&ma, &mb, &mc, &g};
  SF_CUDA_TRY(cudaLaunchKernelExC(&cfg, kernel, args), "launch k_tc_gemm");
  return SF_OK;
}

const void* device_error_gemm() { return &g_device_error; }

}  // namespace sf

extern "C" {

sf_status sf_gemm_abt_bf16(const void* A, const void* B, float* C, int64_t M, int64_t N, int64_t K, int64_t lda,
                           int64_t ldb, int64_t ldc, float alpha, int accumulate, void* stream) {
  sf::clear_error();
  sf::NvtxRange nvtx_range("sf_gemm_abt_bf16");
  return sf::tc_gemm(A, false, B, false, C, M, N, K, lda, ldb, ldc, alpha, accumulate != 0, sf::as_stream(stream),
                     nullptr);
}

sf_status sf_gemm_bf16(const void* A, int a_layout, const void* B, int b_layout, float* C, int64_t M, int64_t N,
                       int64_t K, int64_t lda, int64_t ldb, int64_t ldc, float alpha, int accumulate, void* stream) {
  sf::clear_error();
  sf::NvtxRange nvtx_range("sf_gemm_bf16");
  if ((a_layout != 0 && a_layout != 1) || (b_layout != 0 && b_layout != 1))
    return sf::fail(SF_ERR_INVALID, "a_layout and b_layout must be 0 (K-major) or 1 (MN-major)");
  return sf::tc_gemm(A, a_layout == 1, B, b_layout == 1, C, M, N, K, lda, ldb, ldc, alpha, accumulate != 0,
                     sf::as_stream(stream), nullptr);
}

}  // extern "C"
