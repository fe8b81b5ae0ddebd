// The weight gradient of a linear layer from the 8-bit checkpoint of its
// input: dW = base + dY^T X, X = value * scale, on the tensor cores.
//
// The pair form of tc_gemm.cu (256 x 256 tiles of dW by clusters of two CTAs,
// tcgen05.mma into tensor memory), with X turned into bf16 in one of two places
// (restores(), below).  On the way: a CTA's 64-token slab of the checkpoint (64 x
// 128 values, 8 KB by TMA) is read from shared memory by four converter warps,
// multiplied by its scales and written as the swizzled MN-major operand that
// the MMA reads (16 KB); three such groups take the slabs in turn, and the
// activations are never restored in memory.  Or before: a launch of its own
// restores X in the workspace, and slabs of it are copied by TMA as dY's are.
// With power-of-two scales from 2^-124 on value * scale is exact in bf16.
//
// 8192 tokens, 4096 -> 11008, bf16: 422 us with X restored first (1750 TFLOP/s in a short
// replay, the tensor pipe 80 % busy in its 388 us; 450 to 468 us call after call, under
// the power cap), 519 us converted on the way; 4096 -> 1024
// converted 62 us (tensor pipe 43 %: 64 tiles on 76 pairs).
//
// Sums: the tensor cores cut the low bits of their fp32 accumulator at every
// step, which shrinks a long sum (measured on 4096 tokens 4e-6 of it, on 16384
// 2e-5).  So a span of 512 tokens is summed there, and the epilogue's threads
// add the spans in their registers, rounded to nearest, while the MMAs of the
// next span fill the other accumulator: eight warps hold a tile's 32768 sums a
// CTA, 128 a thread, for which they take registers from the other warps.
//
// Tiles that do not fill a whole wave of pairs are split over the tokens, so
// that all pairs work on them; their parts go through the workspace and a
// second kernel adds them in order.
#include <algorithm>
#include <map>
#include <mutex>

#include "lanes.cuh"
#include "tc_pair.cuh"

namespace sf {
namespace {

struct WgradArgs {
  const __nv_bfloat16* dy;   // [tokens][ldy]
  const void* base;          // [out][ldbase], may be null or dw
  void* dw;                  // [out][lddw]
  int64_t ldy, ldbase, lddw;
  int64_t tokens, out, in;
  int32_t fp32;              // dw and base
  Ck ck;
};

__device__ __forceinline__ float dw_at(const void* p, int fp32, int64_t i) {
  return fp32 ? static_cast<const float*>(p)[i] : __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}

constexpr int kSpan = 8;                       // slabs that one accumulator sums
constexpr int kRing = 6;                       // slabs of dY in flight
constexpr int kRing8 = 6;                      // slabs of the checkpoint
constexpr int kSlots = 4;                      // converted slabs
constexpr int kA = kBM * kBK * 2;              // 16 KB: 128 columns of dY
constexpr int kB8 = 128 * kBK;                 // 8 KB: 128 columns of the checkpoint
constexpr int kB = kBRows * kBK * 2;           // 16 KB: the same in bf16
constexpr int kEpiWarps = 8;
constexpr int kConvWarps = 4, kConvGroups = 3; // converter warps of a slab; the groups take slabs in turn
// a group finds every phase of the barriers that it waits on
static_assert(kRing % kConvGroups == 0 && kRing8 % kConvGroups == 0 && kSlots <= kRing, "the groups' slabs");
template <bool FUSED>
constexpr int kTcThreads = 32 * (4 + (FUSED ? kConvWarps * kConvGroups : 0) + kEpiWarps);
constexpr int kStaging = 2048;                 // an epilogue warp's box: 32 rows of 64 bytes
template <bool FUSED>
constexpr size_t kTcSmem = (size_t)kRing * kA + (FUSED ? (size_t)kRing8 * kB8 + (size_t)kSlots * kB : (size_t)kRing * kB) +
                           kEpiWarps * kStaging + 1024 + 256;
constexpr int64_t kMaxParts = 160;             // parts of split tiles, 256 KB of workspace each
constexpr int64_t kPartFloats = 2 * kBM * kBN;

struct TcArgs {
  int32_t out, in, tokens;
  int32_t n_fast;            // tile order: columns fastest
  int32_t whole, parts;      // tiles before `whole` are one item each, later ones `parts`
  int32_t items;
  int32_t tma;               // dW by tensor stores
  int32_t base_vec;          // base in 16-byte loads
  void* dw;
  const void* base;
  int64_t lddw, ldbase;
  float* ws;
  Ck ck;
};

template <int N>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// 8 consecutive fp32 columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}

// What the second CTA's converters write is read by MMAs that the first CTA's thread issues, and they write again where
// those have read: orders between two CTAs.  A release or an acquire at cluster scope waits for all that its thread has in
// flight, of a converter the next slabs' scales (8192 tokens 4096 -> 1024 in 111 us where one idle warp releases for them,
// 76 with two that take turns).  So the fences here are restricted to shared memory, and cost nothing that shows (61.7 us).
//
// Arrival on a barrier of the first CTA, after this thread's accesses of its own CTA's shared memory and those that it met
// at a barrier.
__device__ __forceinline__ void mbar_arrive_pair(uint32_t cluster_bar) {
  asm volatile("fence.release.sync_restrict::shared::cta.cluster;\n mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}

// Bounded wait for arrivals from either CTA, before this thread's accesses of the pair's shared memory.
__device__ __forceinline__ bool mbar_wait_pair(uint64_t* bar, uint32_t parity) {
  auto test = [&]() {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.relaxed.cluster.shared::cta.b64 p, [%1], %2;\n"
        " selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
  };
  if (!test()) {
    const long long t0 = clock64();
    while (!test()) {
      if (clock64() - t0 > kWaitLimitCycles) {
        atomicOr(&g_device_error, kDevErrTimeout);
        return false;
      }
    }
  }
  asm volatile("fence.acquire.sync_restrict::shared::cluster.cluster;" ::: "memory");
  return true;
}

// An item: a tile of dW and the slabs of tokens to sum.
struct Item {
  int mt, nt, k0, k1, part;      // part < 0: a whole tile, else its place in the workspace
};
__device__ __forceinline__ Item item_of(const TcArgs& g, int it, int m_tiles, int n_tiles, int nk) {
  Item i;
  int t = it;
  i.k0 = 0, i.k1 = nk, i.part = -1;
  if (it >= g.whole) {
    const int j = it - g.whole, p = j % g.parts;
    t = g.whole + j / g.parts;
    i.k0 = (int)((int64_t)nk * p / g.parts);
    i.k1 = (int)((int64_t)nk * (p + 1) / g.parts);
    i.part = j;
  }
  i.mt = g.n_fast ? t / n_tiles : t % m_tiles;
  i.nt = g.n_fast ? t % n_tiles : t / m_tiles;
  return i;
}

// FP32: dW's type.  FUSED: X converted here; else X is a bf16 matrix (map_b), copied like dY.
template <bool FP32, bool FUSED>
__global__ void __launch_bounds__(kTcThreads<FUSED>, 1)
    k_wgrad_tc(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
               const __grid_constant__ CUtensorMap map_c, const TcArgs g, const int a_form) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  // [dY: kRing x 16 KB] [X in bf16: kX x 16 KB] [checkpoint: kRing8 x 8 KB] [staging: 8 x 2 KB] [barriers]
  constexpr int kX = FUSED ? kSlots : kRing;
  const uint32_t ring_a = smem_u32(smem), conv = ring_a + kRing * kA, ring_b = conv + kX * kB;
  const uint32_t staging = ring_b + (FUSED ? kRing8 * kB8 : 0);
  uint64_t* ready = reinterpret_cast<uint64_t*>(smem + kTcSmem<FUSED> - 1024 - 256);   // first CTA: dY and X are there, in both
  uint64_t* empty = ready + kRing;         // the slab's MMAs are done
  uint64_t* land = empty + kRing;          // the CTA's own values landed
  uint64_t* taken = land + kRing8;         // its converters have read them
  uint64_t* tfull = taken + kRing8;        // [2] accumulator b holds a span
  uint64_t* tempty = tfull + 2;            // [2] both CTAs have read accumulator b (first CTA)
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tempty + 2);

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int pair = blockIdx.x / kPair, n_pairs = gridDim.x / kPair;
  if (threadIdx.x == 0) {
    prefetch_tensormap(&map_a);
    prefetch_tensormap(&map_b);
    for (int s = 0; s < kRing; ++s) {
      mbar_init(&ready[s], 1 + (FUSED ? kPair * kConvWarps : 0));      // the copies, both CTAs' converters
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < kRing8; ++s) {
      mbar_init(&land[s], 1);
      mbar_init(&taken[s], kConvWarps);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], kPair * kEpiWarps);
    }
    fence_mbar_init_cluster();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), 2 * kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  griddep_launch_dependents();
  if (!FUSED) griddep_wait();      // X is written by the kernel before

  const int nk = (g.tokens + kBK - 1) / kBK;
  const int m_tiles = (g.out + kPair * kBM - 1) / (kPair * kBM), n_tiles = (g.in + kBN - 1) / kBN;
  if (warp < 4) {
    if (FUSED) regs_down<24>();
    if (warp == 0 && lane == 0) {
      const uint32_t ready_lead = cluster_addr(smem_u32(ready), 0);
      int i = 0, landing = 0;
      bool failed = false;
      for (int it = pair; it < g.items && !failed; it += n_pairs) {
        const Item w = item_of(g, it, m_tiles, n_tiles, nk);
        const int m0 = w.mt * (kPair * kBM) + (int)rank * kBM, nb = w.nt * kBN + (int)rank * kBRows;
        for (int kb = w.k0; kb < w.k1; ++kb, ++i) {
          const int s = i % kRing, s8 = i % kRing8;
          if (FUSED) {
            if (i >= kRing8 && !mbar_wait(&taken[s8], (uint32_t)(i / kRing8 - 1) & 1u)) {
              failed = true;
              break;
            }
            mbar_arrive_expect_tx(&land[s8], kB8);
            tma_load_2d(smem + (ring_b - ring_a) + s8 * kB8, &map_b, &land[s8], nb, kb * kBK);
            landing = i + 1;
          }
          if (i >= kRing && !mbar_wait_cluster(&empty[s], (uint32_t)(i / kRing - 1) & 1u)) {
            failed = true;
            break;
          }
          if (rank == 0) mbar_arrive_expect_tx(&ready[s], kPair * (kA + (FUSED ? 0 : kB)));
          const uint32_t st = ring_a + (uint32_t)s * kA, bar = ready_lead + 8u * (uint32_t)s;
          if (a_form == 2) {
            tma_load_3d_pair(st, &map_a, bar, 0, kb * kBK, m0 >> 6);
          } else {
            tma_load_2d_pair(st, &map_a, bar, m0, kb * kBK);
            tma_load_2d_pair(st + kMnBox, &map_a, bar, m0 + 64, kb * kBK);
          }
          if (!FUSED) tma_load_3d_pair(conv + (uint32_t)s * kB, &map_b, bar, 0, kb * kBK, nb >> 6);
        }
      }
      // the last copies have landed before the pair can exit (immediate unless a wait ran out)
      for (int j = landing > kRing8 ? landing - kRing8 : 0; j < landing; ++j) mbar_wait(&land[j % kRing8], (uint32_t)(j / kRing8) & 1u);
      if (rank == 0)
        for (int j = i > kRing ? i - kRing : 0; j < i; ++j) mbar_wait_cluster(&ready[j % kRing], (uint32_t)(j / kRing) & 1u);
    } else if (warp == 1 && lane == 0 && rank == 0) {
      const uint32_t idesc = kIdesc | (1u << 15) | (1u << 16);      // both operands MN-major
      const uint32_t empty_a = smem_u32(empty), tfull_a = smem_u32(tfull);
      int i = 0, j = 0;
      bool failed = false;
      for (int it = pair; it < g.items && !failed; it += n_pairs) {
        const Item w = item_of(g, it, m_tiles, n_tiles, nk);
        for (int k0 = w.k0; k0 < w.k1 && !failed; k0 += kSpan, ++j) {
          const int b = j & 1, use = j >> 1, k1 = min(k0 + kSpan, w.k1);
          if (use > 0 && !mbar_wait_cluster(&tempty[b], (uint32_t)(use - 1) & 1u)) {
            failed = true;
            break;
          }
          tc_fence_after();
          const uint32_t d_tmem = tmem + (uint32_t)(b * kTmemCols);
          for (int kb = k0; kb < k1; ++kb, ++i) {
            const int s = i % kRing;
            if (!mbar_wait_cluster(&ready[s], (uint32_t)(i / kRing) & 1u)) {
              failed = true;
              break;
            }
            tc_fence_after();
            const uint64_t adesc = umma_desc_mn_sw128(ring_a + (uint32_t)s * kA), bdesc = umma_desc_mn_sw128(conv + (uint32_t)(i % kX) * kB);
#pragma unroll
            for (int k = 0; k < kBK / 16; ++k) tc_mma(d_tmem, adesc + 128u * k, bdesc + 128u * k, idesc, kb != k0 || k != 0 ? 1u : 0u);
            tc_commit_pair(empty_a + 8u * (uint32_t)s);
          }
          tc_commit_pair(tfull_a + 8u * (uint32_t)b);
        }
      }
    }
  } else if (FUSED && warp < 4 + kConvWarps * kConvGroups) {
    if (FUSED) regs_down<48>();
    // A thread's 16 columns of tokens r0, r0 + 16, r0 + 32, r0 + 48 of a slab.  Both sides are swizzled (16-byte unit ^
    // row mod 8); eight neighbouring lanes take four units of two rows that differ in bits 0 and 2, so that neither
    // their loads (units c) nor their stores (2 c, then 2 c + 1) meet in a bank.
    const int group = (warp - 4) / kConvWarps, tid = threadIdx.x & 127;
    const int cc = (tid & 3) | (tid >> 1 & 4), r0 = ((tid >> 4 & 3) ^ 5 * (tid >> 2 & 1)) + (tid >> 6) * 8;
    const uint32_t ready_lead = cluster_addr(smem_u32(ready), 0);
    // the slabs of this group, one ahead
    int it = pair, kb = 0;
    Item w{};
    auto enter = [&]() {
      if (it < g.items) w = item_of(g, it, m_tiles, n_tiles, nk);
      kb = w.k0;
    };
    auto advance = [&]() {
      if (it < g.items && ++kb == w.k1) {
        it += n_pairs;
        enter();
      }
    };
    // A slab's scales, as loaded: turned into fp32 when their values have come, so that nothing waits for them here.
    // Past the last token they are zero or 2^-127, as finite as the zeros that they scale; past the last column the last
    // one's are taken, whose products no output has.
    auto scales = [&](uint32_t (&f)[4]) {
      const int c = min(w.nt * kBN + (int)rank * kBRows + 16 * cc, g.in - 1) >> (g.ck.group_log2 ? g.ck.group_log2 : 31);
      const int t0 = kb * kBK + r0;
      int64_t at[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) at[q] = (int64_t)(t0 + 16 * q) * g.ck.n_groups + c;
      if (g.ck.s8) {
#pragma unroll
        for (int q = 0; q < 4; ++q) f[q] = t0 + 16 * q < g.tokens ? __ldg(g.ck.s8 + at[q]) : 0u;
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q) f[q] = t0 + 16 * q < g.tokens ? __float_as_uint(__ldg(g.ck.s32 + at[q])) : 0u;
      }
    };
    const uint32_t src0 = ring_b + 128u * r0 + 16u * (cc ^ (r0 & 7));
    const uint32_t dst0 = conv + (uint32_t)(cc >> 2) * kMnBox + 128u * r0 + 16u * ((2 * (cc & 3)) ^ (r0 & 7));
    enter();
    for (int k = 0; k < group; ++k) advance();
    uint32_t next[4] = {};
    if (it < g.items) scales(next);
    for (int i = group; it < g.items; i += kConvGroups) {
      const int s = i % kRing, s8 = i % kRing8;
      uint32_t f[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) f[q] = next[q];
#pragma unroll
      for (int k = 0; k < kConvGroups; ++k) advance();
      if (it < g.items) scales(next);
      if (!mbar_wait(&land[s8], (uint32_t)(i / kRing8) & 1u)) break;
      const uint32_t src = src0 + (uint32_t)s8 * kB8, dst = dst0 + (uint32_t)(i % kSlots) * kB;
      int4 v[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] = lds_i4(src + 2048u * q);
      // the slab that the slot held has been multiplied
      if (i >= kSlots && !mbar_wait_pair(&empty[(i - kSlots) % kRing], (uint32_t)((i - kSlots) / kRing) & 1u)) break;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t in[4] = {(uint32_t)v[q].x, (uint32_t)v[q].y, (uint32_t)v[q].z, (uint32_t)v[q].w};
        const float scale = g.ck.s8 ? e8m0_value(f[q]) : __uint_as_float(f[q]);
        const uint64_t f2 = pack_f2(scale, scale);
        uint32_t o[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float2 x = e4m3x2_value(in[e >> 1] >> (16 * (e & 1)) & 0xffffu);
          o[e] = bf16x2_rn(fmul2(pack_f2(x.x, x.y), f2));
        }
        // (16 rows on, the swizzle is the same)
        const uint32_t to = dst + 2048u * q;
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to), "r"(o[0]), "r"(o[1]), "r"(o[2]), "r"(o[3]));
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to ^ 16u), "r"(o[4]), "r"(o[5]), "r"(o[6]), "r"(o[7]));
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        // (not before: a copy into the values' place must find every load of them done, and that they are is certain
        // only once they have been used)
        mbar_arrive_local(&taken[s8]);
        if (rank == 0) mbar_arrive_local(&ready[s]);
        else mbar_arrive_pair(ready_lead + 8u * (uint32_t)s);
      }
    }
  } else {
    if (FUSED) regs_up<152>();
    const int ew = warp - 4 - (FUSED ? kConvWarps * kConvGroups : 0), quarter = warp & 3, half = ew / 4;
    const uint32_t lane_off = (uint32_t)(32 * quarter) << 16;
    const uint32_t buf = staging + (uint32_t)ew * kStaging;
    const uint32_t tempty_lead = cluster_addr(smem_u32(tempty), 0);
    int j = 0;
    bool failed = false;
    for (int it = pair; it < g.items && !failed; it += n_pairs) {
      const Item w = item_of(g, it, m_tiles, n_tiles, nk);
      float acc[128];
#pragma unroll
      for (int e = 0; e < 128; ++e) acc[e] = 0.0f;
      for (int k0 = w.k0; k0 < w.k1; k0 += kSpan, ++j) {
        const int b = j & 1;
        if (!mbar_wait_cluster(&tfull[b], (uint32_t)(j >> 1) & 1u)) {
          failed = true;
          break;
        }
        tc_fence_after();
        const uint32_t at = tmem + (uint32_t)(b * kTmemCols + 128 * half) + lane_off;
#pragma unroll
        for (int q = 0; q < 16; ++q) {
          uint32_t r[8];
          __syncwarp();
          tmem_ld8(at + 8u * q, r);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[8 * q + e] += __uint_as_float(r[e]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (rank == 0) mbar_arrive_local(&tempty[b]);
          else mbar_arrive_remote_release(tempty_lead + 8u * (uint32_t)b);
        }
      }
      if (failed) break;
      const int row_in = (int)rank * kBM + 32 * quarter + lane;      // within the tile
      const int row0 = w.mt * (kPair * kBM) + (int)rank * kBM + 32 * quarter, row = row0 + lane;
      const int col0 = w.nt * kBN + 128 * half;
      if (w.part >= 0) {      // [part][column / 4][row][4]: a warp's rows side by side
        float4* p = reinterpret_cast<float4*>(g.ws) + ((int64_t)w.part * (kBN / 4) + 32 * half) * (kPair * kBM) + row_in;
#pragma unroll
        for (int q = 0; q < 32; ++q)
          p[(int64_t)q * (kPair * kBM)] = make_float4(acc[4 * q], acc[4 * q + 1], acc[4 * q + 2], acc[4 * q + 3]);
        continue;
      }
      constexpr int kUnit = FP32 ? 4 : 8;                            // elements of 16 bytes
      constexpr int kBox = FP32 ? 16 : 32;                           // columns of a staging box
      const int whole = g.in % kUnit ? g.in : INT32_MAX;      // a row's ragged end goes element by element
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int c0 = col0 + 32 * q;
        float v[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] = acc[32 * q + e];
        if (g.base && row < g.out && c0 < g.in) {
          const int n = min(32, g.in - c0);
          if (FP32) {
            const float* p = static_cast<const float*>(g.base) + (int64_t)row * g.ldbase + c0;
            if (g.base_vec && n == 32) {
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float4 u = *reinterpret_cast<const float4*>(p + 4 * e);
                v[4 * e] += u.x, v[4 * e + 1] += u.y, v[4 * e + 2] += u.z, v[4 * e + 3] += u.w;
              }
            } else {
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (e < n) v[e] += p[e];
            }
          } else {
            const uint16_t* p = static_cast<const uint16_t*>(g.base) + (int64_t)row * g.ldbase + c0;
            if (g.base_vec && n == 32) {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const uint4 u = *reinterpret_cast<const uint4*>(p + 8 * e);
                const uint32_t x[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                for (int f = 0; f < 4; ++f) v[8 * e + 2 * f] += __uint_as_float(x[f] << 16), v[8 * e + 2 * f + 1] += __uint_as_float(x[f] & 0xffff0000u);
              }
            } else {
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (e < n) v[e] += __uint_as_float((uint32_t)p[e] << 16);
            }
          }
        }
        if (!g.tma || c0 + 32 > whole) {
          if (row < g.out) {
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              if (c0 + e >= g.in) continue;
              if (FP32) static_cast<float*>(g.dw)[(int64_t)row * g.lddw + c0 + e] = v[e];
              else static_cast<__nv_bfloat16*>(g.dw)[(int64_t)row * g.lddw + c0 + e] = __float2bfloat16_rn(v[e]);
            }
          }
          continue;
        }
        // boxes of 32 rows x 64 bytes, 64-byte swizzled
#pragma unroll
        for (int box = 0; box < 32 / kBox; ++box) {
          if (lane == 0) bulk_wait_read<0>();      // the last store has been read out of it
          __syncwarp();
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            uint32_t o[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if (FP32) o[e] = __float_as_uint(v[16 * box + 4 * u + e]);
              else o[e] = bf16x2_rn(pack_f2(v[8 * u + 2 * e], v[8 * u + 2 * e + 1]));
            }
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(buf + (uint32_t)lane * 64u + (uint32_t)((u ^ (lane >> 1 & 3)) * 16)),
                         "r"(o[0]), "r"(o[1]), "r"(o[2]), "r"(o[3])
                         : "memory");
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            if (row0 < g.out && c0 + kBox * box < g.in) tma_store_2d(&map_c, buf, c0 + kBox * box, row0);
            bulk_commit();
          }
          __syncwarp();
        }
      }
    }
    if (lane == 0) bulk_wait_all();
  }
  tc_fence_before();
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 2 * kTmemCols);
  }
}

// Adds the parts of the split tiles, in order: a block 32 rows x 32 columns of
// a tile, turned in shared memory.
__global__ void __launch_bounds__(256) k_wgrad_join(const TcArgs g, const int m_tiles, const int n_tiles, const int fp32) {
  __shared__ float4 turn[8][33];
  const int tile = g.whole + blockIdx.x / 64, sub = blockIdx.x % 64;
  const int mt = g.n_fast ? tile / n_tiles : tile % m_tiles, nt = g.n_fast ? tile % n_tiles : tile / m_tiles;
  const int r0 = sub / 8 * 32, q0 = sub % 8 * 8;      // rows, and columns / 4, within the tile
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  griddep_wait();
  if (mt * 256 + r0 >= g.out || nt * kBN + 4 * q0 >= g.in) return;
  const float4* p = reinterpret_cast<const float4*>(g.ws) + ((int64_t)(tile - g.whole) * g.parts * (kBN / 4) + q0 + w) * (kPair * kBM) + r0 + lane;
  float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
  for (int i = 0; i < g.parts; ++i, p += kBN / 4 * kPair * kBM) {
    const float4 u = *p;
    v.x += u.x, v.y += u.y, v.z += u.z, v.w += u.w;
  }
  turn[w][lane] = v;
  __syncthreads();
  const int r = threadIdx.x >> 3, q = threadIdx.x & 7;
  const int64_t row = (int64_t)mt * 256 + r0 + r;
  const int col = nt * kBN + 4 * (q0 + q);
  if (row >= g.out) return;
  v = turn[q][r];
  const float x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (col + e >= g.in) continue;
    float y = x[e];
    if (g.base) y += dw_at(g.base, fp32, row * g.ldbase + col + e);
    if (fp32) static_cast<float*>(g.dw)[row * g.lddw + col + e] = y;
    else static_cast<__nv_bfloat16*>(g.dw)[row * g.lddw + col + e] = __float2bfloat16_rn(y);
  }
}

// Map of the checkpoint's values: boxes of 128 columns x 64 tokens.
sf_status make_map_values(CUtensorMap* map, const Ck& ck, int64_t in, int64_t tokens) {
  cuuint64_t dims[2] = {(cuuint64_t)in, (cuuint64_t)tokens};
  cuuint64_t strides[1] = {(cuuint64_t)ck.ld};
  cuuint32_t box[2] = {128, (cuuint32_t)kBK};
  cuuint32_t estr[2] = {1, 1};
  CUresult r = tensor_map_encoder()(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, ck.q, dims, strides, box, estr,
                                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(SF_ERR_CUDA, "cuTensorMapEncodeTiled (checkpoint) failed (%d)", (int)r);
  return SF_OK;
}

// Map of dW's stores: boxes of 32 rows x 64 bytes.
sf_status make_map_dw(CUtensorMap* map, const WgradArgs& a) {
  const size_t size = a.fp32 ? 4 : 2;
  cuuint64_t dims[2] = {(cuuint64_t)a.in, (cuuint64_t)a.out};
  cuuint64_t strides[1] = {(cuuint64_t)(a.lddw * size)};
  cuuint32_t box[2] = {(cuuint32_t)(64 / size), 32};
  cuuint32_t estr[2] = {1, 1};
  CUresult r = tensor_map_encoder()(map, a.fp32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, a.dw, dims, strides,
                                    box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B,
                                    CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(SF_ERR_CUDA, "cuTensorMapEncodeTiled (dW) failed (%d)", (int)r);
  return SF_OK;
}

// Clusters of two CTAs that fit on the device at once (cached per device; one CTA an SM in either form).
sf_status resident_pairs(int* out) {
  static std::mutex mu;
  static std::map<int, int> cache;
  int dev = 0;
  SF_CUDA_TRY(cudaGetDevice(&dev), "cudaGetDevice");
  std::lock_guard<std::mutex> lock(mu);
  auto it = cache.find(dev);
  if (it == cache.end()) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim = {kPair, 1, 1};
    cfg.attrs = at;
    cfg.numAttrs = 1;
    cfg.blockDim = dim3(kTcThreads<true>);
    cfg.gridDim = dim3((unsigned)(kPair * std::max(1, sm_count() / kPair)));
    cfg.dynamicSmemBytes = kTcSmem<true>;
    int n = 0;
    const auto kernel = &k_wgrad_tc<false, true>;
    SF_TRY(allow_dynamic_smem(reinterpret_cast<const void*>(kernel), kTcSmem<true>));
    SF_CUDA_TRY(cudaOccupancyMaxActiveClusters(&n, kernel, &cfg), "cudaOccupancyMaxActiveClusters (k_wgrad_tc)");
    if (n < 1) return fail(SF_ERR_UNSUPPORTED, "no cluster of two CTAs fits on this device");
    it = cache.emplace(dev, n).first;
  }
  *out = it->second;
  return SF_OK;
}

// Tiles that are one item each, and the parts of the others: whole waves of
// tiles, and the rest split so that its rounds of parts take least time (a
// part is at least a span of tokens; a pair's part costs about two slabs more
// for the workspace).
void plan(int64_t tiles, int nk, int pairs, TcArgs* g) {
  const int64_t left = tiles % pairs;
  g->whole = (int32_t)tiles;
  g->parts = 1;
  double best = nk;
  for (int s = 2; left && s <= nk / kSpan && s * left <= kMaxParts; ++s) {
    const double cost = (double)ceil_div<int64_t>(left * s, pairs) * ((double)nk / s + 2.0);
    if (cost < 0.9 * best) {
      best = cost;
      g->parts = s;
      g->whole = (int32_t)(tiles - left);
    }
  }
  g->items = (int32_t)(g->whole + (tiles - g->whole) * g->parts);
}

// 64 x 64 tiles on the CUDA cores, 4 x 4 a thread, for operands that tensor
// copies cannot take (rows off 16 bytes, pinned host memory).
constexpr int kT = 64, kTk = 16;
__global__ void __launch_bounds__(256) k_wgrad_plain(const WgradArgs a, const uint32_t tiles_i) {
  __shared__ float sa[kTk][kT + 4], sb[kTk][kT + 4];
  const uint32_t tile_o = blockIdx.x / tiles_i;
  const int64_t o0 = (int64_t)tile_o * kT, i0 = (int64_t)(blockIdx.x - tile_o * tiles_i) * kT;
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
  float acc[4][4] = {};
  for (int64_t t0 = 0; t0 < a.tokens; t0 += kTk) {
    for (int e = threadIdx.x; e < kTk * kT; e += 256) {
      const int64_t t = t0 + e / kT, o = o0 + e % kT, i = i0 + e % kT;
      sa[e / kT][e % kT] = t < a.tokens && o < a.out ? __bfloat162float(a.dy[t * a.ldy + o]) : 0.0f;
      float x = 0.0f;
      if (t < a.tokens && i < a.in) x = __bfloat162float(__float2bfloat16_rn(e4m3x2_value(a.ck.q[t * a.ck.ld + i]).x * ck_scale(a.ck, t, (int)i)));
      sb[e / kT][e % kT] = x;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kTk; ++k)
#pragma unroll
      for (int y = 0; y < 4; ++y)
#pragma unroll
        for (int x = 0; x < 4; ++x) acc[y][x] = fmaf(sa[k][ty * 4 + y], sb[k][tx * 4 + x], acc[y][x]);
    __syncthreads();
  }
#pragma unroll
  for (int y = 0; y < 4; ++y)
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int64_t o = o0 + ty * 4 + y, i = i0 + tx * 4 + x;
      if (o >= a.out || i >= a.in) continue;
      float v = acc[y][x];
      if (a.base) v += dw_at(a.base, a.fp32, o * a.ldbase + i);
      if (a.fp32) static_cast<float*>(a.dw)[o * a.lddw + i] = v;
      else static_cast<__nv_bfloat16*>(a.dw)[o * a.lddw + i] = __float2bfloat16_rn(v);
    }
}

// Whether X is restored as a bf16 matrix first: more bytes through
// memory, for a product without conversions beside it.  It
// pays where an element is used often enough (restored / converted on the way,
// us): 8192 tokens 4096 -> 11008 422 / 519, 4096 -> 4096 178 / 206, 2048 -> 2048 55 / 62,
// 512 -> 2048 25.4 / 26.1, 256 -> 2048 22.0 / 20.7, 256 -> 11008 55.6 / 58.4; 4096 -> 1792 90.6 / 96.3,
// 4096 -> 1024 61.5 / 62.0, 1024 -> 1024 27.1 / 25.3, 11008 -> 512 106 / 78; 512 tokens 4096 -> 4096
// 21.9 / 23.6, 2048 -> 2048 11.0 / 11.0, 512 -> 2048 10.4 / 10.0; 256 tokens 4096 -> 4096 18.6 / 18.5,
// 4096 -> 1024 9.7 / 9.3.  Of 93 sizes of 512 to 16384 tokens the rule's form is 7 % the slower one at most (2048
// tokens 11008 -> 1792, 61.0 / 65.3).
bool restores(int64_t tokens, int64_t out, int64_t in) { return tokens >= 512 && out >= 2048 && in >= 256; }
int64_t restored_ld(int64_t in) { return ceil_div<int64_t>(in, 64) * 64; }
size_t restored_bytes(int64_t tokens, int64_t out, int64_t in) {
  return restores(tokens, out, in) ? (size_t)tokens * restored_ld(in) * 2 + 255 & ~(size_t)255 : 0;
}

sf_status launch_tc(const WgradArgs& a, const sf_checkpoint* c, void* ws, cudaStream_t st) {
  TcArgs g{};
  g.out = (int32_t)a.out;
  g.in = (int32_t)a.in;
  g.tokens = (int32_t)a.tokens;
  g.n_fast = a.out > a.in;
  g.dw = a.dw;
  g.base = a.base;
  g.lddw = a.lddw;
  g.ldbase = a.ldbase;
  g.ck = a.ck;
  const bool fused = !restores(a.tokens, a.out, a.in);
  g.ws = reinterpret_cast<float*>(static_cast<char*>(ws) + restored_bytes(a.tokens, a.out, a.in));
  const size_t size = a.fp32 ? 4 : 2;
  g.base_vec = a.base && reinterpret_cast<uintptr_t>(a.base) % 16 == 0 && a.ldbase * size % 16 == 0;
  g.tma = reinterpret_cast<uintptr_t>(a.dw) % 16 == 0 && a.lddw * size % 16 == 0 && a.lddw >= a.in && on_current_device(a.dw);
  const int64_t m_tiles = ceil_div<int64_t>(a.out, kPair * kBM), n_tiles = ceil_div<int64_t>(a.in, kBN);
  if (m_tiles * n_tiles > INT32_MAX / 2) return fail(SF_ERR_UNSUPPORTED, "too many tiles");
  int pairs = 0;
  SF_TRY(resident_pairs(&pairs));
  plan(m_tiles * n_tiles, (int)ceil_div<int64_t>(a.tokens, kBK), pairs, &g);
  CUtensorMap ma, mb;
  int a_form = make_map_mn3d(&ma, a.dy, a.out, a.tokens, a.ldy) ? 2 : 1;
  if (a_form == 1) SF_TRY(make_map(&ma, a.dy, a.out, a.tokens, a.ldy, kBK));
  if (fused) {
    SF_TRY(make_map_values(&mb, a.ck, a.in, a.tokens));
  } else {
    const sf_matrix x{ws, a.tokens, a.in, restored_ld(a.in), SF_BF16};
    if (!make_map_mn3d(&mb, ws, x.ld, a.tokens, x.ld)) return fail(SF_ERR_CUDA, "cuTensorMapEncodeTiled (restored checkpoint) failed");
    SF_TRY(checkpoint_load(c, nullptr, nullptr, SF_FP32, 0.0, &x, st));
  }
  CUtensorMap mc = ma;       // unused unless dW is written by tensor stores
  if (g.tma) SF_TRY(make_map_dw(&mc, a));
  const void* kernel = a.fp32 ? (fused ? (const void*)&k_wgrad_tc<true, true> : (const void*)&k_wgrad_tc<true, false>)
                              : (fused ? (const void*)&k_wgrad_tc<false, true> : (const void*)&k_wgrad_tc<false, false>);
  const size_t smem = fused ? kTcSmem<true> : kTcSmem<false>;
  SF_TRY(allow_dynamic_smem(kernel, smem));
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim = {kPair, 1, 1};
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = fused ? 1 : 2;
  cfg.gridDim = dim3((unsigned)(kPair * std::min<int64_t>(g.items, pairs)));
  cfg.blockDim = dim3(fused ? kTcThreads<true> : kTcThreads<false>);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  void* args[] = {&ma, &mb, &mc, &g, &a_form};
  SF_CUDA_TRY(cudaLaunchKernelExC(&cfg, kernel, args), "launch k_wgrad_tc");
  if (g.parts > 1)
    SF_CUDA_TRY(launch_pdl(k_wgrad_join, dim3((unsigned)((m_tiles * n_tiles - g.whole) * 64)), dim3(256), 0, st, g, (int)m_tiles, (int)n_tiles, (int)a.fp32),
                "launch k_wgrad_join");
  return SF_OK;
}

}  // namespace

const void* device_error_wgrad() { return &g_device_error; }

}  // namespace sf

extern "C" {

size_t sf_checkpoint_wgrad_workspace_bytes(int64_t tokens, int64_t out, int64_t in) {
  using namespace sf;
  if (tokens < 0 || out < 1 || in < 1) return 0;
  const int64_t tiles = ceil_div<int64_t>(out, 2 * kBM) * ceil_div<int64_t>(in, kBN);
  const int64_t parts = ceil_div<int64_t>(tokens, kBK) / kSpan;      // of a tile, at most
  const size_t x = restored_bytes(tokens, out, in);
  if (parts < 2) return x;      // never split
  return x + (size_t)(tiles < kMaxParts && parts < kMaxParts ? std::min(kMaxParts, tiles * parts) : kMaxParts) * kPartFloats * sizeof(float);
}

sf_status sf_checkpoint_wgrad(const sf_matrix* dY, const sf_checkpoint* c, const sf_matrix* base, const sf_matrix* dW,
                              void* ws, size_t ws_bytes, void* stream) {
  using namespace sf;
  clear_error();
  NvtxRange nvtx_range("sf_checkpoint_wgrad");
  SF_TRY(check_matrix(dY, "dY", -1, -1, 1u << SF_BF16));
  SF_TRY(check_matrix(dW, "dW", dY->cols, -1, 1u << SF_BF16 | 1u << SF_FP32));
  SF_TRY(check_checkpoint(c, "checkpoint", dY->rows, dW->cols, false));
  if (base) SF_TRY(check_matrix(base, "base", dW->rows, dW->cols, 1u << dW->dtype));
  const int64_t tokens = dY->rows, out = dW->rows, in = dW->cols;
  if (tokens > INT32_MAX / 2 || out > INT32_MAX / 2 || in > INT32_MAX / 2) return fail(SF_ERR_UNSUPPORTED, "tokens, out and in must be below 2^30");
  const size_t need = sf_checkpoint_wgrad_workspace_bytes(tokens, out, in);
  if (need && (!ws || ws_bytes < need || reinterpret_cast<uintptr_t>(ws) % 16))
    return fail(SF_ERR_INVALID, "workspace needs %zu bytes, 16-byte aligned (got %zu)", need, ws_bytes);
  if (!out || !in) return SF_OK;
  WgradArgs a{};
  a.dy = static_cast<const __nv_bfloat16*>(dY->data);
  a.ldy = dY->ld;
  if (base) a.base = base->data, a.ldbase = base->ld;
  a.dw = dW->data;
  a.lddw = dW->ld;
  a.tokens = tokens;
  a.out = out;
  a.in = in;
  a.fp32 = dW->dtype == SF_FP32;
  a.ck = device_ck(c);
  if (need && !on_current_device(ws)) return fail(SF_ERR_INVALID, "ws must be device memory of the current device");
  const sf_matrix scale{c->scale, tokens, a.ck.n_groups, a.ck.n_groups, c->scale_dtype};
  if (overlap(dW, dY) || overlap(dW, &c->values) || overlap(dW, &scale)) return fail(SF_ERR_INVALID, "dW must not lie over dY or the checkpoint");
  if (overlap(dW, base) && !same_matrix(dW, base)) return fail(SF_ERR_INVALID, "dW lies over base with another place or distance of rows");
  if (tokens && dY->ld % 8 == 0 && dY->ld >= out && c->values.ld % 16 == 0 && c->values.ld >= in && reinterpret_cast<uintptr_t>(dY->data) % 16 == 0 &&
      reinterpret_cast<uintptr_t>(c->values.data) % 16 == 0 && tensor_map_encoder() && on_current_device(dY->data) &&
      on_current_device(c->values.data))
    return launch_tc(a, c, ws, as_stream(stream));
  const int64_t tiles_i = ceil_div<int64_t>(in, kT), tiles = ceil_div<int64_t>(out, kT) * tiles_i;
  if (tiles > INT32_MAX) return fail(SF_ERR_UNSUPPORTED, "too many tiles");      // (of 4096 elements each)
  k_wgrad_plain<<<(unsigned)tiles, 256, 0, as_stream(stream)>>>(a, (uint32_t)tiles_i);
  return check_launch("launch k_wgrad_plain");
}

}  // extern "C"
