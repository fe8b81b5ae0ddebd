// The residual's addition and the root-mean-square norm, forward:
//   s = r + dropout(x),  rstd = 1 / sqrt(mean_j s_j^2 + eps),  h = s rstd g
// (SlideFormer, kernel lists of the summaries: fused RMSNorm; the norm is
// Zhang and Sennrich 2019), h in bf16 or fp32 and / or in 8 bits with scales:
// per group of columns (or per row) scale = max(max |h| / 448, 2^-126) and
// q = h / scale rounded to e4m3, whose largest value is 448.
//
// One pass: a row is read once into registers (`tpr` threads a row, up to
// four units of eight columns a thread), s is written, the squares are summed
// over the row by shuffles and one shared-memory step, and h is written from
// the registers.  Bound by HBM: a bf16 row moves 8 bytes a column (x, r, s,
// h).  What it took to get there: registers few enough for 24 and more warps
// an SM (72 a thread in bf16; at 96 the same kernel takes 90 us instead of
// 81), blocks of whole warps rather than powers of two, fp32 arithmetic in pairs, one
// division a scale group.  16384 x 4096 bf16 81 us (6.6 TB/s); 8192 x 12288,
// fp32 stream, e4m3 with 128-column groups 168 us (6.6 TB/s); one row of 4096
// 3.3 us.  Dropout on: 91 us at 16384 x 4096, 169 at 16384 x 4095 (128 off).
// The fp32 and off-unit instances spill 4 to 84 bytes at these limits.
//
// The norm is taken of s in fp32, before s is rounded to its stored type, so
// storing s in bf16 costs h no precision; the backward pass uses the stored s.
#include <cuda_fp8.h>

#include <algorithm>
#include <type_traits>

#include "ptx.cuh"
#include "row_span.h"
#include "rows.cuh"

namespace sf {
namespace {

constexpr int kK = 4;               // units per thread
constexpr int kMaxThreads = 512;
constexpr int64_t kMaxCols = (int64_t)kMaxThreads * kK * 8;   // 16384

struct FwdArgs {
  const void* x;
  const void* r;       // may be null
  void* s;             // may be null
  void* h;             // may be null
  uint8_t* q;          // may be null
  float* scale;
  float* rstd;         // may be null
  const void* gain;
  int64_t ldx, ldr, lds, ldh, ldq;
  int64_t rows;
  int32_t cols, per_row;
  int32_t shift;         // kShifted
  int32_t tpr;           // threads a row: a power of two up to 64, or the whole block (a multiple of 32)
  int32_t rpb;           // rows a block
  int32_t units;         // units a thread, 1..kK
  int32_t gain_fp32;
  int32_t group_log2;    // columns of a scale group; 0: one scale a row
  int32_t n_groups;
  float eps, inv_cols;
  DropConsts d;
};

// A unit's gains (served by L1 after a row or two).  kAligned: gains are aligned
// to their units.
template <int MODE>
__device__ __forceinline__ F8 load_gain(const void* g, int fp32, const Span& s) {
  if (fp32) {
    const float* p = static_cast<const float*>(g) + s.c;
    Unit<float> u;
    if (MODE == kAligned && s.hi == 8) {
      const float4 x = __ldg(reinterpret_cast<const float4*>(p)), y = __ldg(reinterpret_cast<const float4*>(p) + 1);
      u.f[0] = x.x, u.f[1] = x.y, u.f[2] = x.z, u.f[3] = x.w;
      u.f[4] = y.x, u.f[5] = y.y, u.f[6] = y.z, u.f[7] = y.w;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) u.f[i] = i >= s.lo && i < s.hi ? __ldg(p + i) : 0.0f;
    }
    return unpack(u);
  }
  const uint16_t* p = static_cast<const uint16_t*>(g) + s.c;
  Unit<__nv_bfloat16> u;
  if (MODE == kAligned && s.hi == 8) {
    const uint4 w = __ldg(reinterpret_cast<const uint4*>(p));
    u.w[0] = w.x, u.w[1] = w.y, u.w[2] = w.z, u.w[3] = w.w;
  } else if (MODE == kShifted && s.lo == 0 && s.hi == 8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) u.w[i] = (uint32_t)__ldg(p + 2 * i) | (uint32_t)__ldg(p + 2 * i + 1) << 16;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      u.w[i] = (2 * i >= s.lo && 2 * i < s.hi ? (uint32_t)__ldg(p + 2 * i) : 0u) |
               (2 * i + 1 >= s.lo && 2 * i + 1 < s.hi ? (uint32_t)__ldg(p + 2 * i + 1) << 16 : 0u);
  }
  return unpack(u);
}

// A thread's units of a row: first + k * step, those of the whole row's
// threads beside one another, or (`handed`, for ShiftedBits) those of 32 lanes
// (or of a shorter row's).
struct UnitWalk {
  int first, step, lane;      // lane: among those
  __device__ __forceinline__ static UnitWalk of(bool handed, int t, int tpr, int units) {
    const int w = min(tpr, 32), lane = t & (w - 1);
    return handed ? UnitWalk{(t - lane) * units + lane, w, lane} : UnitWalk{t, tpr, lane};
  }
};

// Maximum that keeps a NaN: a NaN in a group must reach its scale.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Sum (or maximum) over the tpr threads of a row, in a fixed order: lanes by
// a butterfly, then the row's warps in turn through shared memory.
template <bool MAX>
__device__ __forceinline__ float row_reduce(float v, int tpr, float* red) {
  for (int o = min(tpr, 32) >> 1; o > 0; o >>= 1) {
    const float w = __shfl_xor_sync(0xffffffffu, v, o);
    v = MAX ? max_nan(v, w) : v + w;
  }
  if (tpr <= 32) return v;
  const int warp = threadIdx.x >> 5, n = tpr >> 5, first = warp - warp % n;
  if ((threadIdx.x & 31) == 0) red[warp] = v;
  __syncthreads();
  float t = red[first];
  for (int i = 1; i < n; ++i) t = MAX ? max_nan(t, red[first + i]) : t + red[first + i];
  return t;
}

// A group's scale, and its reciprocal from the maximum itself: one rounding
// and not two, so that h times it is as near to h / scale as a division.  (The
// scale, to which nothing is rounded, does without a second division.)
__device__ __forceinline__ float group_scale(float amax, float* inv) {
  amax = max_nan(amax, 448.0f * 1.17549435e-38f);
  *inv = __fdiv_rn(448.0f, amax);
  return max_nan(amax * (1.0f / 448.0f), 1.17549435e-38f);
}

// DROP false: no dropout (otherwise as the arguments say); an instance of its
// own for shifted rows, whose hand-over of the generator's words costs
// registers (8192 x 6001 bf16 without dropout: 93 us, in one instance 109;
// with dropout 108 at 80 registers, 120 at 96; fp32 7132 x 9409 195 and 203
// the other way round).
template <typename TA, typename TS, int MODE, bool DROP>
__global__ void __maxnreg__(MODE == kShifted && DROP && sizeof(TA) == 4 ? 96 : sizeof(TA) + sizeof(TS) == 4 && !(MODE == kShifted && DROP) ? 72 : 80) k_add_rmsnorm_fwd(const FwdArgs a) {
  __shared__ float red[2][kMaxThreads / 32];
  __shared__ float group_max[2][MODE == kShifted ? kMaxCols / 32 : 1];      // shifted rows: of a unit's own group, and of the one before
  const int tpr = a.tpr, lane_row = (int)threadIdx.x / tpr, t = (int)threadIdx.x - lane_row * tpr;
  const int64_t row = (int64_t)blockIdx.x * a.rpb + lane_row;
  const bool on = row < a.rows;
  const int m = MODE == kShifted ? (int)(row * a.shift) & 7 : 0;
  const UnitWalk at = UnitWalk::of(MODE == kShifted && DROP, t, tpr, a.units);
  auto span = [&](int k) { return unit_span<MODE>(at.first + k * at.step, m, (MODE != kShifted || k < a.units) && on ? a.cols : 0); };
  F8 s[kK];
  {
    Unit<TA> x[kK];
    Unit<TS> r[kK];
    const TA* xp = row_ptr<TA>(a.x, a.ldx, row);
    const TS* rp = row_ptr<TS>(a.r, a.ldr, row);
#pragma unroll
    for (int k = 0; k < kK; ++k) {
      const Span p = span(k);
      if (!p.some()) continue;
      load_unit<MODE>(xp + p.c, p.lo, p.hi, x[k]);
      if (a.r) load_unit<MODE>(rp + p.c, p.lo, p.hi, r[k]);
    }
    const DropWords words = a.d.threshold ? drop_words(a.d) : DropWords{};
    const uint64_t b0 = (uint64_t)(row * a.per_row + at.first);
    ShiftedBits bits;
    if (MODE == kShifted && DROP && t > at.lane) bits.start(b0 - at.lane - 1, words, a.d);
#pragma unroll
    for (int k = 0; k < kK; ++k) {
#pragma unroll
      for (int i = 0; i < 4; ++i) s[k].p[i] = 0;
      if (MODE == kShifted && k >= a.units) continue;
      uint32_t w[4];
      if (MODE == kShifted && DROP)
        bits.next(b0 + k * at.step, at.lane, min(tpr, 32), m, words, a.d, w);
      if (!span(k).some()) continue;
      s[k] = unpack(x[k]);
      if (DROP && a.d.threshold) {
        if (MODE == kShifted) drop_apply(s[k], w, a.d);
        else drop_unit(s[k], b0 + k * at.step, words, a.d);
      }
      if (a.r) {
        const F8 w = unpack(r[k]);
#pragma unroll
        for (int i = 0; i < 4; ++i) s[k].p[i] = fadd2(s[k].p[i], w.p[i]);
      }
    }
  }
  uint64_t sum2 = 0;
  TS* sp = row_ptr<TS>(a.s, a.lds, row);
#pragma unroll
  for (int k = 0; k < kK; ++k) {
    const Span p = span(k);
    if (a.s && p.some()) store_unit<MODE>(sp + p.c, p.lo, p.hi, s[k]);
#pragma unroll
    for (int i = 0; i < 4; ++i) sum2 = fmadd2(s[k].p[i], s[k].p[i], sum2);
  }
  const float sum = row_reduce<false>(unpack_f2(sum2).x + unpack_f2(sum2).y, tpr, red[0]);
  const float rstd = rsqrtf(fmaf(sum, a.inv_cols, a.eps));
  if (a.rstd && on && t == 0) a.rstd[row] = rstd;
  const uint64_t rstd2 = pack_f2(rstd, rstd);
  float amax = 0.0f;
  TA* hp = row_ptr<TA>(a.h, a.ldh, row);
#pragma unroll
  for (int k = 0; k < kK; ++k) {
    const Span p = span(k);
    if (p.some()) {
      const F8 g = load_gain<MODE>(a.gain, a.gain_fp32, p);
#pragma unroll
      for (int i = 0; i < 4; ++i) s[k].p[i] = fmul2(fmul2(s[k].p[i], rstd2), g.p[i]);
      if (a.h) store_unit<MODE>(hp + p.c, p.lo, p.hi, s[k]);
    }
    if (a.q && k < a.units) {
      // shifted units: those that start a group hold its columns from m on,
      // and before them the last m of the group before
      const int lanes = 1 << (a.group_log2 - 3), u = at.first + k * at.step;
      const bool edge = MODE == kShifted && a.group_log2 && m && (u & (lanes - 1)) == 0;
      float top = 0.0f, carry = 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        // outside a ragged row the sum is 0 and so is the gain
        const float2 v = unpack_f2(s[k].p[i]);
        if (edge) {
          (2 * i < m ? carry : top) = max_nan(2 * i < m ? carry : top, fabsf(v.x));
          (2 * i + 1 < m ? carry : top) = max_nan(2 * i + 1 < m ? carry : top, fabsf(v.y));
        } else {
          top = max_nan(top, max_nan(fabsf(v.x), fabsf(v.y)));
        }
      }
      if (!p.some()) top = 0.0f;
      amax = max_nan(amax, top);
      if (MODE == kShifted && a.group_log2) {
        for (int o = lanes >> 1; o > 0; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
        const int group = u >> (a.group_log2 - 3);
        if (p.some() && (u & (lanes - 1)) == 0) {
          if (group < a.n_groups) group_max[0][lane_row * a.n_groups + group] = top;
          if (edge && u) group_max[1][lane_row * a.n_groups + group - 1] = carry;
        }
      } else if (a.group_log2) {
        for (int o = lanes >> 1; o > 0; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
        float inv;
        const float sc = group_scale(top, &inv);
        if (p.some() && (t & (lanes - 1)) == 0) a.scale[row * a.n_groups + (p.c >> a.group_log2)] = sc;
#pragma unroll
        for (int i = 0; i < 4; ++i) s[k].p[i] = fmul2(s[k].p[i], pack_f2(inv, inv));
      }
    }
  }
  if (!a.q) return;
  if (MODE == kShifted && a.group_log2) {
    __syncthreads();
    // a group's maximum, with its columns in the unit that starts the next one
    auto scale_of = [&](int group, float* inv) {
      float top = group_max[0][lane_row * a.n_groups + group];
      if (m && ((group + 1) << a.group_log2) - m < a.cols) top = max_nan(top, group_max[1][lane_row * a.n_groups + group]);
      return group_scale(top, inv);
    };
#pragma unroll
    for (int k = 0; k < kK; ++k) {
      if (!span(k).some()) continue;
      const int lanes = 1 << (a.group_log2 - 3), u = at.first + k * at.step, group = u >> (a.group_log2 - 3);
      const bool starts = (u & (lanes - 1)) == 0;
      float inv = 0.0f;
      if (group < a.n_groups) {
        const float sc = scale_of(group, &inv);
        if (starts) a.scale[row * a.n_groups + group] = sc;
      }
      float before = inv;
      if (starts && m && u) scale_of(group - 1, &before);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        s[k].p[i] = fmul2(s[k].p[i], pack_f2(starts && 2 * i < m ? before : inv, starts && 2 * i + 1 < m ? before : inv));
    }
  } else if (!a.group_log2) {
    amax = row_reduce<true>(amax, tpr, red[1]);
    float inv;
    const float sc = group_scale(amax, &inv);
    if (on && t == 0) a.scale[row] = sc;
#pragma unroll
    for (int k = 0; k < kK; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) s[k].p[i] = fmul2(s[k].p[i], pack_f2(inv, inv));
  }
#pragma unroll
  for (int k = 0; k < kK; ++k) {
    const Span part = span(k);
    if (!part.some()) continue;
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      // saturating, so |h| / scale just above 448 by rounding stays 448
      const uint32_t lo = __nv_cvt_float2_to_fp8x2(unpack_f2(s[k].p[2 * i]), __NV_SATFINITE, __NV_E4M3);
      const uint32_t hi = __nv_cvt_float2_to_fp8x2(unpack_f2(s[k].p[2 * i + 1]), __NV_SATFINITE, __NV_E4M3);
      w[i] = lo | hi << 16;
    }
    uint8_t* p = row_ptr<uint8_t>(a.q, a.ldq, row) + part.c;
    if (MODE != kScalar && part.lo == 0 && part.hi == 8) {
      *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i >= part.lo && i < part.hi) p[i] = (uint8_t)(w[i >> 2] >> (8 * (i & 3)));
    }
  }
}

// Backward.  With n_j = s_j rstd, the gradients are
//   ds_j = dsum_j + rstd (dh_j g_j - n_j mean_i(dh_i g_i n_i))
//   dresidual = ds,  dx = m o ds f (the forward mask),  dg_j = sum_rows dh_j n_j
// A persistent grid walks the rows; a thread keeps its columns' share of dg
// in registers over all its rows, so dg costs one partial row per block and a
// second small kernel (5 us at 456 x 4096, its launch overlapped), summed in
// block order (no atomics).  This form, with loads into registers, serves few
// rows, short, long and unaligned ones; 16384 x 4096 bf16 with dropout takes
// it 165 us, against 118 us (5.7 TB/s) in the staged form further down.  Its 512
// threads leave 128 registers, of which all instances but bf16 over bf16 spill
// 36 to 424 bytes.
struct BwdArgs {
  const void* dh;
  const void* s;
  const void* dsum;     // may be null
  const void* gain;
  const float* rstd;
  void* dr;             // may be null
  void* dx;             // may be null
  float* part;          // [grid][cols], null without dg
  int32_t ring_dsum;    // staged form: dsum comes through the ring (else from memory, prefetched into L2)
  int64_t lddh, lds, lddsum, lddr, lddx;
  int64_t rows;
  int32_t cols, per_row;
  int32_t shift;         // kShifted
  int32_t tpr, rpb, units;      // as in FwdArgs
  int32_t gain_fp32;
  float inv_cols;
  DropConsts d;
};

// One unit's share of a row's sums: with w = dh s (unscaled), dg gains w rstd
// and the row's dot product sum dh g s gains w g.
__device__ __forceinline__ void bwd_sums(const F8& dh, const F8& s, const F8& g, uint64_t rstd2, F8& acc, uint64_t& dot2) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint64_t w = fmul2(dh.p[i], s.p[i]);
    acc.p[i] = fmadd2(w, rstd2, acc.p[i]);
    dot2 = fmadd2(w, g.p[i], dot2);
  }
}

// ds = dsum + rstd dh g + c s, c = -rstd^3 / cols * (the row's dot product).
__device__ __forceinline__ F8 bwd_unit(const F8& dh, const F8& s, const F8& g, const F8& dsum, uint64_t rstd2, uint64_t c2) {
  F8 v;
#pragma unroll
  for (int i = 0; i < 4; ++i) v.p[i] = fmadd2(fmul2(dh.p[i], g.p[i]), rstd2, fmadd2(s.p[i], c2, dsum.p[i]));
  return v;
}

// A unit from shared memory.
__device__ __forceinline__ void lds_unit(uint32_t p, Unit<__nv_bfloat16>& u) {
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(u.w[0]), "=r"(u.w[1]), "=r"(u.w[2]), "=r"(u.w[3])
               : "r"(p));
}
__device__ __forceinline__ void lds_unit(uint32_t p, Unit<float>& u) {
  const float4 a = lds_f4(p), b = lds_f4(p + 16);
  u.f[0] = a.x, u.f[1] = a.y, u.f[2] = a.z, u.f[3] = a.w;
  u.f[4] = b.x, u.f[5] = b.y, u.f[6] = b.z, u.f[7] = b.w;
}

// Rows that start off a unit (kShifted): the grid's step is a multiple of
// eight rows, so all rows of a thread start the same m columns past a unit and
// its units hold the same columns in each of them.  Their gains are laid out
// once, at the same shift and zero outside the row, in shared memory.
template <typename TA, typename TS, int MODE>
__global__ void __launch_bounds__(kMaxThreads) k_add_rmsnorm_bwd(const BwdArgs a) {
  __shared__ float red[2][kMaxThreads / 32];
  extern __shared__ __align__(16) float comb[];      // with several rows a block, or shifted: [rows of a block][cols + 8 or more]
  const int tpr = a.tpr, rpb = a.rpb, lane_row = (int)threadIdx.x / tpr, t = (int)threadIdx.x - lane_row * tpr;
  const DropWords words = a.d.threshold ? drop_words(a.d) : DropWords{};
  const int m = MODE == kShifted ? (int)(((int64_t)blockIdx.x * rpb + lane_row) * a.shift) & 7 : 0;
  float* mine = comb + lane_row * (8 * a.per_row + 8);
  const UnitWalk at = UnitWalk::of(MODE == kShifted, t, tpr, a.units);
  if (MODE == kShifted) {
    for (int k = 0; k < a.units; ++k) {
      const Span p = unit_span<MODE>(at.first + k * at.step, m, a.cols);
      if (!p.some()) continue;
      Unit<float> u;
      pack(load_gain<MODE>(a.gain, a.gain_fp32, p), u);
      for (int i = 0; i < 8; ++i) mine[p.c + m + i] = u.f[i];
    }
  }
  auto gain_at = [&](const Span& p) {
    if (MODE != kShifted) return load_gain<MODE>(a.gain, a.gain_fp32, p);
    Unit<float> u;
    lds_unit(smem_u32(mine + p.c + m), u);
    return unpack(u);
  };
  F8 acc[kK] = {};
  int parity = 0;
  for (int64_t base = (int64_t)blockIdx.x * rpb; base < a.rows; base += (int64_t)gridDim.x * rpb, parity ^= 1) {
    const int64_t row = base + lane_row;
    auto span = [&](int k) { return unit_span<MODE>(at.first + k * at.step, m, (MODE != kShifted || k < a.units) && row < a.rows ? a.cols : 0); };
    Unit<TA> dh[kK];
    Unit<TS> s[kK], ds[kK];
#pragma unroll
    for (int k = 0; k < kK; ++k) {
      const Span p = span(k);
      if (!p.some()) continue;
      load_unit<MODE>(row_ptr<TA>(a.dh, a.lddh, row) + p.c, p.lo, p.hi, dh[k]);
      load_unit<MODE>(row_ptr<TS>(a.s, a.lds, row) + p.c, p.lo, p.hi, s[k]);
      if (a.dsum) load_unit<MODE>(row_ptr<TS>(a.dsum, a.lddsum, row) + p.c, p.lo, p.hi, ds[k]);
    }
    const float rstd = row < a.rows ? a.rstd[row] : 0.0f;
    const uint64_t rstd2 = pack_f2(rstd, rstd);
    uint64_t dot2 = 0;
#pragma unroll
    for (int k = 0; k < kK; ++k) {
      const Span p = span(k);
      if (p.some()) bwd_sums(unpack(dh[k]), unpack(s[k]), gain_at(p), rstd2, acc[k], dot2);
    }
    // two alternating buffers: the next row's write cannot meet this row's reads
    const float dot = row_reduce<false>(unpack_f2(dot2).x + unpack_f2(dot2).y, tpr, red[parity]);
    const float c = -rstd * (rstd * (rstd * dot * a.inv_cols));
    const uint64_t c2 = pack_f2(c, c);
    const bool drop = a.dx && a.d.threshold;
    const uint64_t b0 = (uint64_t)(row * a.per_row + at.first);
    ShiftedBits bits;
    if (MODE == kShifted && drop && t > at.lane) bits.start(b0 - at.lane - 1, words, a.d);
#pragma unroll
    for (int k = 0; k < kK; ++k) {
      const Span p = span(k);
      uint32_t w[4];
      if (MODE == kShifted && drop && k < a.units)
        bits.next(b0 + k * at.step, at.lane, min(tpr, 32), m, words, a.d, w);
      if (!p.some()) continue;
      F8 v = bwd_unit(unpack(dh[k]), unpack(s[k]), gain_at(p), a.dsum ? unpack(ds[k]) : F8{}, rstd2, c2);
      if (a.dr) store_unit<MODE>(row_ptr<TS>(a.dr, a.lddr, row) + p.c, p.lo, p.hi, v);
      if (a.dx) {
        if (drop) {
          if (MODE == kShifted) drop_apply(v, w, a.d);
          else drop_unit(v, b0 + k * at.step, words, a.d);
        }
        store_unit<MODE>(row_ptr<TA>(a.dx, a.lddx, row) + p.c, p.lo, p.hi, v);
      }
    }
  }
  if (!a.part) return;
  griddep_launch_dependents();
  if (rpb > 1) __syncthreads();      // the gains have been read
  float* part = a.part + (int64_t)blockIdx.x * a.cols;
#pragma unroll
  for (int k = 0; k < kK; ++k) {
    const Span p = unit_span<MODE>(at.first + k * at.step, m, k < a.units ? a.cols : 0);
    if (p.some()) store_unit<kScalar>((rpb == 1 ? part : mine) + p.c, p.lo, p.hi, acc[k]);
  }
  if (rpb == 1) return;
  __syncthreads();
  for (int c = threadIdx.x; c < a.cols; c += blockDim.x) {
    float v = 0.0f;
    for (int r = 0; r < rpb; ++r) v += comb[r * (8 * a.per_row + 8) + c];
    part[c] = v;
  }
}

__device__ __forceinline__ void sts_unit(uint32_t p, const F8& v, __nv_bfloat16) {
  Unit<__nv_bfloat16> u;
  pack(v, u);
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(p), "r"(u.w[0]), "r"(u.w[1]), "r"(u.w[2]), "r"(u.w[3])
               : "memory");
}
__device__ __forceinline__ void sts_unit(uint32_t p, const F8& v, float) {
  asm volatile("st.shared.v2.b64 [%0], {%1, %2};" ::"r"(p), "l"(v.p[0]), "l"(v.p[1]) : "memory");
  asm volatile("st.shared.v2.b64 [%0], {%1, %2};" ::"r"(p + 16), "l"(v.p[2]), "l"(v.p[3]) : "memory");
}
// Bulk copy of shared memory to global memory, of this thread's bulk group.
__device__ __forceinline__ void bulk_store(void* dst, uint32_t src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(src), "r"(bytes) : "memory");
}

// The columns that copy_span leaves out of the matrix's last row, into the row's
// place at `at` (its first column at m).
template <typename T>
__device__ __forceinline__ void load_rest(unsigned char* at, const T* row, uint32_t m, uint32_t cols) {
  for (uint32_t c = copy_span(m, cols, sizeof(T), true).end / sizeof(T); c < m + cols; ++c) reinterpret_cast<T*>(at)[c] = row[c - m];
}

constexpr int kMinStages = 3, kMaxStages = 4;

// The same backward pass with whole rows moved by bulk copies, both ways, so
// that threads address shared memory only.  A ring of `stages` stages of rpb
// rows each (dh, s and dsum): a stage is filled ahead, its row is reduced, the
// outputs overwrite the inputs in place (dx over dh, dresidual over s), a bulk
// store takes them out, and the stage is filled again.  One barrier a row: past
// the barrier of row i's sum every thread has also finished row i - 1's
// outputs, which then leave, and row i - 2's have left, so its stage is
// refilled.  With loads and stores of registers the kernel was bound by
// instruction issue (49 instructions an element, 59 % of the copy rate).
// SHIFT: rows that start off a unit, as above.  A copy brings the 16-byte units
// that hold any of the row (as far as the matrix goes: copy_span), so that units lie
// in shared memory as in memory; of the first and last one, the columns outside the row are set to zero, and
// those inside are written to memory by their threads, the rest by bulk stores
// (16384 x 4095 bf16: 175 us, with dropout 226, against 349 element by element).
template <typename TA, typename TS, int K, bool KEEP, bool SHIFT>
__global__ void __maxnreg__(K == 2 && !SHIFT ? 80 : KEEP && K == 4 ? 168 : 128) k_add_rmsnorm_bwd_ring(const BwdArgs a, const int stages) {
  constexpr int MODE = SHIFT ? kShifted : kAligned;
  __shared__ __align__(16) float red[2][4][kMaxThreads / 32];    // [alternating][row of the block][warp of the row]
  __shared__ __align__(8) uint64_t full[kMaxStages];
  extern __shared__ __align__(128) unsigned char ring[];
  const int tpr = a.tpr, rpb = a.rpb, lane_row = (int)threadIdx.x / tpr, t = (int)threadIdx.x - lane_row * tpr;
  // (a block of 96 threads leaves rows 2 and 3 of red[1] alone: it has one row, so nothing reads them)
  if (threadIdx.x < 2 * 4 * kMaxThreads / 32) (&red[0][0][0])[threadIdx.x] = 0.0f;
  // a row's place holds whole units
  const uint32_t slot = SHIFT ? 8u * a.per_row + 8u : (uint32_t)a.cols;
  const uint32_t row_a = slot * sizeof(TA), row_s = slot * sizeof(TS);
  const uint32_t off_s = row_a * rpb, off_d = off_s + row_s * rpb;
  const bool ring_d = a.dsum && a.ring_dsum;
  const uint32_t stage_bytes = off_d + (ring_d ? row_s * rpb : 0u);
  const uint32_t ring0 = smem_u32(ring);
  const int64_t step = (int64_t)gridDim.x * rpb, first = (int64_t)blockIdx.x * rpb;
  // by the first warp, a lane a row: the copies of the rows from `base` on
  // into stage st ...
  const int m_lane = SHIFT ? (int)((first + threadIdx.x) * a.shift) & 7 : 0;
  auto bring = [&](unsigned char* at, const void* row, uint32_t size, int st, bool last) {
    const CopySpan c = copy_span(m_lane, a.cols, size, last);
    if (SHIFT) bulk_load(at + c.begin, static_cast<const unsigned char*>(row) - m_lane * size + c.begin, c.end - c.begin, &full[st]);
    else bulk_load(at, row, a.cols * size, &full[st]);
  };
  // (ENDS: the matrix's last row may be among them; see copy_span)
  auto fill_rows = [&](int64_t base, int st, auto ends) {
    constexpr bool ENDS = SHIFT && decltype(ends)::value;
    const int n = (int)min((int64_t)rpb, a.rows - base);
    const int64_t row = base + threadIdx.x;
    const bool mine = (int)threadIdx.x < n, last = ENDS && mine && row == a.rows - 1;
    unsigned char* at = ring + (size_t)st * stage_bytes;
    uint32_t bytes = (uint32_t)n * (row_a + row_s + (ring_d ? row_s : 0u));
    if (SHIFT) {
      const CopySpan ca = copy_span(m_lane, a.cols, sizeof(TA), last), cs = copy_span(m_lane, a.cols, sizeof(TS), last);
      bytes = __reduce_add_sync(0xffffffffu, mine ? ca.end - ca.begin + (ring_d ? 2u : 1u) * (cs.end - cs.begin) : 0u);
    }
    if (ENDS) {
      if (last) {      // ordered before the readers by the arrival below
        load_rest(at + threadIdx.x * row_a, row_ptr<TA>(a.dh, a.lddh, row), m_lane, a.cols);
        load_rest(at + off_s + threadIdx.x * row_s, row_ptr<TS>(a.s, a.lds, row), m_lane, a.cols);
        if (ring_d) load_rest(at + off_d + threadIdx.x * row_s, row_ptr<TS>(a.dsum, a.lddsum, row), m_lane, a.cols);
      }
      __syncwarp();
    }
    if (threadIdx.x == 0) mbar_arrive_expect_tx(&full[st], bytes);
    __syncwarp();
    if (mine) {
      bring(at + threadIdx.x * row_a, row_ptr<TA>(a.dh, a.lddh, row), sizeof(TA), st, last);
      bring(at + off_s + threadIdx.x * row_s, row_ptr<TS>(a.s, a.lds, row), sizeof(TS), st, last);
      if (ring_d) bring(at + off_d + threadIdx.x * row_s, row_ptr<TS>(a.dsum, a.lddsum, row), sizeof(TS), st, last);
    }
  };
  // two forms: a test for the last row in every copy costs long rows 3 % (16384 x 4095 bf16, pass after pass, 181 us, with
  // dropout 236; this way 175 and 228), and short ones nothing (32714 x 597 fp32 83 and 93 us either way)
  auto fill = [&](int64_t base, int st) {
    if (!SHIFT || base + rpb >= a.rows) fill_rows(base, st, std::true_type());
    else fill_rows(base, st, std::false_type());
  };
  // ... and those of its outputs to global memory (each lane its own row, so
  // that the lane that fills a row's place knows when it has been read)
  auto take = [&](unsigned char* row, uint32_t at, uint32_t size) {
    const uint32_t u0 = m_lane ? 8 : 0, u1 = (m_lane + a.cols) & ~7;      // whole units
    if (SHIFT) bulk_store(row + (int)(u0 - m_lane) * (int)size, at + u0 * size, (u1 - u0) * size);
    else bulk_store(row, at, a.cols * size);
  };
  auto drain = [&](int64_t base, int st) {
    const int n = (int)min((int64_t)rpb, a.rows - base);
    if ((int)threadIdx.x < n) {
      const uint32_t at = ring0 + (uint32_t)st * stage_bytes;
      const int64_t row = base + threadIdx.x;
      if (a.dx) take(reinterpret_cast<unsigned char*>(row_ptr<TA>(a.dx, a.lddx, row)), at + threadIdx.x * row_a, sizeof(TA));
      if (a.dr) take(reinterpret_cast<unsigned char*>(row_ptr<TS>(a.dr, a.lddr, row)), at + off_s + threadIdx.x * row_s, sizeof(TS));
    }
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
  };
  if (threadIdx.x == 0) {
    for (int i = 0; i < stages; ++i) mbar_init(&full[i], 1);
    fence_mbar_init_cluster();
  }
  __syncthreads();
  if (threadIdx.x < 32)
    for (int i = 0; i < stages; ++i)
      if (first + i * step < a.rows) fill(first + i * step, i);

  const DropWords words = a.d.threshold ? drop_words(a.d) : DropWords{};
  const UnitWalk walk = UnitWalk::of(MODE == kShifted, t, tpr, a.units);
  const int col0 = 8 * walk.first, dcol = 8 * walk.step;
  const int m = SHIFT ? (int)((first + lane_row) * a.shift) & 7 : 0;
  auto span = [&](int k) { return unit_span<MODE>(walk.first + k * walk.step, m, !SHIFT || k < a.units ? a.cols : 0); };
  bool in[K];
  F8 acc[K] = {}, gain[K];      // KEEP: a thread's gains stay in registers
  auto gain_at = [&](int k) {
    return in[k] ? load_gain<MODE>(a.gain, a.gain_fp32, SHIFT ? span(k) : Span{col0 + k * dcol, 0, 8}) : F8{};
  };
#pragma unroll
  for (int k = 0; k < K; ++k) {
    in[k] = SHIFT ? span(k).some() : col0 + k * dcol < a.cols;
    if (KEEP) gain[k] = gain_at(k);
  }
  // of a unit at the row's ends, the columns that are the row's
  auto trim = [&](F8 v, int k) {
    const Span p = span(k);
    if (SHIFT && (p.lo > 0 || p.hi < 8)) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 x = unpack_f2(v.p[i]);
        v.p[i] = pack_f2(2 * i >= p.lo && 2 * i < p.hi ? x.x : 0.0f, 2 * i + 1 >= p.lo && 2 * i + 1 < p.hi ? x.y : 0.0f);
      }
    }
    return v;
  };
  const uint32_t at_a0 = ring0 + (uint32_t)lane_row * row_a + (uint32_t)col0 * sizeof(TA);
  const uint32_t at_s0 = ring0 + off_s + (uint32_t)lane_row * row_s + (uint32_t)col0 * sizeof(TS);
  const uint32_t at_d0 = at_s0 + off_d - off_s;
  const float* rp = a.rstd + first + lane_row;
  float rstd_next = first + lane_row < a.rows ? *rp : 0.0f;
  uint64_t unit = (uint64_t)((first + lane_row) * a.per_row + walk.first);
  uint32_t at = 0;         // offset of the row's stage
  int st = 0, parity = 0;
  uint32_t pass = 0;
  bool dead = false;       // a wait ran out (recorded): go on without waiting, so that all threads still leave together
  int64_t base = first;
  for (; base < a.rows; base += step, parity ^= 1) {
    const bool on = base + lane_row < a.rows;
    const float rstd = rstd_next;
    rp += step;
    if (base + step + lane_row < a.rows) {
      rstd_next = *rp;
      if (a.dsum && !ring_d) {
#pragma unroll
        for (int k = 0; k < K; ++k)
          if (in[k])
            asm volatile("prefetch.global.L2 [%0];" ::"l"(row_ptr<TS>(a.dsum, a.lddsum, base + step + lane_row) + (SHIFT ? span(k).c + span(k).lo : col0 + k * dcol)));
      }
    }
    if (!dead) dead = !mbar_wait_u32(smem_u32(&full[st]), pass);
    const uint64_t rstd2 = pack_f2(rstd, rstd);
    Unit<TA> dh;
    Unit<TS> s, ds;
    uint64_t dot2 = 0;
    if (on) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (!in[k]) continue;
        lds_unit(at_a0 + at + (uint32_t)(k * dcol) * sizeof(TA), dh);
        lds_unit(at_s0 + at + (uint32_t)(k * dcol) * sizeof(TS), s);
        bwd_sums(trim(unpack(dh), k), trim(unpack(s), k), KEEP ? gain[k] : gain_at(k), rstd2, acc[k], dot2);
      }
    }
    // the row's sum: lanes by a butterfly, then all warps of the row (unused
    // places hold 0) in one fixed tree
    float dot = unpack_f2(dot2).x + unpack_f2(dot2).y;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
    if ((threadIdx.x & 31) == 0) red[parity][lane_row][t >> 5] = dot;
    __syncthreads();
    if (threadIdx.x < 32 && base != first) {
      const int prev = st == 0 ? stages - 1 : st - 1;
      drain(base - step, prev);
      // the outputs of the row before that have been read out of its stage
      asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
      if (base - first > step && base + (stages - 2) * step < a.rows)
        fill(base + (stages - 2) * step, prev == 0 ? stages - 1 : prev - 1);
    }
    {
      uint64_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 v = *reinterpret_cast<const float4*>(&red[parity][lane_row][4 * i]);
        w[i] = fadd2(pack_f2(v.x, v.y), pack_f2(v.z, v.w));
      }
      const float2 v = unpack_f2(fadd2(fadd2(w[0], w[1]), fadd2(w[2], w[3])));
      dot = v.x + v.y;
    }
    const float coef = -rstd * (rstd * (rstd * dot * a.inv_cols));
    const uint64_t c2 = pack_f2(coef, coef);
    if (on && (a.dr || a.dx)) {      // (the same for a whole warp)
      const bool drop = SHIFT && a.dx && a.d.threshold;
      ShiftedBits bits;
      if (SHIFT && drop && t > walk.lane) bits.start(unit - walk.lane - 1, words, a.d);
#pragma unroll
      for (int k = 0; k < K; ++k) {
        uint32_t w[4];
        if (SHIFT && drop && 8 * (walk.first - walk.lane + k * walk.step) < a.cols + 7) bits.next(unit + k * walk.step, walk.lane, 32, m, words, a.d, w);
        if (!in[k]) continue;
        const uint32_t pa = at_a0 + at + (uint32_t)(k * dcol) * sizeof(TA), ps = at_s0 + at + (uint32_t)(k * dcol) * sizeof(TS);
        const Span p = span(k);
        const bool whole = !SHIFT || (p.lo == 0 && p.hi == 8);
        lds_unit(pa, dh);
        lds_unit(ps, s);
        if (ring_d) lds_unit(at_d0 + at + (uint32_t)(k * dcol) * sizeof(TS), ds);
        else if (a.dsum && SHIFT) load_unit<MODE>(row_ptr<TS>(a.dsum, a.lddsum, base + lane_row) + p.c, p.lo, p.hi, ds);
        else if (a.dsum) ld_unit(row_ptr<TS>(a.dsum, a.lddsum, base + lane_row) + col0 + k * dcol, ds);
        F8 v = bwd_unit(unpack(dh), unpack(s), KEEP ? gain[k] : gain_at(k), a.dsum ? unpack(ds) : F8{}, rstd2, c2);
        if (a.dr) {
          if (whole) sts_unit(ps, v, TS());
          else store_unit<MODE>(row_ptr<TS>(a.dr, a.lddr, base + lane_row) + p.c, p.lo, p.hi, v);
        }
        if (a.dx) {
          if (a.d.threshold) {
            if (SHIFT) drop_apply(v, w, a.d);
            else drop_unit(v, unit + k * walk.step, words, a.d);
          }
          if (whole) sts_unit(pa, v, TA());
          else store_unit<MODE>(row_ptr<TA>(a.dx, a.lddx, base + lane_row) + p.c, p.lo, p.hi, v);
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    unit += (uint64_t)(step * a.per_row);
    at += stage_bytes;
    if (++st == stages) {
      st = 0;
      at = 0;
      pass ^= 1u;
    }
  }
  if (dead) {      // copies still under way land before their memory is used again or given up (waited for once more, bounded)
    const int64_t n = ceil_div<int64_t>(a.rows - first, step);
    for (int i = 0; i < stages && i < n; ++i) mbar_wait_u32(smem_u32(&full[i]), (uint32_t)((n - 1 - i) / stages) & 1u);
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    drain(base - step, st == 0 ? stages - 1 : st - 1);       // the last row's outputs
    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }
  if (!a.part) return;
  griddep_launch_dependents();
  float* part = a.part + (int64_t)blockIdx.x * a.cols;
  float* comb = reinterpret_cast<float*>(ring);      // every copy has landed, and every store has left
  __syncthreads();
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const Span p = span(k);
    if (in[k]) store_unit<kScalar>((rpb == 1 ? part : comb + lane_row * a.cols) + p.c, p.lo, p.hi, acc[k]);
  }
  if (rpb == 1) return;
  __syncthreads();
  for (int c = threadIdx.x; c < a.cols; c += blockDim.x) {
    float v = 0.0f;
    for (int r = 0; r < rpb; ++r) v += comb[r * a.cols + c];
    part[c] = v;
  }
}

// dg[c] = sum over the blocks' partial rows: 32 columns a block, 32 threads a
// column, each over every 32nd partial, then a tree.
__global__ void __launch_bounds__(1024) k_sum_partials(const float* part, int n_parts, int cols,
                                                       void* __restrict__ out, int out_fp32) {
  __shared__ float red[32][33];
  const int c = blockIdx.x * 32 + threadIdx.x;
  float v = 0.0f;
  griddep_wait();
  if (c < cols) {
#pragma unroll 8
    for (int p = threadIdx.y; p < n_parts; p += 32) v += part[(int64_t)p * cols + c];
  }
  red[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  v = red[threadIdx.x][threadIdx.y];       // column threadIdx.y, partial sum threadIdx.x
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const int col = blockIdx.x * 32 + threadIdx.y;
  if (threadIdx.x == 0 && col < cols) {
    if (out_fp32) static_cast<float*>(out)[col] = v;
    else static_cast<__nv_bfloat16*>(out)[col] = __float2bfloat16_rn(v);
  }
}

// Threads a row: enough that four units a thread cover it, at least 16 with
// scale groups (a group of 128 columns is 16 units); while rows leave SMs
// without work, one unit a thread.  A row of up to 64 threads takes a power of
// two and shares its block of 128; a longer one has a block of its own, of
// whole warps (not rounded up further: 12288 columns take 384 threads, two
// blocks of which fit an SM, where 512 would leave one).
void pick_threads(int64_t rows, int64_t per_row, bool groups, int32_t* tpr, int32_t* rpb, int32_t* n) {
  const int64_t units = rows < 2 * sm_count() ? 1 : kK;
  int64_t t = std::min<int64_t>(ceil_div<int64_t>(per_row, units), kMaxThreads);
  if (t > 64) {
    *tpr = (int32_t)ceil_div<int64_t>(t, 32) * 32;
    *rpb = 1;
  } else {
    int p = groups ? 16 : 4;
    while (p < t) p *= 2;
    *tpr = p;
    *rpb = 128 / p;
  }
  *n = (int32_t)ceil_div<int64_t>(per_row, *tpr);
}

constexpr int kMaxParts = 1024;   // blocks of the backward kernel, and so partial rows of dg

// Blocks of a persistent grid over `blocks` blocks' worth of rows: a multiple
// of eight if there is more than one pass, so that a thread's rows all start
// the same number of columns past a unit.
inline int64_t grid_blocks(int64_t blocks, int64_t resident) {
  const int64_t most = std::min<int64_t>(resident, kMaxParts);
  return blocks <= most ? blocks : std::max<int64_t>(8, most / 8 * 8);
}

constexpr unsigned kTypes = 1u << SF_BF16 | 1u << SF_FP32;

template <typename TA, typename TS>
struct Fwd {
  static const void* ptr(RowMode mode, bool drop) {
    return mode == kAligned           ? (const void*)&k_add_rmsnorm_fwd<TA, TS, kAligned, true>
           : mode == kShifted && drop ? (const void*)&k_add_rmsnorm_fwd<TA, TS, kShifted, true>
           : mode == kShifted         ? (const void*)&k_add_rmsnorm_fwd<TA, TS, kShifted, false>
                                      : (const void*)&k_add_rmsnorm_fwd<TA, TS, kScalar, true>;
  }
};
template <typename TA, typename TS>
struct Bwd {
  static const void* ptr(RowMode mode, bool) {
    return mode == kAligned   ? (const void*)&k_add_rmsnorm_bwd<TA, TS, kAligned>
           : mode == kShifted ? (const void*)&k_add_rmsnorm_bwd<TA, TS, kShifted>
                              : (const void*)&k_add_rmsnorm_bwd<TA, TS, kScalar>;
  }
};
template <template <typename, typename> class K>
const void* pick(int32_t ta, int32_t ts, RowMode mode, bool drop) {
  using B = __nv_bfloat16;
  if (ta == SF_BF16) return ts == SF_BF16 ? K<B, B>::ptr(mode, drop) : K<B, float>::ptr(mode, drop);
  return ts == SF_BF16 ? K<float, B>::ptr(mode, drop) : K<float, float>::ptr(mode, drop);
}
// The mode of a call: kAligned also wants the gains on their units.
template <size_t N>
RowMode call_mode(const sf_matrix* const (&ms)[N], const void* gain, int32_t gain_dtype, int* shift) {
  const RowMode mode = row_mode(ms, shift);
  return mode == kAligned && reinterpret_cast<uintptr_t>(gain) % (8 * dtype_bytes(gain_dtype)) ? kShifted : mode;
}


constexpr size_t kSmemPerSm = 222 << 10;

// Bytes of one row in the staged kernel's ring.
inline size_t ring_row_bytes(int64_t cols, bool shifted, int32_t ta, int32_t ts, bool dsum) {
  return (size_t)(shifted ? (cols + 15) / 8 * 8 : cols) * (dtype_bytes(ta) + (dsum ? 2 : 1) * dtype_bytes(ts));
}

// The staged kernel takes aligned rows of whole units, long enough that a
// block's few copies are worth their set-up and short enough that three fit
// in shared memory (without dsum if need be: 8192 x 12288 bf16, fp32 stream,
// 296 us, against 382 us with loads into registers), when there is more than
// one block's worth of rows an SM.
inline bool ring_fits(int64_t rows, int64_t cols, RowMode mode, int32_t ta, int32_t ts) {
  return (mode == kShifted || (mode == kAligned && cols % 8 == 0)) && cols >= 512 && rows >= 2 * sm_count() &&
         kMinStages * ring_row_bytes(cols, mode == kShifted, ta, ts, false) <= kSmemPerSm - 1024;
}

template <typename TA, typename TS, bool SHIFT>
const void* ring_kernel(int k, bool keep) {
  if (k == 2) return (const void*)&k_add_rmsnorm_bwd_ring<TA, TS, 2, true, SHIFT>;
  // rows too long to keep their gains have over 12288 columns, of which the ring does not hold three in fp32 throughout
  if constexpr (sizeof(TA) + sizeof(TS) < 8)
    if (!keep) return (const void*)&k_add_rmsnorm_bwd_ring<TA, TS, 4, false, SHIFT>;
  return (const void*)&k_add_rmsnorm_bwd_ring<TA, TS, 4, true, SHIFT>;
}
template <typename TA, typename TS>
const void* ring_kernel(int k, bool keep, bool shifted) {
  return shifted ? ring_kernel<TA, TS, true>(k, keep) : ring_kernel<TA, TS, false>(k, keep);
}

// Two units a thread up to 1024 columns, four beyond (16384 x 4096 bf16, all
// outputs: 137 us with four, 149 us with two: fewer barriers' worth of work a
// row outweighs fewer warps), and the gains in registers where a block's
// registers allow (118 us, against 130 us read from L1 in both passes); as many
// blocks an SM as registers and three stages each allow.
sf_status launch_ring(BwdArgs& a, bool shifted, int32_t ta, int32_t ts, cudaStream_t st, int64_t* parts) {
  using B = __nv_bfloat16;
  const int units = a.per_row + (shifted ? 1 : 0);
  const int k = units <= 128 ? 2 : 4;
  const int t = ceil_div(units, k);
  if (t > 64) {
    a.tpr = ceil_div(t, 32) * 32;
    a.rpb = 1;
  } else {
    a.tpr = t > 32 ? 64 : 32;
    a.rpb = 128 / a.tpr;
  }
  a.units = ceil_div(units, a.tpr);
  const int threads = a.tpr * a.rpb;
  const bool keep = threads <= 384;
  const void* kernel = ta == SF_BF16 ? (ts == SF_BF16 ? ring_kernel<B, B>(k, keep, shifted) : ring_kernel<B, float>(k, keep, shifted))
                                     : (ts == SF_BF16 ? ring_kernel<float, B>(k, keep, shifted) : ring_kernel<float, float>(k, keep, shifted));
  a.ring_dsum = a.dsum && kMinStages * a.rpb * ring_row_bytes(a.cols, shifted, ta, ts, true) <= kSmemPerSm - 1024;
  const size_t stage = a.rpb * ring_row_bytes(a.cols, shifted, ta, ts, a.ring_dsum);
  const int per_sm = (int)std::max<size_t>(1, std::min<size_t>((k == 2 && !shifted ? 768 : keep && k == 4 ? 384 : 512) / threads, kSmemPerSm / (kMinStages * stage + 1024)));
  const int stages = (int)std::min<size_t>(kMaxStages, (kSmemPerSm / per_sm - 1024) / stage);
  const size_t smem = stage * stages;
  SF_TRY(allow_dynamic_smem(kernel, smem));
  *parts = grid_blocks(ceil_div<int64_t>(a.rows, a.rpb), (int64_t)sm_count() * per_sm);
  void* args[] = {&a, const_cast<int*>(&stages)};
  SF_CUDA_TRY(cudaLaunchKernel(kernel, dim3((unsigned)*parts), dim3(threads), args, smem, st), "launch k_add_rmsnorm_bwd_ring");
  return SF_OK;
}

sf_status check_gain(const void* gain, int32_t dtype, const char* name) {
  if (!gain) return fail(SF_ERR_INVALID, "%s is NULL", name);
  if (dtype != SF_BF16 && dtype != SF_FP32) return fail(SF_ERR_UNSUPPORTED, "%s: type %d is not taken here", name, (int)dtype);
  return check_aligned(gain, dtype_bytes(dtype), name);
}

sf_status check_cols(int64_t cols) {
  if (cols < 1) return fail(SF_ERR_INVALID, "a row needs at least one column");
  if (cols > kMaxCols) return fail(SF_ERR_UNSUPPORTED, "rows of up to %lld columns are supported (got %lld)", (long long)kMaxCols, (long long)cols);
  return SF_OK;
}

}  // namespace

const void* device_error_norm() { return &g_device_error; }

}  // namespace sf

extern "C" {

sf_status sf_add_rmsnorm_forward(const sf_matrix* x, const sf_matrix* residual, const void* gain, sf_dtype gain_dtype,
                                 double eps, double p, const sf_rng* rng, const sf_matrix* sum, const sf_matrix* h,
                                 const sf_matrix* h8, float* h8_scale, int32_t group, float* rstd, void* stream) {
  using namespace sf;
  clear_error();
  NvtxRange nvtx_range("sf_add_rmsnorm_forward");
  SF_TRY(check_matrix(x, "x", -1, -1, kTypes));
  const int64_t rows = x->rows, cols = x->cols;
  SF_TRY(check_cols(cols));
  SF_TRY(check_gain(gain, gain_dtype, "gain"));
  if (!(eps >= 0.0) || eps > 1e30) return fail(SF_ERR_INVALID, "eps must be finite and >= 0");
  if (residual) SF_TRY(check_matrix(residual, "residual", rows, cols, kTypes));
  if (sum) SF_TRY(check_matrix(sum, "sum", rows, cols, kTypes));
  if (h) SF_TRY(check_matrix(h, "h", rows, cols, kTypes));
  if (h8) SF_TRY(check_matrix(h8, "h8", rows, cols, 1u << SF_E4M3));
  if (!h && !h8) return fail(SF_ERR_INVALID, "h and h8 are both NULL");
  if (h && h->dtype != x->dtype) return fail(SF_ERR_INVALID, "h and x must have one type");
  if (residual && sum && residual->dtype != sum->dtype) return fail(SF_ERR_INVALID, "residual and sum must have one type");
  if (h8) {
    if (!h8_scale) return fail(SF_ERR_INVALID, "h8 needs h8_scale");
    if (group != 0 && group != 32 && group != 64 && group != 128)
      return fail(SF_ERR_INVALID, "group must be 0 (a scale per row), 32, 64 or 128 (got %d)", (int)group);
    SF_TRY(check_aligned(h8_scale, sizeof(float), "h8_scale"));
  }
  SF_TRY(check_aligned(rstd, sizeof(float), "rstd"));
  FwdArgs a{};
  SF_TRY(make_drop_consts(p, rng, &a.d));
  if (!rows) return SF_OK;
  a.x = x->data;
  a.ldx = x->ld;
  if (residual) a.r = residual->data, a.ldr = residual->ld;
  if (sum) a.s = sum->data, a.lds = sum->ld;
  if (h) a.h = h->data, a.ldh = h->ld;
  if (h8) a.q = static_cast<uint8_t*>(h8->data), a.ldq = h8->ld;
  a.scale = h8_scale;
  a.rstd = rstd;
  a.gain = gain;
  a.gain_fp32 = gain_dtype == SF_FP32;
  a.rows = rows;
  a.cols = (int32_t)cols;
  a.per_row = (int32_t)ceil_div<int64_t>(cols, 8);
  a.group_log2 = group == 128 ? 7 : group == 64 ? 6 : group == 32 ? 5 : 0;
  a.n_groups = group ? (int32_t)ceil_div<int64_t>(cols, group) : 1;
  a.eps = (float)eps;
  a.inv_cols = (float)(1.0 / (double)cols);
  const sf_matrix* const all[5] = {x, residual, sum, h, h8};
  RowMode mode = call_mode(all, gain, gain_dtype, &a.shift);
  // a shifted row may touch one unit more, which four units a thread have to cover
  if (mode == kShifted && cols > kMaxCols - 8) mode = kScalar;
  pick_threads(rows, a.per_row + (mode == kShifted ? 1 : 0), h8 != nullptr, &a.tpr, &a.rpb, &a.units);
  const int threads = a.tpr * a.rpb;
  const int64_t grid = ceil_div<int64_t>(rows, a.rpb);
  if (grid > INT32_MAX) return fail(SF_ERR_UNSUPPORTED, "too many rows");
  const int32_t ts = residual ? residual->dtype : sum ? sum->dtype : x->dtype;
  void* args[] = {&a};
  SF_CUDA_TRY(cudaLaunchKernel(pick<Fwd>(x->dtype, ts, mode, a.d.threshold != 0), dim3((unsigned)grid), dim3(threads), args, 0, as_stream(stream)),
              "launch k_add_rmsnorm_fwd");
  return SF_OK;
}

size_t sf_add_rmsnorm_workspace_bytes(int64_t rows, int64_t cols) {
  if (rows < 0 || cols < 1 || cols > sf::kMaxCols) return 0;
  return (size_t)std::max<int64_t>(1, std::min<int64_t>(rows, sf::kMaxParts)) * cols * sizeof(float);
}

sf_status sf_add_rmsnorm_backward(const sf_matrix* dh, const sf_matrix* sum, const void* gain, sf_dtype gain_dtype,
                                  const float* rstd, const sf_matrix* dsum, double p, const sf_rng* rng,
                                  const sf_matrix* dresidual, const sf_matrix* dx, void* dgain, sf_dtype dgain_dtype,
                                  void* ws, size_t ws_bytes, void* stream) {
  using namespace sf;
  clear_error();
  NvtxRange nvtx_range("sf_add_rmsnorm_backward");
  SF_TRY(check_matrix(dh, "dh", -1, -1, kTypes));
  const int64_t rows = dh->rows, cols = dh->cols;
  SF_TRY(check_cols(cols));
  SF_TRY(check_matrix(sum, "sum", rows, cols, kTypes));
  SF_TRY(check_gain(gain, gain_dtype, "gain"));
  if (!rstd && rows) return fail(SF_ERR_INVALID, "rstd is NULL");
  SF_TRY(check_aligned(rstd, sizeof(float), "rstd"));
  if (dsum) SF_TRY(check_matrix(dsum, "dsum", rows, cols, 1u << sum->dtype));
  if (dresidual) SF_TRY(check_matrix(dresidual, "dresidual", rows, cols, 1u << sum->dtype));
  if (dx) SF_TRY(check_matrix(dx, "dx", rows, cols, 1u << dh->dtype));
  if (!dresidual && !dx && !dgain) return fail(SF_ERR_INVALID, "dresidual, dx and dgain are all NULL");
  if (dgain) {
    SF_TRY(check_gain(dgain, dgain_dtype, "dgain"));
    const size_t need = sf_add_rmsnorm_workspace_bytes(rows, cols);
    if (!ws || ws_bytes < need || reinterpret_cast<uintptr_t>(ws) % 16)
      return fail(SF_ERR_INVALID, "workspace needs %zu bytes, 16-byte aligned (got %zu)", need, ws_bytes);
  }
  BwdArgs a{};
  SF_TRY(make_drop_consts(p, rng, &a.d));
  a.dh = dh->data;
  a.lddh = dh->ld;
  a.s = sum->data;
  a.lds = sum->ld;
  if (dsum) a.dsum = dsum->data, a.lddsum = dsum->ld;
  if (dresidual) a.dr = dresidual->data, a.lddr = dresidual->ld;
  if (dx) a.dx = dx->data, a.lddx = dx->ld;
  a.gain = gain;
  a.gain_fp32 = gain_dtype == SF_FP32;
  a.rstd = rstd;
  a.part = dgain ? static_cast<float*>(ws) : nullptr;
  a.rows = rows;
  a.cols = (int32_t)cols;
  a.per_row = (int32_t)ceil_div<int64_t>(cols, 8);
  a.inv_cols = (float)(1.0 / (double)cols);
  const sf_matrix* const all[5] = {dh, sum, dsum, dresidual, dx};
  RowMode mode = call_mode(all, gain, gain_dtype, &a.shift);
  if (mode == kShifted && cols > kMaxCols - 8) mode = kScalar;      // as in the forward pass
  pick_threads(rows, a.per_row + (mode == kShifted ? 1 : 0), false, &a.tpr, &a.rpb, &a.units);
  const int threads = a.tpr * a.rpb, rpb = a.rpb;
  const int64_t grid = grid_blocks(ceil_div<int64_t>(rows, rpb), (int64_t)sm_count() * std::max(1, 512 / threads));
  // a few KB with several rows a block, up to 64 KB shifted
  const size_t smem = mode == kShifted || (dgain && rpb > 1) ? (size_t)rpb * (8 * a.per_row + 8) * sizeof(float) : 0;
  cudaStream_t st = as_stream(stream);
  int64_t parts = grid;
  // bulk copies take this device's own memory only (pinned host rows go the plain way)
  auto local = [](const sf_matrix* m) { return !m || on_current_device(m->data); };
  if (ring_fits(rows, cols, mode, dh->dtype, sum->dtype) && local(dh) && local(sum) && local(dsum) &&
      local(dresidual) && local(dx)) {
    SF_TRY(launch_ring(a, mode == kShifted, dh->dtype, sum->dtype, st, &parts));
  } else if (grid) {
    void* args[] = {&a};
    const void* kernel = pick<Bwd>(dh->dtype, sum->dtype, mode, a.d.threshold != 0);
    if (smem > (48 << 10)) SF_TRY(allow_dynamic_smem(kernel, smem));
    SF_CUDA_TRY(cudaLaunchKernel(kernel, dim3((unsigned)grid), dim3(threads), args, smem, st),
                "launch k_add_rmsnorm_bwd");
  }
  if (dgain) {
    SF_CUDA_TRY(launch_pdl(k_sum_partials, dim3((unsigned)ceil_div<int64_t>(cols, 32)), dim3(32, 32), 0, st, a.part, (int)parts,
                           (int)cols, dgain, (int)(dgain_dtype == SF_FP32)),
                "launch k_sum_partials");
  }
  return SF_OK;
}

}  // extern "C"
