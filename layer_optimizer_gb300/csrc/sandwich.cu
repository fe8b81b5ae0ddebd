// The end of a residual block: the norm after the block, its gate, the
// residual's addition with its scales, and the norm before the next block,
//   n = x rho1 g1,  s = a r + b gate n,  h = s rho2 g2,
// rho = 1 / sqrt(mean(row^2) + eps), and its gradients; x and s kept as 8-bit
// checkpoints where wanted.  (The root-mean-square norm is Zhang and Sennrich
// 2019.)
#include <algorithm>

#include "lanes.cuh"
#include "ptx.cuh"

namespace sf {
namespace {

constexpr int kK = 2;               // steps per thread of the register forms
constexpr int kMaxThreads = 1024;
constexpr int64_t kMaxCols = (int64_t)kMaxThreads * kK * 8;   // 16384

// What both passes take of a call.
struct Vectors {
  const void* g_post;      // may be null
  const void* g_pre;       // may be null
  const void* gate;        // may be null
  int64_t ld_gate, span;
  int32_t gain_fp32, gate_fp32;
  float offset, a, b;      // gain offset, residual and block scales
};

struct FwdArgs {
  const void* x;
  const void* r;       // may be null
  void* s;             // may be null
  void* h;             // may be null
  float* rho1;         // may be null
  float* rho2;         // may be null
  Ck x8, s8;
  int64_t ldx, ldr, lds, ldh, rows;
  int32_t cols, tpr, rpb, steps;
  int32_t wide;        // staged form: rows on wide units, not on units of eight only
  float eps, inv_cols;
  Vectors v;
};

__device__ __forceinline__ const void* gate_row_of(const Vectors& v, int64_t k) {
  return static_cast<const char*>(v.gate) + k * v.ld_gate * (v.gate_fp32 ? 4 : 2);
}
__device__ __forceinline__ const void* gate_row(const Vectors& v, int64_t row) { return gate_row_of(v, row / v.span); }

__device__ __forceinline__ F8 mul8(const F8& a, const F8& b) {
  F8 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r.p[i] = fmul2(a.p[i], b.p[i]);
  return r;
}
__device__ __forceinline__ F8 scale8(const F8& a, float f) {
  F8 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r.p[i] = fmul2(a.p[i], pack_f2(f, f));
  return r;
}
__device__ __forceinline__ float dot8(const F8& a, const F8& b) {
  uint64_t s = fmul2(a.p[0], b.p[0]);
#pragma unroll
  for (int i = 1; i < 4; ++i) s = fmadd2(a.p[i], b.p[i], s);
  const float2 x = unpack_f2(s);
  return x.x + x.y;
}

// One pass: a row's x and r are read once into registers, x's squares summed
// over the row, s formed and summed in turn, and h written from registers.
template <typename TA, typename TS, int LAY>
__global__ void __launch_bounds__(kMaxThreads) k_sandwich_fwd(const FwdArgs a) {
  __shared__ float red[2][2 * (kMaxThreads / 32)];
  const int tpr = a.tpr, lane_row = (int)threadIdx.x / tpr, t = (int)threadIdx.x - lane_row * tpr;
  const int64_t row = (int64_t)blockIdx.x * a.rpb + lane_row;
  const bool on = row < a.rows;
  const int cols = on ? a.cols : 0;
  const Lane l = lane_of<LAY>(t, tpr);
  Unit<TA> x[kK];      // (zero past the row)
  Unit<TS> r[kK];
  const TA* xp = row_ptr<TA>(a.x, a.ldx, row);
  const TS* rp = row_ptr<TS>(a.r, a.ldr, row);
#pragma unroll
  for (int k = 0; k < kK; ++k) {
    x[k] = Unit<TA>{};
    if (l.c0(k) >= cols) continue;
    load_raw<LAY>(xp, l.c0(k), l.dj, cols, x[k]);
    if (a.r) load_raw<LAY>(rp, l.c0(k), l.dj, cols, r[k]);
  }
  const bool post = a.v.g_post != nullptr, x_row = a.x8.q && !a.x8.group_log2;
  float rho1 = 1.0f;
  if (post || x_row) {
    float m[2] = {0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < kK; ++k) {
      const F8 v = unpack(x[k]);
      m[0] += dot8(v, v);
      if (x_row) m[1] = fmaxf(m[1], top8_finite(v));
    }
    row_reduce_n<2, 1>(m, tpr, red[0]);
    if (post) {
      rho1 = rsqrtf(fmaf(m[0], a.inv_cols, a.eps));
      if (a.rho1 && on && t == 0) a.rho1[row] = rho1;
    }
    if (x_row && on && t == 0) a.x8.s8[row] = (uint8_t)e8m0_of(m[1]);
    if (a.x8.q) {
#pragma unroll
      for (int k = 0; k < kK; ++k)
        if (k < a.steps) ck_store8<LAY>(a.x8, row, l.c0(k), l.dj, cols, unpack(x[k]), e8m0_of(m[1]));
    }
  } else if (a.x8.q) {
#pragma unroll
    for (int k = 0; k < kK; ++k)
      if (k < a.steps) ck_store8<LAY>(a.x8, row, l.c0(k), l.dj, cols, unpack(x[k]), 1);
  }
  if (!a.s && !a.h && !a.s8.q && !a.rho2) return;
  float m[2] = {0.0f, 0.0f};
  const bool s_row = a.s8.q && !a.s8.group_log2;
  F8 s[kK];
#pragma unroll
  for (int k = 0; k < kK; ++k) {
    s[k] = zero8();
    if (l.c0(k) >= cols) continue;
    F8 n = unpack(x[k]);
    if (post) n = mul8(scale8(n, rho1), load_vec<LAY>(a.v.g_post, a.v.gain_fp32, l.c0(k), l.dj, cols, a.v.offset));
    if (a.v.gate) n = mul8(n, load_vec<LAY>(gate_row(a.v, row), a.v.gate_fp32, l.c0(k), l.dj, cols, 0.0f));
    n = scale8(n, a.v.b);
    if (a.r) {
#pragma unroll
      for (int i = 0; i < 4; ++i) n.p[i] = fmadd2(unpack(r[k]).p[i], pack_f2(a.v.a, a.v.a), n.p[i]);
    }
    s[k] = n;
    if (a.s) store8<LAY>(row_ptr<TS>(a.s, a.lds, row), l.c0(k), l.dj, cols, n);
    m[0] += dot8(n, n);
    if (s_row) m[1] = fmaxf(m[1], top8_finite(n));
  }
  const bool pre = a.h || a.rho2;
  if (pre || s_row) row_reduce_n<2, 1>(m, tpr, red[1]);
  if (s_row && on && t == 0) a.s8.s8[row] = (uint8_t)e8m0_of(m[1]);
  if (a.s8.q) {
#pragma unroll
    for (int k = 0; k < kK; ++k)
      if (k < a.steps) ck_store8<LAY>(a.s8, row, l.c0(k), l.dj, cols, s[k], e8m0_of(m[1]));
  }
  if (!pre) return;
  const float rho2 = rsqrtf(fmaf(m[0], a.inv_cols, a.eps));
  if (a.rho2 && on && t == 0) a.rho2[row] = rho2;
  if (!a.h) return;
#pragma unroll
  for (int k = 0; k < kK; ++k) {
    if (l.c0(k) >= cols) continue;
    const F8 g = load_vec<LAY>(a.v.g_pre, a.v.gain_fp32, l.c0(k), l.dj, cols, a.v.offset);
    store8<LAY>(row_ptr<TA>(a.h, a.ldh, row), l.c0(k), l.dj, cols, mul8(scale8(s[k], rho2), g));
  }
}

// The same with rows brought by bulk copies, for aligned rows of whole units:
// a block takes neighbouring rows one after the other, `stages` of them on
// their way into shared memory, so that loads never wait for a row's sums.
// What the rows share (b gate g1, g2) stays in registers while the gate row is
// the same.
constexpr int kRingThreads = 768, kMaxStages = 8;

// A block's sum of a value per lane and, where wanted, maximum of another one.
// red: up to kRingThreads / 32 floats of each, those of warps that the block
// has not zero; alternating between calls.
constexpr int kRed = kRingThreads / 32;
__device__ __forceinline__ float block_sum(float v, float* top, float (&red)[2][kRed]) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (top) *top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(*top)));      // magnitudes order as their bits
  if ((threadIdx.x & 31) == 0) {
    red[0][threadIdx.x >> 5] = v;
    if (top) red[1][threadIdx.x >> 5] = *top;
  }
  __syncthreads();
  uint64_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 x = *reinterpret_cast<const float4*>(&red[0][4 * i]);
    w[i] = fadd2(pack_f2(x.x, x.y), pack_f2(x.z, x.w));
  }
  w[0] = fadd2(fadd2(w[0], w[1]), fadd2(w[2], w[3]));
  if (blockDim.x > 512) {
#pragma unroll
    for (int i = 4; i < kRed / 4; ++i) {
      const float4 x = *reinterpret_cast<const float4*>(&red[0][4 * i]);
      w[0] = fadd2(w[0], fadd2(pack_f2(x.x, x.y), pack_f2(x.z, x.w)));
    }
  }
  if (top) {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < kRed; ++i) m = fmaxf(m, red[1][i]);
    *top = m;
  }
  const float2 x = unpack_f2(w[0]);
  return x.x + x.y;
}
// What a maximum over finite values starts from: infinity where one is not.
__device__ __forceinline__ float top_or_inf(float top) { return top <= kLargest ? top : __uint_as_float(0x7f800000u); }

template <typename T>
struct LdsWide;      // 16 columns from shared memory
template <>
struct LdsWide<__nv_bfloat16> : Wide<__nv_bfloat16> {
  __device__ __forceinline__ explicit LdsWide(uint32_t p) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int4 v = lds_i4(p + 16 * i);
      w[i] = make_uint4(v.x, v.y, v.z, v.w);
    }
  }
};
template <>
struct LdsWide<float> : Wide<float> {
  __device__ __forceinline__ explicit LdsWide(uint32_t p) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int4 v = lds_i4(p + 16 * i);
      w[i] = make_uint4(v.x, v.y, v.z, v.w);
    }
  }
};

// A row in shared memory: the 16-byte words that hold any of it, so that its
// first column lies as far into the first word as in memory.  Of the matrix's
// last row, past which memory may end, the last word's bytes come by ordinary
// loads.
__device__ __forceinline__ uint32_t lead_of(const void* row) { return (uint32_t)reinterpret_cast<uintptr_t>(row) & 15u; }
__host__ __device__ __forceinline__ uint32_t slot_bytes(int64_t cols, uint32_t size) { return (uint32_t)(cols * size + 30) & ~15u; }
struct Bring {
  const void* row;
  uint32_t bytes;      // of the row
  bool last;
  __device__ __forceinline__ uint32_t copied() const { return (lead_of(row) + bytes + (last ? 0u : 15u)) & ~15u; }
  __device__ __forceinline__ void rest(unsigned char* to) const {      // before the arrival
    const unsigned char* from = static_cast<const unsigned char*>(row) - lead_of(row);
    for (uint32_t i = copied(); i < lead_of(row) + bytes; ++i) to[i] = from[i];
  }
  __device__ __forceinline__ void copy(unsigned char* to, uint64_t* bar) const {
    if (copied()) bulk_load(to, static_cast<const unsigned char*>(row) - lead_of(row), copied(), bar);
  }
};
// Brings N rows' worth of operands into their slots, by one thread.
template <int N>
__device__ __forceinline__ void bring_rows(const Bring (&b)[N], unsigned char* const (&to)[N], uint64_t* bar) {
  uint32_t bytes = 0;
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (b[i].bytes) {
      bytes += b[i].copied();
      b[i].rest(to[i]);
    }
  mbar_arrive_expect_tx(bar, bytes);
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (b[i].bytes) b[i].copy(to[i], bar);
}

// 16 columns of a thread in either lay.  c0: its first; strided ones are 32 apart.
template <int LAY>
__device__ __forceinline__ int first16(int t, int T, int k) {
  return LAY == kUnits ? 16 * (t + k * T) : ((t >> 5) + k * (T >> 5)) * 512 + (t & 31);
}
__device__ __forceinline__ float lds_value(uint32_t p, __nv_bfloat16) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(p));
  return __uint_as_float((uint32_t)v << 16);
}
__device__ __forceinline__ float lds_value(uint32_t p, float) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(p));
  return v;
}
// From shared memory, at the address of column 0 (c0 below cols; strided columns past it read as zero).
template <typename T, int LAY>
__device__ __forceinline__ void lds16(uint32_t p, int c0, int cols, F8 (&v)[2]) {
  if constexpr (LAY == kUnits) {
    const LdsWide<T> u(p + c0 * (uint32_t)sizeof(T));
    v[0] = u.half(0), v[1] = u.half(1);
  } else {
    float x[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) x[e] = c0 + 32 * e < cols ? lds_value(p + (c0 + 32 * e) * (uint32_t)sizeof(T), T()) : 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e >> 2].p[e & 3] = pack_f2(x[2 * e], x[2 * e + 1]);
  }
}
template <typename T, int LAY>
__device__ __forceinline__ void put16(T* row, int c0, int cols, const F8& lo, const F8& hi, bool wide) {
  if constexpr (LAY == kUnits) {
    store16(row + c0, lo, hi, wide);
  } else {
    store8<kStrided>(row, c0, 32, cols, lo);
    store8<kStrided>(row, c0 + 256, 32, cols, hi);
  }
}
template <int LAY>
__device__ __forceinline__ void vec16(const void* p, int fp32, int c0, int cols, float add, F8 (&v)[2]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) v[h] = load_vec<LAY>(p, fp32, c0 + (LAY == kUnits ? 8 : 256) * h, LAY == kUnits ? 1 : 32, cols, add);
}

// C: wide units a thread.  With one of them g2 stays in registers too.
template <typename TA, typename TS, int LAY, int C, int REGS>
__global__ void __maxnreg__(REGS) k_sandwich_fwd_ring(const FwdArgs a, const int stages) {
  __shared__ __align__(16) float red[2][2][2][kRed];      // [row mod 2][which sum][sums, maxima]
  __shared__ float redx[kRed];
  __shared__ __align__(8) uint64_t full[kMaxStages];
  extern __shared__ __align__(128) unsigned char ring[];
  const int t = threadIdx.x, T = blockDim.x;
  for (int i = t; i < 8 * kRed; i += T) (&red[0][0][0][0])[i] = 0.0f;
  const uint32_t row_x = slot_bytes(a.cols, sizeof(TA)), stage_bytes = row_x + (a.r ? slot_bytes(a.cols, sizeof(TS)) : 0u);
  const uint32_t ring0 = smem_u32(ring);
  const int64_t first = a.rows * blockIdx.x / gridDim.x, end = a.rows * (blockIdx.x + 1) / gridDim.x;
  auto fill = [&](int64_t row, int st) {      // by one thread
    unsigned char* at = ring + (size_t)st * stage_bytes;
    const bool last = row == a.rows - 1;
    const Bring b[2] = {{row_ptr<TA>(a.x, a.ldx, row), (uint32_t)a.cols * (uint32_t)sizeof(TA), last},
                        {row_ptr<TS>(a.r, a.ldr, row), a.r ? (uint32_t)a.cols * (uint32_t)sizeof(TS) : 0u, last}};
    unsigned char* const to[2] = {at, at + row_x};
    bring_rows(b, to, &full[st]);
  };
  if (t == 0) {
    for (int i = 0; i < stages; ++i) mbar_init(&full[i], 1);
    fence_mbar_init_cluster();
    for (int i = 0; i < stages && first + i < end; ++i) fill(first + i, i);
  }
  __syncthreads();
  const bool post = a.v.g_post != nullptr;
  const bool x_row = a.x8.q && !a.x8.group_log2, s_row = a.s8.q && !a.s8.group_log2;
  F8 w[C][2], g2[2];
  auto vec = [&](const void* p, int fp32, int c, float add, F8 (&v)[2]) { vec16<LAY>(p, fp32, c, a.cols, add, v); };
  auto col = [&](int k) { return first16<LAY>(t, T, k); };
  if (C == 1 && a.h && col(0) < a.cols) vec(a.v.g_pre, a.v.gain_fp32, col(0), a.v.offset, g2);
  int64_t gate_end = first;      // rows from here on take another gate row
  int64_t gate_at = a.v.gate ? first / a.v.span : 0;
  int st = 0, parity = 0;
  uint32_t phase = 0;
  bool dead = false;      // a wait ran out (recorded): go on without waiting, so that all threads still leave together
  for (int64_t row = first; row < end; ++row, parity ^= 1) {
    if (row == gate_end) {
      gate_end = a.v.gate ? (gate_at + 1) * a.v.span : end;
#pragma unroll
      for (int k = 0; k < C; ++k) {
        const int c = col(k);
        if (c >= a.cols) continue;
        const uint64_t b2 = pack_f2(a.v.b, a.v.b);
        w[k][0] = w[k][1] = F8{{b2, b2, b2, b2}};
        F8 v[2];
        if (post) {
          vec(a.v.g_post, a.v.gain_fp32, c, a.v.offset, v);
          w[k][0] = mul8(w[k][0], v[0]), w[k][1] = mul8(w[k][1], v[1]);
        }
        if (a.v.gate) {
          vec(static_cast<const char*>(a.v.gate) + gate_at * a.v.ld_gate * (a.v.gate_fp32 ? 4 : 2), a.v.gate_fp32, c, 0.0f, v);
          w[k][0] = mul8(w[k][0], v[0]), w[k][1] = mul8(w[k][1], v[1]);
        }
      }
      ++gate_at;
    }
    if (!dead) dead = !mbar_wait_u32(smem_u32(&full[st]), phase);
    const uint32_t at = ring0 + (uint32_t)st * stage_bytes + (LAY == kUnits ? 0u : lead_of(row_ptr<TA>(a.x, a.ldx, row)));
    const uint32_t at_r = ring0 + (uint32_t)st * stage_bytes + row_x + (LAY == kUnits ? 0u : lead_of(row_ptr<TS>(a.r, a.ldr, row)));
    float rho1 = 1.0f;
    if (post || a.x8.q) {
      float sum = 0.0f, top[1] = {0.0f};
#pragma unroll
      for (int k = 0; k < C; ++k) {
        const int c = col(k);
        if constexpr (LAY == kUnits) {
          const bool on = c < a.cols;      // (the others read the row's start and drop it)
          const LdsWide<TA> u(at + (on ? c : 0) * (uint32_t)sizeof(TA));
          const F8 lo = u.half(0), hi = u.half(1);
          const float part = dot8(lo, lo) + dot8(hi, hi);
          sum += on ? part : 0.0f;
          if (x_row) top[0] = on ? fmaxf(top[0], top_or_inf(u.top())) : top[0];
          else if (a.x8.q) ck_store16(a.x8, row, c, a.cols, lo, hi, on ? u.top() : 0.0f, 1, a.wide);
        } else {
          F8 x[2];
          lds16<TA, LAY>(at, c, a.cols, x);
          sum += dot8(x[0], x[0]) + dot8(x[1], x[1]);
          if (x_row) top[0] = fmaxf(top[0], fmaxf(top8(x[0]), top8(x[1])));
          else if (a.x8.q) ck_store16_strided(a.x8, row, c, a.cols, x, 1);
        }
      }
      if (post || x_row) sum = block_sum(sum, x_row ? top : nullptr, red[parity][0]);
      if (post) {
        rho1 = rsqrtf(fmaf(sum, a.inv_cols, a.eps));
        if (a.rho1 && t == 0) a.rho1[row] = rho1;
      }
      if (x_row) {
        if (top[0] > kLargest) {      // (the same for the block)
          top[0] = 0.0f;
#pragma unroll
          for (int k = 0; k < C; ++k) {
            const int c = col(k);
            if (c >= a.cols) continue;
            F8 x[2];
            lds16<TA, LAY>(at, c, a.cols, x);
            top[0] = fmaxf(top[0], fmaxf(top8_finite(x[0]), top8_finite(x[1])));
          }
          row_reduce_n<1, 0>(top, T, redx);
        }
        const uint32_t code = e8m0_of(top[0]);
        if (t == 0) a.x8.s8[row] = (uint8_t)code;
#pragma unroll
        for (int k = 0; k < C; ++k) {
          const int c = col(k);
          if (c >= a.cols) continue;
          F8 x[2];
          lds16<TA, LAY>(at, c, a.cols, x);
          if (LAY == kUnits) ck_store16(a.x8, row, c, a.cols, x[0], x[1], 0.0f, code, a.wide);
          else ck_store16_strided(a.x8, row, c, a.cols, x, code);
        }
      }
    }
    F8 s[C][2];
    float sum = 0.0f, top[1] = {0.0f};
#pragma unroll
    for (int k = 0; k < C; ++k) {
      const int c = col(k);
      s[k][0] = s[k][1] = zero8();
      if (c < a.cols) {
        F8 v[2];
        lds16<TA, LAY>(at, c, a.cols, v);
#pragma unroll
        for (int h = 0; h < 2; ++h) s[k][h] = mul8(scale8(v[h], rho1), w[k][h]);
        if (a.r) {
          lds16<TS, LAY>(at_r, c, a.cols, v);
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[k][h].p[i] = fmadd2(v[h].p[i], pack_f2(a.v.a, a.v.a), s[k][h].p[i]);
        }
        if (a.s) put16<TS, LAY>(row_ptr<TS>(a.s, a.lds, row), c, a.cols, s[k][0], s[k][1], a.wide);
      }
      sum += dot8(s[k][0], s[k][0]) + dot8(s[k][1], s[k][1]);
      if (s_row) top[0] = fmaxf(top[0], fmaxf(top8(s[k][0]), top8(s[k][1])));
      else if (a.s8.q && LAY == kUnits) ck_store16(a.s8, row, c, a.cols, s[k][0], s[k][1], fmaxf(top8(s[k][0]), top8(s[k][1])), 1, a.wide);
      else if (a.s8.q) ck_store16_strided(a.s8, row, c, a.cols, s[k], 1);
    }
    // (a barrier in any case: the row has been read out of its stage)
    const float rho2 = rsqrtf(fmaf(block_sum(sum, s_row ? top : nullptr, red[parity][1]), a.inv_cols, a.eps));
    if (t == 0) {
      if (row + stages < end) fill(row + stages, st);
      if (a.rho2) a.rho2[row] = rho2;
    }
    if (s_row) {
      if (top[0] > kLargest) {
        top[0] = 0.0f;
#pragma unroll
        for (int k = 0; k < C; ++k) top[0] = fmaxf(top[0], fmaxf(top8_finite(s[k][0]), top8_finite(s[k][1])));
        __syncthreads();      // redx may still be read
        row_reduce_n<1, 0>(top, T, redx);
      }
      const uint32_t code = e8m0_of(top[0]);
      if (t == 0) a.s8.s8[row] = (uint8_t)code;
#pragma unroll
      for (int k = 0; k < C; ++k) {
        if (LAY == kUnits) ck_store16(a.s8, row, col(k), a.cols, s[k][0], s[k][1], 0.0f, code, a.wide);
        else ck_store16_strided(a.s8, row, col(k), a.cols, s[k], code);
      }
    }
    if (a.h) {
#pragma unroll
      for (int k = 0; k < C; ++k) {
        const int c = col(k);
        if (c >= a.cols) continue;
        if (C > 1) vec(a.v.g_pre, a.v.gain_fp32, c, a.v.offset, g2);
        put16<TA, LAY>(row_ptr<TA>(a.h, a.ldh, row), c, a.cols, mul8(scale8(s[k][0], rho2), g2[0]), mul8(scale8(s[k][1], rho2), g2[1]), a.wide);
      }
    }
    if (++st == stages) {
      st = 0;
      phase ^= 1u;
    }
  }
  if (dead && t == 0) {      // copies still under way land before their memory is given up (waited for once more, bounded)
    const int64_t n = end - first;
    for (int i = 0; i < stages && i < n; ++i) mbar_wait(&full[i], (uint32_t)((n - 1 - i) / stages) & 1u);
  }
  if (dead) __syncthreads();
}

// Backward.  With w = b gate g1 (the factor of x's norm in s) a row's sums
//   A = sum dh g2 s,  B = sum w x (dsum + rho2 dh g2),  D = sum w x s
// come from one pass over the row, and then
//   c = -rho2^3 A / cols,  d = dsum + rho2 dh g2 + c s
//   c1 = -rho1^3 (B + c D) / cols,  dx = rho1 w d + c1 x
// since sum w x d = B + c D: one reduction a row, not two.
//
// Gradients of the gains and the gate.  With t = b d x rho1 and T_k its sum
// over the rows of gate row k,  dgate_k = g1 T_k  and  dg1 = sum_k gate_k T_k,
// so a thread holds one sum for both (and one for dg2), over rows of one gate
// row after the other.
//
// Work items: gate row k's rows in P parts; a worker (the threads of a row)
// takes the items w, w + workers, ...  Where the gate has fewer rows than
// there are workers, every worker has one item at most: its T is a partial row
// (tpart), joined by k_sandwich_join.  Else P = 1 and a worker has several:
// each T is complete, goes into dgate at once, and times its gate row into the
// worker's partial dg1 (kept in the workspace, this worker's own row).
struct BwdArgs {
  const void* dh;         // may be null
  const void* dsum;       // may be null
  const void* x;          // may be null, as may x8.q: at most one of the two
  const void* s;
  void* dr;               // may be null
  void* dx;               // may be null
  void* dgate;            // several items a worker: written here (else by the join)
  Ck x8, s8;
  const float* rho1;
  const float* rho2;
  float* tpart;           // [workers][cols] or null: T of the worker's item, or its share of dg1
  float* ppart;           // [workers][cols] or null: dg2
  int64_t lddh, lddsum, ldx, lds, lddr, lddx, lddgate;
  int64_t rows, span, items;      // span: rows of an undivided item (gate_span, or all rows)
  int64_t workers;
  int32_t parts;          // P
  int32_t many;           // several items a worker
  int32_t dgate_fp32;
  int32_t cols, tpr, rpb;
  int32_t wide;           // staged form: rows on wide units, not on units of eight only
  float inv_cols;
  Vectors v;
};

template <int LAY>
__device__ __forceinline__ void store_any(void* row, int fp32, int c0, int dj, int cols, const F8& v) {
  if (fp32) store8<LAY>(static_cast<float*>(row), c0, dj, cols, v);
  else store8<LAY>(static_cast<__nv_bfloat16*>(row), c0, dj, cols, v);
}

constexpr int kBwdThreads = 1024, kBwdFew = 256, kBwdK = 2;

// T: most threads of a block.  Up to 4096 columns kBwdFew, with 128 registers a thread; 1024 have 64 and spill.
template <typename TA, typename TS, int LAY, int T>
__global__ void __launch_bounds__(T, T == kBwdFew ? 2 : 1) k_sandwich_bwd(const BwdArgs a) {
  __shared__ float red[2][3 * (T / 32)];
  const int tpr = a.tpr, lane_row = (int)threadIdx.x / tpr, t = (int)threadIdx.x - lane_row * tpr;
  const int64_t worker = (int64_t)blockIdx.x * a.rpb + lane_row;
  const Lane l = lane_of<LAY>(t, tpr);
  const bool post = a.v.g_post != nullptr, have_x = a.x || a.x8.q, pre = a.dh != nullptr;
  F8 accT[kBwdK] = {}, accP[kBwdK] = {};
  int parity = 0;
  const int64_t rounds = ceil_div<int64_t>(a.items, a.workers), most = ceil_div<int64_t>(a.span, a.parts);
  for (int64_t round = 0; round < rounds; ++round) {
    const int64_t item = worker + round * a.workers;
    const bool has = worker < a.workers && item < a.items;
    const int64_t k = has ? item / a.parts : 0;
    const int64_t len = min(a.span, a.rows - k * a.span), p = has ? item - k * a.parts : 0;
    const int64_t r0 = k * a.span + len * p / a.parts, r1 = has ? k * a.span + len * (p + 1) / a.parts : r0;
    const void* gate = a.v.gate ? gate_row(a.v, k * a.span) : nullptr;
    for (int64_t i = 0; i < most; ++i, parity ^= 1) {
      const int64_t row = r0 + i;
      const int cols = row < r1 ? a.cols : 0;
      F8 dn[kBwdK], s[kBwdK], x[kBwdK], e[kBwdK];      // dh, s, x, dsum
      const float rho2 = cols && pre ? a.rho2[row] : 0.0f, rho1 = cols && post ? a.rho1[row] : 1.0f;
#pragma unroll
      for (int q = 0; q < kBwdK; ++q) {
        dn[q] = s[q] = x[q] = e[q] = zero8();
        const int c0 = l.c0(q);
        if (c0 >= cols) continue;
        if (pre) {
          dn[q] = load8<LAY>(row_ptr<TA>(a.dh, a.lddh, row), c0, l.dj, cols);
          s[q] = a.s8.q ? load8<LAY>(a.s8, row, c0, l.dj, cols) : load8<LAY>(row_ptr<TS>(a.s, a.lds, row), c0, l.dj, cols);
        }
        if (a.dsum) e[q] = load8<LAY>(row_ptr<TS>(a.dsum, a.lddsum, row), c0, l.dj, cols);
        if (a.x8.q) x[q] = load8<LAY>(a.x8, row, c0, l.dj, cols);
        else if (a.x) x[q] = load8<LAY>(row_ptr<TA>(a.x, a.ldx, row), c0, l.dj, cols);
      }
      float m[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int q = 0; q < kBwdK; ++q) {
        const int c0 = l.c0(q);
        if (c0 >= cols) continue;
        if (pre) {
          const F8 g2 = load_vec<LAY>(a.v.g_pre, a.v.gain_fp32, c0, l.dj, cols, a.v.offset);
#pragma unroll
          for (int i4 = 0; i4 < 4; ++i4) {
            accP[q].p[i4] = fmadd2(fmul2(dn[q].p[i4], s[q].p[i4]), pack_f2(rho2, rho2), accP[q].p[i4]);
            dn[q].p[i4] = fmul2(dn[q].p[i4], g2.p[i4]);
          }
          m[0] += dot8(dn[q], s[q]);
#pragma unroll
          for (int i4 = 0; i4 < 4; ++i4) e[q].p[i4] = fmadd2(dn[q].p[i4], pack_f2(rho2, rho2), e[q].p[i4]);
        }
        if (post) {
          F8 w = load_vec<LAY>(a.v.g_post, a.v.gain_fp32, c0, l.dj, cols, a.v.offset);
          if (gate) w = mul8(w, load_vec<LAY>(gate, a.v.gate_fp32, c0, l.dj, cols, 0.0f));
          w = mul8(w, x[q]);
          m[1] += dot8(w, e[q]);
          m[2] += dot8(w, s[q]);
        }
      }
      if (pre || post) row_reduce_n<3, 3>(m, tpr, red[parity]);
      const float c = pre ? -rho2 * (rho2 * (rho2 * m[0] * a.inv_cols)) : 0.0f;
      const float c1 = post ? -rho1 * (rho1 * (rho1 * a.v.b * fmaf(c, m[2], m[1]) * a.inv_cols)) : 0.0f;
      const float tf = a.v.b * rho1;
#pragma unroll
      for (int q = 0; q < kBwdK; ++q) {
        const int c0 = l.c0(q);
        if (c0 >= cols) continue;
        F8 d = e[q];
        if (pre) {
#pragma unroll
          for (int i4 = 0; i4 < 4; ++i4) d.p[i4] = fmadd2(s[q].p[i4], pack_f2(c, c), d.p[i4]);
        }
        if (a.dr) store8<LAY>(row_ptr<TS>(a.dr, a.lddr, row), c0, l.dj, cols, scale8(d, a.v.a));
        d = scale8(d, tf);      // b d rho1
        if (have_x) {
#pragma unroll
          for (int i4 = 0; i4 < 4; ++i4) accT[q].p[i4] = fmadd2(d.p[i4], x[q].p[i4], accT[q].p[i4]);
        }
        if (a.dx) {
          if (gate) d = mul8(d, load_vec<LAY>(gate, a.v.gate_fp32, c0, l.dj, cols, 0.0f));
          if (post) {
            d = mul8(d, load_vec<LAY>(a.v.g_post, a.v.gain_fp32, c0, l.dj, cols, a.v.offset));
#pragma unroll
            for (int i4 = 0; i4 < 4; ++i4) d.p[i4] = fmadd2(x[q].p[i4], pack_f2(c1, c1), d.p[i4]);
          }
          store8<LAY>(row_ptr<TA>(a.dx, a.lddx, row), c0, l.dj, cols, d);
        }
      }
    }
    if (a.many && has) {
#pragma unroll
      for (int q = 0; q < kBwdK; ++q) {
        const int c0 = l.c0(q);
        if (c0 >= a.cols) continue;
        if (a.dgate) {
          F8 v = accT[q];
          if (post) v = mul8(v, load_vec<LAY>(a.v.g_post, a.v.gain_fp32, c0, l.dj, a.cols, a.v.offset));
          store_any<LAY>(static_cast<char*>(a.dgate) + k * a.lddgate * (a.dgate_fp32 ? 4 : 2), a.dgate_fp32, c0, l.dj, a.cols, v);
        }
        if (a.tpart) {
          // this worker's own row, written and read by the same threads
          float* part = a.tpart + worker * a.cols;
          F8 v = round ? load8<kStrided>(part, c0, l.dj, a.cols) : zero8();
          const F8 g = load_vec<LAY>(gate, a.v.gate_fp32, c0, l.dj, a.cols, 0.0f);
#pragma unroll
          for (int i4 = 0; i4 < 4; ++i4) v.p[i4] = fmadd2(accT[q].p[i4], g.p[i4], v.p[i4]);
          store8<kStrided>(part, c0, l.dj, a.cols, v);
        }
        accT[q] = zero8();
      }
    }
  }
  griddep_launch_dependents();
  if (worker >= a.workers) return;
#pragma unroll
  for (int q = 0; q < kBwdK; ++q) {
    const int c0 = l.c0(q);
    if (c0 >= a.cols) continue;
    if (a.tpart && !a.many) store8<kStrided>(a.tpart + worker * a.cols, c0, l.dj, a.cols, accT[q]);
    if (a.ppart) store8<kStrided>(a.ppart + worker * a.cols, c0, l.dj, a.cols, accP[q]);
  }
}

// The same backward pass with rows brought by bulk copies, as in the forward
// form: a block is one worker, a thread holds a wide unit's sums, w and g2 in
// registers.  A row is read from shared memory twice, for its sums and, past
// the one barrier, for its outputs (dsum + rho2 dh g2 stays in registers
// between); past that barrier every thread is also done with the row before,
// whose stage is filled again.  For calls with dh, dsum or none, and x and s both in
// full or both as checkpoints (KEPT).
// 16 e4m3 values from shared memory, times their scale; wide: on 16 bytes (else on eight).
__device__ __forceinline__ void lds16_e4m3(uint32_t p, float scale, bool wide, F8 (&v)[2]) {
  uint32_t w[4];
  if (wide) {
    const int4 q = lds_i4(p);
    w[0] = (uint32_t)q.x, w[1] = (uint32_t)q.y, w[2] = (uint32_t)q.z, w[3] = (uint32_t)q.w;
  } else {
    const uint2 a = lds_u2(p), b = lds_u2(p + 8);
    w[0] = a.x, w[1] = a.y, w[2] = b.x, w[3] = b.y;
  }
  const uint64_t s2 = pack_f2(scale, scale);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 x = e4m3x2_value(w[i >> 1] >> (16 * (i & 1)) & 0xffffu);
    v[i >> 2].p[i & 3] = fmul2(pack_f2(x.x, x.y), s2);
  }
}
// In the second lay, the row's scales from shared memory too.
__device__ __forceinline__ void lds16_e4m3_strided(uint32_t p, int c0, int cols, const float* scales, int group_log2, F8 (&v)[2]) {
  const int shift = group_log2 ? group_log2 : 31;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int c = c0 + 64 * i, d = c + 32;
    uint16_t q0 = 0, q1 = 0;
    if (c < cols) asm volatile("{.reg .b32 t; ld.shared.u8 t, [%1]; cvt.u16.u32 %0, t;}" : "=h"(q0) : "r"(p + c));
    if (d < cols) asm volatile("{.reg .b32 t; ld.shared.u8 t, [%1]; cvt.u16.u32 %0, t;}" : "=h"(q1) : "r"(p + d));
    const float2 x = e4m3x2_value((uint32_t)q0 | (uint32_t)q1 << 8);
    v[i >> 2].p[i & 3] = fmul2(pack_f2(x.x, x.y), pack_f2(c < cols ? scales[c >> shift] : 0.0f, d < cols ? scales[d >> shift] : 0.0f));
  }
}

constexpr int kBwdRingThreads = 512, kBwdRingRegs = 128;

template <typename TA, typename TS, int LAY, bool KEPT, bool POST>
__global__ void __launch_bounds__(kBwdRingThreads) k_sandwich_bwd_ring(const BwdArgs a, const int stages) {
  constexpr int kWarps = kBwdRingThreads / 32, N = POST ? 3 : 1;
  __shared__ __align__(16) float red[2][N][kWarps];
  __shared__ __align__(8) uint64_t full[kMaxStages];
  extern __shared__ __align__(128) unsigned char ring[];
  // (KEPT, strided: the scales of three rows in turn, of x and of s)
  __shared__ float scl[KEPT && LAY == kStrided ? 3 : 1][2][KEPT && LAY == kStrided ? 16 * kBwdRingThreads / 32 : 1];
  const int t = threadIdx.x, c = first16<LAY>(t, blockDim.x, 0);
  const bool on = c < a.cols;
  for (int i = t; i < 2 * N * kWarps; i += blockDim.x) (&red[0][0][0])[i] = 0.0f;
  const uint32_t slot_a = slot_bytes(a.cols, sizeof(TA)), slot_s = slot_bytes(a.cols, sizeof(TS)), slot_8 = slot_bytes(a.cols, 1);
  const uint32_t off_e = slot_a, off_x = off_e + (a.dsum ? slot_s : 0u), off_s = off_x + (KEPT ? slot_8 : slot_a);
  const uint32_t stage_bytes = off_s + (KEPT ? slot_8 : slot_s);
  const uint32_t ring0 = smem_u32(ring);
  // this worker's rows (n of them, below 2^29): the part of a gate row, or every workers-th gate row
  const int worker = blockIdx.x, workers = gridDim.x, span = (int)a.span, rows = (int)a.rows;
  int row, n, left;      // the next row, the number of rows, those left in its item
  if (a.many) {
    const int items = (int)a.items, mine = (items - worker + workers - 1) / workers;
    n = mine * span - (worker + (mine - 1) * workers == items - 1 ? items * span - rows : 0);
    row = worker * span;
    left = min(span, rows - row);
  } else {
    const int k = worker / a.parts, p = worker - k * a.parts, len = min(span, rows - k * span);
    row = k * span + (int)((int64_t)len * p / a.parts);
    left = n = k * span + (int)((int64_t)len * (p + 1) / a.parts) - row;
  }
  const int row0 = row;
  auto row_at = [&](int j) {
    if (!a.many) return row0 + j;
    const int q = j / span;
    return (worker + q * workers) * span + j - q * span;
  };
  auto fill = [&](int j, int st) {      // by one thread
    const int64_t r = row_at(j);
    unsigned char* at = ring + (size_t)st * stage_bytes;
    const bool last = r == a.rows - 1;
    const uint32_t size_a = (uint32_t)a.cols * (uint32_t)sizeof(TA), size_s = (uint32_t)a.cols * (uint32_t)sizeof(TS);
    const Bring b[4] = {{row_ptr<TA>(a.dh, a.lddh, r), size_a, last},
                        {row_ptr<TS>(a.dsum, a.lddsum, r), a.dsum ? size_s : 0u, last},
                        {KEPT ? (const void*)(a.x8.q + r * a.x8.ld) : row_ptr<TA>(a.x, a.ldx, r), KEPT ? (uint32_t)a.cols : size_a, last},
                        {KEPT ? (const void*)(a.s8.q + r * a.s8.ld) : row_ptr<TS>(a.s, a.lds, r), KEPT ? (uint32_t)a.cols : size_s, last}};
    unsigned char* const to[4] = {at, at + off_e, at + off_x, at + off_s};
    bring_rows(b, to, &full[st]);
  };
  if (t == 0) {
    for (int i = 0; i < stages; ++i) mbar_init(&full[i], 1);
    fence_mbar_init_cluster();
    for (int i = 0; i < stages && i < n; ++i) fill(i, i);
  }
  __syncthreads();
  F8 accT[2] = {}, accP[2] = {}, w[2], g2[2];
  auto vec = [&](const void* p, int fp32, float add, F8 (&v)[2]) { vec16<LAY>(p, fp32, c, a.cols, add, v); };
  constexpr int kNext = LAY == kUnits ? 8 : 256, kApart = LAY == kUnits ? 1 : 32;      // of a thread's columns
  auto load_w = [&](const void* gate) {      // gate g1
    const uint64_t one = pack_f2(1.0f, 1.0f);
    w[0] = w[1] = F8{{one, one, one, one}};
    if (!on) return;
    F8 v[2];
    if (POST) vec(a.v.g_post, a.v.gain_fp32, a.v.offset, w);
    if (gate) {
      vec(gate, a.v.gate_fp32, 0.0f, v);
      w[0] = mul8(w[0], v[0]), w[1] = mul8(w[1], v[1]);
    }
  };
  if (on) vec(a.v.g_pre, a.v.gain_fp32, a.v.offset, g2);
  // a gate row's T is complete (several items a worker)
  auto flush = [&](int gate_row, bool first) {
    const void* gate = gate_row_of(a.v, gate_row);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int ch = c + kNext * h;
      if (on && a.dgate) {
        F8 v = accT[h];
        if (POST) v = mul8(v, load_vec<LAY>(a.v.g_post, a.v.gain_fp32, ch, kApart, a.cols, a.v.offset));
        store_any<LAY>(static_cast<char*>(a.dgate) + (int64_t)gate_row * a.lddgate * (a.dgate_fp32 ? 4 : 2), a.dgate_fp32, ch, kApart, a.cols, v);
      }
      if (on && a.tpart) {      // this worker's own row, written and read by the same threads (on 16 bytes at least: no wide access)
        float* part = a.tpart + (int64_t)worker * a.cols;
        F8 v = first ? zero8() : load8<kStrided>(part, ch, kApart, a.cols);
        const F8 g = load_vec<LAY>(gate, a.v.gate_fp32, ch, kApart, a.cols, 0.0f);
#pragma unroll
        for (int i = 0; i < 4; ++i) v.p[i] = fmadd2(accT[h].p[i], g.p[i], v.p[i]);
        store8<kStrided>(part, ch, kApart, a.cols, v);
      }
      accT[h] = zero8();
    }
  };
  // a row's rhos and scales come one row ahead
  float rho1_next = 1.0f, rho2_next = 0.0f;
  uint32_t sx_next = 0, ss_next = 0;
  // (strided: a thread brings one group's, for all)
  auto scale_raw = [&](const Ck& ck, int64_t r) {
    const int64_t i = r * ck.n_groups + (LAY == kStrided ? min(t, ck.n_groups - 1) : ck.group_log2 && on ? c >> ck.group_log2 : 0);
    return ck.s8 ? (uint32_t)ck.s8[i] : __float_as_uint(ck.s32[i]);
  };
  auto scale_value = [](const Ck& ck, uint32_t raw) { return ck.s8 ? e8m0_value(raw) : __uint_as_float(raw); };
  auto prefetch = [&](int64_t r) {
    if (POST) rho1_next = a.rho1[r];
    rho2_next = a.rho2[r];
    if (KEPT && LAY == kUnits) sx_next = scale_raw(a.x8, r), ss_next = scale_raw(a.s8, r);
  };
  if (n > 0) prefetch(row);
  auto put_scales = [&](int j) {      // row j's, fetched before
    if constexpr (KEPT && LAY == kStrided) {
      if (t < a.x8.n_groups) scl[j % 3][0][t] = scale_value(a.x8, sx_next);
      if (t < a.s8.n_groups) scl[j % 3][1][t] = scale_value(a.s8, ss_next);
    }
  };
  auto fetch_scales = [&](int j) {
    if (KEPT && LAY == kStrided && j < n) sx_next = scale_raw(a.x8, row_at(j)), ss_next = scale_raw(a.s8, row_at(j));
  };
  if constexpr (KEPT && LAY == kStrided) {
    fetch_scales(0);
    put_scales(0);
    fetch_scales(1);
    __syncthreads();
  }
  int gate_row = a.many ? worker : worker / a.parts;
  load_w(a.v.gate ? gate_row_of(a.v, gate_row) : nullptr);
  int st = 0;
  uint32_t phase = 0;
  bool dead = false;      // a wait ran out (recorded): go on without waiting, so that all threads still leave together
  for (int j = 0; j < n; ++j) {
    const float rho1 = rho1_next, rho2 = rho2_next;
    const float sx = scale_value(a.x8, sx_next), ss = scale_value(a.s8, ss_next);
    const int64_t r = row;
    const bool last = --left == 0;      // of its item
    row = last ? (gate_row + workers) * span : row + 1;
    if (j + 1 < n) prefetch(row);
    if (!dead) dead = !mbar_wait_u32(smem_u32(&full[st]), phase);
    const uint32_t base = ring0 + (uint32_t)st * stage_bytes;
    const uint32_t at_dh = base + (LAY == kUnits ? 0u : lead_of(row_ptr<TA>(a.dh, a.lddh, r)));
    const uint32_t at_e = base + off_e + (LAY == kUnits ? 0u : lead_of(row_ptr<TS>(a.dsum, a.lddsum, r)));
    const uint32_t at_x = base + off_x + (KEPT ? lead_of(a.x8.q + r * a.x8.ld) : LAY == kUnits ? 0u : lead_of(row_ptr<TA>(a.x, a.ldx, r)));
    const uint32_t at_s = base + off_s + (KEPT ? lead_of(a.s8.q + r * a.s8.ld) : LAY == kUnits ? 0u : lead_of(row_ptr<TS>(a.s, a.lds, r)));
    auto load_s = [&](F8 (&s)[2]) {
      if constexpr (!KEPT) lds16<TS, LAY>(at_s, c, a.cols, s);
      else if constexpr (LAY == kUnits) lds16_e4m3(at_s + c, ss, a.wide, s);
      else lds16_e4m3_strided(at_s, c, a.cols, scl[j % 3][1], a.s8.group_log2, s);
    };
    auto load_x = [&](F8 (&x)[2]) {
      if constexpr (!KEPT) lds16<TA, LAY>(at_x, c, a.cols, x);
      else if constexpr (LAY == kUnits) lds16_e4m3(at_x + c, sx, a.wide, x);
      else lds16_e4m3_strided(at_x, c, a.cols, scl[j % 3][0], a.x8.group_log2, x);
    };
    const uint64_t rho2_2 = pack_f2(rho2, rho2);
    F8 e[2] = {};
    float m[N] = {};
    if (on) {
      F8 dn[2], s[2], x[2];
      lds16<TA, LAY>(at_dh, c, a.cols, dn);
      if (a.dsum) lds16<TS, LAY>(at_e, c, a.cols, e);
      load_s(s);
      if (POST) load_x(x);
      uint64_t q[N] = {};
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint64_t ds = fmul2(dn[h].p[i], s[h].p[i]);
          accP[h].p[i] = fmadd2(ds, rho2_2, accP[h].p[i]);
          q[0] = fmadd2(ds, g2[h].p[i], q[0]);
          e[h].p[i] = fmadd2(fmul2(dn[h].p[i], g2[h].p[i]), rho2_2, e[h].p[i]);
          if constexpr (POST) {
            const uint64_t wx = fmul2(w[h].p[i], x[h].p[i]);
            q[1] = fmadd2(wx, e[h].p[i], q[1]);
            q[2] = fmadd2(wx, s[h].p[i], q[2]);
          }
        }
#pragma unroll
      for (int i = 0; i < N; ++i) m[i] = unpack_f2(q[i]).x + unpack_f2(q[i]).y;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
      for (int i = 0; i < N; ++i) m[i] += __shfl_xor_sync(0xffffffffu, m[i], o);
    if ((t & 31) == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) red[j & 1][i][t >> 5] = m[i];
    }
    put_scales(j + 1);      // (of the three places the one that the last row before this barrier no longer reads)
    __syncthreads();
    fetch_scales(j + 2);
    if (t == 0 && j > 0 && j - 1 + stages < n) fill(j - 1 + stages, st == 0 ? stages - 1 : st - 1);      // the stage of the row before
#pragma unroll
    for (int i = 0; i < N; ++i) {
      uint64_t v = 0;
#pragma unroll
      for (int q = 0; q < kWarps / 4; ++q) {
        if (q == 2 && blockDim.x <= 256) break;
        const float4 f = *reinterpret_cast<const float4*>(&red[j & 1][i][4 * q]);
        v = fadd2(v, fadd2(pack_f2(f.x, f.y), pack_f2(f.z, f.w)));
      }
      m[i] = unpack_f2(v).x + unpack_f2(v).y;
    }
    const float c0 = -rho2 * (rho2 * (rho2 * m[0] * a.inv_cols));
    const float tf = a.v.b * rho1;
    float c1 = 0.0f;
    if constexpr (POST) c1 = -rho1 * (rho1 * (tf * fmaf(c0, m[2], m[1]) * a.inv_cols));
    if (on) {
      F8 s[2], x[2];
      load_s(s);
      load_x(x);
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i) e[h].p[i] = fmadd2(s[h].p[i], pack_f2(c0, c0), e[h].p[i]);
      if (a.dr) put16<TS, LAY>(row_ptr<TS>(a.dr, a.lddr, r), c, a.cols, scale8(e[0], a.v.a), scale8(e[1], a.v.a), a.wide);
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint64_t bd = fmul2(e[h].p[i], pack_f2(tf, tf));
          accT[h].p[i] = fmadd2(bd, x[h].p[i], accT[h].p[i]);
          e[h].p[i] = POST ? fmadd2(bd, w[h].p[i], fmul2(x[h].p[i], pack_f2(c1, c1))) : fmul2(bd, w[h].p[i]);
        }
      if (a.dx) put16<TA, LAY>(row_ptr<TA>(a.dx, a.lddx, r), c, a.cols, e[0], e[1], a.wide);
    }
    if (last && a.many) {
      flush(gate_row, gate_row == worker);
      gate_row += workers;
      if (j + 1 < n) {
        left = min(span, rows - row);
        load_w(gate_row_of(a.v, gate_row));
      }
    }
    if (++st == stages) {
      st = 0;
      phase ^= 1u;
    }
  }
  if (dead && t == 0) {      // copies still under way land before their memory is given up (waited for once more, bounded)
    for (int j = max(0, n - stages); j < n; ++j) mbar_wait(&full[j % stages], (uint32_t)(j / stages) & 1u);
  }
  if (dead) __syncthreads();
  griddep_launch_dependents();
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (on && a.tpart && !a.many) store8<kStrided>(a.tpart + (int64_t)worker * a.cols, c + kNext * h, kApart, a.cols, accT[h]);
    if (on && a.ppart) store8<kStrided>(a.ppart + (int64_t)worker * a.cols, c + kNext * h, kApart, a.cols, accP[h]);
  }
}

// Joins the partial rows, 32 columns and 32 threads a column a block, in a
// fixed order.  blockIdx.y 0: dg2 = sum of ppart.  1: dg1 and dgate from tpart:
// with one item a worker (gate rows x parts partial T), dgate_k = g1 T_k and
// dg1 = sum gate_k T_k; else tpart holds shares of dg1.
struct JoinArgs {
  const float* tpart;
  const float* ppart;
  void* dg1;              // may be null
  void* dg2;              // may be null
  void* dgate;            // may be null: none, or already written
  int64_t workers, lddgate, gate_rows;
  int32_t parts, many, cols, dgain_fp32, dgate_fp32;
  Vectors v;
};

__device__ __forceinline__ float vec_at(const void* v, int fp32, int64_t i) {
  return fp32 ? static_cast<const float*>(v)[i] : __uint_as_float((uint32_t)static_cast<const uint16_t*>(v)[i] << 16);
}
__device__ __forceinline__ void put_at(void* v, int fp32, int64_t i, float x) {
  if (fp32) static_cast<float*>(v)[i] = x;
  else static_cast<__nv_bfloat16*>(v)[i] = __float2bfloat16_rn(x);
}

// The sum over the block's 32 rows of threads, for each column; valid in lanes 0 of warp = column.
__device__ __forceinline__ float join32(float v, float (&red)[32][33]) {
  __syncthreads();
  red[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  v = red[threadIdx.x][threadIdx.y];       // column threadIdx.y, partial sum threadIdx.x
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__global__ void __launch_bounds__(1024) k_sandwich_join(const JoinArgs a) {
  __shared__ float red[32][33];
  const int c = blockIdx.x * 32 + threadIdx.x, out = blockIdx.x * 32 + threadIdx.y;
  const bool on = c < a.cols, writes = threadIdx.x == 0 && out < a.cols;
  griddep_wait();
  const bool shares = a.many || !a.v.gate;
  if (blockIdx.y == 0 || shares) {
    const float* part = blockIdx.y == 0 ? a.ppart : a.tpart;
    void* dst = blockIdx.y == 0 ? a.dg2 : a.dg1;
    if (!dst) return;
    float v = 0.0f;
    if (on) {
#pragma unroll 8
      for (int64_t p = threadIdx.y; p < a.workers; p += 32) v += part[p * a.cols + c];
    }
    v = join32(v, red);
    if (writes) put_at(dst, a.dgain_fp32, out, v);
    return;
  }
  if (!a.tpart) return;
  const float g1c = on && a.v.g_post ? vec_at(a.v.g_post, a.v.gain_fp32, c) + a.v.offset : 1.0f;
  float dg1 = 0.0f;
  if (a.gate_rows >= 32) {      // a gate row's parts by one thread
    for (int64_t k = threadIdx.y; k < a.gate_rows; k += 32) {
      float v = 0.0f;
      if (on) {
        for (int p = 0; p < a.parts; ++p) v += a.tpart[(k * a.parts + p) * a.cols + c];
        if (a.dgate) put_at(a.dgate, a.dgate_fp32, k * a.lddgate + c, g1c * v);
        dg1 = fmaf(vec_at(a.v.gate, a.v.gate_fp32, k * a.v.ld_gate + c), v, dg1);
      }
    }
    dg1 = join32(dg1, red);
  } else {
    for (int64_t k = 0; k < a.gate_rows; ++k) {
      float v = 0.0f;
      if (on) {
#pragma unroll 4
        for (int p = threadIdx.y; p < a.parts; p += 32) v += a.tpart[(k * a.parts + p) * a.cols + c];
      }
      v = join32(v, red);
      if (writes) {
        const float g1 = a.v.g_post ? vec_at(a.v.g_post, a.v.gain_fp32, out) + a.v.offset : 1.0f;
        if (a.dgate) put_at(a.dgate, a.dgate_fp32, k * a.lddgate + out, g1 * v);
        dg1 = fmaf(vec_at(a.v.gate, a.v.gate_fp32, k * a.v.ld_gate + out), v, dg1);
      }
    }
  }
  if (a.dg1 && writes) put_at(a.dg1, a.dgain_fp32, out, dg1);
}

constexpr unsigned kTypes = 1u << SF_BF16 | 1u << SF_FP32;

// Rows of the workspace's partial sums: more of them where rows are short.
int64_t max_workers(int64_t cols) { return std::min<int64_t>(8192, std::max<int64_t>(1024, (1 << 21) / cols)); }

template <template <typename, typename, int> class K, typename... A>
const void* pick_kernel(int32_t ta, int32_t ts, Lay lay, A... args) {
  using B = __nv_bfloat16;
  if (ta == SF_BF16) {
    if (ts == SF_BF16) return lay == kUnits ? K<B, B, kUnits>::ptr(args...) : K<B, B, kStrided>::ptr(args...);
    return lay == kUnits ? K<B, float, kUnits>::ptr(args...) : K<B, float, kStrided>::ptr(args...);
  }
  if (ts == SF_BF16) return lay == kUnits ? K<float, B, kUnits>::ptr(args...) : K<float, B, kStrided>::ptr(args...);
  return lay == kUnits ? K<float, float, kUnits>::ptr(args...) : K<float, float, kStrided>::ptr(args...);
}
template <typename TA, typename TS, int LAY>
struct Fwd {
  static const void* ptr() { return (const void*)&k_sandwich_fwd<TA, TS, LAY>; }
};
template <typename TA, typename TS, int LAY>
struct Bwd {
  static const void* ptr() { return (const void*)&k_sandwich_bwd<TA, TS, LAY, kBwdThreads>; }
};
template <typename TA, typename TS, int LAY>
struct BwdFew {
  static const void* ptr() { return (const void*)&k_sandwich_bwd<TA, TS, LAY, kBwdFew>; }
};

// The staged form: wide units a thread, registers.
constexpr int kFwdRegs1 = 80, kFwdRegs2 = 128;
template <typename TA, typename TS>
const void* fwd_ring(int c, Lay lay) {
  if (lay == kUnits) return c == 1 ? (const void*)&k_sandwich_fwd_ring<TA, TS, kUnits, 1, kFwdRegs1> : (const void*)&k_sandwich_fwd_ring<TA, TS, kUnits, 2, kFwdRegs2>;
  return c == 1 ? (const void*)&k_sandwich_fwd_ring<TA, TS, kStrided, 1, kFwdRegs1> : (const void*)&k_sandwich_fwd_ring<TA, TS, kStrided, 2, kFwdRegs2>;
}
template <typename TA, typename TS, int LAY>
const void* bwd_ring(bool kept, bool post) {
  return kept ? (post ? (const void*)&k_sandwich_bwd_ring<TA, TS, LAY, true, true> : (const void*)&k_sandwich_bwd_ring<TA, TS, LAY, true, false>)
              : (post ? (const void*)&k_sandwich_bwd_ring<TA, TS, LAY, false, true> : (const void*)&k_sandwich_bwd_ring<TA, TS, LAY, false, false>);
}
template <typename TA, typename TS, int LAY>
struct BwdRing {
  static const void* ptr(bool kept, bool post) { return bwd_ring<TA, TS, LAY>(kept, post); }
};
constexpr size_t kSmemPerSm = 224 << 10, kSmemBlock = 2 << 10;      // a block's static and reserved shared memory
constexpr size_t kSmemScales = 6 << 10;        // of three rows
constexpr int kRingMinCols = 1024, kBwdMinCols = 256;

struct RingShape {
  int c = 0, threads = 0, per_sm = 0, stages = 0;
};
// One or two wide units a thread, whichever lets more threads, or as many in
// more blocks, reside on an SM (bf16, 4 x 4096-token batches' worth of data: 8192
// columns in two blocks of 256 threads 127 us, in one of 512 169; 12288 with an
// fp32 stream in one of 768 threads 201 us, in one of 384 244).  At least three
// stages each, two in long rows.  False where rows are too long, or too few or short
// for it to pay (65536 x 512: 63 us, 51 with loads into registers; 32768 x 1024 50 and 54).
bool ring_shape(int64_t rows, int64_t cols, size_t stage, int regs1, int regs2, RingShape* best) {
  if (cols < kRingMinCols || rows < 2 * sm_count()) return false;
  for (int c = 1; c <= 2; ++c) {
    RingShape s;
    s.c = c;
    s.threads = ceil_div(ceil_div(ceil_div((int)cols, 16), c), 32) * 32;
    const int regs = c == 1 ? regs1 : regs2;
    int n = std::min(65536 / (regs * s.threads), 2048 / s.threads);
    while (n > 1 && kSmemPerSm / n < kSmemBlock + 3 * stage) --n;
    if (s.threads > kRingThreads || n < 1) continue;
    s.per_sm = n;
    s.stages = (int)std::min<size_t>(kMaxStages, (kSmemPerSm / n - kSmemBlock) / stage);
    if (s.stages < 2) continue;
    const int now = s.threads * n, was = best->threads * best->per_sm;
    if (now > was || (now == was && n > best->per_sm)) *best = s;
  }
  return best->c > 0;
}

sf_status check_vector(const void* v, int32_t dtype, const char* name) {
  if (!v) return SF_OK;
  if (dtype != SF_BF16 && dtype != SF_FP32) return fail(SF_ERR_UNSUPPORTED, "%s: type %d is not taken here", name, (int)dtype);
  return check_aligned(v, dtype_bytes(dtype), name);
}

// The configuration and the vectors that both passes share.
sf_status check_common(const sf_sandwich* p, int64_t rows, int64_t cols, const void* gain_post, const void* gain_pre,
                       int32_t gain_dtype, const sf_matrix* gate, Vectors* v) {
  if (!p) return fail(SF_ERR_INVALID, "the configuration is NULL");
  if (cols < 1) return fail(SF_ERR_INVALID, "a row needs at least one column");
  if (cols > kMaxCols) return fail(SF_ERR_UNSUPPORTED, "rows of up to %lld columns are supported (got %lld)", (long long)kMaxCols, (long long)cols);
  if (!(p->eps >= 0.0) || p->eps > 1e30) return fail(SF_ERR_INVALID, "eps must be finite and >= 0");
  const double f[3] = {p->residual_scale, p->block_scale, p->gain_offset};
  for (double x : f)
    if (!(x >= -1e30 && x <= 1e30)) return fail(SF_ERR_INVALID, "residual_scale, block_scale and gain_offset must be finite");
  if (p->gate_span < 0) return fail(SF_ERR_INVALID, "gate_span must be >= 0");
  SF_TRY(check_vector(gain_post, gain_dtype, "gain_post"));
  SF_TRY(check_vector(gain_pre, gain_dtype, "gain_pre"));
  *v = Vectors{};
  v->span = p->gate_span && p->gate_span < rows ? p->gate_span : std::max<int64_t>(1, rows);
  if (gate) {
    SF_TRY(check_matrix(gate, "gate", rows ? ceil_div<int64_t>(rows, v->span) : p->gate_span ? 0 : 1, cols, kTypes));
    v->gate = gate->data;
    v->ld_gate = gate->ld;
    v->gate_fp32 = gate->dtype == SF_FP32;
  }
  v->g_post = gain_post;
  v->g_pre = gain_pre;
  v->gain_fp32 = gain_dtype == SF_FP32;
  v->offset = (float)p->gain_offset;
  v->a = (float)p->residual_scale;
  v->b = (float)p->block_scale;
  return SF_OK;
}

}  // namespace

int read_and_clear_device_error_sandwich() {
  int v = 0, z = 0;
  if (cudaMemcpyFromSymbol(&v, g_device_error, sizeof v) != cudaSuccess) return 0;
  if (v) cudaMemcpyToSymbol(g_device_error, &z, sizeof z);
  return v;
}

}  // namespace sf

extern "C" {

sf_status sf_sandwich_norm_forward(const sf_sandwich* p, const sf_matrix* x, const sf_matrix* residual,
                                   const void* gain_post, const void* gain_pre, sf_dtype gain_dtype,
                                   const sf_matrix* gate, const sf_matrix* sum, const sf_matrix* h,
                                   const sf_checkpoint* x8, const sf_checkpoint* sum8, float* rstd_post,
                                   float* rstd_pre, void* stream) {
  using namespace sf;
  clear_error();
  NvtxRange nvtx_range("sf_sandwich_norm_forward");
  SF_TRY(check_matrix(x, "x", -1, -1, kTypes));
  const int64_t rows = x->rows, cols = x->cols;
  FwdArgs a{};
  SF_TRY(check_common(p, rows, cols, gain_post, gain_pre, gain_dtype, gate, &a.v));
  if (residual) SF_TRY(check_matrix(residual, "residual", rows, cols, kTypes));
  if (sum) SF_TRY(check_matrix(sum, "sum", rows, cols, kTypes));
  if (h) SF_TRY(check_matrix(h, "h", rows, cols, 1u << x->dtype));
  if (residual && sum && residual->dtype != sum->dtype) return fail(SF_ERR_INVALID, "residual and sum must have one type");
  if (x8) SF_TRY(check_checkpoint(x8, "x8", rows, cols, true));
  if (sum8) SF_TRY(check_checkpoint(sum8, "sum8", rows, cols, true));
  if (!sum && !h && !x8 && !sum8) return fail(SF_ERR_INVALID, "sum, h, x8 and sum8 are all NULL");
  if ((h || rstd_pre) && !gain_pre) return fail(SF_ERR_INVALID, "h and rstd_pre need gain_pre");
  if (rstd_post && !gain_post) return fail(SF_ERR_INVALID, "rstd_post needs gain_post");
  SF_TRY(check_aligned(rstd_post, sizeof(float), "rstd_post"));
  SF_TRY(check_aligned(rstd_pre, sizeof(float), "rstd_pre"));
  if (!rows) return SF_OK;
  a.x = x->data;
  a.ldx = x->ld;
  if (residual) a.r = residual->data, a.ldr = residual->ld;
  if (sum) a.s = sum->data, a.lds = sum->ld;
  if (h) a.h = h->data, a.ldh = h->ld;
  a.x8 = device_ck(x8);
  a.s8 = device_ck(sum8);
  a.rho1 = rstd_post;
  a.rho2 = rstd_pre;
  a.rows = rows;
  a.cols = (int32_t)cols;
  a.eps = (float)p->eps;
  a.inv_cols = (float)(1.0 / (double)cols);
  const bool units = on_units(x) && on_units(residual) && on_units(sum) && on_units(h) && on_units(gate) && on_units(x8) &&
                     on_units(sum8) && on_units(gain_post, gain_dtype) && on_units(gain_pre, gain_dtype);
  const int32_t ts = residual ? residual->dtype : sum ? sum->dtype : x->dtype;
  void* args[] = {&a, nullptr};
  // bulk copies take this device's own memory only
  RingShape ring;
  const size_t stage = slot_bytes(cols, dtype_bytes(x->dtype)) + (residual ? slot_bytes(cols, dtype_bytes(ts)) : 0);
  const Lay lay = units && cols % 16 == 0 ? kUnits : kStrided;
  a.wide = on_wide(sum) && on_wide(h) && on_wide(x8) && on_wide(sum8);
  if (ring_shape(rows, cols, stage, kFwdRegs1, kFwdRegs2, &ring) && (sum || h || sum8 || rstd_pre) && on_bulk(x) && on_bulk(residual)) {
    using B = __nv_bfloat16;
    const void* kernel = x->dtype == SF_BF16 ? (ts == SF_BF16 ? fwd_ring<B, B>(ring.c, lay) : fwd_ring<B, float>(ring.c, lay))
                                             : (ts == SF_BF16 ? fwd_ring<float, B>(ring.c, lay) : fwd_ring<float, float>(ring.c, lay));
    SF_TRY(allow_dynamic_smem(kernel, stage * ring.stages));
    args[1] = &ring.stages;
    SF_CUDA_TRY(cudaLaunchKernel(kernel, dim3((unsigned)std::min<int64_t>(rows, (int64_t)sm_count() * ring.per_sm)), dim3(ring.threads), args,
                                 stage * ring.stages, as_stream(stream)),
                "launch k_sandwich_fwd_ring");
    return SF_OK;
  }
  // as many threads a row as two steps need; one step while rows leave SMs without work
  const int64_t n = ceil_div<int64_t>(cols, 8);
  const int64_t t = std::min<int64_t>(ceil_div<int64_t>(n, rows < 2 * sm_count() ? 1 : kK), kMaxThreads);      // (1024 x 2 x 8 columns)
  if (t > 64) {
    a.tpr = (int32_t)ceil_div<int64_t>(t, 32) * 32;
    a.rpb = 1;
  } else {
    int w = 16;
    while (w < t) w *= 2;
    a.tpr = w;
    a.rpb = 128 / w;
  }
  a.steps = (int32_t)ceil_div<int64_t>(n, a.tpr);
  const int64_t grid = ceil_div<int64_t>(rows, a.rpb);
  if (grid > INT32_MAX) return fail(SF_ERR_UNSUPPORTED, "too many rows");
  SF_CUDA_TRY(cudaLaunchKernel(pick_kernel<Fwd>(x->dtype, ts, units ? kUnits : kStrided), dim3((unsigned)grid),
                               dim3(a.tpr * a.rpb), args, 0, as_stream(stream)),
              "launch k_sandwich_fwd");
  return SF_OK;
}

size_t sf_sandwich_norm_workspace_bytes(int64_t rows, int64_t cols) {
  if (rows < 0 || cols < 1 || cols > sf::kMaxCols) return 0;
  return 2 * (size_t)std::max<int64_t>(1, std::min<int64_t>(rows, sf::max_workers(cols))) * cols * sizeof(float);
}

sf_status sf_sandwich_norm_backward(const sf_sandwich* p, const sf_matrix* dh, const sf_matrix* dsum, const sf_matrix* x,
                                    const sf_checkpoint* x8, const sf_matrix* sum, const sf_checkpoint* sum8,
                                    const void* gain_post, const void* gain_pre, sf_dtype gain_dtype,
                                    const sf_matrix* gate, const float* rstd_post, const float* rstd_pre,
                                    const sf_matrix* dresidual, const sf_matrix* dx, void* dgain_post, void* dgain_pre,
                                    sf_dtype dgain_dtype, const sf_matrix* dgate, void* ws, size_t ws_bytes,
                                    void* stream) {
  using namespace sf;
  clear_error();
  NvtxRange nvtx_range("sf_sandwich_norm_backward");
  const sf_matrix* first = dh ? dh : dsum;
  if (!first) return fail(SF_ERR_INVALID, "dh and dsum are both NULL");
  SF_TRY(check_matrix(first, dh ? "dh" : "dsum", -1, -1, kTypes));
  const int64_t rows = first->rows, cols = first->cols;
  BwdArgs a{};
  SF_TRY(check_common(p, rows, cols, gain_post, gain_pre, gain_dtype, gate, &a.v));
  if (x && x8) return fail(SF_ERR_INVALID, "x and x8 are both given");
  if (sum && sum8) return fail(SF_ERR_INVALID, "sum and sum8 are both given");
  if (!dresidual && !dx && !dgain_post && !dgain_pre && !dgate) return fail(SF_ERR_INVALID, "no gradient is wanted");
  // one type for dh, dx and x, another for dsum, dresidual and the sum
  const sf_matrix* act[3] = {dh, dx, x};
  const sf_matrix* str[3] = {dsum, dresidual, sum};
  const char* act_name[3] = {"dh", "dx", "x"};
  const char* str_name[3] = {"dsum", "dresidual", "sum"};
  int32_t ta = -1, ts = -1;
  for (int i = 0; i < 3; ++i) {
    if (act[i]) {
      SF_TRY(check_matrix(act[i], act_name[i], rows, cols, ta < 0 ? kTypes : 1u << ta));
      ta = act[i]->dtype;
    }
    if (str[i]) {
      SF_TRY(check_matrix(str[i], str_name[i], rows, cols, ts < 0 ? kTypes : 1u << ts));
      ts = str[i]->dtype;
    }
  }
  if (ta < 0) ta = ts;
  if (ts < 0) ts = ta;
  if (x8) SF_TRY(check_checkpoint(x8, "x8", rows, cols, false));
  if (sum8) SF_TRY(check_checkpoint(sum8, "sum8", rows, cols, false));
  SF_TRY(check_vector(dgain_post, dgain_dtype, "dgain_post"));
  SF_TRY(check_vector(dgain_pre, dgain_dtype, "dgain_pre"));
  if (dh) {
    if (!gain_pre) return fail(SF_ERR_INVALID, "dh needs gain_pre");
    if (!sum && !sum8) return fail(SF_ERR_INVALID, "dh needs sum or sum8");
    if (rows && !rstd_pre) return fail(SF_ERR_INVALID, "dh needs rstd_pre");
  }
  if (dgain_pre && !dh) return fail(SF_ERR_INVALID, "dgain_pre needs dh");
  if (dgain_post && !gain_post) return fail(SF_ERR_INVALID, "dgain_post needs gain_post");
  if (dgate && !gate) return fail(SF_ERR_INVALID, "dgate needs gate");
  const bool wants_t = dgain_post || dgate;
  if (((gain_post && dx) || wants_t) && !x && !x8) return fail(SF_ERR_INVALID, "dx, dgain_post and dgate need x or x8");
  if (gain_post && (dx || wants_t) && rows && !rstd_post) return fail(SF_ERR_INVALID, "the norm after the block needs rstd_post");
  SF_TRY(check_aligned(rstd_post, sizeof(float), "rstd_post"));
  SF_TRY(check_aligned(rstd_pre, sizeof(float), "rstd_pre"));
  if (dgate) SF_TRY(check_matrix(dgate, "dgate", gate->rows, cols, kTypes));
  if (wants_t || dgain_pre) {
    const size_t need = sf_sandwich_norm_workspace_bytes(rows, cols);
    if (!ws || ws_bytes < need || reinterpret_cast<uintptr_t>(ws) % 16)
      return fail(SF_ERR_INVALID, "workspace needs %zu bytes, 16-byte aligned (got %zu)", need, ws_bytes);
  }
  // where only the residual's gradient is wanted, the branch is left out
  if (!dx && !wants_t) a.v.g_post = nullptr, x = nullptr, x8 = nullptr;
  if (!dh) a.v.g_pre = nullptr, sum = nullptr, sum8 = nullptr;
  if (dh) a.dh = dh->data, a.lddh = dh->ld;
  if (dsum) a.dsum = dsum->data, a.lddsum = dsum->ld;
  if (x) a.x = x->data, a.ldx = x->ld;
  if (sum) a.s = sum->data, a.lds = sum->ld;
  if (dresidual) a.dr = dresidual->data, a.lddr = dresidual->ld;
  if (dx) a.dx = dx->data, a.lddx = dx->ld;
  a.x8 = device_ck(x8);
  a.s8 = device_ck(sum8);
  a.rho1 = rstd_post;
  a.rho2 = rstd_pre;
  a.rows = rows;
  a.cols = (int32_t)cols;
  a.inv_cols = (float)(1.0 / (double)cols);
  const bool units = on_units(dh) && on_units(dsum) && on_units(x) && on_units(sum) && on_units(dresidual) && on_units(dx) &&
                     on_units(x8) && on_units(sum8) && on_units(gate) && on_units(dgate) && on_units(a.v.g_post, gain_dtype) &&
                     on_units(a.v.g_pre, gain_dtype);
  // the staged form: as many blocks an SM as registers and three stages (of long rows two) allow
  const bool kept = x8 && sum8;
  const Lay lay = units && cols % 16 == 0 ? kUnits : kStrided;
  const size_t stage = slot_bytes(cols, dtype_bytes(ta)) + (dsum ? slot_bytes(cols, dtype_bytes(ts)) : 0) +
                       (kept ? 2 * slot_bytes(cols, 1) : slot_bytes(cols, dtype_bytes(ta)) + slot_bytes(cols, dtype_bytes(ts)));
  int ring_threads = 0, ring_blocks = 0, ring_stages = 0;
  if (dh && (kept || (x && sum)) && cols >= kBwdMinCols && cols <= 16 * kBwdRingThreads && rows >= 2 * sm_count() && rows < (1 << 29) &&
      on_bulk(dh) && on_bulk(dsum) && on_bulk(x) && on_bulk(sum) && (!kept || (on_bulk(&x8->values) && on_bulk(&sum8->values)))) {
    a.wide = on_wide(x8) && on_wide(sum8) && on_wide(dresidual) && on_wide(dx);
    ring_threads = (int)ceil_div<int64_t>(ceil_div<int64_t>(cols, 16), 32) * 32;
    ring_blocks = std::min(32, 65536 / (kBwdRingRegs * ring_threads));
    const size_t block = kSmemBlock + (kept && lay == kStrided ? kSmemScales : 0);
    while (ring_blocks > 1 && kSmemPerSm / ring_blocks < block + 3 * stage) --ring_blocks;
    ring_stages = (int)std::min<size_t>(kMaxStages, (kSmemPerSm / ring_blocks - block) / stage);
  }
  const bool staged = ring_stages >= 2;
  const int64_t n = ceil_div<int64_t>(cols, 8);
  const int64_t t = ceil_div<int64_t>(n, rows < 2 * sm_count() && n <= kBwdThreads ? 1 : kBwdK);
  if (t > 64) {
    a.tpr = (int32_t)ceil_div<int64_t>(t, 32) * 32;
    a.rpb = 1;
  } else {
    int w = 4;
    while (w < t) w *= 2;
    a.tpr = w;
    a.rpb = 128 / w;
  }
  if (staged) a.tpr = ring_threads, a.rpb = 1;
  const int threads = a.tpr * a.rpb;
  // items: gate rows (without a gate one, all rows) in parts
  a.span = gate ? a.v.span : std::max<int64_t>(1, rows);
  const int64_t gate_rows = gate ? gate->rows : 1;
  const int64_t most = std::min<int64_t>(max_workers(cols), (int64_t)sm_count() * (staged ? ring_blocks : std::max(1, 512 / threads)) * a.rpb);
  a.many = gate_rows > most;
  a.parts = !rows || !gate_rows ? 0 : a.many ? 1 : (int32_t)std::min(most / gate_rows, rows / gate_rows);
  a.items = gate_rows * a.parts;
  a.workers = std::min(a.items, most);
  float* part = static_cast<float*>(ws);
  if (dgain_pre) a.ppart = part;
  if (wants_t && (!a.many || dgain_post)) a.tpart = part + a.workers * cols;
  if (dgate) {
    a.dgate_fp32 = dgate->dtype == SF_FP32;
    if (a.many) a.dgate = dgate->data, a.lddgate = dgate->ld;
  }
  cudaStream_t st = as_stream(stream);
  if (rows && staged) {
    const void* kernel = pick_kernel<BwdRing>(ta, ts, lay, kept, a.v.g_post != nullptr);
    SF_TRY(allow_dynamic_smem(kernel, stage * ring_stages));
    void* args[] = {&a, &ring_stages};
    SF_CUDA_TRY(cudaLaunchKernel(kernel, dim3((unsigned)a.workers), dim3(threads), args, stage * ring_stages, st), "launch k_sandwich_bwd_ring");
  } else if (rows) {
    void* args[] = {&a};
    SF_CUDA_TRY(cudaLaunchKernel(threads <= kBwdFew ? pick_kernel<BwdFew>(ta, ts, units ? kUnits : kStrided) : pick_kernel<Bwd>(ta, ts, units ? kUnits : kStrided), dim3((unsigned)ceil_div<int64_t>(a.workers, a.rpb)),
                                 dim3(threads), args, 0, st),
                "launch k_sandwich_bwd");
  }
  if (dgain_pre || a.tpart) {
    JoinArgs j{};
    j.tpart = a.tpart;
    j.ppart = a.ppart;
    j.dg1 = dgain_post;
    j.dg2 = dgain_pre;
    if (dgate && !a.many) j.dgate = dgate->data, j.lddgate = dgate->ld;
    j.workers = a.workers;
    j.gate_rows = gate_rows;
    j.parts = a.parts;
    j.many = a.many;
    j.cols = a.cols;
    j.dgain_fp32 = dgain_dtype == SF_FP32;
    j.dgate_fp32 = a.dgate_fp32;
    j.v = a.v;
    SF_CUDA_TRY(launch_pdl(k_sandwich_join, dim3((unsigned)ceil_div<int64_t>(cols, 32), a.tpart ? 2 : 1), dim3(32, 32), 0, st, j),
                "launch k_sandwich_join");
  }
  return SF_OK;
}

}  // extern "C"
