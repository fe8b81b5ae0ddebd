// The end of a residual block: the norm after the block, its gate, the
// residual's addition with its scales, and the norm before the next block,
//   n = x rho1 g1,  s = a r + b gate n,  h = s rho2 g2,
// rho = 1 / sqrt(mean(row^2) + eps), and its gradients; x and s kept as 8-bit
// checkpoints where wanted.  (The root-mean-square norm is Zhang and Sennrich
// 2019.)
#include "sandwich.cuh"

namespace sf {
namespace {

constexpr int kK = 2;               // steps per thread of the register form
constexpr int kMaxThreads = 1024;
constexpr int kRingMinCols = 1024;

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
constexpr int kRingThreads = 768;

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

// C: wide units a thread.  With one of them g2 stays in registers too.
//
// 16384 x 4096 bf16 with a gate and both checkpoints 113 us, 0.87 of the copy rate (614 MB
// of DRAM traffic; an instruction is issued in 0.62 of the cycles, from 24 warps an SM); 8192 x 12288 with an
// fp32 stream 187 us, 0.95; 16384 x 4095 129 us, with both checkpoints 236.
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
  const int first = (int)(a.rows * blockIdx.x / gridDim.x), end = (int)(a.rows * (blockIdx.x + 1) / gridDim.x);
  auto fill = [&](int row, int st) {      // by one thread
    unsigned char* at = ring + (size_t)st * stage_bytes;
    if constexpr (LAY == kUnits) {      // (few instructions: the thread's warp is waited for)
      const uint32_t bytes_x = (uint32_t)a.cols * sizeof(TA), bytes_r = a.r ? (uint32_t)a.cols * sizeof(TS) : 0u;
      mbar_arrive_expect_tx(&full[st], bytes_x + bytes_r);
      bulk_load(at, short_row<TA>(a.x, a.ldx, row), bytes_x, &full[st]);
      if (a.r) bulk_load(at + row_x, short_row<TS>(a.r, a.ldr, row), bytes_r, &full[st]);
      return;
    }
    const bool last = row == a.rows - 1;
    const Bring b[2] = {{short_row<TA>(a.x, a.ldx, row), (uint32_t)a.cols * (uint32_t)sizeof(TA), last},
                        {short_row<TS>(a.r, a.ldr, row), a.r ? (uint32_t)a.cols * (uint32_t)sizeof(TS) : 0u, last}};
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
  const int span = (int)a.v.span;
  int gate_end = first;      // rows from here on take another gate row
  int gate_at = a.v.gate ? first / span : 0;
  int st = 0, parity = 0;
  uint32_t phase = 0;
  bool dead = false;      // a wait ran out (recorded): go on without waiting, so that all threads still leave together
  for (int row = first; row < end; ++row, parity ^= 1) {
    if (row == gate_end) {
      gate_end = a.v.gate ? (gate_at + 1) * span : end;
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
          vec(gate_row_of(a.v, gate_at), a.v.gate_fp32, c, 0.0f, v);
          w[k][0] = mul8(w[k][0], v[0]), w[k][1] = mul8(w[k][1], v[1]);
        }
      }
      ++gate_at;
    }
    if (!dead) dead = !mbar_wait_u32(smem_u32(&full[st]), phase);
    const uint32_t at = ring0 + (uint32_t)st * stage_bytes + (LAY == kUnits ? 0u : lead_of(short_row<TA>(a.x, a.ldx, row)));
    const uint32_t at_r = ring0 + (uint32_t)st * stage_bytes + row_x + (LAY == kUnits ? 0u : lead_of(short_row<TS>(a.r, a.ldr, row)));
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
        const Lds16<TA, LAY> x(at, c, a.cols);
#pragma unroll
        for (int h = 0; h < 2; ++h) s[k][h] = mul8(scale8(x.half(h), rho1), w[k][h]);
        if (a.r) {
          const Lds16<TS, LAY> r(at_r, c, a.cols);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const F8 v = r.half(h);
#pragma unroll
            for (int i = 0; i < 4; ++i) s[k][h].p[i] = fmadd2(v.p[i], pack_f2(a.v.a, a.v.a), s[k][h].p[i]);
          }
        }
        if (a.s) put16<TS, LAY>(short_row<TS>(a.s, a.lds, row), c, a.cols, s[k][0], s[k][1], a.wide);
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
        put16<TA, LAY>(short_row<TA>(a.h, a.ldh, row), c, a.cols, mul8(scale8(s[k][0], rho2), g2[0]), mul8(scale8(s[k][1], rho2), g2[1]), a.wide);
      }
    }
    if (++st == stages) {
      st = 0;
      phase ^= 1u;
    }
  }
  if (dead && t == 0) {      // copies still under way land before their memory is given up (waited for once more, bounded)
    const int n = end - first;
    for (int i = 0; i < stages && i < n; ++i) mbar_wait(&full[i], (uint32_t)((n - 1 - i) / stages) & 1u);
  }
  if (dead) __syncthreads();
}

template <typename TA, typename TS, int LAY>
struct Fwd {
  static const void* ptr() { return (const void*)&k_sandwich_fwd<TA, TS, LAY>; }
};
// The staged form: wide units a thread, registers.
constexpr int kFwdRegs1 = 80, kFwdRegs2 = 128;
template <typename TA, typename TS>
const void* fwd_ring(int c, Lay lay) {
  if (lay == kUnits) return c == 1 ? (const void*)&k_sandwich_fwd_ring<TA, TS, kUnits, 1, kFwdRegs1> : (const void*)&k_sandwich_fwd_ring<TA, TS, kUnits, 2, kFwdRegs2>;
  return c == 1 ? (const void*)&k_sandwich_fwd_ring<TA, TS, kStrided, 1, kFwdRegs1> : (const void*)&k_sandwich_fwd_ring<TA, TS, kStrided, 2, kFwdRegs2>;
}
struct RingShape {
  int c = 0, threads = 0, per_sm = 0, stages = 0;
};
// One or two wide units a thread, whichever lets more threads, or as many in
// more blocks, reside on an SM (bf16, 4 x 4096-token batches' worth of data: 8192
// columns in two blocks of 256 threads 127 us, in one of 512 169; 12288 with an
// fp32 stream in one of 768 threads 201 us, in one of 384 244, when this was chosen).  At least three
// stages each, two in long rows.  False where rows are too long, or too few or short
// for it to pay (65536 x 512: 63 us, 51 with loads into registers; 32768 x 1024 50 and 54).
bool ring_shape(int64_t rows, int64_t cols, size_t stage, int regs1, int regs2, RingShape* best) {
  if (cols < kRingMinCols || rows < 2 * sm_count() || rows >= 1 << 29) return false;
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

}  // namespace

const void* device_error_sandwich_fwd() { return &g_device_error; }

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
  // (a gate row that several rows take must outlast them)
  for (const sf_matrix* out : {sum, h})
    if (overlap(out, gate) && !(gate->rows == rows && same_matrix(out, gate)))
      return fail(SF_ERR_INVALID, "sum and h may lie over the gate only as the same matrix, with a gate row for each row");
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
  const bool short_lds = short_ld(x) && short_ld(residual) && short_ld(sum) && short_ld(h);
  if (ring_shape(rows, cols, stage, kFwdRegs1, kFwdRegs2, &ring) && (sum || h || sum8 || rstd_pre) && short_lds && on_bulk(x) && on_bulk(residual)) {
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

}  // extern "C"
