// The staged form of the backward pass of a residual block's end, instantiated
// for one lay each by sandwich_bwd_units.cu and sandwich_bwd_strided.cu.
#pragma once

#include "sandwich_bwd.cuh"

namespace sf {
namespace {

// The same backward pass with rows brought by bulk copies, as in the forward
// form: a block is one worker, a thread holds a wide unit's sums, w and g2 in
// registers.  A row is read from shared memory twice, for its sums and, past
// the one barrier, for its outputs (dsum + rho2 dh g2 stays in registers
// between); past that barrier every thread is also done with the row before,
// whose stage is filled again.  For calls with dh, dsum or none, and x and s both in
// full or both as checkpoints (KEPT).
//
// 16384 x 4096 from both checkpoints with four gate rows 143 us, about 9 of them the
// join, 0.69 of the copy rate: 128 registers a thread leave 16 warps an SM, which issue
// 0.53 of an instruction a cycle.  From bf16 152 us, odd rows (16384 x 4095) 211, from checkpoints 294.

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
  const bool whole = whole512(c0, cols);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int c = c0 + 64 * i, d = c + 32;
    uint32_t q0 = 0, q1 = 0;
    if (whole || c < cols) asm volatile("ld.shared.u8 %0, [%1];" : "=r"(q0) : "r"(p + c));
    if (whole || d < cols) asm volatile("ld.shared.u8 %0, [%1];" : "=r"(q1) : "r"(p + d));
    const float2 x = e4m3x2_value(q0 | q1 << 8);
    // (a column past the row: 0 times the last scale)
    v[i >> 2].p[i & 3] = fmul2(pack_f2(x.x, x.y), pack_f2(scales[(whole ? c : min(c, cols - 1)) >> shift], scales[(whole ? d : min(d, cols - 1)) >> shift]));
  }
}

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
    const int r = row_at(j);
    unsigned char* at = ring + (size_t)st * stage_bytes;
    const bool last = r == a.rows - 1;
    const uint32_t size_a = (uint32_t)a.cols * (uint32_t)sizeof(TA), size_s = (uint32_t)a.cols * (uint32_t)sizeof(TS);
    if (LAY == kUnits && (!KEPT || a.wide)) {      // (few instructions: the thread's warp is waited for)
      mbar_arrive_expect_tx(&full[st], size_a + (a.dsum ? size_s : 0u) + (KEPT ? 2u * a.cols : size_a + size_s));
      bulk_load(at, short_row<TA>(a.dh, a.lddh, r), size_a, &full[st]);
      if (a.dsum) bulk_load(at + off_e, short_row<TS>(a.dsum, a.lddsum, r), size_s, &full[st]);
      if (KEPT) {
        bulk_load(at + off_x, short_row<uint8_t>(a.x8.q, a.x8.ld, r), a.cols, &full[st]);
        bulk_load(at + off_s, short_row<uint8_t>(a.s8.q, a.s8.ld, r), a.cols, &full[st]);
      } else {
        bulk_load(at + off_x, short_row<TA>(a.x, a.ldx, r), size_a, &full[st]);
        bulk_load(at + off_s, short_row<TS>(a.s, a.lds, r), size_s, &full[st]);
      }
      return;
    }
    const Bring b[4] = {{short_row<TA>(a.dh, a.lddh, r), size_a, last},
                        {short_row<TS>(a.dsum, a.lddsum, r), a.dsum ? size_s : 0u, last},
                        {KEPT ? (const void*)short_row<uint8_t>(a.x8.q, a.x8.ld, r) : short_row<TA>(a.x, a.ldx, r), KEPT ? (uint32_t)a.cols : size_a, last},
                        {KEPT ? (const void*)short_row<uint8_t>(a.s8.q, a.s8.ld, r) : short_row<TS>(a.s, a.lds, r), KEPT ? (uint32_t)a.cols : size_s, last}};
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
#pragma unroll
      for (int h = 0; h < 2; ++h) v[h] = load8_any<LAY>(gate, a.v.gate_fp32, c + (LAY == kUnits ? 8 : 256) * h, LAY == kUnits ? 1 : 32, a.cols);
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
      if (on && a.tpart) {      // (before dgate, which may be the gate's own memory) this worker's own row, written and read by the same threads (on 16 bytes at least: no wide access)
        float* part = a.tpart + (int64_t)worker * a.cols;
        F8 v = first ? zero8() : load8<kStrided>(part, ch, kApart, a.cols);
        const F8 g = load8_any<LAY>(gate, a.v.gate_fp32, ch, kApart, a.cols);
#pragma unroll
        for (int i = 0; i < 4; ++i) v.p[i] = fmadd2(accT[h].p[i], g.p[i], v.p[i]);
        store8<kStrided>(part, ch, kApart, a.cols, v);
      }
      if (on && a.dgate) {
        F8 v = accT[h];
        if (POST) v = mul8(v, load_vec<LAY>(a.v.g_post, a.v.gain_fp32, ch, kApart, a.cols, a.v.offset));
        store_any<LAY>(static_cast<char*>(a.dgate) + (int64_t)gate_row * a.lddgate * (a.dgate_fp32 ? 4 : 2), a.dgate_fp32, ch, kApart, a.cols, v);
      }
      accT[h] = zero8();
    }
  };
  // a row's rhos and scales come one row ahead
  float rho1_next = 1.0f, rho2_next = 0.0f;
  uint32_t sx_next = 0, ss_next = 0;
  // (strided: a thread brings one group's, for all)
  auto scale_raw = [&](const Ck& ck, uint32_t r) {
    const uint64_t i = (uint64_t)r * (uint32_t)ck.n_groups + (LAY == kStrided ? min(t, ck.n_groups - 1) : ck.group_log2 && on ? c >> ck.group_log2 : 0);
    return ck.s8 ? (uint32_t)ck.s8[i] : __float_as_uint(ck.s32[i]);
  };
  auto scale_value = [](const Ck& ck, uint32_t raw) { return ck.s8 ? e8m0_value(raw) : __uint_as_float(raw); };
  auto prefetch = [&](int r) {
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
    const int r = row;
    const bool last = --left == 0;      // of its item
    row = last ? (gate_row + workers) * span : row + 1;
    if (j + 1 < n) prefetch(row);
    if (!dead) dead = !mbar_wait_u32(smem_u32(&full[st]), phase);
    const uint32_t base = ring0 + (uint32_t)st * stage_bytes;
    const uint32_t at_dh = base + (LAY == kUnits ? 0u : lead_of(short_row<TA>(a.dh, a.lddh, r)));
    const uint32_t at_e = base + off_e + (LAY == kUnits ? 0u : lead_of(short_row<TS>(a.dsum, a.lddsum, r)));
    const uint32_t at_x = base + off_x + (KEPT ? lead_of(short_row<uint8_t>(a.x8.q, a.x8.ld, r)) : LAY == kUnits ? 0u : lead_of(short_row<TA>(a.x, a.ldx, r)));
    const uint32_t at_s = base + off_s + (KEPT ? lead_of(short_row<uint8_t>(a.s8.q, a.s8.ld, r)) : LAY == kUnits ? 0u : lead_of(short_row<TS>(a.s, a.lds, r)));
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
      if (a.dr) put16<TS, LAY>(short_row<TS>(a.dr, a.lddr, r), c, a.cols, scale8(e[0], a.v.a), scale8(e[1], a.v.a), a.wide);
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint64_t bd = fmul2(e[h].p[i], pack_f2(tf, tf));
          accT[h].p[i] = fmadd2(bd, x[h].p[i], accT[h].p[i]);
          e[h].p[i] = POST ? fmadd2(bd, w[h].p[i], fmul2(x[h].p[i], pack_f2(c1, c1))) : fmul2(bd, w[h].p[i]);
        }
      if (a.dx) put16<TA, LAY>(short_row<TA>(a.dx, a.lddx, r), c, a.cols, e[0], e[1], a.wide);
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

template <typename TA, typename TS, int LAY>
const void* bwd_ring(bool kept, bool post) {
  return kept ? (post ? (const void*)&k_sandwich_bwd_ring<TA, TS, LAY, true, true> : (const void*)&k_sandwich_bwd_ring<TA, TS, LAY, true, false>)
              : (post ? (const void*)&k_sandwich_bwd_ring<TA, TS, LAY, false, true> : (const void*)&k_sandwich_bwd_ring<TA, TS, LAY, false, false>);
}
template <int LAY>
const void* bwd_ring_of(int32_t ta, int32_t ts, bool kept, bool post) {
  using B = __nv_bfloat16;
  if (ta == SF_BF16) return ts == SF_BF16 ? bwd_ring<B, B, LAY>(kept, post) : bwd_ring<B, float, LAY>(kept, post);
  return ts == SF_BF16 ? bwd_ring<float, B, LAY>(kept, post) : bwd_ring<float, float, LAY>(kept, post);
}

}  // namespace
}  // namespace sf
