// The backward pass of the end of a residual block: the form with loads into
// registers, the join of the partial sums, and the entry point.
#include "sandwich_bwd.cuh"

namespace sf {
namespace {

constexpr int kBwdMinCols = 256;

constexpr int kBwdThreads = 1024, kBwdFew = 256, kBwdK = 2;

// T: most threads of a block.  Up to 4096 columns (2048 where rows are few, of one step a thread) kBwdFew, with 128
// registers a thread; 1024 have 64 and spill over 1.2 KB.
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
          if (gate) w = mul8(w, load8_any<LAY>(gate, a.v.gate_fp32, c0, l.dj, cols));
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
          if (gate) d = mul8(d, load8_any<LAY>(gate, a.v.gate_fp32, c0, l.dj, cols));
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
        if (a.tpart) {      // (before dgate, which may be the gate's own memory)
          // this worker's own row, written and read by the same threads
          float* part = a.tpart + worker * a.cols;
          F8 v = round ? load8<kStrided>(part, c0, l.dj, a.cols) : zero8();
          const F8 g = load8_any<LAY>(gate, a.v.gate_fp32, c0, l.dj, a.cols);
#pragma unroll
          for (int i4 = 0; i4 < 4; ++i4) v.p[i4] = fmadd2(accT[q].p[i4], g.p[i4], v.p[i4]);
          store8<kStrided>(part, c0, l.dj, a.cols, v);
        }
        if (a.dgate) {
          F8 v = accT[q];
          if (post) v = mul8(v, load_vec<LAY>(a.v.g_post, a.v.gain_fp32, c0, l.dj, a.cols, a.v.offset));
          store_any<LAY>(static_cast<char*>(a.dgate) + k * a.lddgate * (a.dgate_fp32 ? 4 : 2), a.dgate_fp32, c0, l.dj, a.cols, v);
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
  __shared__ float red[4][32][33];
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
    v = join32(v, red[0]);
    if (writes) put_at(dst, a.dgain_fp32, out, v);
    return;
  }
  if (!a.tpart) return;
  const float g1c = on && a.v.g_post ? vec_at(a.v.g_post, a.v.gain_fp32, c) + a.v.offset : 1.0f;
  float dg1 = 0.0f;
  // A gate row's parts by one thread, unless gate rows are few and their parts many (21 gate rows of 28 parts: the backward
  // pass over 5003 x 2003 took 61 us so, and 82 with the rows one after the other by the whole block).
  if (a.gate_rows >= 32 || a.parts <= 32) {
    for (int64_t k = threadIdx.y; k < a.gate_rows; k += 32) {
      float v = 0.0f;
      if (on) {
#pragma unroll 8
        for (int p = 0; p < a.parts; ++p) v += a.tpart[(k * a.parts + p) * a.cols + c];
        dg1 = fmaf(vec_at(a.v.gate, a.v.gate_fp32, k * a.v.ld_gate + c), v, dg1);      // (before: dgate may be the gate's own memory)
        if (a.dgate) put_at(a.dgate, a.dgate_fp32, k * a.lddgate + c, g1c * v);
      }
    }
    dg1 = join32(dg1, red[0]);
  } else {      // four gate rows at a time
    const float g1 = writes && a.v.g_post ? vec_at(a.v.g_post, a.v.gain_fp32, out) + a.v.offset : 1.0f;
    for (int64_t k0 = 0; k0 < a.gate_rows; k0 += 4) {
      float v[4] = {};
      if (on) {
#pragma unroll 4
        for (int p = threadIdx.y; p < a.parts; p += 32)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (k0 + i < a.gate_rows) v[i] += a.tpart[((k0 + i) * a.parts + p) * a.cols + c];
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 4; ++i) red[i][threadIdx.y][threadIdx.x] = v[i];
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] = red[i][threadIdx.x][threadIdx.y];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
        const int64_t k = k0 + i;
        if (!writes || k >= a.gate_rows) continue;
        dg1 = fmaf(vec_at(a.v.gate, a.v.gate_fp32, k * a.v.ld_gate + out), v[i], dg1);
        if (a.dgate) put_at(a.dgate, a.dgate_fp32, k * a.lddgate + out, g1 * v[i]);
      }
    }
  }
  if (a.dg1 && writes) put_at(a.dg1, a.dgain_fp32, out, dg1);
}

// Rows of the workspace's partial sums: more of them where rows are short.
int64_t max_workers(int64_t cols) { return std::min<int64_t>(8192, std::max<int64_t>(1024, (1 << 21) / cols)); }

template <typename TA, typename TS, int LAY>
struct Bwd {
  static const void* ptr() { return (const void*)&k_sandwich_bwd<TA, TS, LAY, kBwdThreads>; }
};
template <typename TA, typename TS, int LAY>
struct BwdFew {
  static const void* ptr() { return (const void*)&k_sandwich_bwd<TA, TS, LAY, kBwdFew>; }
};

}  // namespace
}  // namespace sf

extern "C" {

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
  // (the gate is read again for its products and for dgain_post; a row of it before the same row of dgate is written)
  if (overlap(dresidual, gate) || overlap(dx, gate)) return fail(SF_ERR_INVALID, "dresidual and dx must not lie over the gate");
  if (overlap(dgate, gate) && !same_matrix(dgate, gate)) return fail(SF_ERR_INVALID, "dgate lies over the gate with another type, place or distance of rows");
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
      short_ld(dh) && short_ld(dsum) && short_ld(x) && short_ld(sum) && short_ld(dresidual) && short_ld(dx) &&
      (!kept || (short_ld(&x8->values) && short_ld(&sum8->values))) && on_bulk(dh) && on_bulk(dsum) && on_bulk(x) && on_bulk(sum) && (!kept || (on_bulk(&x8->values) && on_bulk(&sum8->values)))) {
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
    const bool post = a.v.g_post != nullptr;
    const void* kernel = lay == kUnits ? bwd_ring_units(ta, ts, kept, post) : bwd_ring_strided(ta, ts, kept, post);
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
