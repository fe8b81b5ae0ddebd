// Dropout with the residual's addition, from a counter-based generator:
//   y = r + m o x f,   m_ij = [bits_ij >= t],  f = 65536 / (65536 - t)
// The mask is a function of (seed, offset, row, column), so it is computed
// where it is used and never stored: the backward pass is the same call on
// the gradient, and the norm kernels apply the same mask inside their pass.
//
// Elementwise, one read of x (and r) and one write of y; HBM bounds it.  A
// block takes 1024 consecutive units of eight columns, four loads of each
// operand in flight a thread (a persistent grid with two resident blocks an SM
// was 40 % slower), and products and additions go two at a time, so that the
// generator's 2.5 wide multiplications an element stay in the shadow of the
// loads: 16384 x 4096 bf16 with a bf16 residual 59.8 us, 6.7 TB/s, the copy
// rate.  In rows that start off a unit, each unit's bits come from two
// evaluations, its own and the neighbouring lane's (16384 x 4095: 100 us).
#include <algorithm>

#include "rows.cuh"

namespace sf {
namespace {

constexpr int kThreads = 256;
constexpr int kUnits = 4;   // units in flight per thread

struct DropoutArgs {
  const void* x;
  const void* r;
  void* y;
  int64_t ldx, ldr, ldy;
  int64_t units;        // rows * per_row
  int64_t per_row;      // units a row may touch
  int64_t counters;     // generator units per row
  int32_t cols;         // (not FLAT)
  int32_t shift;        // kShifted
  int32_t per_thread;   // units a thread takes, 1..kUnits
  uint32_t div_mul;     // b / per_row = (mulhi(b, div_mul) + b) >> div_shift for b < 2^31
  int32_t div_shift;    // (Granlund and Montgomery, "Division by invariant integers using multiplication", 1994)
  DropConsts d;
};

// A block takes per_thread * 256 consecutive units.  FLAT: dense rows of whole
// units, so a unit's place follows from its index; otherwise one division a
// unit finds its row.
template <typename TX, typename TY, bool RES, int MODE, bool FLAT>
__global__ void __launch_bounds__(kThreads) k_dropout(const DropoutArgs a) {
  const DropWords words = drop_words(a.d);
  const int lane = threadIdx.x & 31;
  // shifted: a warp's units are consecutive, so that the lanes can hand the
  // generator's words on; otherwise a block's are
  const int64_t b0 = (int64_t)blockIdx.x * (a.per_thread * kThreads) + (MODE == kShifted ? (threadIdx.x - lane) * a.per_thread + lane : threadIdx.x);
  constexpr int kStep = MODE == kShifted ? 32 : kThreads;
  Unit<TX> x[kUnits];
  Unit<TY> r[kUnits];
  // the k-th unit's row, unit of the row, the row's shift, and its columns
  auto place = [&](int k, int64_t& row, int& u, int& m) {
    const int64_t b = b0 + k * kStep;
    if (k >= a.per_thread || b >= a.units) return Span{0, 0, 0};
    row = a.units <= INT32_MAX ? (int64_t)((__umulhi((uint32_t)b, a.div_mul) + (uint32_t)b) >> a.div_shift) : b / a.per_row;
    u = (int)(b - row * a.per_row);
    m = MODE == kShifted ? (int)(row * a.shift) & 7 : 0;
    return unit_span<MODE>(u, m, a.cols);
  };
#pragma unroll
  for (int k = 0; k < kUnits; ++k) {
    if (FLAT) {
      const int64_t b = b0 + k * kStep;
      if (k >= a.per_thread || b >= a.units) continue;
      ld_unit(static_cast<const TX*>(a.x) + 8 * b, x[k]);
      if (RES) ld_unit(static_cast<const TY*>(a.r) + 8 * b, r[k]);
    } else {
      int64_t row = 0;
      int u = 0, m = 0;
      const Span s = place(k, row, u, m);
      if (!s.some()) continue;
      load_unit<MODE>(row_ptr<TX>(a.x, a.ldx, row) + s.c, s.lo, s.hi, x[k]);
      if (RES) load_unit<MODE>(row_ptr<TY>(a.r, a.ldr, row) + s.c, s.lo, s.hi, r[k]);
    }
  }
  ShiftedBits bits;
  if (MODE == kShifted && a.d.threshold) {
    // the counter before the warp's first unit's, if that does not begin a row
    int64_t row = 0;
    int u = 0, m = 0;
    place(0, row, u, m);
    const int64_t before = __shfl_sync(0xffffffffu, u ? row * a.counters + u - 1 : (int64_t)-1, 0);
    if (before >= 0) bits.start((uint64_t)before, words, a.d);
  }
#pragma unroll
  for (int k = 0; k < kUnits; ++k) {
    const int64_t b = b0 + k * kStep;
    int64_t row = 0;
    int u = 0, m = 0;
    uint32_t w[4];
    Span s = {0, 0, 8};
    if (FLAT) {
      if (k >= a.per_thread || b >= a.units) continue;
    } else {
      s = place(k, row, u, m);
      if (MODE == kShifted && a.d.threshold && k < a.per_thread)
        bits.next((uint64_t)(row * a.counters + u), lane, 32, m, words, a.d, w);
      if (!s.some()) continue;
    }
    F8 v = unpack(x[k]);
    if (a.d.threshold) {
      if (MODE == kShifted) drop_apply(v, w, a.d);
      else drop_unit(v, (uint64_t)(FLAT ? b : row * a.counters + u), words, a.d);
    }
    if (RES) {
      const F8 w = unpack(r[k]);
#pragma unroll
      for (int i = 0; i < 4; ++i) v.p[i] = fadd2(v.p[i], w.p[i]);
    }
    store_unit<MODE>(FLAT ? static_cast<TY*>(a.y) + 8 * b : row_ptr<TY>(a.y, a.ldy, row) + s.c, s.lo, s.hi, v);
  }
}

template <typename TX, typename TY, bool RES>
const void* pick(RowMode mode, bool flat) {
  return flat               ? (const void*)&k_dropout<TX, TY, RES, kAligned, true>
         : mode == kAligned ? (const void*)&k_dropout<TX, TY, RES, kAligned, false>
         : mode == kShifted ? (const void*)&k_dropout<TX, TY, RES, kShifted, false>
                            : (const void*)&k_dropout<TX, TY, RES, kScalar, false>;
}
template <typename TX, typename TY>
const void* pick(bool res, RowMode mode, bool flat) {
  return res ? pick<TX, TY, true>(mode, flat) : pick<TX, TY, false>(mode, flat);
}

}  // namespace

sf_status make_drop_consts(double p, const sf_rng* rng, DropConsts* out) {
  if (!(p >= 0.0 && p <= 1.0)) return fail(SF_ERR_INVALID, "p must lie in [0, 1] (got %g)", p);
  const uint32_t t = (uint32_t)(p * 65536.0 + 0.5);
  if (t && !rng) return fail(SF_ERR_INVALID, "p > 0 needs a generator (rng is NULL)");
  *out = DropConsts{};
  if (!t) return SF_OK;
  SF_TRY(check_aligned(rng->device_offset, sizeof(uint64_t), "device_offset"));
  uint32_t k0 = (uint32_t)rng->seed, k1 = (uint32_t)(rng->seed >> 32);
  for (int r = 0; r < 10; ++r, k0 += 0x9E3779B9u, k1 += 0xBB67AE85u) {
    out->key[2 * r] = k0;
    out->key[2 * r + 1] = k1;
  }
  out->offset = rng->offset;
  out->device_offset = rng->device_offset;
  out->threshold = t;
  out->factor = t < 65536 ? (float)(65536.0 / (65536.0 - t)) : 0.0f;
  return SF_OK;
}

}  // namespace sf

extern "C" {

sf_status sf_dropout(const sf_matrix* x, const sf_matrix* residual, const sf_matrix* y, double p, const sf_rng* rng,
                     void* stream) {
  using namespace sf;
  clear_error();
  NvtxRange nvtx_range("sf_dropout");
  constexpr unsigned kTypes = 1u << SF_BF16 | 1u << SF_FP32;
  SF_TRY(check_matrix(x, "x", -1, -1, kTypes));
  SF_TRY(check_matrix(y, "y", x->rows, x->cols, kTypes));
  if (residual) {
    SF_TRY(check_matrix(residual, "residual", x->rows, x->cols, kTypes));
    if (residual->dtype != y->dtype) return fail(SF_ERR_INVALID, "residual and y must have one type");
  }
  DropoutArgs a{};
  SF_TRY(make_drop_consts(p, rng, &a.d));
  if (!x->rows || !x->cols) return SF_OK;
  a.x = x->data;
  a.r = residual ? residual->data : nullptr;
  a.y = y->data;
  a.ldx = x->ld;
  a.ldr = residual ? residual->ld : 0;
  a.ldy = y->ld;
  const sf_matrix* const all[3] = {x, residual, y};
  const RowMode mode = row_mode(all, &a.shift);
  auto dense = [&](const sf_matrix* m) { return !m || m->ld == m->cols || m->rows == 1; };
  const bool flat = mode == kAligned && x->cols % 8 == 0 && dense(x) && dense(residual) && dense(y);
  if (!flat && x->cols > INT32_MAX / 2)
    return fail(SF_ERR_UNSUPPORTED, "rows of over 2^30 columns need dense, aligned matrices and a multiple of 8 columns");
  a.cols = (int32_t)std::min<int64_t>(x->cols, INT32_MAX);
  a.counters = ceil_div<int64_t>(x->cols, 8);
  a.per_row = a.counters + (mode == kShifted ? 1 : 0);
  a.units = a.per_row * x->rows;
  while ((int64_t)1 << a.div_shift < a.per_row) ++a.div_shift;
  if (a.div_shift < 32)
    a.div_mul = (uint32_t)((((uint64_t)1 << 32) * (((uint64_t)1 << a.div_shift) - (uint64_t)a.per_row)) / (uint64_t)a.per_row + 1);
  // one unit a thread while that leaves SMs idle, else four loads in flight
  a.per_thread = (int32_t)std::clamp<int64_t>(a.units / ((int64_t)kThreads * sm_count() * 4), 1, kUnits);
  const int64_t grid = ceil_div<int64_t>(a.units, (int64_t)kThreads * a.per_thread);
  if (grid > INT32_MAX) return fail(SF_ERR_UNSUPPORTED, "sizes too large");
  using B = __nv_bfloat16;
  const void* k = x->dtype == SF_BF16
                      ? (y->dtype == SF_BF16 ? pick<B, B>(residual, mode, flat) : pick<B, float>(residual, mode, flat))
                      : (y->dtype == SF_BF16 ? pick<float, B>(residual, mode, flat) : pick<float, float>(residual, mode, flat));
  void* args[] = {&a};
  SF_CUDA_TRY(cudaLaunchKernel(k, dim3((unsigned)grid), dim3(kThreads), args, 0, as_stream(stream)), "launch k_dropout");
  return SF_OK;
}

}  // extern "C"
