// Dropout with the residual's addition, from a counter-based generator:
//   y = r + m o x f,   m_ij = [bits_ij >= t],  f = 65536 / (65536 - t)
// The mask is a function of (seed, offset, row, column), so it is computed
// where it is used and never stored: the backward pass is the same call on
// the gradient, and the norm kernels apply the same mask inside their pass.
//
// Elementwise, one read of x (and r) and one write of y; bound by HBM where
// the 2.5 wide multiplications an element that the generator costs stay
// below the multiplier's rate.
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
  int64_t units;        // rows * units_per_row
  int64_t per_row;      // units per row
  int64_t cols;
  int32_t per_thread;   // units a thread takes, 1..kUnits
  DropConsts d;
};

// A block takes per_thread * 256 consecutive units.  FLAT: dense rows of whole
// units, so a unit's place follows from its index; otherwise one division a
// unit finds its row.
template <typename TX, typename TY, bool RES, bool VEC, bool FLAT>
__global__ void __launch_bounds__(kThreads) k_dropout(const DropoutArgs a) {
  const DropWords words = drop_words(a.d);
  const int64_t b0 = (int64_t)blockIdx.x * (a.per_thread * kThreads) + threadIdx.x;
  Unit<TX> x[kUnits];
  Unit<TY> r[kUnits];
  // the unit's row and first column; columns of it (0 past the end)
  auto place = [&](int k, int64_t& row, int64_t& c) {
    const int64_t b = b0 + k * kThreads;
    if (k >= a.per_thread || b >= a.units) return 0;
    if (FLAT) {
      row = 0;
      c = 8 * b;
      return 8;
    }
    row = a.units <= INT32_MAX ? (int64_t)((uint32_t)b / (uint32_t)a.per_row) : b / a.per_row;
    c = 8 * (b - row * a.per_row);
    return (int)min((int64_t)8, a.cols - c);
  };
#pragma unroll
  for (int k = 0; k < kUnits; ++k) {
    int64_t row, c;
    const int n = place(k, row, c);
    if (!n) continue;
    load_unit<VEC>(row_ptr<TX>(a.x, a.ldx, row) + c, n, x[k]);
    if (RES) load_unit<VEC>(row_ptr<TY>(a.r, a.ldr, row) + c, n, r[k]);
  }
#pragma unroll
  for (int k = 0; k < kUnits; ++k) {
    int64_t row, c;
    const int n = place(k, row, c);
    if (!n) continue;
    F8 v = unpack(x[k]);
    if (a.d.threshold) drop_unit(v, (uint64_t)(b0 + k * kThreads), words, a.d);
    if (RES) {
      const F8 w = unpack(r[k]);
#pragma unroll
      for (int i = 0; i < 4; ++i) v.p[i] = add2(v.p[i], w.p[i]);
    }
    store_unit<VEC>(row_ptr<TY>(a.y, a.ldy, row) + c, n, v);
  }
}

template <typename TX, typename TY, bool RES>
const void* pick(bool vec, bool flat) {
  return flat  ? (const void*)&k_dropout<TX, TY, RES, true, true>
         : vec ? (const void*)&k_dropout<TX, TY, RES, true, false>
               : (const void*)&k_dropout<TX, TY, RES, false, false>;
}
template <typename TX, typename TY>
const void* pick(bool res, bool vec, bool flat) {
  return res ? pick<TX, TY, true>(vec, flat) : pick<TX, TY, false>(vec, flat);
}

}  // namespace

sf_status make_drop_consts(double p, const sf_rng* rng, DropConsts* out) {
  if (!(p >= 0.0 && p <= 1.0)) return fail(SF_ERR_INVALID, "p must lie in [0, 1] (got %g)", p);
  const uint32_t t = (uint32_t)(p * 65536.0 + 0.5);
  if (t && !rng) return fail(SF_ERR_INVALID, "p > 0 needs a generator (rng is NULL)");
  *out = DropConsts{};
  if (!t) return SF_OK;
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
  a.cols = x->cols;
  a.per_row = ceil_div<int64_t>(x->cols, 8);
  a.units = a.per_row * x->rows;
  const bool vec = units_aligned(x) && units_aligned(residual) && units_aligned(y);
  auto dense = [&](const sf_matrix* m) { return !m || m->ld == m->cols || m->rows == 1; };
  const bool flat = vec && x->cols % 8 == 0 && dense(x) && dense(residual) && dense(y);
  // one unit a thread while that leaves SMs idle, else four loads in flight
  a.per_thread = (int32_t)std::clamp<int64_t>(a.units / ((int64_t)kThreads * sm_count() * 4), 1, kUnits);
  const int64_t grid = ceil_div<int64_t>(a.units, (int64_t)kThreads * a.per_thread);
  if (grid > INT32_MAX) return fail(SF_ERR_UNSUPPORTED, "sizes too large");
  using B = __nv_bfloat16;
  const void* k = x->dtype == SF_BF16
                      ? (y->dtype == SF_BF16 ? pick<B, B>(residual, vec, flat) : pick<B, float>(residual, vec, flat))
                      : (y->dtype == SF_BF16 ? pick<float, B>(residual, vec, flat) : pick<float, float>(residual, vec, flat));
  void* args[] = {&a};
  SF_CUDA_TRY(cudaLaunchKernel(k, dim3((unsigned)grid), dim3(kThreads), args, 0, as_stream(stream)), "launch k_dropout");
  return SF_OK;
}

}  // extern "C"
