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
  int64_t step_rows, step_units;   // the grid's stride as rows and units of a row
  DropConsts d;
};

template <typename TX, typename TY, bool RES, bool VEC>
__global__ void __launch_bounds__(kThreads) k_dropout(const DropoutArgs a) {
  const DropKey key = drop_key(a.d);
  const int64_t stride = (int64_t)gridDim.x * kThreads;
  int64_t b = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  int64_t row = b / a.per_row, u = b - row * a.per_row;
  while (b < a.units) {
    Unit<TX> x[kUnits];
    Unit<TY> r[kUnits];
    int64_t rows[kUnits], cols[kUnits], at[kUnits];
    int n[kUnits];
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
      at[k] = b;
      rows[k] = row;
      cols[k] = 8 * u;
      n[k] = b < a.units ? (int)min((int64_t)8, a.cols - 8 * u) : 0;
      if (n[k]) {
        load_unit<VEC>(row_ptr<TX>(a.x, a.ldx, row) + 8 * u, n[k], x[k]);
        if (RES) load_unit<VEC>(row_ptr<TY>(a.r, a.ldr, row) + 8 * u, n[k], r[k]);
      }
      // the next unit of this thread, without a division
      b += stride;
      row += a.step_rows;
      u += a.step_units;
      if (u >= a.per_row) {
        u -= a.per_row;
        ++row;
      }
    }
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
      if (!n[k]) continue;
      float v[8];
      unpack(x[k], v);
      if (a.d.threshold) drop_unit(v, (uint64_t)at[k], key, a.d.threshold, a.d.factor);
      if (RES) {
        float w[8];
        unpack(r[k], w);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += w[i];
      }
      store_unit<VEC>(row_ptr<TY>(a.y, a.ldy, rows[k]) + cols[k], n[k], v);
    }
  }
}

template <typename TX, typename TY>
const void* pick(bool res, bool vec) {
  if (res) return vec ? (const void*)&k_dropout<TX, TY, true, true> : (const void*)&k_dropout<TX, TY, true, false>;
  return vec ? (const void*)&k_dropout<TX, TY, false, true> : (const void*)&k_dropout<TX, TY, false, false>;
}

}  // namespace

sf_status make_drop_consts(double p, const sf_rng* rng, DropConsts* out) {
  if (!(p >= 0.0 && p <= 1.0)) return fail(SF_ERR_INVALID, "p must lie in [0, 1] (got %g)", p);
  const uint32_t t = (uint32_t)(p * 65536.0 + 0.5);
  if (t && !rng) return fail(SF_ERR_INVALID, "p > 0 needs a generator (rng is NULL)");
  *out = DropConsts{};
  if (!t) return SF_OK;
  out->seed = rng->seed;
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
  const int64_t want = ceil_div<int64_t>(a.units, (int64_t)kThreads * kUnits);
  // one unit a thread while that leaves SMs idle, then up to eight resident blocks an SM
  const int64_t most = (int64_t)sm_count() * 8;
  const int64_t grid = want > most ? most : std::min(ceil_div<int64_t>(a.units, kThreads), most);
  const int64_t stride = grid * kThreads;
  a.step_rows = stride / a.per_row;
  a.step_units = stride % a.per_row;
  const void* k = x->dtype == SF_BF16
                      ? (y->dtype == SF_BF16 ? pick<__nv_bfloat16, __nv_bfloat16>(residual, vec)
                                             : pick<__nv_bfloat16, float>(residual, vec))
                      : (y->dtype == SF_BF16 ? pick<float, __nv_bfloat16>(residual, vec) : pick<float, float>(residual, vec));
  void* args[] = {&a};
  SF_CUDA_TRY(cudaLaunchKernel(k, dim3((unsigned)grid), dim3(kThreads), args, 0, as_stream(stream)), "launch k_dropout");
  return SF_OK;
}

}  // extern "C"
