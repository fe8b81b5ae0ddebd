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
// h) for about 20 instructions.  The norm is taken of s in fp32, before s is
// rounded to its stored type, so storing s in bf16 costs h no precision; the
// backward pass uses the stored s.
#include <cuda_fp8.h>

#include <algorithm>

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
  int32_t tpr_log2;
  int32_t gain_fp32;
  int32_t group_lanes;   // lanes (units) of a scale group; 0: one scale a row
  int32_t n_groups;
  float eps, inv_cols;
  DropConsts d;
};

// Eight gains from column c on (served by L1 after a row or two).
__device__ __forceinline__ void load_gain(const void* g, int fp32, int64_t c, int n, float (&v)[8]) {
  if (fp32) {
    const float* p = static_cast<const float*>(g) + c;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? __ldg(p + i) : 0.0f;
  } else {
    const uint16_t* p = static_cast<const uint16_t*>(g) + c;
    if (n == 8 && (reinterpret_cast<uintptr_t>(p) & 15u) == 0) {
      const uint4 w = __ldg(reinterpret_cast<const uint4*>(p));
      const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(u[i] << 16);
        v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = i < n ? __uint_as_float((uint32_t)__ldg(p + i) << 16) : 0.0f;
    }
  }
}

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
  const int warp = threadIdx.x >> 5, n = tpr >> 5, first = warp & ~(n - 1);
  if ((threadIdx.x & 31) == 0) red[warp] = v;
  __syncthreads();
  float t = red[first];
  for (int i = 1; i < n; ++i) t = MAX ? max_nan(t, red[first + i]) : t + red[first + i];
  return t;
}

__device__ __forceinline__ float group_scale(float amax) { return max_nan(__fdiv_rn(amax, 448.0f), 1.17549435e-38f); }

template <typename TA, typename TS, bool VEC>
__global__ void __launch_bounds__(kMaxThreads) k_add_rmsnorm_fwd(const FwdArgs a) {
  __shared__ float red[2][kMaxThreads / 32];
  const int tpr = 1 << a.tpr_log2, t = threadIdx.x & (tpr - 1);
  const int64_t row = (int64_t)blockIdx.x * (blockDim.x >> a.tpr_log2) + (threadIdx.x >> a.tpr_log2);
  const bool on = row < a.rows;
  int n[kK];
  float s[kK][8];
  {
    Unit<TA> x[kK];
    Unit<TS> r[kK];
#pragma unroll
    for (int k = 0; k < kK; ++k) {
      const int c = 8 * (t + k * tpr);
      n[k] = on ? max(0, min(8, a.cols - c)) : 0;
      if (n[k]) {
        load_unit<VEC>(row_ptr<TA>(a.x, a.ldx, row) + c, n[k], x[k]);
        if (a.r) load_unit<VEC>(row_ptr<TS>(a.r, a.ldr, row) + c, n[k], r[k]);
      }
    }
    const DropKey key = a.d.threshold ? drop_key(a.d) : DropKey{};
#pragma unroll
    for (int k = 0; k < kK; ++k) {
#pragma unroll
      for (int i = 0; i < 8; ++i) s[k][i] = 0.0f;
      if (!n[k]) continue;
      unpack(x[k], s[k]);
      if (a.d.threshold)
        drop_unit(s[k], (uint64_t)(row * a.per_row + t + k * tpr), key, a.d.threshold, a.d.factor);
      if (a.r) {
        float w[8];
        unpack(r[k], w);
#pragma unroll
        for (int i = 0; i < 8; ++i) s[k][i] += w[i];
      }
    }
  }
  float sum = 0.0f;
#pragma unroll
  for (int k = 0; k < kK; ++k) {
    const int c = 8 * (t + k * tpr);
    if (a.s && n[k]) store_unit<VEC>(row_ptr<TS>(a.s, a.lds, row) + c, n[k], s[k]);
#pragma unroll
    for (int i = 0; i < 8; ++i) sum = fmaf(s[k][i], s[k][i], sum);
  }
  sum = row_reduce<false>(sum, tpr, red[0]);
  const float rstd = rsqrtf(fmaf(sum, a.inv_cols, a.eps));
  if (a.rstd && on && t == 0) a.rstd[row] = rstd;
  float amax = 0.0f;
#pragma unroll
  for (int k = 0; k < kK; ++k) {
    const int c = 8 * (t + k * tpr);
    if (n[k]) {
      float g[8];
      load_gain(a.gain, a.gain_fp32, c, n[k], g);
#pragma unroll
      for (int i = 0; i < 8; ++i) s[k][i] = s[k][i] * rstd * g[i];
      if (a.h) store_unit<VEC>(row_ptr<TA>(a.h, a.ldh, row) + c, n[k], s[k]);
    }
    if (a.q) {
      float m = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) m = max_nan(m, fabsf(i < n[k] ? s[k][i] : 0.0f));
      amax = max_nan(amax, m);
      if (a.group_lanes) {
        for (int o = a.group_lanes >> 1; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
        const float sc = group_scale(m), inv = __fdiv_rn(1.0f, sc);
        if (n[k]) {
          if ((t & (a.group_lanes - 1)) == 0) a.scale[row * a.n_groups + (t + k * tpr) / a.group_lanes] = sc;
#pragma unroll
          for (int i = 0; i < 8; ++i) s[k][i] *= inv;
        }
      }
    }
  }
  if (!a.q) return;
  if (!a.group_lanes) {
    amax = row_reduce<true>(amax, tpr, red[1]);
    const float sc = group_scale(amax), inv = __fdiv_rn(1.0f, sc);
    if (on && t == 0) a.scale[row] = sc;
#pragma unroll
    for (int k = 0; k < kK; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) s[k][i] *= inv;
  }
#pragma unroll
  for (int k = 0; k < kK; ++k) {
    if (!n[k]) continue;
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      // saturating, so |h| / scale just above 448 by rounding stays 448
      const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(s[k][4 * i], s[k][4 * i + 1]), __NV_SATFINITE, __NV_E4M3);
      const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(s[k][4 * i + 2], s[k][4 * i + 3]), __NV_SATFINITE, __NV_E4M3);
      w[i] = lo | hi << 16;
    }
    uint8_t* p = row_ptr<uint8_t>(a.q, a.ldq, row) + 8 * (t + k * tpr);
    if (VEC && n[k] == 8) {
      *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n[k]) p[i] = (uint8_t)(w[i >> 2] >> (8 * (i & 3)));
    }
  }
}

// Backward.  With n_j = s_j rstd, the gradients are
//   ds_j = dsum_j + rstd (dh_j g_j - n_j mean_i(dh_i g_i n_i))
//   dresidual = ds,  dx = m o ds f (the forward mask),  dg_j = sum_rows dh_j n_j
// A persistent grid walks the rows; a thread keeps its columns' share of dg
// in registers over all its rows, so dg costs one partial row per block and a
// second small kernel, summed in block order (no atomics).
struct BwdArgs {
  const void* dh;
  const void* s;
  const void* dsum;     // may be null
  const void* gain;
  const float* rstd;
  void* dr;             // may be null
  void* dx;             // may be null
  float* part;          // [grid][cols], null without dg
  int64_t lddh, lds, lddsum, lddr, lddx;
  int64_t rows;
  int32_t cols, per_row;
  int32_t tpr_log2;
  int32_t gain_fp32;
  float inv_cols;
  DropConsts d;
};

template <typename TA, typename TS, bool VEC>
__global__ void __launch_bounds__(kMaxThreads) k_add_rmsnorm_bwd(const BwdArgs a) {
  __shared__ float red[2][kMaxThreads / 32];
  extern __shared__ float comb[];      // [rows of a block][cols], only with several rows a block
  const int tpr = 1 << a.tpr_log2, t = threadIdx.x & (tpr - 1), rpb = blockDim.x >> a.tpr_log2;
  const int lane_row = threadIdx.x >> a.tpr_log2;
  const DropKey key = a.d.threshold ? drop_key(a.d) : DropKey{};
  float acc[kK][8];
#pragma unroll
  for (int k = 0; k < kK; ++k)
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[k][i] = 0.0f;
  int parity = 0;
  for (int64_t base = (int64_t)blockIdx.x * rpb; base < a.rows; base += (int64_t)gridDim.x * rpb, parity ^= 1) {
    const int64_t row = base + lane_row;
    const bool on = row < a.rows;
    Unit<TA> dh[kK];
    Unit<TS> s[kK], ds[kK];
    int n[kK];
#pragma unroll
    for (int k = 0; k < kK; ++k) {
      const int c = 8 * (t + k * tpr);
      n[k] = on ? max(0, min(8, a.cols - c)) : 0;
      if (n[k]) {
        load_unit<VEC>(row_ptr<TA>(a.dh, a.lddh, row) + c, n[k], dh[k]);
        load_unit<VEC>(row_ptr<TS>(a.s, a.lds, row) + c, n[k], s[k]);
        if (a.dsum) load_unit<VEC>(row_ptr<TS>(a.dsum, a.lddsum, row) + c, n[k], ds[k]);
      }
    }
    const float rstd = on ? a.rstd[row] : 0.0f;
    float dot = 0.0f;
#pragma unroll
    for (int k = 0; k < kK; ++k) {
      if (!n[k]) continue;
      float u[8], v[8], g[8];
      unpack(dh[k], u);
      unpack(s[k], v);
      load_gain(a.gain, a.gain_fp32, 8 * (t + k * tpr), n[k], g);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float w = u[i] * (v[i] * rstd);
        acc[k][i] += w;
        dot = fmaf(w, g[i], dot);
      }
    }
    // two alternating buffers: the next row's write cannot meet this row's reads
    dot = row_reduce<false>(dot, tpr, red[parity]);
    const float mean = dot * a.inv_cols;
#pragma unroll
    for (int k = 0; k < kK; ++k) {
      if (!n[k]) continue;
      const int c = 8 * (t + k * tpr);
      float u[8], v[8], g[8];
      unpack(dh[k], u);
      unpack(s[k], v);
      load_gain(a.gain, a.gain_fp32, c, n[k], g);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = rstd * (u[i] * g[i] - (v[i] * rstd) * mean);
      if (a.dsum) {
        unpack(ds[k], u);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += u[i];
      }
      if (a.dr) store_unit<VEC>(row_ptr<TS>(a.dr, a.lddr, row) + c, n[k], v);
      if (a.dx) {
        if (a.d.threshold)
          drop_unit(v, (uint64_t)(row * a.per_row + t + k * tpr), key, a.d.threshold, a.d.factor);
        store_unit<VEC>(row_ptr<TA>(a.dx, a.lddx, row) + c, n[k], v);
      }
    }
  }
  if (!a.part) return;
  float* part = a.part + (int64_t)blockIdx.x * a.cols;
  if (rpb == 1) {
#pragma unroll
    for (int k = 0; k < kK; ++k) {
      const int c = 8 * (t + k * tpr);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (c + i < a.cols) part[c + i] = acc[k][i];
    }
    return;
  }
#pragma unroll
  for (int k = 0; k < kK; ++k) {
    const int c = 8 * (t + k * tpr);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < a.cols) comb[lane_row * a.cols + c + i] = acc[k][i];
  }
  __syncthreads();
  for (int c = threadIdx.x; c < a.cols; c += blockDim.x) {
    float v = 0.0f;
    for (int r = 0; r < rpb; ++r) v += comb[r * a.cols + c];
    part[c] = v;
  }
}

// dg[c] = sum over the blocks' partial rows: 32 columns a block, 32 threads a
// column, each over every 32nd partial, then a tree.
__global__ void __launch_bounds__(1024) k_sum_partials(const float* __restrict__ part, int n_parts, int cols,
                                                       void* __restrict__ out, int out_fp32) {
  __shared__ float red[32][33];
  const int c = blockIdx.x * 32 + threadIdx.x;
  float v = 0.0f;
  if (c < cols)
    for (int p = threadIdx.y; p < n_parts; p += 32) v += part[(int64_t)p * cols + c];
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
// without work, one unit a thread.
int pick_tpr_log2(int64_t rows, int64_t per_row, bool groups) {
  int l = groups ? 4 : 2;
  while (((int64_t)kK << l) < per_row) ++l;
  while (rows < 2 * sm_count() && ((int64_t)1 << l) < per_row && l < 9) ++l;
  return l;
}

constexpr int kMaxParts = 1024;   // blocks of the backward kernel, and so partial rows of dg
constexpr unsigned kTypes = 1u << SF_BF16 | 1u << SF_FP32;

template <template <typename, typename, bool> class K>
const void* pick(int32_t ta, int32_t ts, bool vec) {
  using B = __nv_bfloat16;
  if (ta == SF_BF16)
    return ts == SF_BF16 ? (vec ? K<B, B, true>::ptr() : K<B, B, false>::ptr())
                         : (vec ? K<B, float, true>::ptr() : K<B, float, false>::ptr());
  return ts == SF_BF16 ? (vec ? K<float, B, true>::ptr() : K<float, B, false>::ptr())
                       : (vec ? K<float, float, true>::ptr() : K<float, float, false>::ptr());
}
template <typename TA, typename TS, bool VEC>
struct Fwd {
  static const void* ptr() { return (const void*)&k_add_rmsnorm_fwd<TA, TS, VEC>; }
};
template <typename TA, typename TS, bool VEC>
struct Bwd {
  static const void* ptr() { return (const void*)&k_add_rmsnorm_bwd<TA, TS, VEC>; }
};

sf_status check_gain(const void* gain, int32_t dtype, const char* name) {
  if (!gain) return fail(SF_ERR_INVALID, "%s is NULL", name);
  if (dtype != SF_BF16 && dtype != SF_FP32) return fail(SF_ERR_UNSUPPORTED, "%s: type %d is not taken here", name, (int)dtype);
  if (reinterpret_cast<uintptr_t>(gain) % dtype_bytes(dtype)) return fail(SF_ERR_INVALID, "%s is not aligned to its type", name);
  return SF_OK;
}

sf_status check_cols(int64_t cols) {
  if (cols < 1) return fail(SF_ERR_INVALID, "a row needs at least one column");
  if (cols > kMaxCols) return fail(SF_ERR_UNSUPPORTED, "rows of up to %lld columns are supported (got %lld)", (long long)kMaxCols, (long long)cols);
  return SF_OK;
}

}  // namespace
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
  }
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
  a.group_lanes = group / 8;
  a.n_groups = group ? (int32_t)ceil_div<int64_t>(cols, group) : 1;
  a.eps = (float)eps;
  a.inv_cols = (float)(1.0 / (double)cols);
  a.tpr_log2 = pick_tpr_log2(rows, a.per_row, h8 != nullptr);
  const int threads = std::max(128, 1 << a.tpr_log2);
  const int64_t grid = ceil_div<int64_t>(rows, threads >> a.tpr_log2);
  if (grid > INT32_MAX) return fail(SF_ERR_UNSUPPORTED, "too many rows");
  const bool vec = units_aligned(x) && units_aligned(residual) && units_aligned(sum) && units_aligned(h) && units_aligned(h8);
  const int32_t ts = residual ? residual->dtype : sum ? sum->dtype : x->dtype;
  void* args[] = {&a};
  SF_CUDA_TRY(cudaLaunchKernel(pick<Fwd>(x->dtype, ts, vec), dim3((unsigned)grid), dim3(threads), args, 0, as_stream(stream)),
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
  a.tpr_log2 = pick_tpr_log2(rows, a.per_row, false);
  const int threads = std::max(128, 1 << a.tpr_log2), rpb = threads >> a.tpr_log2;
  const int64_t blocks = ceil_div<int64_t>(rows, rpb);
  const int64_t resident = (int64_t)sm_count() * std::max(1, 512 / threads);
  const int64_t grid = std::min({blocks, resident, (int64_t)kMaxParts});
  const size_t smem = dgain && rpb > 1 ? (size_t)rpb * cols * sizeof(float) : 0;   // <= 16 KB: rpb * cols <= 4096
  const bool vec = units_aligned(dh) && units_aligned(sum) && units_aligned(dsum) && units_aligned(dresidual) && units_aligned(dx);
  cudaStream_t st = as_stream(stream);
  if (grid) {
    void* args[] = {&a};
    SF_CUDA_TRY(cudaLaunchKernel(pick<Bwd>(dh->dtype, sum->dtype, vec), dim3((unsigned)grid), dim3(threads), args, smem, st),
                "launch k_add_rmsnorm_bwd");
  }
  if (dgain) {
    k_sum_partials<<<(unsigned)ceil_div<int64_t>(cols, 32), dim3(32, 32), 0, st>>>(a.part, (int)grid, (int)cols, dgain,
                                                                                  dgain_dtype == SF_FP32);
    SF_TRY(check_launch("k_sum_partials"));
  }
  return SF_OK;
}

}  // extern "C"
