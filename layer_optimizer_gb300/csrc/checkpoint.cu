// 8-bit checkpoints of a matrix: written (values and scales in one pass) and
// read back, optionally times a factor per row and a gain per column.
//
// Both move three bytes an element with bf16 on the other side and are bound by HBM.
#include <algorithm>

#include "lanes.cuh"

namespace sf {
namespace {

// Steps a thread holds in registers; of narrow accesses one, whose eight loads
// an operand keep memory busy with more threads.  Loading, two (16384 x 4088 bf16 with
// the norm's factors 69 us; four, of 119 registers, 101; one 87).
template <int LAY>
constexpr int kK = LAY == kUnits ? 4 : 1;
template <int LAY>
constexpr int kLoadK = LAY == kUnits ? 2 : 1;
constexpr int kMaxThreads = 512;

struct CkArgs {
  const void* x;         // store: the matrix; load: unused
  void* y;               // load: the matrix
  int64_t ldx;
  int64_t rows;
  int64_t cols;
  Ck ck;
  int32_t tpr, rpb, steps;      // threads a row, rows a block, segments of tpr * kK * 8 columns a row
  const float* row_factor;
  const void* gain;
  int32_t gain_fp32;
  float gain_offset;
};

// A row's segments of tpr * kK * 8 columns in turn.  One scale a row: of a
// row longer than a segment the maximum is taken first, in a pass of its own.
template <typename T, int LAY>
__global__ void __launch_bounds__(kMaxThreads) k_checkpoint_store(const CkArgs a) {
  __shared__ float red[kMaxThreads / 32];
  const int tpr = a.tpr, lane_row = (int)threadIdx.x / tpr, t = (int)threadIdx.x - lane_row * tpr;
  const int64_t row = (int64_t)blockIdx.x * a.rpb + lane_row;
  const bool on = row < a.rows;
  const Lane l = lane_of<LAY>(t, tpr);
  const int64_t seg = (int64_t)tpr * kK<LAY> * 8;
  const T* x = row_ptr<T>(a.x, a.ldx, on ? row : 0);
  const bool one = a.ck.group_log2 == 0;
  auto left = [&](int64_t s) { return on ? (int)min(a.cols - s * seg, seg) : 0; };      // columns of segment s
  uint32_t code = 1;
  Unit<T> v[kK<LAY>];
  auto load = [&](int64_t s, int n) {
#pragma unroll
    for (int k = 0; k < kK<LAY>; ++k) {
      v[k] = Unit<T>{};
      if (l.c0(k) < n) load_raw<LAY>(x + s * seg, l.c0(k), l.dj, n, v[k]);
    }
  };
  float top[1] = {0.0f};
  if (one) {
    for (int64_t s = 0; s < a.steps; ++s) {
      load(s, left(s));
#pragma unroll
      for (int k = 0; k < kK<LAY>; ++k) top[0] = fmaxf(top[0], top8_finite(unpack(v[k])));
    }
    row_reduce_n<1, 0>(top, tpr, red);
    code = e8m0_of(top[0]);
    if (on && t == 0) a.ck.s8[row] = (uint8_t)code;
  }
  for (int64_t s = 0; s < a.steps; ++s) {
    const int n = left(s);
    if (!one || a.steps > 1) load(s, n);
    Ck ck = a.ck;
    ck.q += s * seg;
    if (!one) ck.s8 += (s * seg) >> ck.group_log2;
#pragma unroll
    for (int k = 0; k < kK<LAY>; ++k) ck_store8<LAY>(ck, row, l.c0(k), l.dj, n, unpack(v[k]), code);
  }
}

template <typename T, int LAY>
__global__ void __launch_bounds__(kMaxThreads) k_checkpoint_load(const CkArgs a) {
  const int tpr = a.tpr, lane_row = (int)threadIdx.x / tpr, t = (int)threadIdx.x - lane_row * tpr;
  const int64_t row = (int64_t)blockIdx.x * a.rpb + lane_row;
  if (row >= a.rows) return;
  const Lane l = lane_of<LAY>(t, tpr);
  const int64_t seg = (int64_t)tpr * kLoadK<LAY> * 8;
  const float f = a.row_factor ? a.row_factor[row] : 1.0f;
  const uint64_t f2 = pack_f2(f, f);
  for (int64_t s = 0; s < a.steps; ++s) {
    const int n = (int)min(a.cols - s * seg, seg);
    Ck ck = a.ck;
    ck.q += s * seg;
    const int64_t at = ck.group_log2 ? (s * seg) >> ck.group_log2 : 0;
    if (ck.s8) ck.s8 += at;
    else ck.s32 += at;
    F8 v[kLoadK<LAY>];
#pragma unroll
    for (int k = 0; k < kLoadK<LAY>; ++k)
      if (l.c0(k) < n) v[k] = load8<LAY>(ck, row, l.c0(k), l.dj, n);
#pragma unroll
    for (int k = 0; k < kLoadK<LAY>; ++k) {
      if (l.c0(k) >= n) continue;
      if (a.row_factor) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[k].p[i] = fmul2(v[k].p[i], f2);
      }
      if (a.gain) {
        const void* g = static_cast<const char*>(a.gain) + s * seg * (a.gain_fp32 ? 4 : 2);
        const F8 w = load_vec<LAY>(g, a.gain_fp32, l.c0(k), l.dj, n, a.gain_offset);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[k].p[i] = fmul2(v[k].p[i], w.p[i]);
      }
      store8<LAY>(row_ptr<T>(a.y, a.ldx, row) + s * seg, l.c0(k), l.dj, n, v[k]);
    }
  }
}

// The wide forms, for rows of whole 16-byte units of values: a thread takes 16
// columns of four rows (fp32 stores: of two), all its loads under way before
// the first is used.
struct WideShape {
  int32_t tx_log2, segs;      // threads across a row's units, blocks across a row
  __device__ __forceinline__ void place(int rows, int64_t* row, int* c) const {
    const int64_t b = blockIdx.x / segs;
    const int seg = (int)(blockIdx.x - b * segs), tx = threadIdx.x & ((1 << tx_log2) - 1);
    *row = (b << (8 - tx_log2)) * rows + (threadIdx.x >> tx_log2);      // the first; the others 256 >> tx_log2 further each
    *c = ((seg << tx_log2) + tx) * 16;
  }
};
constexpr int kWideThreads = 256;

// With scale groups.  bf16 33 us at 16384 x 4096, groups of 128 (6.1 TB/s), bound by HBM.
template <typename T>
__global__ void __launch_bounds__(kWideThreads) k_checkpoint_store_wide(const CkArgs a, const WideShape shape) {
  constexpr int kRows = sizeof(T) == 2 ? 4 : 2;
  int64_t row;
  int c;
  shape.place(kRows, &row, &c);
  const int64_t step = kWideThreads >> shape.tx_log2;
  Wide<T> v[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    v[i] = Wide<T>{};
    if (c < a.cols && row + i * step < a.rows) v[i].load(row_ptr<T>(a.x, a.ldx, row + i * step) + c);
  }
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int64_t r = row + i * step;
    ck_store16(a.ck, r, c, r < a.rows ? (int)a.cols : 0, v[i].half(0), v[i].half(1), v[i].top(), 0, true);
  }
}

// bf16 with the norm's factors 33 us at 16384 x 4096 (6.2 TB/s), bound by HBM.
template <typename T>
__global__ void __launch_bounds__(kWideThreads) k_checkpoint_load_wide(const CkArgs a, const WideShape shape) {
  constexpr int kRows = 4;
  int64_t row;
  int c;
  shape.place(kRows, &row, &c);
  if (c >= a.cols) return;
  const int64_t step = kWideThreads >> shape.tx_log2;
  const int group = a.ck.group_log2 ? c >> a.ck.group_log2 : 0;
  uint4 q[kRows];
  uint32_t s[kRows];
  float f[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i)
    if (row + i * step < a.rows) q[i] = ld_once(a.ck.q + (row + i * step) * a.ck.ld + c);
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int64_t r = min(row + i * step, a.rows - 1);
    s[i] = a.ck.s8 ? a.ck.s8[r * a.ck.n_groups + group] : __float_as_uint(a.ck.s32[r * a.ck.n_groups + group]);
    f[i] = a.row_factor ? a.row_factor[r] : 1.0f;
  }
  F8 g[2];
  if (a.gain) {
#pragma unroll
    for (int h = 0; h < 2; ++h) g[h] = load_vec<kUnits>(a.gain, a.gain_fp32, c + 8 * h, 1, (int)a.cols, a.gain_offset);
  }
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int64_t r = row + i * step;
    if (r >= a.rows) continue;
    const float scale = a.ck.s8 ? e8m0_value(s[i]) : __uint_as_float(s[i]);
    const uint32_t w[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
    F8 o[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      F8 v;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 x = e4m3x2_value(w[2 * h + (e >> 1)] >> (16 * (e & 1)) & 0xffffu);
        v.p[e] = fmul2(pack_f2(x.x, x.y), pack_f2(scale, scale));
        if (a.row_factor) v.p[e] = fmul2(v.p[e], pack_f2(f[i], f[i]));
        if (a.gain) v.p[e] = fmul2(v.p[e], g[h].p[e]);
      }
      o[h] = v;
    }
    store16(row_ptr<T>(a.y, a.ldx, r) + c, o[0], o[1], true);
  }
}

// Rows off their units, a warp for 512 columns of a row: lane, lane + 32, ..,
// at constant distances, all loads under way before the first is used, and
// nothing shared between warps.  16384 x 4095 bf16: stored with groups of 128 in 54 us (3.7
// TB/s; 173 by the form above), loaded with the norm's factors in 68 (152); fp32, with groups
// of 64, stored in 64 (190).
constexpr int kRowWarps = 8;      // neighbouring rows of a block

template <bool WHOLE>
__device__ __forceinline__ void load_chunk(const __nv_bfloat16* p, int left, F8 (&v)[2]) {
  const uint16_t* q = reinterpret_cast<const uint16_t*>(p);
  uint32_t w[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) w[j] = WHOLE || 32 * j < left ? q[32 * j] : 0u;
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j >> 2].p[j & 3] = pack_f2(__uint_as_float(w[2 * j] << 16), __uint_as_float(w[2 * j + 1] << 16));
}
template <bool WHOLE>
__device__ __forceinline__ void load_chunk(const float* p, int left, F8 (&v)[2]) {
  float w[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) w[j] = WHOLE || 32 * j < left ? p[32 * j] : 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j >> 2].p[j & 3] = pack_f2(w[2 * j], w[2 * j + 1]);
}
template <bool WHOLE>
__device__ __forceinline__ void store_chunk(__nv_bfloat16* p, int left, const F8 (&v)[2]) {
  uint16_t* q = reinterpret_cast<uint16_t*>(p);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    Unit<__nv_bfloat16> u;
    pack(v[h], u);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (WHOLE || 32 * (8 * h + j) < left) q[32 * (8 * h + j)] = (uint16_t)(u.w[j >> 1] >> (16 * (j & 1)));
  }
}
template <bool WHOLE>
__device__ __forceinline__ void store_chunk(float* p, int left, const F8 (&v)[2]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float2 x = unpack_f2(v[j >> 2].p[j & 3]);
    if (WHOLE || 64 * j < left) p[64 * j] = x.x;
    if (WHOLE || 64 * j + 32 < left) p[64 * j + 32] = x.y;
  }
}

template <typename T, bool WHOLE>
__device__ __forceinline__ void store_rows_chunk(const CkArgs& a, int64_t row, int c) {
  F8 v[2];
  load_chunk<WHOLE>(row_ptr<T>(a.x, a.ldx, row) + c, (int)a.cols - c, v);
  ck_store16_strided<WHOLE>(a.ck, row, c, (int)a.cols, v, 1);
}
// With scale groups.
template <typename T>
__global__ void __launch_bounds__(32 * kRowWarps) k_checkpoint_store_rows(const CkArgs a, const uint32_t chunks) {
  const uint32_t block = blockIdx.x / chunks, chunk = blockIdx.x - block * chunks;
  const int64_t row = (int64_t)block * kRowWarps + (threadIdx.x >> 5);
  if (row >= a.rows) return;
  const int c = (int)(chunk * 512 + (threadIdx.x & 31));
  if (chunk * 512 + 512 <= a.cols) store_rows_chunk<T, true>(a, row, c);
  else store_rows_chunk<T, false>(a, row, c);
}

// One scale a row: a block for a row of up to 32 warps' columns, held in registers while their
// maximum is joined.  16384 x 4095 bf16 61 us (147 by the form above), fp32 53 (148).
// Not for short rows (60000 x 257 32 us against 53, 65536 x 129 35 against 26).
constexpr int kRowScaleCols = 512 * 32, kRowScaleMin = 192;
template <typename T>
__global__ void __launch_bounds__(1024) k_checkpoint_store_row_scale(const CkArgs a) {
  __shared__ uint32_t red[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = warp * 512 + lane, cols = (int)a.cols;
  const int64_t row = blockIdx.x;
  const T* p = row_ptr<T>(a.x, a.ldx, row) + c;
  const bool whole = warp * 512 + 512 <= cols;
  F8 v[2];
  if (whole) load_chunk<true>(p, 0, v);
  else load_chunk<false>(p, cols - c, v);
  // magnitudes order as their bits
  const uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(fmaxf(top8_finite(v[0]), top8_finite(v[1]))));
  if (lane == 0) red[warp] = top;
  __syncthreads();
  const uint32_t code = e8m0_of(__uint_as_float(__reduce_max_sync(0xffffffffu, lane < blockDim.x >> 5 ? red[lane] : 0u)));
  if (threadIdx.x == 0) a.ck.s8[row] = (uint8_t)code;
  if (whole) ck_store16_strided<true>(a.ck, row, c, cols, v, code);
  else ck_store16_strided<false>(a.ck, row, c, cols, v, code);
}

template <typename T, bool WHOLE>
__device__ __forceinline__ void load_rows_chunk(const CkArgs& a, int64_t row, int c) {
  const int left = (int)a.cols - c, lane = threadIdx.x & 31;
  const uint8_t* p = a.ck.q + row * a.ck.ld + c;
  uint32_t q[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) q[j] = WHOLE || 32 * j < left ? p[32 * j] : 0u;
  // the scale of the lane's block of 32 columns (of lane j: block j)
  const int64_t at = row * a.ck.n_groups + (a.ck.group_log2 ? min((c - lane + 32 * (lane & 15)) >> a.ck.group_log2, a.ck.n_groups - 1) : 0);
  const float mine = a.ck.s8 ? e8m0_value(a.ck.s8[at]) : a.ck.s32[at];
  const float f = a.row_factor ? a.row_factor[row] : 1.0f;
  F8 g[2];
  if (a.gain) {
#pragma unroll
    for (int h = 0; h < 2; ++h) g[h] = load_vec<kStrided>(a.gain, a.gain_fp32, c + 256 * h, 32, (int)a.cols, a.gain_offset);
  }
  F8 v[2];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float2 x = e4m3x2_value(q[2 * j] | q[2 * j + 1] << 8);
    uint64_t y = fmul2(pack_f2(x.x, x.y), pack_f2(__shfl_sync(0xffffffffu, mine, 2 * j), __shfl_sync(0xffffffffu, mine, 2 * j + 1)));
    if (a.row_factor) y = fmul2(y, pack_f2(f, f));
    if (a.gain) y = fmul2(y, g[j >> 2].p[j & 3]);
    v[j >> 2].p[j & 3] = y;
  }
  store_chunk<WHOLE>(row_ptr<T>(a.y, a.ldx, row) + c, left, v);
}
template <typename T>
__global__ void __launch_bounds__(32 * kRowWarps) k_checkpoint_load_rows(const CkArgs a, const uint32_t chunks) {
  const uint32_t block = blockIdx.x / chunks, chunk = blockIdx.x - block * chunks;
  const int64_t row = (int64_t)block * kRowWarps + (threadIdx.x >> 5);
  if (row >= a.rows) return;
  const int c = (int)(chunk * 512 + (threadIdx.x & 31));
  if (chunk * 512 + 512 <= a.cols) load_rows_chunk<T, true>(a, row, c);
  else load_rows_chunk<T, false>(a, row, c);
}

// Threads a row: a power of two up to 64 (at least 16, a group of 128 columns), or whole warps.
void pick_shape(CkArgs& a, int held) {
  const int64_t units = ceil_div<int64_t>(a.cols, 8);
  const int64_t per = a.rows < 2 * sm_count() ? 1 : held;
  const int64_t t = std::min<int64_t>(ceil_div<int64_t>(units, per), kMaxThreads);
  if (t > 64) {
    a.tpr = (int32_t)ceil_div<int64_t>(t, 32) * 32;
    a.rpb = 1;
  } else {
    int p = 16;
    while (p < t) p *= 2;
    a.tpr = p;
    a.rpb = 128 / p;
  }
  a.steps = (int32_t)ceil_div<int64_t>(units, (int64_t)a.tpr * held);
}

template <template <typename, int> class K>
const void* pick_kernel(int32_t dtype, Lay lay) {
  using B = __nv_bfloat16;
  if (dtype == SF_BF16) return lay == kUnits ? K<B, kUnits>::ptr() : K<B, kStrided>::ptr();
  return lay == kUnits ? K<float, kUnits>::ptr() : K<float, kStrided>::ptr();
}
template <typename T, int LAY>
struct Store {
  static const void* ptr() { return (const void*)&k_checkpoint_store<T, LAY>; }
};
template <typename T, int LAY>
struct Load {
  static const void* ptr() { return (const void*)&k_checkpoint_load<T, LAY>; }
};

constexpr unsigned kTypes = 1u << SF_BF16 | 1u << SF_FP32;

sf_status launch_wide(const void* kernel, CkArgs& a, int rows, cudaStream_t stream, const char* what) {
  WideShape s;
  const int64_t units = a.cols / 16;
  s.tx_log2 = 3;      // a group of 128 columns
  while (s.tx_log2 < 8 && (1 << s.tx_log2) < units) ++s.tx_log2;
  s.segs = (int32_t)ceil_div<int64_t>(units, 1 << s.tx_log2);
  const int64_t grid = ceil_div<int64_t>(a.rows, (int64_t)rows * (kWideThreads >> s.tx_log2)) * s.segs;
  if (grid > INT32_MAX) return fail(SF_ERR_UNSUPPORTED, "too many rows");
  void* args[] = {&a, &s};
  SF_CUDA_TRY(cudaLaunchKernel(kernel, dim3((unsigned)grid), dim3(kWideThreads), args, 0, stream), what);
  return SF_OK;
}

sf_status launch(const void* kernel, CkArgs& a, cudaStream_t stream, const char* what) {
  const int64_t grid = ceil_div<int64_t>(a.rows, a.rpb);
  if (grid > INT32_MAX) return fail(SF_ERR_UNSUPPORTED, "too many rows");
  void* args[] = {&a};
  SF_CUDA_TRY(cudaLaunchKernel(kernel, dim3((unsigned)grid), dim3(a.tpr * a.rpb), args, 0, stream), what);
  return SF_OK;
}

// Whether the form for rows off their units takes a call: not short rows, which leave its
// lanes without work (us, so / by the form above; stored and loaded: 65536 x 129 43 / 46
// and 32 / 32, 60000 x 257 40 / 83 and 30 / 57, 200000 x 33 126 / 70 and 93 / 46).
bool takes_rows(const CkArgs& a) {
  return a.cols > 128 && ceil_div<int64_t>(a.rows, kRowWarps) * ceil_div<int64_t>(a.cols, 512) <= INT32_MAX;
}
sf_status launch_rows(const void* kernel, CkArgs& a, cudaStream_t stream, const char* what) {
  uint32_t chunks = (uint32_t)ceil_div<int64_t>(a.cols, 512);
  void* args[] = {&a, &chunks};
  SF_CUDA_TRY(cudaLaunchKernel(kernel, dim3((unsigned)(ceil_div<int64_t>(a.rows, kRowWarps) * chunks)), dim3(32 * kRowWarps), args, 0, stream), what);
  return SF_OK;
}

}  // namespace

sf_status checkpoint_load(const sf_checkpoint* c, const float* row_factor, const void* gain, int32_t gain_dtype,
                          double gain_offset, const sf_matrix* y, cudaStream_t stream) {
  SF_TRY(check_matrix(y, "y", -1, -1, kTypes));
  SF_TRY(check_checkpoint(c, "checkpoint", y->rows, y->cols, false));
  SF_TRY(check_aligned(row_factor, sizeof(float), "row_factor"));
  if (gain) {
    if (gain_dtype != SF_BF16 && gain_dtype != SF_FP32) return fail(SF_ERR_UNSUPPORTED, "gain: type %d is not taken here", (int)gain_dtype);
    SF_TRY(check_aligned(gain, dtype_bytes(gain_dtype), "gain"));
    if (!(gain_offset >= -1e30 && gain_offset <= 1e30)) return fail(SF_ERR_INVALID, "gain_offset must be finite");
  }
  if (y->cols > INT32_MAX / 2) return fail(SF_ERR_UNSUPPORTED, "rows of fewer than 2^30 columns are supported");
  if (!y->rows || !y->cols) return SF_OK;
  CkArgs a{};
  a.y = y->data;
  a.ldx = y->ld;
  a.rows = y->rows;
  a.cols = y->cols;
  a.ck = device_ck(c);
  a.row_factor = row_factor;
  a.gain = gain;
  a.gain_fp32 = gain_dtype == SF_FP32;
  a.gain_offset = (float)gain_offset;
  if (on_wide(y) && on_wide(c) && (!gain || on_units(gain, gain_dtype)))
    return launch_wide(y->dtype == SF_BF16 ? (const void*)&k_checkpoint_load_wide<__nv_bfloat16> : (const void*)&k_checkpoint_load_wide<float>, a, 4, stream,
                       "launch k_checkpoint_load_wide");
  const Lay lay = on_units(y) && on_units(c) && (!gain || on_units(gain, gain_dtype)) ? kUnits : kStrided;
  if (lay == kStrided && takes_rows(a))
    return launch_rows(y->dtype == SF_BF16 ? (const void*)&k_checkpoint_load_rows<__nv_bfloat16> : (const void*)&k_checkpoint_load_rows<float>, a, stream,
                       "launch k_checkpoint_load_rows");
  pick_shape(a, lay == kUnits ? kLoadK<kUnits> : kLoadK<kStrided>);
  return launch(pick_kernel<Load>(y->dtype, lay), a, stream, "launch k_checkpoint_load");
}

}  // namespace sf

extern "C" {

sf_status sf_checkpoint_store(const sf_matrix* x, const sf_checkpoint* out, void* stream) {
  using namespace sf;
  clear_error();
  NvtxRange nvtx_range("sf_checkpoint_store");
  SF_TRY(check_matrix(x, "x", -1, -1, kTypes));
  SF_TRY(check_checkpoint(out, "checkpoint", x->rows, x->cols, true));
  if (x->cols > INT32_MAX / 2) return fail(SF_ERR_UNSUPPORTED, "rows of fewer than 2^30 columns are supported");
  if (!x->rows || !x->cols) return SF_OK;
  CkArgs a{};
  a.x = x->data;
  a.ldx = x->ld;
  a.rows = x->rows;
  a.cols = x->cols;
  a.ck = device_ck(out);
  if (out->group && on_wide(x) && on_wide(out))
    return launch_wide(x->dtype == SF_BF16 ? (const void*)&k_checkpoint_store_wide<__nv_bfloat16> : (const void*)&k_checkpoint_store_wide<float>, a,
                       x->dtype == SF_BF16 ? 4 : 2, as_stream(stream), "launch k_checkpoint_store_wide");
  const Lay lay = on_units(x) && on_units(out) ? kUnits : kStrided;
  if (lay == kStrided && !out->group && a.cols >= kRowScaleMin && a.cols <= kRowScaleCols && a.rows <= INT32_MAX) {
    const void* kernel = x->dtype == SF_BF16 ? (const void*)&k_checkpoint_store_row_scale<__nv_bfloat16> : (const void*)&k_checkpoint_store_row_scale<float>;
    void* args[] = {&a};
    SF_CUDA_TRY(cudaLaunchKernel(kernel, dim3((unsigned)a.rows), dim3(32 * (unsigned)ceil_div<int64_t>(a.cols, 512)), args, 0, as_stream(stream)),
                "launch k_checkpoint_store_row_scale");
    return SF_OK;
  }
  if (lay == kStrided && out->group && takes_rows(a))
    return launch_rows(x->dtype == SF_BF16 ? (const void*)&k_checkpoint_store_rows<__nv_bfloat16> : (const void*)&k_checkpoint_store_rows<float>, a,
                       as_stream(stream), "launch k_checkpoint_store_rows");
  pick_shape(a, lay == kUnits ? kK<kUnits> : kK<kStrided>);
  return launch(pick_kernel<Store>(x->dtype, lay), a, as_stream(stream), "launch k_checkpoint_store");
}

sf_status sf_checkpoint_load(const sf_checkpoint* c, const float* row_factor, const void* gain, sf_dtype gain_dtype,
                             double gain_offset, const sf_matrix* y, void* stream) {
  sf::clear_error();
  sf::NvtxRange nvtx_range("sf_checkpoint_load");
  return sf::checkpoint_load(c, row_factor, gain, gain_dtype, gain_offset, y, sf::as_stream(stream));
}

}  // extern "C"
