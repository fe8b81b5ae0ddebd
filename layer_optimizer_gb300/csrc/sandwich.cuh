// What the two passes of the end of a residual block share: the call's vectors,
// rows in shared memory, checks of arguments.  The forward pass is in
// sandwich_fwd.cu, the backward pass in sandwich_bwd.cu and (its staged form)
// sandwich_bwd_ring.cuh.
#pragma once

#include <algorithm>

#include "lanes.cuh"
#include "ptx.cuh"

namespace sf {
namespace {

constexpr int kMaxStages = 8;
constexpr int64_t kMaxCols = 16384;
constexpr size_t kSmemPerSm = 224 << 10, kSmemBlock = 2 << 10;      // a block's static and reserved shared memory
constexpr size_t kSmemScales = 6 << 10;        // of three rows


constexpr unsigned kTypes = 1u << SF_BF16 | 1u << SF_FP32;

// What both passes take of a call.
struct Vectors {
  const void* g_post;      // may be null
  const void* g_pre;       // may be null
  const void* gate;        // may be null
  int64_t ld_gate, span;
  int32_t gain_fp32, gate_fp32;
  float offset, a, b;      // gain offset, residual and block scales
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

// Row `row` of a matrix with fewer than 2^31 rows and columns between rows: one
// 32 x 32 -> 64 bit multiplication instead of a 64-bit one.
template <typename T>
__device__ __forceinline__ T* short_row(void* base, int64_t ld, uint32_t row) {
  return static_cast<T*>(base) + (uint64_t)row * (uint32_t)ld;
}
template <typename T>
__device__ __forceinline__ const T* short_row(const void* base, int64_t ld, uint32_t row) {
  return static_cast<const T*>(base) + (uint64_t)row * (uint32_t)ld;
}

// Host side: whether short_row() does for `m` (null passes).
inline bool short_ld(const sf_matrix* m) { return !m || m->ld < (int64_t)1 << 31; }

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
// Whether all 512 columns of a warp in the second lay are the row's (the same for the warp).
__device__ __forceinline__ bool whole512(int c0, int cols) { return (c0 | 31) + 480 < cols; }

// From shared memory, at the address of column 0 (c0 below cols; strided
// columns past it read as zero); in the first lay kept as stored until used.
template <typename T, int LAY>
struct Lds16;
template <typename T>
struct Lds16<T, kUnits> : LdsWide<T> {
  __device__ __forceinline__ Lds16(uint32_t p, int c0, int) : LdsWide<T>(p + c0 * (uint32_t)sizeof(T)) {}
};
template <typename T>
struct Lds16<T, kStrided> {
  F8 v[2];
  __device__ __forceinline__ Lds16(uint32_t p, int c0, int cols) {
    float x[16];
    const uint32_t at = p + c0 * (uint32_t)sizeof(T);
    if (whole512(c0, cols)) {
#pragma unroll
      for (int e = 0; e < 16; ++e) x[e] = lds_value(at + 32 * e * (uint32_t)sizeof(T), T());
    } else {
#pragma unroll
      for (int e = 0; e < 16; ++e) x[e] = c0 + 32 * e < cols ? lds_value(at + 32 * e * (uint32_t)sizeof(T), T()) : 0.0f;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e >> 2].p[e & 3] = pack_f2(x[2 * e], x[2 * e + 1]);
  }
  __device__ __forceinline__ F8 half(int h) const { return v[h]; }
};
template <typename T, int LAY>
__device__ __forceinline__ void lds16(uint32_t p, int c0, int cols, F8 (&v)[2]) {
  const Lds16<T, LAY> u(p, c0, cols);
  v[0] = u.half(0), v[1] = u.half(1);
}
__device__ __forceinline__ void put8_strided(__nv_bfloat16* p, const F8& v) {
  Unit<__nv_bfloat16> u;
  pack(v, u);
  uint16_t* q = reinterpret_cast<uint16_t*>(p);
#pragma unroll
  for (int j = 0; j < 8; ++j) q[32 * j] = (uint16_t)(u.w[j >> 1] >> (16 * (j & 1)));
}
__device__ __forceinline__ void put8_strided(float* p, const F8& v) {
  Unit<float> u;
  pack(v, u);
#pragma unroll
  for (int j = 0; j < 8; ++j) p[32 * j] = u.f[j];
}
template <typename T, int LAY>
__device__ __forceinline__ void put16(T* row, int c0, int cols, const F8& lo, const F8& hi, bool wide) {
  if constexpr (LAY == kUnits) {
    store16(row + c0, lo, hi, wide);
  } else {
    if (whole512(c0, cols)) {
      put8_strided(row + c0, lo);
      put8_strided(row + c0 + 256, hi);
    } else {
      store8<kStrided>(row, c0, 32, cols, lo);
      store8<kStrided>(row, c0 + 256, 32, cols, hi);
    }
  }
}
template <int LAY>
__device__ __forceinline__ void vec16(const void* p, int fp32, int c0, int cols, float add, F8 (&v)[2]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) v[h] = load_vec<LAY>(p, fp32, c0 + (LAY == kUnits ? 8 : 256) * h, LAY == kUnits ? 1 : 32, cols, add);
}

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
inline sf_status check_vector(const void* v, int32_t dtype, const char* name) {
  if (!v) return SF_OK;
  if (dtype != SF_BF16 && dtype != SF_FP32) return fail(SF_ERR_UNSUPPORTED, "%s: type %d is not taken here", name, (int)dtype);
  return check_aligned(v, dtype_bytes(dtype), name);
}

// The configuration and the vectors that both passes share.
inline sf_status check_common(const sf_sandwich* p, int64_t rows, int64_t cols, const void* gain_post, const void* gain_pre,
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
}  // namespace sf
