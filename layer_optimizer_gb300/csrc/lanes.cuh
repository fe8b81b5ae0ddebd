// How the threads of a row share its columns, for the kernels around a
// residual block and its 8-bit checkpoints: eight columns a thread and step,
// in one of two lays.
//
//   kUnits    column c0 + j: eight neighbouring columns, one wide access (16
//             bytes in bf16, 32 in fp32, 8 in e4m3).  Needs every row to start
//             on such a unit.
//   kStrided  column c0 + j w of a chunk of 8 w columns, w neighbouring lanes
//             (32, or a shorter row's threads) taking neighbouring columns:
//             narrow accesses, but each a contiguous run of w elements, so any
//             alignment and row length reads whole sectors.
//
// A scale group (32, 64 or 128 columns) lies within group / 8 neighbouring
// lanes in the first lay and within one chunk in the second (or is the whole
// of a shorter row).
#pragma once

#include <cuda_fp8.h>

#include "rows.cuh"

namespace sf {

enum Lay : int { kUnits = 0, kStrided = 1 };

// A thread's columns at step k: c0 + j dj for j = 0..7, those below cols.
struct Lane {
  int first, step, dj;
  __device__ __forceinline__ int c0(int k) const { return first + k * step; }
};
template <int LAY>
__device__ __forceinline__ Lane lane_of(int t, int tpr) {
  if (LAY == kUnits) return Lane{8 * t, 8 * tpr, 1};
  const int w = min(tpr, 32);
  return Lane{(t / w) * 8 * w + t % w, 8 * tpr, w};
}

// The device form of an 8-bit checkpoint.
struct Ck {
  uint8_t* q;            // null: none
  uint8_t* s8;           // e8m0 scales, or ...
  const float* s32;      // ... fp32 ones (read only)
  int64_t ld;
  int32_t group_log2;    // 0: one scale a row
  int32_t n_groups;
};

__device__ __forceinline__ F8 zero8() { return F8{}; }

// Eight columns from c0 on (those below cols; the others read as zero), as they
// are stored: unpack() turns them into fp32.
template <int LAY>
__device__ __forceinline__ void load_raw(const __nv_bfloat16* row, int c0, int dj, int cols, Unit<__nv_bfloat16>& u) {
  if (LAY == kUnits) {
    load_unit<kAligned>(row + c0, 0, min(8, cols - c0), u);
  } else {
    const uint16_t* p = reinterpret_cast<const uint16_t*>(row);
    uint32_t v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = c0 + j * dj < cols ? p[c0 + j * dj] : 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) u.w[i] = v[2 * i] | v[2 * i + 1] << 16;
  }
}
template <int LAY>
__device__ __forceinline__ void load_raw(const float* row, int c0, int dj, int cols, Unit<float>& u) {
  if (LAY == kUnits) {
    load_unit<kAligned>(row + c0, 0, min(8, cols - c0), u);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) u.f[j] = c0 + j * dj < cols ? row[c0 + j * dj] : 0.0f;
  }
}
template <int LAY, typename T>
__device__ __forceinline__ F8 load8(const T* row, int c0, int dj, int cols) {
  Unit<T> u;
  load_raw<LAY>(row, c0, dj, cols, u);
  return unpack(u);
}
template <int LAY>
__device__ __forceinline__ void store8(__nv_bfloat16* row, int c0, int dj, int cols, const F8& v) {
  if (LAY == kUnits) {
    store_unit<kAligned>(row + c0, 0, min(8, cols - c0), v);
    return;
  }
  Unit<__nv_bfloat16> u;
  pack(v, u);
  uint16_t* p = reinterpret_cast<uint16_t*>(row);
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (c0 + j * dj < cols) p[c0 + j * dj] = (uint16_t)(u.w[j >> 1] >> (16 * (j & 1)));
}
template <int LAY>
__device__ __forceinline__ void store8(float* row, int c0, int dj, int cols, const F8& v) {
  if (LAY == kUnits) {
    store_unit<kAligned>(row + c0, 0, min(8, cols - c0), v);
    return;
  }
  Unit<float> u;
  pack(v, u);
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (c0 + j * dj < cols) row[c0 + j * dj] = u.f[j];
}

// A vector that every row reads (a gain, a row of a gate), in fp32 plus `add`.
template <int LAY>
__device__ __forceinline__ F8 load_vec(const void* v, int fp32, int c0, int dj, int cols, float add) {
  Unit<float> u;
  if (LAY == kUnits && c0 + 8 <= cols) {
    if (fp32) {
      const float4 x = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(v) + c0)),
                   y = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(v) + c0) + 1);
      u.f[0] = x.x, u.f[1] = x.y, u.f[2] = x.z, u.f[3] = x.w;
      u.f[4] = y.x, u.f[5] = y.y, u.f[6] = y.z, u.f[7] = y.w;
    } else {
      const uint4 w = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(v) + c0));
      Unit<__nv_bfloat16> b;
      b.w[0] = w.x, b.w[1] = w.y, b.w[2] = w.z, b.w[3] = w.w;
      pack(unpack(b), u);
    }
  } else {      // all eight under way before the first is used
    const int d = LAY == kUnits ? 1 : dj;
    uint32_t raw[8];
    if (fp32) {
#pragma unroll
      for (int j = 0; j < 8; ++j) raw[j] = __float_as_uint(__ldg(static_cast<const float*>(v) + min(c0 + j * d, cols - 1)));
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) raw[j] = (uint32_t)__ldg(static_cast<const uint16_t*>(v) + min(c0 + j * d, cols - 1)) << 16;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) u.f[j] = c0 + j * d < cols ? __uint_as_float(raw[j]) : 0.0f;
  }
  F8 r = unpack(u);
  const uint64_t a = pack_f2(add, add);
#pragma unroll
  for (int i = 0; i < 4; ++i) r.p[i] = fadd2(r.p[i], a);
  return r;
}

// 2^(code - 127); code 255 is NaN.
__device__ __forceinline__ float e8m0_value(uint32_t code) {
  return __uint_as_float(code == 0 ? 0x00400000u : code == 255 ? 0x7fffffffu : code << 23);
}
// The code of the smallest 2^k, k >= -126, with amax <= 448 2^k = 1.75 2^(k + 8), for a finite amax >= 0.
__device__ __forceinline__ uint32_t e8m0_of(float amax) {
  const uint32_t b = __float_as_uint(amax);
  return (uint32_t)max(1, (int)(b >> 23) - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0));
}
// Its reciprocal, exact (codes 1..247).
__device__ __forceinline__ float e8m0_inverse(uint32_t code) { return __uint_as_float((254u - code) << 23); }

__device__ __forceinline__ float ck_scale(const Ck& k, int64_t row, int c) {
  const int64_t i = row * k.n_groups + (k.group_log2 ? c >> k.group_log2 : 0);
  return k.s8 ? e8m0_value(k.s8[i]) : k.s32[i];
}

__device__ __forceinline__ float2 e4m3x2_value(uint32_t two) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// Eight columns of a checkpoint's row, times their scales.
template <int LAY>
__device__ __forceinline__ F8 load8(const Ck& k, int64_t row, int c0, int dj, int cols) {
  F8 v;
  const uint8_t* p = k.q + row * k.ld;
  if (LAY == kUnits) {
    uint32_t w[2] = {0, 0};
    if (c0 + 8 <= cols) {
      asm volatile("ld.global.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "l"(p + c0));
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (c0 + j < cols) w[j >> 2] |= (uint32_t)p[c0 + j] << (8 * (j & 3));
    }
    const float s = ck_scale(k, row, c0);
    const uint64_t s2 = pack_f2(s, s);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 x = e4m3x2_value(w[i >> 1] >> (16 * (i & 1)) & 0xffffu);
      v.p[i] = fmul2(pack_f2(x.x, x.y), s2);
    }
    return v;
  }
  uint32_t x[8];
  float s[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j] = c0 + j * dj < cols ? p[c0 + j * dj] : 0u;
  if (k.group_log2 == 0) {
    s[0] = ck_scale(k, row, 0);
#pragma unroll
    for (int j = 1; j < 8; ++j) s[j] = s[0];
  } else {      // one access a warp and group
    const int64_t base = row * k.n_groups;
    if (k.s8) {
      uint32_t code[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) code[j] = c0 + j * dj < cols ? k.s8[base + ((c0 + j * dj) >> k.group_log2)] : 0u;
#pragma unroll
      for (int j = 0; j < 8; ++j) s[j] = e8m0_value(code[j]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) s[j] = c0 + j * dj < cols ? k.s32[base + ((c0 + j * dj) >> k.group_log2)] : 0.0f;
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 y = e4m3x2_value(x[2 * i] | x[2 * i + 1] << 8);
    v.p[i] = fmul2(pack_f2(y.x, y.y), pack_f2(s[2 * i], s[2 * i + 1]));
  }
  return v;
}

constexpr float kLargest = 3.402823466e38f;

// The largest magnitude of a thread's eight values (those past the row are
// zero), NaN left out; NaN where there is nothing else.
__device__ __forceinline__ float top8(const F8& v) {
  float t[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = unpack_f2(v.p[i]);
    t[i] = fmaxf(fabsf(x.x), fabsf(x.y));
  }
  return fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3]));
}
// The same of the finite ones.
__device__ __forceinline__ float top8_finite(const F8& v) {
  float top = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float2 x = unpack_f2(v.p[j >> 1]);
    const float a = fabsf(j & 1 ? x.y : x.x);
    top = a <= kLargest ? fmaxf(top, a) : top;
  }
  return top;
}

// v / scale in e4m3, four codes a word.  A NaN stays one; an infinity becomes
// one only where EXACT (v - v is 0 or NaN), which costs a subtraction a value:
// rounded down, its zero is -0, whose addition leaves a zero's sign as it is.
template <bool EXACT>
__device__ __forceinline__ uint32_t e4m3_pair(uint64_t v, uint64_t inv) {
  const uint64_t x = EXACT ? fmadd2(v, inv, fsub2_down(v, v)) : fmul2(v, inv);
  return __nv_cvt_float2_to_fp8x2(unpack_f2(x), __NV_SATFINITE, __NV_E4M3);
}
template <bool EXACT>
__device__ __forceinline__ void e4m3_codes(const F8& v, float inv, uint32_t (&w)[2]) {
  const uint64_t i2 = pack_f2(inv, inv);
#pragma unroll
  for (int i = 0; i < 2; ++i) w[i] = e4m3_pair<EXACT>(v.p[2 * i], i2) | e4m3_pair<EXACT>(v.p[2 * i + 1], i2) << 16;
}

// Writes a thread's eight columns of a checkpoint's row.  Scale groups: every lane of the warp calls it together
// (a thread without columns with c0 >= cols and v zero); one scale a row: `row_code` is its code, and the row's
// first thread writes it elsewhere.
template <int LAY>
__device__ __forceinline__ void ck_store8(const Ck& k, int64_t row, int c0, int dj, int cols, const F8& v, uint32_t row_code) {
  uint8_t* p = k.q + row * k.ld;
  uint32_t w[2];
  if (LAY == kUnits) {
    uint32_t code = row_code;
    bool infinite = !k.group_log2;      // (one scale a row: the caller has left infinities out of it)
    if (k.group_log2) {
      const int lanes = 1 << (k.group_log2 - 3);
      float top = top8(v);
      for (int o = lanes >> 1; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      infinite = __any_sync(0xffffffffu, !(top <= kLargest));      // (NaN where a thread has nothing else)
      if (infinite) {
        top = top8_finite(v);
        for (int o = lanes >> 1; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      }
      code = e8m0_of(top);
      if (c0 < cols && (c0 & ((1 << k.group_log2) - 1)) == 0) k.s8[row * k.n_groups + (c0 >> k.group_log2)] = (uint8_t)code;
    }
    if (c0 >= cols) return;
    if (infinite) e4m3_codes<true>(v, e8m0_inverse(code), w);
    else e4m3_codes<false>(v, e8m0_inverse(code), w);
    if (c0 + 8 <= cols) {
      asm volatile("st.global.v2.u32 [%0], {%1, %2};" ::"l"(p + c0), "r"(w[0]), "r"(w[1]) : "memory");
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (c0 + j < cols) p[c0 + j] = (uint8_t)(w[j >> 2] >> (8 * (j & 3)));
    }
    return;
  }
  // the chunk's groups: 1 << (group_log2 - log2 dj) elements of each thread
  uint32_t code[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) code[j] = row_code;
  if (k.group_log2) {
    float top[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float2 x = unpack_f2(v.p[j >> 1]);
      const float a = fabsf(j & 1 ? x.y : x.x);
      top[j] = a <= kLargest ? a : 0.0f;
    }
    // elements of a group: dj = 32: 1, 2 or 4; shorter rows up to all eight
    const int per = min(8, (1 << k.group_log2) / dj);
#pragma unroll
    for (int s = 1; s < 8; s *= 2) {
      if (s < per) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if ((j & s) == 0) top[j] = top[j | s] = fmaxf(top[j], top[j | s]);
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (j % per) {
        code[j] = code[j - 1];
        continue;
      }
      float t = top[j];
      if (dj == 32) t = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(t)));      // magnitudes order as their bits
      else
        for (int o = dj >> 1; o > 0; o >>= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, o));
      code[j] = e8m0_of(t);
      const int c = c0 + j * dj;
      if (c < cols && (c & ((1 << k.group_log2) - 1)) == 0) k.s8[row * k.n_groups + (c >> k.group_log2)] = (uint8_t)code[j];
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint64_t inv = pack_f2(e8m0_inverse(code[2 * i]), e8m0_inverse(code[2 * i + 1]));
    const uint32_t two = e4m3_pair<true>(v.p[i], inv);
    const int c = c0 + 2 * i * dj;
    if (c < cols) p[c] = (uint8_t)two;
    if (c + dj < cols) p[c + dj] = (uint8_t)(two >> 8);
  }
}

// Wide units: 16 columns of a thread, of rows whose places all are multiples of
// 32 bytes (16 of e4m3 values).
__device__ __forceinline__ uint4 ld_once(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
__device__ __forceinline__ void ld_once32(const void* p, uint4& a, uint4& b) {
  asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w)
               : "l"(p));
}
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// 16 columns as stored, and as two F8.
template <typename T>
struct Wide {
  static constexpr int kParts = sizeof(T);      // 16-byte words
  uint4 w[kParts];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < kParts; i += 2) ld_once32(p + i * 16 / sizeof(T), w[i], w[i + 1]);
  }
  __device__ __forceinline__ F8 half(int i) const {
    if constexpr (sizeof(T) == 2) {
      Unit<__nv_bfloat16> u;
      u.w[0] = w[i].x, u.w[1] = w[i].y, u.w[2] = w[i].z, u.w[3] = w[i].w;
      return unpack(u);
    } else {
      Unit<float> u;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        u.f[4 * j] = __uint_as_float(w[2 * i + j].x), u.f[4 * j + 1] = __uint_as_float(w[2 * i + j].y);
        u.f[4 * j + 2] = __uint_as_float(w[2 * i + j].z), u.f[4 * j + 3] = __uint_as_float(w[2 * i + j].w);
      }
      return unpack(u);
    }
  }
  // The largest magnitude; not at most kLargest where not all are finite (fp32: unless only NaN are not).
  __device__ __forceinline__ float top() const {
    if constexpr (sizeof(T) == 2) {      // magnitudes of bf16 values order as their bits do
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 2; ++i)
        m = max_u16x2(max_u16x2(m, w[i].x & 0x7fff7fffu), max_u16x2(max_u16x2(w[i].y & 0x7fff7fffu, w[i].z & 0x7fff7fffu), w[i].w & 0x7fff7fffu));
      return __uint_as_float(max(m & 0xffff0000u, m << 16));
    } else {
      return fmaxf(top8(half(0)), top8(half(1)));
    }
  }
};

// Writes 16 columns of a checkpoint's row, as ck_store8 writes eight.  top: what
// Wide::top() or top8() say of both halves.  wide: rows on wide units (else on units of eight).
__device__ __forceinline__ void ck_store16(const Ck& k, int64_t row, int c, int cols, const F8& lo, const F8& hi, float top, uint32_t row_code, bool wide) {
  uint32_t code = row_code;
  bool infinite = !k.group_log2;
  if (k.group_log2) {
    infinite = __any_sync(0xffffffffu, !(top <= kLargest));
    if (infinite) top = c < cols ? fmaxf(top8_finite(lo), top8_finite(hi)) : 0.0f;
#pragma unroll
    for (int o = 1; o < 8; o *= 2) {      // a group of 32, 64 or 128 columns: 2, 4 or 8 lanes
      const float other = __shfl_xor_sync(0xffffffffu, top, o);
      top = fmaxf(top, 16 * o < 1 << k.group_log2 ? other : 0.0f);
    }
    code = e8m0_of(top);
    if (c < cols && (c & ((1 << k.group_log2) - 1)) == 0)
      k.s8[row * k.n_groups + (c >> k.group_log2)] = (uint8_t)code;
  }
  if (c >= cols) return;
  const float inv = e8m0_inverse(code);
  uint32_t w[2], x[2];
  if (infinite) e4m3_codes<true>(lo, inv, w), e4m3_codes<true>(hi, inv, x);
  else e4m3_codes<false>(lo, inv, w), e4m3_codes<false>(hi, inv, x);
  uint8_t* p = k.q + row * k.ld + c;
  if (wide) {
    asm volatile("st.global.v4.u32 [%0], {%1, %2, %3, %4};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(x[0]), "r"(x[1]) : "memory");
  } else {
    asm volatile("st.global.v2.u32 [%0], {%1, %2};" ::"l"(p), "r"(w[0]), "r"(w[1]) : "memory");
    asm volatile("st.global.v2.u32 [%0], {%1, %2};" ::"l"(p + 8), "r"(x[0]), "r"(x[1]) : "memory");
  }
}

__device__ __forceinline__ void store16(__nv_bfloat16* p, const F8& lo, const F8& hi, bool wide) {
  Unit<__nv_bfloat16> a, b;
  pack(lo, a);
  pack(hi, b);
  if (!wide) {
    st_unit(p, a);
    st_unit(p + 8, b);
    return;
  }
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a.w[0]), "r"(a.w[1]), "r"(a.w[2]), "r"(a.w[3]), "r"(b.w[0]),
               "r"(b.w[1]), "r"(b.w[2]), "r"(b.w[3])
               : "memory");
}
__device__ __forceinline__ void store16(float* p, const F8& lo, const F8& hi, bool) {
  Unit<float> a, b;
  pack(lo, a);
  pack(hi, b);
  st_unit(p, a);
  st_unit(p + 8, b);
}

// 16 columns of a thread in the second lay: lane, lane + 32, .. of a warp's 512.
// WHOLE: none is past the row.
template <bool WHOLE = false>
__device__ __forceinline__ void ck_store16_strided(const Ck& k, int64_t row, int c0, int cols, const F8 (&v)[2], uint32_t row_code) {
  uint8_t* p = k.q + row * k.ld;
  const int per = k.group_log2 ? 1 << (k.group_log2 - 5) : 16;      // a group's blocks of 32 columns
  uint32_t code = row_code;
#pragma unroll
  for (int b = 0; b < 4; ++b) {      // four blocks at a time: a group, or several
    float top[4];
    uint32_t codes[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 x = unpack_f2(v[b >> 1].p[2 * (b & 1) + (e >> 1)]);
      const float a = fabsf(e & 1 ? x.y : x.x);
      top[e] = a <= kLargest ? a : 0.0f;
      codes[e] = row_code;
    }
    if (k.group_log2) {
      if (per > 1) top[0] = fmaxf(top[0], top[1]), top[2] = fmaxf(top[2], top[3]);
      if (per > 2) top[0] = fmaxf(top[0], top[2]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (e % per == 0) {
          code = e8m0_of(__uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top[e]))));      // magnitudes order as their bits
          const int c = c0 + 32 * (4 * b + e);
          if ((WHOLE || c < cols) && (threadIdx.x & 31) == 0) k.s8[row * k.n_groups + (c >> k.group_log2)] = (uint8_t)code;
        }
        codes[e] = code;
      }
    }
#pragma unroll
    for (int e = 0; e < 4; e += 2) {
      const uint32_t two = e4m3_pair<true>(v[b >> 1].p[2 * (b & 1) + (e >> 1)], pack_f2(e8m0_inverse(codes[e]), e8m0_inverse(codes[e + 1])));
      const int c = c0 + 32 * (4 * b + e);
      if (WHOLE || c < cols) p[c] = (uint8_t)two;
      if (WHOLE || c + 32 < cols) p[c + 32] = (uint8_t)(two >> 8);
    }
  }
}

// Whether each row of `m` (null passes) starts on a wide unit, and ends on one.
inline bool on_wide(const sf_matrix* m) {
  if (!m || m->rows < 1) return true;
  const uintptr_t unit = m->dtype == SF_E4M3 ? 16 : 32;
  return m->cols % 16 == 0 && reinterpret_cast<uintptr_t>(m->data) % unit == 0 && (m->rows == 1 || m->ld % 16 == 0);
}
inline bool on_wide(const sf_checkpoint* c) { return !c || on_wide(&c->values); }
// Whether bulk copies can bring its rows: 16-byte aligned, in this device's own memory.
inline bool on_bulk(const sf_matrix* m) { return !m || (reinterpret_cast<uintptr_t>(m->data) % 16 == 0 && on_current_device(m->data)); }

// The sums (or, from index SUMS on, the maxima) of N values over the tpr
// threads of a row, in a fixed order: lanes by a butterfly, then the row's
// warps in turn through shared memory (red: [warps of a block][N], the caller
// alternates between two).  With tpr > 32 all threads of the block call it.
template <int N, int SUMS>
__device__ __forceinline__ void row_reduce_n(float (&v)[N], int tpr, float* red) {
  for (int o = min(tpr, 32) >> 1; o > 0; o >>= 1) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float w = __shfl_xor_sync(0xffffffffu, v[i], o);
      v[i] = i < SUMS ? v[i] + w : fmaxf(v[i], w);
    }
  }
  if (tpr <= 32) return;
  const int warp = threadIdx.x >> 5, n = tpr >> 5, first = warp - warp % n;
  if ((threadIdx.x & 31) == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) red[warp * N + i] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float t = red[first * N + i];
    for (int j = 1; j < n; ++j) t = i < SUMS ? t + red[(first + j) * N + i] : fmaxf(t, red[(first + j) * N + i]);
    v[i] = t;
  }
}

// Host side.  Checks a checkpoint argument of rows x cols; `writes`: scales must be e8m0.
inline sf_status check_checkpoint(const sf_checkpoint* c, const char* name, int64_t rows, int64_t cols, bool writes) {
  if (!c) return fail(SF_ERR_INVALID, "%s is NULL", name);
  SF_TRY(check_matrix(&c->values, name, rows, cols, 1u << SF_E4M3));
  if (c->group != 0 && c->group != 32 && c->group != 64 && c->group != 128)
    return fail(SF_ERR_INVALID, "%s: group must be 0 (a scale per row), 32, 64 or 128 (got %d)", name, (int)c->group);
  if (c->scale_dtype != SF_E8M0 && (writes || c->scale_dtype != SF_FP32))
    return fail(SF_ERR_UNSUPPORTED, "%s: scales of type %d are not taken here", name, (int)c->scale_dtype);
  if (c->values.rows && c->values.cols && !c->scale) return fail(SF_ERR_INVALID, "%s: scale is NULL", name);
  return check_aligned(c->scale, dtype_bytes(c->scale_dtype), name);
}

inline Ck device_ck(const sf_checkpoint* c) {
  Ck k{};
  if (!c) return k;
  k.q = static_cast<uint8_t*>(c->values.data);
  k.ld = c->values.ld;
  if (c->scale_dtype == SF_E8M0) k.s8 = static_cast<uint8_t*>(c->scale);
  else k.s32 = static_cast<const float*>(c->scale);
  k.group_log2 = c->group == 128 ? 7 : c->group == 64 ? 6 : c->group == 32 ? 5 : 0;
  k.n_groups = c->group ? (int32_t)ceil_div<int64_t>(c->values.cols, c->group) : 1;
  return k;
}

// Whether each row of `m` (null passes) starts on a unit of eight elements.
inline bool on_units(const sf_matrix* m) {
  if (!m || m->rows < 1) return true;
  return reinterpret_cast<uintptr_t>(m->data) % (8 * dtype_bytes(m->dtype)) == 0 && (m->rows == 1 || m->ld % 8 == 0);
}
inline bool on_units(const sf_checkpoint* c) { return !c || on_units(&c->values); }
inline bool on_units(const void* v, int32_t dtype) { return reinterpret_cast<uintptr_t>(v) % (8 * dtype_bytes(dtype)) == 0; }

}  // namespace sf
