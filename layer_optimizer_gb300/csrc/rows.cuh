// Row-wise access shared by the dropout and norm kernels: a thread's unit is
// eight consecutive columns of a row (one 16-byte load in bf16, one 32-byte
// load in fp32), and the counter-based generator gives one unit's random
// bits per evaluation.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "common.h"
#include "pairs.cuh"

namespace sf {

template <typename T>
struct Unit;
template <>
struct Unit<__nv_bfloat16> {
  uint32_t w[4];
};
template <>
struct Unit<float> {
  float f[8];
};

// Eight fp32 values as four pairs: additions, products and fused
// multiply-adds run on both values of a pair at once (each rounded to nearest
// as two scalar ones would be), which halves the instructions of kernels that
// would otherwise be bound by issue and not by memory.
struct F8 {
  uint64_t p[4];
};

__device__ __forceinline__ F8 unpack(const Unit<__nv_bfloat16>& u) {
  F8 v;
#pragma unroll
  for (int i = 0; i < 4; ++i) v.p[i] = pack_f2(__uint_as_float(u.w[i] << 16), __uint_as_float(u.w[i] & 0xFFFF0000u));
  return v;
}
__device__ __forceinline__ F8 unpack(const Unit<float>& u) {
  F8 v;
#pragma unroll
  for (int i = 0; i < 4; ++i) v.p[i] = pack_f2(u.f[2 * i], u.f[2 * i + 1]);
  return v;
}
__device__ __forceinline__ void pack(const F8& v, Unit<__nv_bfloat16>& u) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = unpack_f2(v.p[i]);
    const __nv_bfloat162 h = __floats2bfloat162_rn(x.x, x.y);   // round to nearest even
    u.w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
}
__device__ __forceinline__ void pack(const F8& v, Unit<float>& u) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = unpack_f2(v.p[i]);
    u.f[2 * i] = x.x;
    u.f[2 * i + 1] = x.y;
  }
}

// Whole-unit accesses.  Not the read-only path: outputs may be their inputs.
__device__ __forceinline__ void ld_unit(const __nv_bfloat16* p, Unit<__nv_bfloat16>& u) {
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(u.w[0]), "=r"(u.w[1]), "=r"(u.w[2]), "=r"(u.w[3])
               : "l"(p));
}
__device__ __forceinline__ void ld_unit(const float* p, Unit<float>& u) {
  asm volatile("ld.global.L1::no_allocate.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=f"(u.f[0]), "=f"(u.f[1]), "=f"(u.f[2]), "=f"(u.f[3]), "=f"(u.f[4]), "=f"(u.f[5]), "=f"(u.f[6]),
                 "=f"(u.f[7])
               : "l"(p));
}
__device__ __forceinline__ void st_unit(__nv_bfloat16* p, const Unit<__nv_bfloat16>& u) {
  asm volatile("st.global.v4.u32 [%0], {%1, %2, %3, %4};" ::"l"(p), "r"(u.w[0]), "r"(u.w[1]), "r"(u.w[2]), "r"(u.w[3])
               : "memory");
}
__device__ __forceinline__ void st_unit(float* p, const Unit<float>& u) {
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(u.f[0]), "f"(u.f[1]),
               "f"(u.f[2]), "f"(u.f[3]), "f"(u.f[4]), "f"(u.f[5]), "f"(u.f[6]), "f"(u.f[7])
               : "memory");
}

// How a matrix's rows meet its units in memory:
//   kAligned  every row starts on a unit: unit u holds columns 8 u .. 8 u + 7;
//   kShifted  row i starts m = i * shift mod 8 columns past a unit, m the same
//             for all operands (dense rows of an odd length, for example): unit
//             u holds columns 8 u - m .. 8 u - m + 7, so that whole units are
//             one access here too (16384 x 4095 bf16: norm with dropout 169 us,
//             against 278 us element by element);
//   kScalar   anything else, element by element.
enum RowMode : int { kScalar = 0, kAligned = 1, kShifted = 2 };

// The first column of a unit, and which of its eight lie in the row.
struct Span {
  int c, lo, hi;
  __device__ __forceinline__ bool some() const { return hi > lo; }
};
template <int MODE>
__device__ __forceinline__ Span unit_span(int u, int m, int cols) {
  Span s;
  s.c = 8 * u - (MODE == kShifted ? m : 0);
  s.lo = MODE == kShifted ? max(0, -s.c) : 0;
  s.hi = min(8, cols - s.c);
  return s;
}

// The columns lo .. hi - 1 of a unit; the others read as zero.
template <int MODE>
__device__ __forceinline__ void load_unit(const __nv_bfloat16* p, int lo, int hi, Unit<__nv_bfloat16>& u) {
  if (MODE != kScalar && lo == 0 && hi == 8) {
    ld_unit(p, u);
    return;
  }
  const uint16_t* q = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t a = 2 * i >= lo && 2 * i < hi ? q[2 * i] : 0u, b = 2 * i + 1 >= lo && 2 * i + 1 < hi ? q[2 * i + 1] : 0u;
    u.w[i] = a | (b << 16);
  }
}
template <int MODE>
__device__ __forceinline__ void load_unit(const float* p, int lo, int hi, Unit<float>& u) {
  if (MODE != kScalar && lo == 0 && hi == 8) {
    ld_unit(p, u);
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) u.f[i] = i >= lo && i < hi ? p[i] : 0.0f;
}
template <int MODE>
__device__ __forceinline__ void store_unit(__nv_bfloat16* p, int lo, int hi, const F8& v) {
  Unit<__nv_bfloat16> u;
  pack(v, u);
  if (MODE != kScalar && lo == 0 && hi == 8) {
    st_unit(p, u);
    return;
  }
  uint16_t* q = reinterpret_cast<uint16_t*>(p);
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i >= lo && i < hi) q[i] = (uint16_t)(u.w[i >> 1] >> (16 * (i & 1)));
}
template <int MODE>
__device__ __forceinline__ void store_unit(float* p, int lo, int hi, const F8& v) {
  Unit<float> u;
  pack(v, u);
  if (MODE != kScalar && lo == 0 && hi == 8) {
    st_unit(p, u);
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i >= lo && i < hi) p[i] = u.f[i];
}

// Dropout's constants: an element is kept where its 16 random bits are at
// least `threshold` = round(65536 p), and kept values are multiplied by
// factor = 65536 / (65536 - threshold), so the expectation is exact for the
// probability threshold / 65536 that is really used (within 2^-17 of p).
// threshold = 0: no dropout.
struct DropConsts {
  uint32_t key[20];                // the rounds' keys, from the seed
  uint64_t offset;
  const uint64_t* device_offset;   // added to offset when not null
  float factor;
  uint32_t threshold;
};

sf_status make_drop_consts(double p, const sf_rng* rng, DropConsts* out);

// The upper counter half, the same for a whole call.
struct DropWords {
  uint32_t c2, c3;
};
__device__ __forceinline__ DropWords drop_words(const DropConsts& d) {
  uint64_t off = d.offset;
  if (d.device_offset) off += *d.device_offset;
  return DropWords{(uint32_t)off, (uint32_t)(off >> 32)};
}

// Philox-4x32 with 10 rounds (Salmon, Moraes, Dror, Shaw: "Parallel random
// numbers: as easy as 1, 2, 3", 2011): 128 bits for the unit with index b,
// 16 per column.  Eight columns share one evaluation, so a column costs 2.5
// 32 x 32 -> 64 multiplications; with 32 bits a column (twice that) the
// bf16 kernels would be bound by the multiplier and not by memory.  The round
// keys come ready from the host: a fifth of the generator's instructions.
__device__ __forceinline__ void drop_bits(uint64_t b, const DropWords& w2, const DropConsts& d, uint32_t (&w)[4]) {
  uint32_t c0 = (uint32_t)b, c1 = (uint32_t)(b >> 32), c2 = w2.c2, c3 = w2.c3;
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t m0 = (uint64_t)c0 * 0xD2511F53u, m1 = (uint64_t)c2 * 0xCD9E8D57u;
    const uint32_t n0 = (uint32_t)(m1 >> 32) ^ c1 ^ d.key[2 * r], n2 = (uint32_t)(m0 >> 32) ^ c3 ^ d.key[2 * r + 1];
    c0 = n0;
    c1 = (uint32_t)m1;
    c2 = n2;
    c3 = (uint32_t)m0;
  }
  w[0] = c0, w[1] = c1, w[2] = c2, w[3] = c3;
}

// Applies the mask with a unit's 128 bits.
__device__ __forceinline__ void drop_apply(F8& v, const uint32_t (&w)[4], const DropConsts& d) {
  // half >= threshold, compared in the upper half of a word (threshold >= 1
  // here, 65536 included); a dropped element is 0 whatever its value
  const uint32_t limit = ((d.threshold - 1) << 16) | 0xFFFFu;
  const uint64_t f = pack_f2(d.factor, d.factor);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 x = unpack_f2(fmul2(v.p[j], f));
    v.p[j] = pack_f2((w[j] << 16) > limit ? x.x : 0.0f, w[j] > limit ? x.y : 0.0f);
  }
}
__device__ __forceinline__ void drop_unit(F8& v, uint64_t b, const DropWords& w2, const DropConsts& d) {
  uint32_t w[4];
  drop_bits(b, w2, d, w);
  drop_apply(v, w, d);
}

// The bits of units whose columns start m below counter b's eight: they come
// from the counters b - 1 and b.  `width` neighbouring lanes take neighbouring
// units, and lane 0 the one after the last lane's of the call before, so each
// counter is evaluated once and handed to the next lane (16384 x 4095 bf16,
// dropout and addition 100 us, with two evaluations a unit 123).  All lanes of a warp call `next` together.
struct ShiftedBits {
  uint32_t carry[4];      // lane 0: the words of the counter before its next unit's
  __device__ __forceinline__ void start(uint64_t before, const DropWords& w2, const DropConsts& d) { drop_bits(before, w2, d, carry); }
  __device__ __forceinline__ void next(uint64_t b, int lane, int width, int m, const DropWords& w2, const DropConsts& d, uint32_t (&w)[4]) {
    uint32_t x[9];
    drop_bits(b, w2, d, w);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t from_left = __shfl_sync(0xffffffffu, w[i], lane == 0 ? width - 1 : lane - 1, width);
      x[i] = lane == 0 ? carry[i] : from_left;
      x[4 + i] = w[i];
      carry[i] = from_left;
    }
    // eight halves from half 8 - m (1..8) of the sixteen on
    const int from = 8 - m;
    x[8] = 0;
#pragma unroll
    for (int i = 0; i < 5; ++i) x[i] = from & 8 ? x[i + 4] : x[i];
#pragma unroll
    for (int i = 0; i < 7; ++i) x[i] = from & 4 ? x[i + 2] : x[i];
#pragma unroll
    for (int i = 0; i < 6; ++i) x[i] = from & 2 ? x[i + 1] : x[i];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(x[i], x[i + 1], from & 1 ? 16 : 0);
  }
};

// A matrix argument as the kernels see it.
template <typename T>
__device__ __forceinline__ T* row_ptr(void* base, int64_t ld, int64_t row) {
  return static_cast<T*>(base) + row * ld;
}
template <typename T>
__device__ __forceinline__ const T* row_ptr(const void* base, int64_t ld, int64_t row) {
  return static_cast<const T*>(base) + row * ld;
}

// The mode that all of `ms` (null entries skipped) allow together, and the
// columns (mod 8) by which each row starts further past a unit than the one
// before.
template <size_t N>
inline RowMode row_mode(const sf_matrix* const (&ms)[N], int* shift) {
  *shift = -1;
  for (const sf_matrix* m : ms) {
    if (!m || m->rows < 1) continue;
    if (reinterpret_cast<uintptr_t>(m->data) % (8 * dtype_bytes(m->dtype))) return kScalar;
    if (m->rows == 1) continue;
    const int d = (int)(m->ld & 7);
    if (*shift >= 0 && *shift != d) return kScalar;
    *shift = d;
  }
  if (*shift < 0) *shift = 0;
  return *shift ? kShifted : kAligned;
}

}  // namespace sf
