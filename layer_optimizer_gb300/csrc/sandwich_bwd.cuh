// The backward pass of a residual block's end: what its forms share.
#pragma once

#include "sandwich.cuh"

namespace sf {

// Backward.  With w = b gate g1 (the factor of x's norm in s) a row's sums
//   A = sum dh g2 s,  B = sum w x (dsum + rho2 dh g2),  D = sum w x s
// come from one pass over the row, and then
//   c = -rho2^3 A / cols,  d = dsum + rho2 dh g2 + c s
//   c1 = -rho1^3 (B + c D) / cols,  dx = rho1 w d + c1 x
// since sum w x d = B + c D: one reduction a row, not two.
//
// Gradients of the gains and the gate.  With t = b d x rho1 and T_k its sum
// over the rows of gate row k,  dgate_k = g1 T_k  and  dg1 = sum_k gate_k T_k,
// so a thread holds one sum for both (and one for dg2), over rows of one gate
// row after the other.
//
// Work items: gate row k's rows in P parts; a worker (the threads of a row)
// takes the items w, w + workers, ...  Where the gate has fewer rows than
// there are workers, every worker has one item at most: its T is a partial row
// (tpart), joined by k_sandwich_join.  Else P = 1 and a worker has several:
// each T is complete, goes into dgate at once, and times its gate row into the
// worker's partial dg1 (kept in the workspace, this worker's own row).
struct BwdArgs {
  const void* dh;         // may be null
  const void* dsum;       // may be null
  const void* x;          // may be null, as may x8.q: at most one of the two
  const void* s;
  void* dr;               // may be null
  void* dx;               // may be null
  void* dgate;            // several items a worker: written here (else by the join)
  Ck x8, s8;
  const float* rho1;
  const float* rho2;
  float* tpart;           // [workers][cols] or null: T of the worker's item, or its share of dg1
  float* ppart;           // [workers][cols] or null: dg2
  int64_t lddh, lddsum, ldx, lds, lddr, lddx, lddgate;
  int64_t rows, span, items;      // span: rows of an undivided item (gate_span, or all rows)
  int64_t workers;
  int32_t parts;          // P
  int32_t many;           // several items a worker
  int32_t dgate_fp32;
  int32_t cols, tpr, rpb;
  int32_t wide;           // staged form: rows on wide units, not on units of eight only
  float inv_cols;
  Vectors v;
};

namespace {

// A gate's row: not by the read-only path, since dgate may be the same memory
// (each row of it is read and written by one worker only).
template <int LAY>
__device__ __forceinline__ F8 load8_any(const void* row, int fp32, int c0, int dj, int cols) {
  if (LAY == kUnits && c0 + 8 <= cols) {
    if (fp32) {
      const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(row) + c0);
      const float4 x = p[0], y = p[1];
      return F8{{pack_f2(x.x, x.y), pack_f2(x.z, x.w), pack_f2(y.x, y.y), pack_f2(y.z, y.w)}};
    }
    const uint4 w = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(row) + c0);
    Unit<__nv_bfloat16> u;
    u.w[0] = w.x, u.w[1] = w.y, u.w[2] = w.z, u.w[3] = w.w;
    return unpack(u);
  }
  return fp32 ? load8<kStrided>(static_cast<const float*>(row), c0, dj, cols) : load8<kStrided>(static_cast<const __nv_bfloat16*>(row), c0, dj, cols);
}
template <int LAY>
__device__ __forceinline__ void store_any(void* row, int fp32, int c0, int dj, int cols, const F8& v) {
  if (fp32) store8<LAY>(static_cast<float*>(row), c0, dj, cols, v);
  else store8<LAY>(static_cast<__nv_bfloat16*>(row), c0, dj, cols, v);
}

constexpr int kBwdRingThreads = 512, kBwdRingRegs = 128;

}  // namespace

// The staged form's kernels in either lay (kept: x and s as checkpoints).
const void* bwd_ring_units(int32_t ta, int32_t ts, bool kept, bool post);
const void* bwd_ring_strided(int32_t ta, int32_t ts, bool kept, bool post);

}  // namespace sf
