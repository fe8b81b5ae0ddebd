// The weight gradient of a linear layer from the 8-bit checkpoint of its
// input: dW = base + dY^T X, X = value * scale.
#include <algorithm>

#include "lanes.cuh"

namespace sf {
namespace {

struct WgradArgs {
  const __nv_bfloat16* dy;   // [tokens][ldy]
  const void* base;          // [out][ldbase], may be null or dw
  void* dw;                  // [out][lddw]
  int64_t ldy, ldbase, lddw;
  int64_t tokens, out, in;
  int32_t fp32;              // dw and base
  Ck ck;
};

__device__ __forceinline__ float dw_at(const void* p, int fp32, int64_t i) {
  return fp32 ? static_cast<const float*>(p)[i] : __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}

// 64 x 64 tiles on the CUDA cores, 4 x 4 a thread, for operands that tensor
// copies cannot take (rows off 16 bytes, pinned host memory).
constexpr int kT = 64, kTk = 16;
__global__ void __launch_bounds__(256) k_wgrad_plain(const WgradArgs a) {
  __shared__ float sa[kTk][kT + 4], sb[kTk][kT + 4];
  const int64_t o0 = (int64_t)blockIdx.y * kT, i0 = (int64_t)blockIdx.x * kT;
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
  float acc[4][4] = {};
  for (int64_t t0 = 0; t0 < a.tokens; t0 += kTk) {
    for (int e = threadIdx.x; e < kTk * kT; e += 256) {
      const int64_t t = t0 + e / kT, o = o0 + e % kT, i = i0 + e % kT;
      sa[e / kT][e % kT] = t < a.tokens && o < a.out ? __bfloat162float(a.dy[t * a.ldy + o]) : 0.0f;
      float x = 0.0f;
      if (t < a.tokens && i < a.in) x = __bfloat162float(__float2bfloat16_rn(e4m3x2_value(a.ck.q[t * a.ck.ld + i]).x * ck_scale(a.ck, t, (int)i)));
      sb[e / kT][e % kT] = x;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kTk; ++k)
#pragma unroll
      for (int y = 0; y < 4; ++y)
#pragma unroll
        for (int x = 0; x < 4; ++x) acc[y][x] = fmaf(sa[k][ty * 4 + y], sb[k][tx * 4 + x], acc[y][x]);
    __syncthreads();
  }
#pragma unroll
  for (int y = 0; y < 4; ++y)
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int64_t o = o0 + ty * 4 + y, i = i0 + tx * 4 + x;
      if (o >= a.out || i >= a.in) continue;
      float v = acc[y][x];
      if (a.base) v += dw_at(a.base, a.fp32, o * a.ldbase + i);
      if (a.fp32) static_cast<float*>(a.dw)[o * a.lddw + i] = v;
      else static_cast<__nv_bfloat16*>(a.dw)[o * a.lddw + i] = __float2bfloat16_rn(v);
    }
}

}  // namespace
}  // namespace sf

extern "C" {

size_t sf_checkpoint_wgrad_workspace_bytes(int64_t tokens, int64_t out, int64_t in) {
  (void)tokens, (void)out, (void)in;
  return 0;
}

sf_status sf_checkpoint_wgrad(const sf_matrix* dY, const sf_checkpoint* c, const sf_matrix* base, const sf_matrix* dW,
                              void* ws, size_t ws_bytes, void* stream) {
  using namespace sf;
  clear_error();
  NvtxRange nvtx_range("sf_checkpoint_wgrad");
  SF_TRY(check_matrix(dY, "dY", -1, -1, 1u << SF_BF16));
  SF_TRY(check_matrix(dW, "dW", dY->cols, -1, 1u << SF_BF16 | 1u << SF_FP32));
  SF_TRY(check_checkpoint(c, "checkpoint", dY->rows, dW->cols, false));
  if (base) SF_TRY(check_matrix(base, "base", dW->rows, dW->cols, 1u << dW->dtype));
  const int64_t tokens = dY->rows, out = dW->rows, in = dW->cols;
  if (tokens > INT32_MAX / 2 || out > INT32_MAX / 2 || in > INT32_MAX / 2) return fail(SF_ERR_UNSUPPORTED, "tokens, out and in must be below 2^30");
  const size_t need = sf_checkpoint_wgrad_workspace_bytes(tokens, out, in);
  if (need && (!ws || ws_bytes < need || reinterpret_cast<uintptr_t>(ws) % 16))
    return fail(SF_ERR_INVALID, "workspace needs %zu bytes, 16-byte aligned (got %zu)", need, ws_bytes);
  if (!out || !in) return SF_OK;
  WgradArgs a{};
  a.dy = static_cast<const __nv_bfloat16*>(dY->data);
  a.ldy = dY->ld;
  if (base) a.base = base->data, a.ldbase = base->ld;
  a.dw = dW->data;
  a.lddw = dW->ld;
  a.tokens = tokens;
  a.out = out;
  a.in = in;
  a.fp32 = dW->dtype == SF_FP32;
  a.ck = device_ck(c);
  const int64_t gx = ceil_div<int64_t>(in, kT), gy = ceil_div<int64_t>(out, kT);
  if (gy > 65535) return fail(SF_ERR_UNSUPPORTED, "out is too large");
  k_wgrad_plain<<<dim3((unsigned)gx, (unsigned)gy), 256, 0, as_stream(stream)>>>(a);
  return check_launch("launch k_wgrad_plain");
}

}  // extern "C"
