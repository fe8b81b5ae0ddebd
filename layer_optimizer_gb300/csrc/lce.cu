// Fused linear cross-entropy: loss and gradients of the softmax
// cross-entropy of a linear output layer, chunked over tokens so that the
// full logits tensor is never held.
//
// SlideFormer ("An Efficient Heterogeneous Co-Design for Fine-Tuning on a
// Single GPU"; the summaries' kernel lists, "Fused LinearCrossEntropy")
// fuses the output projection with the loss and computes the gradients in
// small blocks, so the logits (tokens x vocabulary, larger than every other
// activation for big vocabularies) never exist in full.  For each chunk of
// tokens c:
//   Z_c  = H_c W^T                      tensor cores, fp32 [chunk][V]
//   lse  = logsumexp over each row of Z_c, from (max, sum exp) pairs the
//          logits GEMM's epilogue writes per row and 256-column tile, and
//          the rows' losses
//   G_c  = (softmax(Z_c) - onehot(y_c)) / n  rounded to bf16 [chunk][V]
//   dH_c = G_c W                        tensor cores, W read MN-major
//   dW  += G_c^T H_c                    tensor cores, G_c and H_c read MN-major
// n is the number of tokens whose label is not ignore_index.  The three
// products run on the tensor-core GEMM (tc_gemm.cu), which reads either
// layout of an operand, so no transposed copy of W, G or H is made; the row
// statistics and the gradient are fp32 CUDA-core kernels.  Memory: one
// chunk of logits (fp32) and one of the bf16 gradient instead of N x V.
#include <cuda_bf16.h>

#include <algorithm>

#include "common.h"
#include "ptx.cuh"

namespace sf {
namespace {

// Number n of labelled tokens (label != ignore and in [0, V)); a label that
// is neither is counted as unlabelled and flagged.  inv_n = 1/n (0 if n = 0).
__global__ void __launch_bounds__(1024) k_lce_count(const int32_t* __restrict__ labels, int64_t N, int64_t V,
                                                    int32_t ignore, int64_t* __restrict__ n_out,
                                                    float* __restrict__ inv_n) {
  __shared__ int64_t red[1024];
  int64_t c = 0;
  bool bad = false;
  for (int64_t i = threadIdx.x; i < N; i += blockDim.x) {
    const int32_t y = labels[i];
    if (y == ignore) continue;
    if (y < 0 || y >= V) bad = true;
    else ++c;
  }
  if (bad) atomicOr(&g_device_error, kDevErrIndex);
  red[threadIdx.x] = c;
  __syncthreads();
  for (int s = blockDim.x / 2; s > 0; s >>= 1) {
    if ((int)threadIdx.x < s) red[threadIdx.x] += red[threadIdx.x + s];
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    *n_out = red[0];
    *inv_n = red[0] > 0 ? (float)(1.0 / (double)red[0]) : 0.0f;
  }
}

__device__ __forceinline__ bool labelled(int32_t y, int32_t ignore, int64_t V) {
  return y != ignore && y >= 0 && y < V;
}

// (m, s) pairs meaning "s = sum of exp(x - m)" combined into one.
__device__ __forceinline__ void combine_stats(float& m, float& s, float m2, float s2) {
  if (m2 == -INFINITY) return;
  if (m == -INFINITY) {
    m = m2;
    s = s2;
    return;
  }
  const float mn = fmaxf(m, m2);
  s = s * expf(m - mn) + s2 * expf(m2 - mn);
  m = mn;
}

// One warp per row of the chunk: lse = log sum_j exp(z_j) from the logits
// GEMM's per-tile (max, sum of exp) pairs, combined in a fixed order (lanes
// over tiles, then a butterfly); the row's loss lse - z[y] (0 for an
// unlabelled token).
__global__ void __launch_bounds__(256) k_lce_lse(const float2* __restrict__ stats, int n_tiles, int64_t rows,
                                                 const float* __restrict__ Z, int64_t V,
                                                 const int32_t* __restrict__ labels, int32_t ignore,
                                                 float* __restrict__ lse, float* __restrict__ row_loss) {
  const int lane = threadIdx.x & 31;
  const int64_t r = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (r >= rows) return;
  float m = -INFINITY, s = 0.0f;
  for (int t = lane; t < n_tiles; t += 32) {
    const float2 p = stats[r * n_tiles + t];
    combine_stats(m, s, p.x, p.y);
  }
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const float m2 = __shfl_xor_sync(0xffffffffu, m, o), s2 = __shfl_xor_sync(0xffffffffu, s, o);
    // the same pair order on both lanes of the exchange: lower lane first
    if (lane & o) {
      float mm = m2, ss = s2;
      combine_stats(mm, ss, m, s);
      m = mm;
      s = ss;
    } else {
      combine_stats(m, s, m2, s2);
    }
  }
  if (lane == 0) {
    const float l = m + logf(s);
    lse[r] = l;
    const int32_t y = labels[r];
    row_loss[r] = labelled(y, ignore, V) ? l - Z[r * V + y] : 0.0f;
  }
}

// The gradient: g = (exp(z - lse) - [j == y]) * inv_n (0 for an unlabelled
// row), rounded to bf16, G [rows][V].  A CTA takes 8192 columns of one row:
// each thread 8 float4 loads of Z in flight (read once, streaming) and
// 8-byte stores of 4 bf16.  V is a multiple of 8.
constexpr int kGradCols = 256 * 4 * 8;
__global__ void __launch_bounds__(256) k_lce_grad(const float* __restrict__ Z, int64_t rows, int64_t V,
                                                  const float* __restrict__ lse, const int32_t* __restrict__ labels,
                                                  int32_t ignore, const float* __restrict__ inv_n,
                                                  __nv_bfloat16* __restrict__ G) {
  const float sc = *inv_n;
  const int64_t j0 = (int64_t)blockIdx.x * kGradCols + 4 * threadIdx.x;
  for (int64_t r = blockIdx.y; r < rows; r += gridDim.y) {
    const int32_t y = labels[r];
    const bool on = labelled(y, ignore, V);
    const float l = lse[r];
    const float* zr = Z + r * V;
    __nv_bfloat16* gr = G + r * V;
    float4 z[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int64_t j = j0 + 1024 * u;
      z[u] = (on && j < V) ? __ldcs(reinterpret_cast<const float4*>(zr + j)) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int64_t j = j0 + 1024 * u;
      if (j < V) {
        float g0 = 0.0f, g1 = 0.0f, g2 = 0.0f, g3 = 0.0f;
        if (on) {
          g0 = (expf(z[u].x - l) - (j == y ? 1.0f : 0.0f)) * sc;
          g1 = (expf(z[u].y - l) - (j + 1 == y ? 1.0f : 0.0f)) * sc;
          g2 = (expf(z[u].z - l) - (j + 2 == y ? 1.0f : 0.0f)) * sc;
          g3 = (expf(z[u].w - l) - (j + 3 == y ? 1.0f : 0.0f)) * sc;
        }
        const __nv_bfloat162 lo = __floats2bfloat162_rn(g0, g1), hi = __floats2bfloat162_rn(g2, g3);
        uint2 w;
        w.x = *reinterpret_cast<const uint32_t*>(&lo);
        w.y = *reinterpret_cast<const uint32_t*>(&hi);
        *reinterpret_cast<uint2*>(gr + j) = w;
      }
    }
  }
}

// loss = sum of the rows' losses * inv_n, in fp64 and a fixed order.
__global__ void __launch_bounds__(1024) k_lce_loss(const float* __restrict__ row_loss, int64_t N,
                                                   const float* __restrict__ inv_n, double* __restrict__ loss) {
  __shared__ double red[1024];
  double a = 0.0;
  for (int64_t i = threadIdx.x; i < N; i += blockDim.x) a += (double)row_loss[i];
  red[threadIdx.x] = a;
  __syncthreads();
  for (int s = blockDim.x / 2; s > 0; s >>= 1) {
    if ((int)threadIdx.x < s) red[threadIdx.x] += red[threadIdx.x + s];
    __syncthreads();
  }
  if (threadIdx.x == 0) *loss = red[0] * (double)*inv_n;
}

struct LcePlan {
  size_t off_z, off_g, off_lse, off_rowloss, off_n, off_stats, bytes;
};

// Workspace of one call: the chunk's logits and gradient, its row statistics,
// the row losses of all tokens, the labelled-token count (no dependence on D:
// nothing is transposed).
LcePlan plan_lce(int64_t N, int64_t V, int64_t chunk) {
  LcePlan p;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = (off + bytes + 255) / 256 * 256;
    return o;
  };
  p.off_z = take((size_t)chunk * V * 4);
  p.off_g = take((size_t)chunk * V * 2);
  p.off_lse = take((size_t)chunk * 4);
  p.off_rowloss = take((size_t)N * 4);
  p.off_n = take(16);
  p.off_stats = take((size_t)chunk * ((V + kTcTileN - 1) / kTcTileN) * 8);
  p.bytes = off;
  return p;
}

// ---- the form by pieces of the vocabulary --------------------------------
//
// The loss over all tokens and pieces of the vocabulary, for training steps
// whose chunk x V logits would not fit beside the model:
//   0. The n labelled tokens' rows of H are copied together (a token without a
//      label has no loss and no gradient, so it costs nothing further, and a
//      NaN in it reaches nothing).  n stays on the device: the products below
//      read it there.
//   1. Z = H W^T once, every tile reduced in the GEMM's epilogue to (max, sum
//      exp) per row and the labels' logits: the logits never leave tensor
//      memory.  The last piece's exponentials stay in the workspace (short
//      rows apart, whose logits are cheaper to compute again).
//   2. lse, the tokens' losses, the loss; the last piece's exponentials become
//      its gradient G = softmax - onehot in bf16.  The factor scale / n stays
//      out of G: a label's entry is close to -1 / n for every token, and its
//      rounding to bf16 would scale the whole gradient by up to 2^-9 (measured:
//      dW off by 0.35 % with the factor in G, 0.17 % without).
//   3. Per piece, the last first: dH += f G W_piece, dW_piece = f G^T H, f =
//      scale / n in fp32; for the others G is formed first, as the epilogue of
//      Z once more.
// 8 - 2 / P times n D V flops for P pieces (8192 x 4096 x 128256: 19.2 ms with
// 16 pieces in 0.40 GB, 17.9 with 4 in 0.80, 16.9 with 2 in 1.32, 15.0 with one
// in 2.2; the token-chunk form takes 28.5 ms in 0.40 GB, 16.4 in 3.6), against 6 when a token chunk's
// logits are kept, but the workspace is one n x piece block of bf16 whatever
// V, every row of dW is written once, in bf16 if asked (the type that the
// AdamW step takes), and dW is not read back for accumulation.  Up to 16 tokens
// take another form (lce_few.cuh).

constexpr int kPairsGb300 = 76;                       // CTA pairs of the GEMM's persistent grid (152 SMs)
constexpr size_t kPieceBudget = (size_t)1 << 30;      // bytes of G that the default piece may take

struct GatherArgs {
  const uint16_t* H;       // [N][ldh]
  int64_t ldh, N, D, V;
  const int32_t* labels;
  int32_t ignore;
  double grad_scale;
  uint16_t* Hc;            // [N][ldc]: the labelled rows in order, then zeros up to a multiple of 64 rows
  int64_t ldc;
  int32_t* label_c;        // [N]: their labels
  int32_t* token;          // [N]: their token
  int32_t* place;          // [N]: each token's row in Hc, or -1
  int32_t* n_out;
  float* factor;           // grad_scale / n (0 if n = 0)
  uint32_t* counter;       // set to 0 for k_lce_rows
  float* loss;             // set to 0 (the answer if n = 0); may be null
  float* token_loss;       // set to 0 at unlabelled tokens; may be null
  void* dH;                // unlabelled tokens' rows set to 0; may be null
  int64_t lddh;
  int32_t dh_fp32;
};

// One block per 8 tokens, a warp each.  Every block counts the labels before
// its own and all labels (N words from L2), so no second launch and no order
// between blocks is needed.
__global__ void __launch_bounds__(256) k_lce_gather(const GatherArgs a) {
  __shared__ int before_w[8], all_w[8], mine[8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t0 = (int64_t)blockIdx.x * 8;
  griddep_launch_dependents();
  // this warp's row on its way to L2 while the labels are counted
  if (t0 + warp < a.N)
    for (int64_t c = 64 * lane; c < a.D; c += 64 * 32)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(a.H + (t0 + warp) * a.ldh + c));
  int before = 0, all = 0;
  bool bad = false;
#pragma unroll 8
  for (int64_t i = threadIdx.x; i < a.N; i += 256) {
    const int32_t y = a.labels[i];
    const bool on = labelled(y, a.ignore, a.V);
    all += on;
    before += on && i < t0;
    bad |= !on && y != a.ignore;
  }
  if (bad && blockIdx.x == 0) atomicOr(&g_device_error, kDevErrIndex);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    before += __shfl_xor_sync(0xffffffffu, before, o);
    all += __shfl_xor_sync(0xffffffffu, all, o);
  }
  const int64_t tok = t0 + warp;
  const int32_t y = tok < a.N ? a.labels[tok] : a.ignore;
  const bool on = tok < a.N && labelled(y, a.ignore, a.V);
  if (lane == 0) {
    before_w[warp] = before;
    all_w[warp] = all;
    mine[warp] = on;
  }
  __syncthreads();
  int n = 0, r = 0;
#pragma unroll
  for (int w = 0; w < 8; ++w) {
    n += all_w[w];
    r += before_w[w] + (w < warp ? mine[w] : 0);
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    *a.n_out = n;
    *a.factor = n > 0 ? (float)(a.grad_scale / (double)n) : 0.0f;
    *a.counter = 0;
    if (a.loss) *a.loss = 0.0f;
  }
  if (tok < a.N) {
    if (lane == 0) {
      a.place[tok] = on ? r : -1;
      if (on) {
        a.label_c[r] = y;
        a.token[r] = (int32_t)tok;
      } else if (a.token_loss) {
        a.token_loss[tok] = 0.0f;
      }
    }
    // rows are 16-byte aligned; the last unit may hold columns beyond D, of the row's own padding
    const int units = (int)((a.D + 7) / 8);
    if (on) {
      const uint4* from = reinterpret_cast<const uint4*>(a.H + tok * a.ldh);
      uint4* to = reinterpret_cast<uint4*>(a.Hc + (int64_t)r * a.ldc);
#pragma unroll 8
      for (int u = lane; u < units; u += 32) {
        if (u * 8 + 8 <= a.D) {
          to[u] = from[u];
        } else {
          for (int c = u * 8; c < a.D; ++c) a.Hc[(int64_t)r * a.ldc + c] = a.H[tok * a.ldh + c];
        }
      }
    } else if (a.dH) {
      if (a.dh_fp32) {
        float* p = static_cast<float*>(a.dH) + tok * a.lddh;
        for (int c = lane; c < a.D; c += 32) p[c] = 0.0f;
      } else {
        uint16_t* p = static_cast<uint16_t*>(a.dH) + tok * a.lddh;
        for (int c = lane; c < a.D; c += 32) p[c] = 0;
      }
    }
  }
  // the rows after the last labelled one, up to a whole K slab of dW's product
  const int64_t end = min(a.N, (int64_t)(n + 63) / 64 * 64);
  for (int64_t q = n + blockIdx.x; q < end; q += gridDim.x)
    for (int c = threadIdx.x; c < a.D; c += 256) a.Hc[q * a.ldc + c] = 0;
}

struct RowsArgs {
  const float2* stats;     // [N][n_tiles]
  int32_t n_tiles;
  const int32_t* n_dev;
  const float* label_logit;
  const int32_t* label_c;
  const int32_t* token;
  __nv_bfloat16* G;        // [N][ldg], the last piece; may be null (no gradients)
  int64_t ldg;
  int32_t cols, col0;      // its columns
  int32_t span;            // columns of a block
  float* lse;              // [N]
  float* row_loss;         // [N]
  float* token_loss;       // by token; may be null
  float* loss;             // may be null
  uint32_t* counter;
  int64_t N;
};

// One block per labelled row and span of columns: the row's lse from its tile
// statistics, and the span of G, holding exp(z - tile maximum), becomes the
// gradient: times exp(tile maximum - lse); the label's column comes from its
// fp32 logit, because exp(z - lse) - 1 cancels where the model is
// sure.  The span's loads are in flight while lse is taken (each block of a
// row takes it again: a few hundred values).  4 bytes an element of G, against
// 2 D flops for computing z again.  The blocks of the first span write the
// row's loss, and the last of them sums all losses in a fixed order.
constexpr int kSpanUnits = 8;
__global__ void __launch_bounds__(256) k_lce_rows(const RowsArgs a) {
  __shared__ float red_m[8], red_s[8];
  __shared__ bool last;
  griddep_launch_dependents();
  griddep_wait();
  const int n = *a.n_dev;
  const int64_t r = blockIdx.x;
  const int c0 = blockIdx.y * a.span + 8 * (int)threadIdx.x, c1 = min(a.cols, ((int)blockIdx.y + 1) * a.span);
  if (r >= n) {
    // rows that a K slab of dW's product still reads
    if (a.G && r < (n + 63) / 64 * 64)
      for (int c = c0; c < c1; c += 2048) *reinterpret_cast<uint4*>(a.G + r * a.ldg + c) = make_uint4(0, 0, 0, 0);
    return;
  }
  uint4 v[kSpanUnits];
  if (a.G) {
#pragma unroll
    for (int u = 0; u < kSpanUnits; ++u)
      if (c0 + 2048 * u < c1) v[u] = *reinterpret_cast<const uint4*>(a.G + r * a.ldg + c0 + 2048 * u);
  }
  const float2* st = a.stats + r * a.n_tiles;
  float m = -INFINITY, s = 0.0f;
  // the maximum first, so that the exponentials do not wait for one another
#pragma unroll 4
  for (int t = threadIdx.x; t < a.n_tiles; t += 256) m = fmaxf(m, st[t].x);
#pragma unroll 4
  for (int t = threadIdx.x; t < a.n_tiles; t += 256) {
    const float2 p = st[t];
    s += p.x == -INFINITY ? 0.0f : p.y * expf(p.x - m);
  }
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    float m2 = __shfl_xor_sync(0xffffffffu, m, o), s2 = __shfl_xor_sync(0xffffffffu, s, o);
    if (threadIdx.x & o) {
      combine_stats(m2, s2, m, s);
      m = m2;
      s = s2;
    } else {
      combine_stats(m, s, m2, s2);
    }
  }
  if ((threadIdx.x & 31) == 0) {
    red_m[threadIdx.x >> 5] = m;
    red_s[threadIdx.x >> 5] = s;
  }
  __syncthreads();
  m = red_m[0];
  s = red_s[0];
#pragma unroll
  for (int w = 1; w < 8; ++w) combine_stats(m, s, red_m[w], red_s[w]);
  const float l = m + logf(s), zy = a.label_logit[r];
  if (a.G) {
    const int y = a.label_c[r] - a.col0;
    const float gy = expm1f(zy - l);
#pragma unroll
    for (int u = 0; u < kSpanUnits; ++u) {
      const int c = c0 + 2048 * u;
      if (c >= c1) break;
      const float tm = st[(a.col0 + c) / kTcStatCols].x;
      const float k = exp2_approx(((tm == -INFINITY ? 0.0f : tm) - l) * kLog2e);
      const uint64_t k2 = pack_f2(k, k);
      const uint32_t in[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
      uint32_t out[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        out[i] = bf16x2_rn(fmul2(pack_f2(__uint_as_float(in[i] << 16), __uint_as_float(in[i] & 0xFFFF0000u)), k2));
      if ((unsigned)(y - c) < 8u) {
        const uint32_t g = __bfloat16_as_ushort(__float2bfloat16_rn(gy));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (y - c == 2 * i) out[i] = (out[i] & 0xFFFF0000u) | g;
          if (y - c == 2 * i + 1) out[i] = (out[i] & 0xFFFFu) | g << 16;
        }
      }
      *reinterpret_cast<uint4*>(a.G + r * a.ldg + c) = make_uint4(out[0], out[1], out[2], out[3]);
    }
  }
  if (blockIdx.y != 0) return;
  if (threadIdx.x == 0) {
    a.lse[r] = l;
    a.row_loss[r] = l - zy;
    if (a.token_loss) {
      // labels that change during the call can leave rows without a token
      const int32_t t = a.token[r];
      if (t >= 0 && t < a.N) a.token_loss[t] = l - zy;
      else atomicOr(&g_device_error, kDevErrIndex);
    }
    __threadfence();
    last = atomicAdd(a.counter, 1u) == (uint32_t)(n - 1);
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  __shared__ double sums[8];
  double t = 0.0;
  for (int i = threadIdx.x; i < n; i += 256) t += (double)__ldcg(a.row_loss + i);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
  if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = t;
  __syncthreads();
  if (threadIdx.x == 0 && a.loss) {
    t = 0.0;
    for (int w = 0; w < 8; ++w) t += sums[w];
    *a.loss = (float)(t / (double)n);
  }
}

// out [M][N] = sum over the parts [S][M][ld], rounded to bf16 or kept in fp32;
// with `place`, out's row r is the parts' row place[r], zero where that is -1.
// ld is a multiple of 4; out rows are 16-byte aligned.  For few groups of many
// parts, G = 8 or 32 threads share a group of four columns, each over every G-th
// part, and their sums are added in order (6 tokens, 64 columns, 62 parts: the whole loss 46 us, with one thread a
// group 57).
template <int G>
__global__ void __launch_bounds__(256) k_lce_sum_parts(const float* parts, int S, int64_t M, int64_t N, int64_t ld,
                                                       const int32_t* place, void* out, int64_t ldo, int fp32) {
  constexpr int kGroups = 256 / G;
  __shared__ float4 sums[G][G == 1 ? 1 : kGroups];
  griddep_launch_dependents();
  griddep_wait();
  const int x = threadIdx.x % kGroups, y = threadIdx.x / kGroups;
  const int64_t per_row = (N + 3) / 4, total = M * per_row;
  for (int64_t base = (int64_t)blockIdx.x * kGroups; base < total; base += (int64_t)gridDim.x * kGroups) {
    const int64_t i = base + x, r = i / per_row, c = 4 * (i - r * per_row);
    const int64_t from = i >= total ? -1 : place ? (int64_t)place[r] : r;
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (from >= 0) {
#pragma unroll 4
      for (int s = y; s < S; s += G) {
        const float4 w = __ldcs(reinterpret_cast<const float4*>(parts + ((int64_t)s * M + from) * ld + c));
        v.x += w.x;
        v.y += w.y;
        v.z += w.z;
        v.w += w.w;
      }
    }
    if (G > 1) {
      __syncthreads();
      sums[y][x] = v;
      __syncthreads();
      if (y > 0) continue;
#pragma unroll
      for (int q = 1; q < G; ++q) {
        const float4 w = sums[q][x];
        v.x += w.x;
        v.y += w.y;
        v.z += w.z;
        v.w += w.w;
      }
    }
    if (i >= total) continue;
    const float e[4] = {v.x, v.y, v.z, v.w};
    const int n = (int)min((int64_t)4, N - c);
    if (fp32) {
      float* p = static_cast<float*>(out) + r * ldo + c;
      if (n == 4) *reinterpret_cast<float4*>(p) = v;
      else
        for (int q = 0; q < n; ++q) p[q] = e[q];
    } else {
      __nv_bfloat16* p = static_cast<__nv_bfloat16*>(out) + r * ldo + c;
      if (n == 4) {
        const __nv_bfloat162 lo = __floats2bfloat162_rn(e[0], e[1]), hi = __floats2bfloat162_rn(e[2], e[3]);
        *reinterpret_cast<uint2*>(p) =
            make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
      } else {
        for (int q = 0; q < n; ++q) p[q] = __float2bfloat16_rn(e[q]);
      }
    }
  }
}

// Parts of a product's sum over K, so that few output tiles still fill the
// grid: the number that minimises waves x slabs per item, with 24 slabs
// (about 6 us) charged for writing and adding the parts.
int pick_splits(int64_t M, int64_t N, int64_t K) {
  const int64_t tiles = ceil_div<int64_t>(M, 256) * ceil_div<int64_t>(N, 256), slabs = ceil_div<int64_t>(K, 64);
  int best = 1;
  int64_t cost = ceil_div<int64_t>(tiles, kPairsGb300) * slabs;
  for (int s = 2; s <= 64 && s <= slabs && tiles * s <= 2 * kPairsGb300; ++s) {
    const int64_t c = ceil_div<int64_t>(tiles * s, kPairsGb300) * ceil_div<int64_t>(slabs, s) + 24;
    if (c < cost) {
      cost = c;
      best = s;
    }
  }
  return best;
}

// Whether the last piece's exponentials are kept (written once, read and
// written again by the rows kernel) or its logits computed again, which is
// cheaper for short rows and many logits.  Kept / again, us: 4000 x 64000
// logits of rows of 256 599 / 522, of 512 734 / 689, of 768 897 / 909; rows
// of 64 by 65536 outputs, 2048 tokens 311 / 273, 1024 tokens 170 / 171, 512
// tokens 88 / 102.
inline bool keeps_exponentials(int64_t N, int64_t D, int64_t cols) { return D > 512 || N * cols <= (int64_t)1 << 26; }

struct VocabPlan {
  int64_t pieces, piece, ldg, ldd, ldc;
  int n_tiles;
  int s_dh;                 // parts of dH's sum over a piece
  bool dh_direct;           // dH goes to its rows from the product's epilogue
  size_t off_h, off_g, off_stats, off_rows, off_words, off_dh, off_dw, bytes;
};

VocabPlan plan_vocab(int64_t N, int64_t D, int64_t V, int64_t piece) {
  VocabPlan p;
  if (piece <= 0) {
    // as many columns as the budget holds, in pieces of equal size
    const int64_t most = std::max<int64_t>(2048, (int64_t)(kPieceBudget / 2) / N / 256 * 256);
    piece = ceil_div<int64_t>(ceil_div<int64_t>(V, ceil_div<int64_t>(V, most)), 256) * 256;
  }
  piece = std::min(piece, ceil_div<int64_t>(V, 256) * 256);      // any piece of at least V is the whole vocabulary
  p.pieces = ceil_div<int64_t>(V, piece);
  p.piece = std::min(piece, V);
  p.ldg = ceil_div<int64_t>(p.piece, 64) * 64;
  p.ldd = ceil_div<int64_t>(D, 4) * 4;
  p.ldc = ceil_div<int64_t>(D, 8) * 8;
  p.n_tiles = (int)ceil_div<int64_t>(V, kTcStatCols);
  p.s_dh = pick_splits(N, D, p.piece);
  // the last piece may be shorter than a part count chosen for whole ones
  const int64_t last = V - (p.pieces - 1) * p.piece;
  p.s_dh = (int)std::min<int64_t>(p.s_dh, ceil_div<int64_t>(last, 64));
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = (off + bytes + 255) / 256 * 256;
    return o;
  };
  p.dh_direct = p.pieces == 1 && p.s_dh == 1;
  p.off_h = take((size_t)N * p.ldc * 2);
  p.off_g = take((size_t)N * p.ldg * 2);
  p.off_stats = take((size_t)N * p.n_tiles * 8);
  p.off_rows = take((size_t)N * 4 * 6);          // labels, tokens, places, label logits, lse, losses
  p.off_words = take(16);                        // n, factor, counter
  p.off_dh = take(p.dh_direct ? 0 : (size_t)p.s_dh * N * p.ldd * 4);
  // dW goes to its rows straight from the epilogue only where they are whole
  // 16-byte units: a tensor store writes whole ones
  const bool ragged = D % 8 != 0;
  const int s1 = pick_splits(p.piece, D, N), s2 = pick_splits(last, D, N);
  p.off_dw = take(std::max(s1 > 1 || ragged ? (size_t)s1 * p.piece * p.ldd * 4 : 0,
                           s2 > 1 || ragged ? (size_t)s2 * last * p.ldd * 4 : 0));
  p.bytes = off;
  return p;
}

sf_status sum_parts(const float* parts, int S, int64_t M, int64_t N, int64_t ld, const int32_t* place, void* out,
                    int64_t ldo, bool fp32, cudaStream_t s) {
  // threads a group: more than one where there are too few groups to fill the
  // SMs (512 x 2048, nine parts, 262144 groups: the loss 5 % slower with eight)
  const int64_t groups = M * ceil_div<int64_t>(N, 4);
  const int g = groups >= (int64_t)sm_count() * 512 || S < 8 ? 1 : S < 64 ? 8 : 32;
  const int64_t want = ceil_div<int64_t>(groups, 256 / g);
  SF_CUDA_TRY(launch_pdl(g == 32 ? k_lce_sum_parts<32> : g == 8 ? k_lce_sum_parts<8> : k_lce_sum_parts<1>,
                         dim3((unsigned)std::min<int64_t>(want, (int64_t)sm_count() * 8)), dim3(256), 0, s, parts, S, M, N, ld,
                         place, out, ldo, (int)fp32),
              "launch k_lce_sum_parts");
  return SF_OK;
}

}  // namespace
}  // namespace sf

#include "lce_few.cuh"

namespace sf {

const void* device_error_lce() { return &g_device_error; }

}  // namespace sf

extern "C" {

size_t lce_workspace_bytes(int64_t n_tokens, int64_t d, int64_t vocab, int64_t chunk) {
  if (n_tokens < 1 || d < 1 || vocab < 1 || chunk < 1) return 0;
  return sf::plan_lce(n_tokens, vocab, std::min(chunk, (n_tokens + 7) / 8 * 8)).bytes;
}

sf_status lce_forward_backward(const void* H, const void* W, const int32_t* labels, int64_t N, int64_t D, int64_t V,
                               int64_t chunk, int32_t ignore_index, double* loss, float* dH, float* dW, void* ws,
                               size_t ws_bytes, void* stream_) {
  sf::clear_error();
  sf::NvtxRange nvtx_range("lce_forward_backward");
  if (!H || !W || !labels) return sf::fail(SF_ERR_INVALID, "H, W or labels is NULL");
  if (N < 1 || D < 1 || V < 1) return sf::fail(SF_ERR_INVALID, "N, D, V must be >= 1");
  if (D % 8 || V % 8) return sf::fail(SF_ERR_UNSUPPORTED, "D and V must be multiples of 8 (16-byte rows)");
  if (chunk < 8 || chunk % 8) return sf::fail(SF_ERR_INVALID, "chunk must be a positive multiple of 8");
  if ((reinterpret_cast<uintptr_t>(H) % 16) || (reinterpret_cast<uintptr_t>(W) % 16))
    return sf::fail(SF_ERR_UNSUPPORTED, "H and W need 16-byte aligned bases");
  if ((dH && reinterpret_cast<uintptr_t>(dH) % 16) || (dW && reinterpret_cast<uintptr_t>(dW) % 16))
    return sf::fail(SF_ERR_UNSUPPORTED, "dH and dW need 16-byte aligned bases");
  chunk = std::min(chunk, (N + 7) / 8 * 8);
  if (V > (int64_t)INT32_MAX / 2 || N > (int64_t)INT32_MAX || D > (int64_t)INT32_MAX / 2)
    return sf::fail(SF_ERR_UNSUPPORTED, "sizes too large");
  const sf::LcePlan p = sf::plan_lce(N, V, chunk);
  if (!ws || ws_bytes < p.bytes || (reinterpret_cast<uintptr_t>(ws) % 256))
    return sf::fail(SF_ERR_INVALID, "workspace needs %zu bytes, 256-byte aligned (got %zu)", p.bytes, ws_bytes);
  cudaStream_t s = sf::as_stream(stream_);
  char* w = static_cast<char*>(ws);
  float* Z = reinterpret_cast<float*>(w + p.off_z);
  __nv_bfloat16* G = reinterpret_cast<__nv_bfloat16*>(w + p.off_g);
  float* lse = reinterpret_cast<float*>(w + p.off_lse);
  float* row_loss = reinterpret_cast<float*>(w + p.off_rowloss);
  int64_t* n_valid = reinterpret_cast<int64_t*>(w + p.off_n);
  float* inv_n = reinterpret_cast<float*>(w + p.off_n + 8);
  float2* stats = reinterpret_cast<float2*>(w + p.off_stats);
  const int n_vt = (int)((V + sf::kTcTileN - 1) / sf::kTcTileN);
  const uint16_t* Hb = static_cast<const uint16_t*>(H);
  const bool grads = dH || dW;

  sf::k_lce_count<<<1, 1024, 0, s>>>(labels, N, V, ignore_index, n_valid, inv_n);
  SF_TRY(sf::check_launch("k_lce_count"));
  for (int64_t c0 = 0; c0 < N; c0 += chunk) {
    const int64_t rows = std::min(chunk, N - c0);
    SF_TRY(sf::tc_gemm(Hb + c0 * D, false, W, false, Z, rows, V, D, D, D, V, 1.0f, false, s, stats));
    sf::k_lce_lse<<<(unsigned)sf::ceil_div<int64_t>(rows, 8), 256, 0, s>>>(stats, n_vt, rows, Z, V, labels + c0,
                                                                             ignore_index, lse, row_loss + c0);
    SF_TRY(sf::check_launch("k_lce_lse"));
    if (!grads) continue;
    const dim3 grid((unsigned)sf::ceil_div<int64_t>(V, sf::kGradCols), (unsigned)std::min<int64_t>(rows, 65535));
    sf::k_lce_grad<<<grid, 256, 0, s>>>(Z, rows, V, lse, labels + c0, ignore_index, inv_n, G);
    SF_TRY(sf::check_launch("k_lce_grad"));
    // dH_c = G_c W: G_c K-major [rows][V]; W is [V][D] = B stored [K][N]
    if (dH) SF_TRY(sf::tc_gemm(G, false, W, true, dH + c0 * D, rows, D, V, V, D, D, 1.0f, false, s));
    // dW += G_c^T H_c: A = G_c^T stored [K = rows][M = V], B = H_c^T stored [K][N = D]
    if (dW) SF_TRY(sf::tc_gemm(G, true, Hb + c0 * D, true, dW, V, D, rows, V, D, D, 1.0f, c0 > 0, s));
  }
  if (loss) {
    sf::k_lce_loss<<<1, 1024, 0, s>>>(row_loss, N, inv_n, loss);
    SF_TRY(sf::check_launch("k_lce_loss"));
  }
  return SF_OK;
}

size_t lce_vocab_workspace_bytes(int64_t n_tokens, int64_t d, int64_t vocab, int64_t piece) {
  if (n_tokens < 1 || d < 1 || vocab < 1 || piece < 0 || piece % sf::kTcTileN) return 0;
  return sf::few_tokens(n_tokens, d) ? sf::plan_few(n_tokens, d, vocab).bytes : sf::plan_vocab(n_tokens, d, vocab, piece).bytes;
}

sf_status lce_vocab_forward_backward(const sf_matrix* H, const sf_matrix* W, const int32_t* labels, int64_t piece,
                                     int32_t ignore_index, double grad_scale, float* loss, float* token_loss,
                                     const sf_matrix* dH, const sf_matrix* dW, void* ws, size_t ws_bytes,
                                     void* stream_) {
  using namespace sf;
  clear_error();
  NvtxRange nvtx_range("lce_vocab_forward_backward");
  constexpr unsigned kIn = 1u << SF_BF16, kOut = 1u << SF_BF16 | 1u << SF_FP32;
  SF_TRY(check_matrix(H, "H", -1, -1, kIn));
  const int64_t N = H->rows, D = H->cols;
  SF_TRY(check_matrix(W, "W", -1, D, kIn));
  const int64_t V = W->rows;
  if (N < 1 || D < 1 || V < 1) return fail(SF_ERR_INVALID, "H and W need at least one row and column");
  if (!labels) return fail(SF_ERR_INVALID, "labels is NULL");
  if (N > INT32_MAX / 2 || D > INT32_MAX / 2 || V > INT32_MAX / 4) return fail(SF_ERR_UNSUPPORTED, "sizes too large");
  if (piece < 0 || piece % kTcTileN) return fail(SF_ERR_INVALID, "piece must be 0 or a positive multiple of 256");
  SF_TRY(check_aligned(labels, sizeof(int32_t), "labels"));
  SF_TRY(check_aligned(loss, sizeof(float), "loss"));
  SF_TRY(check_aligned(token_loss, sizeof(float), "token_loss"));
  if (!(grad_scale - grad_scale == 0.0)) return fail(SF_ERR_INVALID, "grad_scale must be finite");
  const sf_matrix* const ins[2] = {H, W};
  for (const sf_matrix* m : ins)
    if (m->ld % 8 || reinterpret_cast<uintptr_t>(m->data) % 16 || m->ld < D)
      return fail(SF_ERR_UNSUPPORTED, "H and W need 16-byte aligned bases and rows (ld a multiple of 8)");
  if (dH) SF_TRY(check_matrix(dH, "dH", N, D, kOut));
  if (dW) SF_TRY(check_matrix(dW, "dW", V, D, kOut));
  const sf_matrix* const outs[2] = {dH, dW};
  for (const sf_matrix* m : outs)
    if (m && (m->ld * (int64_t)dtype_bytes(m->dtype) % 16 || reinterpret_cast<uintptr_t>(m->data) % 16 || m->ld < D))
      return fail(SF_ERR_UNSUPPORTED, "dH and dW need 16-byte aligned bases and rows");
  const size_t need = lce_vocab_workspace_bytes(N, D, V, piece);
  if (!ws || ws_bytes < need || reinterpret_cast<uintptr_t>(ws) % 256)
    return fail(SF_ERR_INVALID, "workspace needs %zu bytes, 256-byte aligned (got %zu)", need, ws_bytes);
  if (!tensor_map_encoder()) return fail(SF_ERR_UNSUPPORTED, "cuTensorMapEncodeTiled is not available");
  // tensor maps and bulk stores may only address this device's own memory
  const void* const dev[5] = {H->data, W->data, ws, dH ? dH->data : ws, dW ? dW->data : ws};
  for (const void* q : dev)
    if (!on_current_device(q))
      return fail(SF_ERR_INVALID, "H, W, dH, dW and the workspace must be device memory of the current device");
  cudaStream_t s = as_stream(stream_);
  char* w = static_cast<char*>(ws);
  if (few_tokens(N, D)) {
    const FewPlan p = plan_few(N, D, V);
    FewArgs a{};
    a.H = static_cast<const uint16_t*>(H->data);
    a.W = static_cast<const uint16_t*>(W->data);
    a.ldh = H->ld;
    a.ldw = W->ld;
    a.V = V;
    a.labels = labels;
    a.N = (int32_t)N;
    a.D = (int32_t)D;
    a.ignore = ignore_index;
    a.n_stats = p.n_stats;
    a.grad_scale = grad_scale;
    a.z = reinterpret_cast<float*>(w);
    a.stats = reinterpret_cast<float2*>(w + p.off_stats);
    a.label_logit = reinterpret_cast<float*>(w + p.off_logit);
    a.loss = loss;
    a.token_loss = token_loss;
    a.part = dH ? reinterpret_cast<float*>(w + p.off_part) : nullptr;
    if (dW) a.dW = dW->data, a.lddw = dW->ld, a.dw_fp32 = dW->dtype == SF_FP32;
    a.rows_part = dH || dW ? p.rows_part : 0;
    k_lce_few_logits<<<p.n_stats, 256, 0, s>>>(a);
    SF_TRY(check_launch("k_lce_few_logits"));
    const dim3 grid = dH || dW ? dim3((unsigned)p.blocks, (unsigned)ceil_div<int64_t>(D, 512)) : dim3(1);
    SF_CUDA_TRY(launch_pdl(k_lce_few_grads, grid, dim3(256), 0, s, a), "launch k_lce_few_grads");
    if (dH) SF_TRY(sum_parts(a.part, p.blocks, N, D, D, nullptr, dH->data, dH->ld, dH->dtype == SF_FP32, s));
    return SF_OK;
  }
  const VocabPlan p = plan_vocab(N, D, V, piece);
  uint16_t* Hc = reinterpret_cast<uint16_t*>(w + p.off_h);
  __nv_bfloat16* G = reinterpret_cast<__nv_bfloat16*>(w + p.off_g);
  float2* stats = reinterpret_cast<float2*>(w + p.off_stats);
  int32_t* label_c = reinterpret_cast<int32_t*>(w + p.off_rows);
  int32_t* token = label_c + N;
  int32_t* place = token + N;
  float* label_logit = reinterpret_cast<float*>(place + N);
  float* lse = label_logit + N;
  float* row_loss = lse + N;
  int32_t* n_dev = reinterpret_cast<int32_t*>(w + p.off_words);
  float* factor = reinterpret_cast<float*>(n_dev + 1);
  uint32_t* counter = reinterpret_cast<uint32_t*>(n_dev + 2);
  float* acc_dh = reinterpret_cast<float*>(w + p.off_dh);
  float* acc_dw = reinterpret_cast<float*>(w + p.off_dw);
  const uint16_t* Wb = static_cast<const uint16_t*>(W->data);
  const bool grads = dH || dW;

  GatherArgs ga{};
  ga.H = static_cast<const uint16_t*>(H->data);
  ga.ldh = H->ld;
  ga.N = N;
  ga.D = D;
  ga.V = V;
  ga.labels = labels;
  ga.ignore = ignore_index;
  ga.grad_scale = grad_scale;
  ga.Hc = Hc;
  ga.ldc = p.ldc;
  ga.label_c = label_c;
  ga.token = token;
  ga.place = place;
  ga.n_out = n_dev;
  ga.factor = factor;
  ga.counter = counter;
  ga.loss = loss;
  ga.token_loss = token_loss;
  if (dH && p.dh_direct) {
    ga.dH = dH->data;
    ga.lddh = dH->ld;
    ga.dh_fp32 = dH->dtype == SF_FP32;
  }
  k_lce_gather<<<(unsigned)ceil_div<int64_t>(N, 8), 256, 0, s>>>(ga);
  SF_TRY(check_launch("k_lce_gather"));

  // the logits of columns [v0, v0 + cols)
  TcJob z;
  z.checked = z.chained = true;
  z.A = Hc;
  z.lda = p.ldc;
  z.ldb = W->ld;
  z.M = N;
  z.m_dev = n_dev;
  z.K = D;
  z.labels = label_c;
  z.C = G;
  z.ldc = p.ldg;
  z.row_stats = stats;
  z.stats_ld = p.n_tiles;
  z.label_logit = label_logit;
  z.lse = lse;
  const int64_t last0 = (p.pieces - 1) * p.piece;      // the last piece's first column
  // columns from here on keep their exponentials
  const int64_t kept0 = grads && keeps_exponentials(N, D, V - last0) ? last0 : V;
  z.epi = kTcStats;
  if (kept0 > 0) {
    z.B = Wb;
    z.N = kept0;
    SF_TRY(tc_gemm(z, s));
  }
  if (kept0 < V) {
    z.B = Wb + kept0 * W->ld;
    z.N = V - kept0;
    z.col0 = (int32_t)kept0;
    z.store = true;
    SF_TRY(tc_gemm(z, s));
  }
  RowsArgs ra{};
  ra.stats = stats;
  ra.n_tiles = p.n_tiles;
  ra.n_dev = n_dev;
  ra.label_logit = label_logit;
  ra.label_c = label_c;
  ra.token = token;
  ra.lse = lse;
  ra.row_loss = row_loss;
  ra.token_loss = token_loss;
  ra.loss = loss;
  ra.counter = counter;
  ra.N = N;
  ra.span = 2048;
  int64_t spans = 1;
  if (kept0 < V) {
    ra.G = G;
    ra.ldg = p.ldg;
    ra.cols = (int32_t)(V - kept0);
    ra.col0 = (int32_t)kept0;
    // few rows: short spans, so that there are blocks for every SM
    while (ra.span < 2048 * kSpanUnits && N * ceil_div<int64_t>(ra.cols, 2 * ra.span) >= 1024) ra.span *= 2;
    spans = ceil_div<int64_t>(ra.cols, ra.span);
  }
  SF_CUDA_TRY(launch_pdl(k_lce_rows, dim3((unsigned)N, (unsigned)spans), dim3(256), 0, s, ra), "launch k_lce_rows");
  if (!grads) return SF_OK;

  for (int64_t q = p.pieces - 1; q >= 0; --q) {
    const int64_t v0 = q * p.piece, cols = std::min(p.piece, V - v0);
    const bool first = q == p.pieces - 1;
    if (!first || kept0 == V) {
      z.epi = kTcGrad;
      z.B = Wb + v0 * W->ld;
      z.N = cols;
      z.col0 = (int32_t)v0;
      SF_TRY(tc_gemm(z, s));
    }
    if (dH) {
      // dH += G W_piece: W is [K = cols][N = D] as stored
      TcJob j;
      j.checked = j.chained = true;
      j.A = G;
      j.lda = p.ldg;
      j.B = Wb + v0 * W->ld;
      j.ldb = W->ld;
      j.b_mn = true;
      j.M = N;
      j.m_dev = n_dev;
      j.scale = factor;
      j.N = D;
      j.K = cols;
      if (p.dh_direct) {
        j.epi = kTcRows;
        j.row_map = token;
        j.out_fp32 = dH->dtype == SF_FP32;
        j.C = dH->data;
        j.ldc = dH->ld;
      } else {
        j.epi = kTcSplit;
        j.splits = p.s_dh;
        j.accumulate = !first;
        j.C = acc_dh;
        j.ldc = p.ldd;
      }
      SF_TRY(tc_gemm(j, s));
    }
    if (dW) {
      // dW_piece = G^T H: G is [K = n][M = cols], H is [K = n][N = D] as stored
      TcJob j;
      j.checked = j.chained = true;
      j.A = G;
      j.lda = p.ldg;
      j.a_mn = true;
      j.B = Hc;
      j.ldb = p.ldc;
      j.b_mn = true;
      j.M = cols;
      j.N = D;
      j.K = N;
      j.k_dev = n_dev;
      j.scale = factor;
      const bool fp32 = dW->dtype == SF_FP32;
      void* out = static_cast<char*>(dW->data) + v0 * dW->ld * (int64_t)dtype_bytes(dW->dtype);
      j.splits = pick_splits(cols, D, N);
      if (j.splits == 1 && !fp32 && D % 8 == 0) {
        j.epi = kTcBf16;
        j.C = out;
        j.ldc = dW->ld;
        SF_TRY(tc_gemm(j, s));
      } else if (j.splits == 1 && fp32 && D % 4 == 0) {
        j.epi = kTcSplit;            // one part, straight to its place
        j.C = out;
        j.ldc = dW->ld;
        SF_TRY(tc_gemm(j, s));
      } else {
        j.epi = kTcSplit;
        j.C = acc_dw;
        j.ldc = p.ldd;
        SF_TRY(tc_gemm(j, s));
        SF_TRY(sum_parts(acc_dw, j.splits, cols, D, p.ldd, nullptr, out, dW->ld, fp32, s));
      }
    }
  }
  if (dH && !p.dh_direct)
    SF_TRY(sum_parts(acc_dh, p.s_dh, N, D, p.ldd, place, dH->data, dH->ld, dH->dtype == SF_FP32, s));
  return SF_OK;
}

}  // extern "C"
