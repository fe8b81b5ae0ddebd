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
//   1. Z = H W^T once, every tile reduced in the GEMM's epilogue to (max, sum
//      exp) per row and the labels' logits: the logits never leave tensor
//      memory.  The last piece's exponentials stay in the workspace.
//   2. lse, the tokens' losses, n and the loss.
//   3. Per piece, the last first: G = (softmax - onehot) * scale / n in bf16
//      (the last piece: its exponentials rescaled; the others: Z again, with
//      the gradient as the epilogue), dH += G W_piece, dW_piece = G^T H.
// 8 - 2 / P times N D V flops for P pieces, against 6 when a token chunk's
// logits are kept, but the workspace is one N x piece block of bf16 whatever
// V, every row of dW is written once, in bf16 if asked (the type that the
// AdamW step takes), and W is streamed P-independent times.

constexpr int kPairsGb300 = 76;                       // CTA pairs of the GEMM's persistent grid (152 SMs)
constexpr size_t kPieceBudget = (size_t)512 << 20;    // bytes of G that the default piece may take
constexpr float kLog2eF = 1.44269504f;

__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// One warp per row: lse from the row's tile statistics (as k_lce_lse), its
// loss; lse = +infinity marks an unlabelled row for the gradient.  The last
// block to finish sums the losses in a fixed order and sets the gradient's
// factor, so no further launch is needed.
__global__ void __launch_bounds__(256) k_lce_finish(const float2* __restrict__ stats, int n_tiles, int64_t N, int64_t V,
                                                    const float* __restrict__ label_logit,
                                                    const int32_t* __restrict__ labels, int32_t ignore,
                                                    double grad_scale, float* __restrict__ lse, float* row_loss,
                                                    float* __restrict__ token_loss, float* __restrict__ factor,
                                                    float* __restrict__ loss, uint32_t* counter) {
  const int lane = threadIdx.x & 31;
  const int64_t r = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (r < N) {
    float m = -INFINITY, s = 0.0f;
    for (int t = lane; t < n_tiles; t += 32) {
      const float2 p = stats[r * n_tiles + t];
      combine_stats(m, s, p.x, p.y);
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      float m2 = __shfl_xor_sync(0xffffffffu, m, o), s2 = __shfl_xor_sync(0xffffffffu, s, o);
      if (lane & o) {
        combine_stats(m2, s2, m, s);
        m = m2;
        s = s2;
      } else {
        combine_stats(m, s, m2, s2);
      }
    }
    if (lane == 0) {
      const int32_t y = labels[r];
      const bool on = labelled(y, ignore, V);
      if (!on && y != ignore) atomicOr(&g_device_error, kDevErrIndex);
      const float l = m + logf(s), a = on ? l - label_logit[r] : 0.0f;
      lse[r] = on ? l : INFINITY;
      row_loss[r] = a;
      if (token_loss) token_loss[r] = a;
    }
  }
  __shared__ bool last;
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    last = atomicAdd(counter, 1u) == gridDim.x - 1;
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  __shared__ double sums[256];
  __shared__ int64_t counts[256];
  double a = 0.0;
  int64_t c = 0;
  for (int64_t i = threadIdx.x; i < N; i += 256) {
    if (!labelled(labels[i], ignore, V)) continue;
    ++c;
    a += (double)__ldcg(row_loss + i);
  }
  sums[threadIdx.x] = a;
  counts[threadIdx.x] = c;
  __syncthreads();
  for (int h = 128; h > 0; h >>= 1) {
    if ((int)threadIdx.x < h) {
      sums[threadIdx.x] += sums[threadIdx.x + h];
      counts[threadIdx.x] += counts[threadIdx.x + h];
    }
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    const double n = (double)counts[0];
    *factor = n > 0 ? (float)(grad_scale / n) : 0.0f;
    if (loss) *loss = n > 0 ? (float)(sums[0] / n) : 0.0f;
  }
}

// G, holding exp(z - tile maximum), becomes the gradient: times
// exp(tile maximum - lse) * factor; the label's column from its fp32 logit,
// because exp(z - lse) - 1 cancels where the model is sure.  Eight columns a
// thread; 4 bytes an element, against 2 D flops for computing z again.
__global__ void __launch_bounds__(256) k_lce_rescale(__nv_bfloat16* __restrict__ G, int64_t ldg, int64_t rows, int cols,
                                                     int col0, const float2* __restrict__ stats, int n_tiles,
                                                     const float* __restrict__ lse,
                                                     const float* __restrict__ label_logit,
                                                     const int32_t* __restrict__ labels,
                                                     const float* __restrict__ factor) {
  const int j = 8 * (blockIdx.x * 256 + threadIdx.x);
  if (j >= cols) return;
  const float f = *factor;
  for (int64_t r = blockIdx.y; r < rows; r += gridDim.y) {
    uint4* p = reinterpret_cast<uint4*>(G + r * ldg + j);
    const float l = lse[r];
    if (l == INFINITY) {
      *p = make_uint4(0, 0, 0, 0);
      continue;
    }
    const uint4 w = *p;
    const float m = stats[r * n_tiles + (col0 + j) / kTcTileN].x;
    const float k = exp2_fast(((m == -INFINITY ? 0.0f : m) - l) * kLog2eF) * f;
    const uint32_t in[4] = {w.x, w.y, w.z, w.w};
    const int y = labels[r] - col0 - j;
    uint32_t out[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float a = __uint_as_float(in[i] << 16) * k, b = __uint_as_float(in[i] & 0xFFFF0000u) * k;
      if (y == 2 * i) a = (exp2_fast((label_logit[r] - l) * kLog2eF) - 1.0f) * f;
      if (y == 2 * i + 1) b = (exp2_fast((label_logit[r] - l) * kLog2eF) - 1.0f) * f;
      const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
      out[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *p = make_uint4(out[0], out[1], out[2], out[3]);
  }
}

// out [M][N] = sum over the parts [S][M][ld] in part order, rounded to bf16
// or kept in fp32.  ld is a multiple of 4; out rows are 16-byte aligned.
__global__ void __launch_bounds__(256) k_lce_sum_parts(const float* __restrict__ parts, int S, int64_t M, int64_t N,
                                                       int64_t ld, void* __restrict__ out, int64_t ldo, int fp32) {
  const int64_t per_row = (N + 3) / 4, total = M * per_row;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t r = i / per_row, c = 4 * (i - r * per_row);
    float4 v = __ldcs(reinterpret_cast<const float4*>(parts + r * ld + c));
    for (int s = 1; s < S; ++s) {
      const float4 w = __ldcs(reinterpret_cast<const float4*>(parts + ((int64_t)s * M + r) * ld + c));
      v.x += w.x;
      v.y += w.y;
      v.z += w.z;
      v.w += w.w;
    }
    const float x[4] = {v.x, v.y, v.z, v.w};
    const int n = (int)min((int64_t)4, N - c);
    if (fp32) {
      float* p = static_cast<float*>(out) + r * ldo + c;
      if (n == 4) *reinterpret_cast<float4*>(p) = v;
      else
        for (int q = 0; q < n; ++q) p[q] = x[q];
    } else {
      __nv_bfloat16* p = static_cast<__nv_bfloat16*>(out) + r * ldo + c;
      if (n == 4) {
        const __nv_bfloat162 lo = __floats2bfloat162_rn(x[0], x[1]), hi = __floats2bfloat162_rn(x[2], x[3]);
        *reinterpret_cast<uint2*>(p) =
            make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
      } else {
        for (int q = 0; q < n; ++q) p[q] = __float2bfloat16_rn(x[q]);
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

struct VocabPlan {
  int64_t pieces, piece, ldg, ldd;
  int n_tiles;
  int s_dh;                 // parts of dH's sum over a piece
  size_t off_g, off_stats, off_lse, off_logit, off_loss, off_words, off_dh, off_dw, bytes;
};

VocabPlan plan_vocab(int64_t N, int64_t D, int64_t V, int64_t piece) {
  VocabPlan p;
  if (piece <= 0) {
    // as many columns as the budget holds, in pieces of equal size
    const int64_t most = std::max<int64_t>(2048, (int64_t)(kPieceBudget / 2) / N / 256 * 256);
    piece = ceil_div<int64_t>(ceil_div<int64_t>(V, ceil_div<int64_t>(V, most)), 256) * 256;
  }
  p.pieces = ceil_div<int64_t>(V, piece);
  p.piece = std::min(piece, V);
  p.ldg = ceil_div<int64_t>(p.piece, 64) * 64;
  p.ldd = ceil_div<int64_t>(D, 4) * 4;
  p.n_tiles = (int)ceil_div<int64_t>(V, kTcTileN);
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
  p.off_g = take((size_t)N * p.ldg * 2);
  p.off_stats = take((size_t)N * p.n_tiles * 8);
  p.off_lse = take((size_t)N * 4);
  p.off_logit = take((size_t)N * 4);
  p.off_loss = take((size_t)N * 4);
  p.off_words = take(16);
  // a product goes to its output straight from the epilogue only where the
  // output's rows are whole 16-byte units: a tensor store writes whole ones
  const bool ragged = D % 8 != 0;
  p.off_dh = take(p.pieces > 1 || p.s_dh > 1 || ragged ? (size_t)p.s_dh * N * p.ldd * 4 : 0);
  const int s1 = pick_splits(p.piece, D, N), s2 = pick_splits(last, D, N);
  p.off_dw = take(std::max(s1 > 1 || ragged ? (size_t)s1 * p.piece * p.ldd * 4 : 0,
                           s2 > 1 || ragged ? (size_t)s2 * last * p.ldd * 4 : 0));
  p.bytes = off;
  return p;
}

sf_status sum_parts(const float* parts, int S, int64_t M, int64_t N, int64_t ld, void* out, int64_t ldo, bool fp32,
                    cudaStream_t s) {
  const int64_t want = ceil_div<int64_t>(M * ceil_div<int64_t>(N, 4), 256);
  k_lce_sum_parts<<<(unsigned)std::min<int64_t>(want, (int64_t)sm_count() * 8), 256, 0, s>>>(parts, S, M, N, ld, out,
                                                                                         ldo, fp32);
  return check_launch("k_lce_sum_parts");
}

}  // namespace

int read_and_clear_device_error_lce() {
  int v = 0, z = 0;
  if (cudaMemcpyFromSymbol(&v, g_device_error, sizeof v) != cudaSuccess) return 0;
  if (v) cudaMemcpyToSymbol(g_device_error, &z, sizeof z);
  return v;
}

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
  return sf::plan_vocab(n_tokens, d, vocab, piece).bytes;
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
  if (N > INT32_MAX / 2 || D > INT32_MAX / 2 || V > INT32_MAX / 2) return fail(SF_ERR_UNSUPPORTED, "sizes too large");
  if (piece < 0 || piece % kTcTileN) return fail(SF_ERR_INVALID, "piece must be 0 or a positive multiple of 256");
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
  const VocabPlan p = plan_vocab(N, D, V, piece);
  if (!ws || ws_bytes < p.bytes || reinterpret_cast<uintptr_t>(ws) % 256)
    return fail(SF_ERR_INVALID, "workspace needs %zu bytes, 256-byte aligned (got %zu)", p.bytes, ws_bytes);
  cudaStream_t s = as_stream(stream_);
  char* w = static_cast<char*>(ws);
  __nv_bfloat16* G = reinterpret_cast<__nv_bfloat16*>(w + p.off_g);
  float2* stats = reinterpret_cast<float2*>(w + p.off_stats);
  float* lse = reinterpret_cast<float*>(w + p.off_lse);
  float* label_logit = reinterpret_cast<float*>(w + p.off_logit);
  float* row_loss = reinterpret_cast<float*>(w + p.off_loss);
  float* factor = reinterpret_cast<float*>(w + p.off_words);
  uint32_t* counter = reinterpret_cast<uint32_t*>(w + p.off_words + 4);
  float* acc_dh = reinterpret_cast<float*>(w + p.off_dh);
  float* acc_dw = reinterpret_cast<float*>(w + p.off_dw);
  const uint16_t* Wb = static_cast<const uint16_t*>(W->data);
  const bool grads = dH || dW;

  // the logits of columns [v0, v0 + cols)
  TcJob z;
  z.A = H->data;
  z.lda = H->ld;
  z.ldb = W->ld;
  z.M = N;
  z.K = D;
  z.labels = labels;
  z.C = G;
  z.ldc = p.ldg;
  z.row_stats = stats;
  z.stats_ld = p.n_tiles;
  z.label_logit = label_logit;
  z.lse = lse;
  z.factor = factor;
  const int64_t last0 = (p.pieces - 1) * p.piece;      // the last piece's first column
  const int64_t kept0 = grads ? last0 : V;             // columns from here on keep their exponentials
  z.epi = kTcStats;
  z.zero = counter;
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
  k_lce_finish<<<(unsigned)ceil_div<int64_t>(N, 8), 256, 0, s>>>(stats, p.n_tiles, N, V, label_logit, labels,
                                                                 ignore_index, grad_scale, lse, row_loss, token_loss,
                                                                 factor, loss, counter);
  SF_TRY(check_launch("k_lce_finish"));
  if (!grads) return SF_OK;

  auto whole = [&](const sf_matrix* m) { return D * (int64_t)dtype_bytes(m->dtype) % 16 == 0; };
  const bool dh_direct = dH && p.s_dh == 1 && (p.pieces == 1 || dH->dtype == SF_FP32) && whole(dH);
  for (int64_t q = p.pieces - 1; q >= 0; --q) {
    const int64_t v0 = q * p.piece, cols = std::min(p.piece, V - v0);
    const bool first = q == p.pieces - 1;
    if (first) {
      const dim3 grid((unsigned)ceil_div<int64_t>(cols, 2048), (unsigned)std::min<int64_t>(N, 65535));
      k_lce_rescale<<<grid, 256, 0, s>>>(G, p.ldg, N, (int)cols, (int)v0, stats, p.n_tiles, lse, label_logit, labels,
                                         factor);
      SF_TRY(check_launch("k_lce_rescale"));
    } else {
      z.epi = kTcGrad;
      z.B = Wb + v0 * W->ld;
      z.N = cols;
      z.col0 = (int32_t)v0;
      SF_TRY(tc_gemm(z, s));
    }
    if (dH) {
      // dH += G W_piece: W is [K = cols][N = D] as stored
      TcJob j;
      j.A = G;
      j.lda = p.ldg;
      j.B = Wb + v0 * W->ld;
      j.ldb = W->ld;
      j.b_mn = true;
      j.M = N;
      j.N = D;
      j.K = cols;
      j.accumulate = !first;
      if (dh_direct) {
        j.epi = dH->dtype == SF_FP32 ? kTcF32 : kTcBf16;
        j.C = dH->data;
        j.ldc = dH->ld;
      } else {
        j.epi = kTcSplit;
        j.splits = p.s_dh;
        j.C = acc_dh;
        j.ldc = p.ldd;
      }
      SF_TRY(tc_gemm(j, s));
    }
    if (dW) {
      // dW_piece = G^T H: G is [K = N][M = cols], H is [K = N][N = D] as stored
      TcJob j;
      j.A = G;
      j.lda = p.ldg;
      j.a_mn = true;
      j.B = H->data;
      j.ldb = H->ld;
      j.b_mn = true;
      j.M = cols;
      j.N = D;
      j.K = N;
      void* out = static_cast<char*>(dW->data) + v0 * dW->ld * (int64_t)dtype_bytes(dW->dtype);
      j.splits = pick_splits(cols, D, N);
      if (j.splits == 1 && whole(dW)) {
        j.epi = dW->dtype == SF_FP32 ? kTcF32 : kTcBf16;
        j.C = out;
        j.ldc = dW->ld;
        SF_TRY(tc_gemm(j, s));
      } else {
        j.epi = kTcSplit;
        j.C = acc_dw;
        j.ldc = p.ldd;
        SF_TRY(tc_gemm(j, s));
        SF_TRY(sum_parts(acc_dw, j.splits, cols, D, p.ldd, out, dW->ld, dW->dtype == SF_FP32, s));
      }
    }
  }
  if (dH && !dh_direct)
    SF_TRY(sum_parts(acc_dh, p.s_dh, N, D, p.ldd, dH->data, dH->ld, dH->dtype == SF_FP32, s));
  return SF_OK;
}

}  // extern "C"
