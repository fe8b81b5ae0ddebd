// The vocabulary-piece cross-entropy for at most 16 tokens: three launches that
// stream W, instead of six around the tiled products, whose 256-row tiles would
// be nearly empty.  Bound by W and dW (2 bytes an entry read twice and written
// once) and, where those are small, by latencies that add up: the second kernel reads W only once the
// statistics are joined and z has become g (19 of 24 us at 16 x 1024 x 8000, for data worth 5).
//   k_lce_few_logits  z = W h for 16 tokens at a time on the warp-level tensor
//                     instruction (16 tokens fill one of its operands; the
//                     products are far from bounding anything), z kept in fp32
//                     [V][16], statistics per block;
//   k_lce_few_grads   every block joins the statistics and turns its rows of z
//                     into the gradient g = softmax - onehot in bf16; dW's rows
//                     leave once, dH's sums over the block's rows as one part;
//   k_lce_sum_parts   dH.
// Operands go from memory straight to registers in 16-byte loads: the order of
// the summed index, and which column of the output a lane's fragment stands
// for, are free to choose, so fragments are what the lanes have loaded.
// Against the tiled products: 16 x 1024 x 8000 24 us (39), 6 x 64 x 74225 23
// (57), 1 x 4096 x 32000 180 (229; W twice at the copy rate and dW at the 4 TB/s
// of writing alone: 144), 16 x 4096 x 128256 652 (645).  Fetching the next
// rows into L2 ahead was slower (198 us at 1 x 4096 x 32000).
#pragma once

namespace sf {
namespace {

constexpr int kFewTokens = 16;

struct FewArgs {
  const uint16_t* H;       // [N][ldh]
  const uint16_t* W;       // [V][ldw]
  int64_t ldh, ldw, V;
  const int32_t* labels;
  int32_t N, D, ignore;
  int32_t n_stats;         // blocks of the first kernel
  double grad_scale;
  float* z;                // [V][16]
  float2* stats;           // [n_stats][16]
  float* label_logit;      // [16]
  float* loss;             // may be null
  float* token_loss;       // may be null
  float* part;             // [parts][N][D]; null without dH
  void* dW;                // [V][lddw]; may be null
  int64_t lddw;
  int32_t dw_fp32;
  int64_t rows_part;       // rows of a block of the second kernel, a multiple of 16
};

// C[16 x 8] += A[16 x 16] B[16 x 8], bf16 in, fp32 sums.  With g = lane / 4 and
// t = lane % 4, a0..a3 hold A's rows g, g + 8, g, g + 8 at k = 2t (+ 1), and
// for a2, a3 8 more; b0, b1 B's column g at k = 2t (+ 1) and 8 more; c0..c3
// C's rows g, g, g + 8, g + 8 at columns 2t, 2t + 1, 2t, 2t + 1.
__device__ __forceinline__ void mma16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                      uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 ldg16(const uint16_t* p, bool on) {
  return on ? __ldg(reinterpret_cast<const uint4*>(p)) : make_uint4(0, 0, 0, 0);
}

// Half j of both 16-byte words, as a pair.
__device__ __forceinline__ uint32_t halves(const uint4& a, const uint4& b, int j) {
  const uint32_t x = j < 2 ? a.x : j < 4 ? a.y : j < 6 ? a.z : a.w, y = j < 2 ? b.x : j < 4 ? b.y : j < 6 ? b.z : b.w;
  return __byte_perm(x, y, j & 1 ? 0x7632 : 0x5410);
}

// Warps share a block's rows and columns: `kw` of the eight split D (in steps
// of 32 columns), the others take rows of their own, 32 a warp.
__host__ __device__ inline int few_k_warps(int D) { return D > 128 ? 8 : D > 64 ? 4 : D > 32 ? 2 : 1; }

__global__ void __launch_bounds__(256, 2) k_lce_few_logits(const FewArgs a) {
  __shared__ float part[8][32][kFewTokens];
  __shared__ float2 joined[8][kFewTokens];
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int kw = few_k_warps(a.D), sets = 8 / kw, set = warp / kw, slice = warp % kw;
  // an unlabelled token's row counts as zero
  const bool on0 = g < a.N && labelled(a.labels[g], a.ignore, a.V);
  const bool on1 = g + 8 < a.N && labelled(a.labels[g + 8], a.ignore, a.V);
  if (blockIdx.x == 0 && threadIdx.x < (unsigned)a.N) {
    const int32_t y = a.labels[threadIdx.x];
    if (y != a.ignore && !labelled(y, a.ignore, a.V)) atomicOr(&g_device_error, kDevErrIndex);
  }
  const uint16_t* h0 = a.H + g * a.ldh + 8 * t;
  const uint16_t* h1 = h0 + 8 * a.ldh;
  // this thread's tokens and its rows' statistics in the summing step
  const int tok = 2 * (threadIdx.x & 7), at = threadIdx.x >> 3;
  int32_t y[2];
  for (int i = 0; i < 2; ++i) y[i] = tok + i < a.N ? a.labels[tok + i] : -1;
  float m[2] = {-INFINITY, -INFINITY}, s[2] = {0.0f, 0.0f};
  for (int64_t item = blockIdx.x; item * 32 * sets < a.V; item += gridDim.x) {
    const int64_t v0 = (item * sets + set) * 32;
    float c[2][2][4] = {};
    bool in[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) in[i] = v0 + g + 8 * i < a.V;
    const uint16_t* w = a.W + (v0 + g) * a.ldw + 8 * t;
#pragma unroll 2
    for (int k0 = 32 * slice; k0 < a.D; k0 += 32 * kw) {
      const bool some = k0 + 8 * t < a.D;
      const uint4 x0 = ldg16(h0 + k0, on0 && some), x1 = ldg16(h1 + k0, on1 && some);
      uint4 r[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) r[i] = ldg16(w + 8 * i * a.ldw + k0, in[i] && some);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        mma16(c[i][0], r[2 * i].x, r[2 * i + 1].x, r[2 * i].y, r[2 * i + 1].y, x0.x, x0.y);
        mma16(c[i][0], r[2 * i].z, r[2 * i + 1].z, r[2 * i].w, r[2 * i + 1].w, x0.z, x0.w);
        mma16(c[i][1], r[2 * i].x, r[2 * i + 1].x, r[2 * i].y, r[2 * i + 1].y, x1.x, x1.y);
        mma16(c[i][1], r[2 * i].z, r[2 * i + 1].z, r[2 * i].w, r[2 * i + 1].w, x1.z, x1.w);
      }
    }
    __syncthreads();      // the item before has been summed
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        *reinterpret_cast<float2*>(&part[warp][16 * i + g][8 * j + 2 * t]) = make_float2(c[i][j][0], c[i][j][1]);
        *reinterpret_cast<float2*>(&part[warp][16 * i + g + 8][8 * j + 2 * t]) = make_float2(c[i][j][2], c[i][j][3]);
      }
    __syncthreads();
    for (int q = 0; q < sets; ++q) {
      const int64_t v = (item * sets + q) * 32 + at;
      if (v >= a.V) break;
      float z[2] = {0.0f, 0.0f};
      for (int k = 0; k < kw; ++k) {
        const float2 p = *reinterpret_cast<const float2*>(&part[q * kw + k][at][tok]);
        z[0] += p.x;
        z[1] += p.y;
      }
      *reinterpret_cast<float2*>(a.z + v * kFewTokens + tok) = make_float2(z[0], z[1]);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float mn = fmaxf(m[i], z[i]), ref = mn == -INFINITY ? 0.0f : mn;
        s[i] = s[i] * expf(m[i] - ref) + expf(z[i] - ref);
        m[i] = mn;
        if (y[i] == v) a.label_logit[tok + i] = z[i];
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (m[i] == -INFINITY && s[i] != 0.0f) m[i] = 0.0f;     // nothing but NaN: it must not be left out
#pragma unroll
    for (int o = 8; o < 32; o <<= 1) combine_stats(m[i], s[i], __shfl_xor_sync(0xffffffffu, m[i], o), __shfl_xor_sync(0xffffffffu, s[i], o));
    if (lane < 8) joined[warp][tok + i] = make_float2(m[i], s[i]);
  }
  __syncthreads();
  if (threadIdx.x < kFewTokens) {
    float2 p = joined[0][threadIdx.x];
    for (int w = 1; w < 8; ++w) combine_stats(p.x, p.y, joined[w][threadIdx.x].x, joined[w][threadIdx.x].y);
    a.stats[(int64_t)blockIdx.x * kFewTokens + threadIdx.x] = p;
  }
}

// Column chunks of 64 a warp; with fewer than eight of them, the other warps
// take 16-row groups of their own.
__host__ __device__ inline int few_row_warps(int D) { return D > 256 ? 1 : D > 128 ? 2 : D > 64 ? 4 : 8; }

constexpr int kFewRows = 128;      // rows of z turned into g at a time

__global__ void __launch_bounds__(256, 2) k_lce_few_grads(const FewArgs a) {
  __shared__ float2 joined[8][kFewTokens];
  __shared__ float lse[kFewTokens], zy[kFewTokens];
  __shared__ int32_t label[kFewTokens];      // -1: none
  // g by row and by token, rows padded so that fragments meet no bank twice
  __shared__ __align__(16) uint16_t gr[kFewRows][24], gt[kFewTokens][kFewRows + 8];
  __shared__ float sums[8][32][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  griddep_launch_dependents();
  if (threadIdx.x < kFewTokens) {
    const int32_t y = threadIdx.x < (unsigned)a.N ? a.labels[threadIdx.x] : -1;
    label[threadIdx.x] = threadIdx.x < (unsigned)a.N && labelled(y, a.ignore, a.V) ? y : -1;
  }
  __syncthreads();
  int n = 0;
  for (int i = 0; i < kFewTokens; ++i) n += label[i] >= 0;
  const float f = n ? (float)(a.grad_scale / n) : 0.0f;
  const int rw = few_row_warps(a.D), set = warp % rw;
  const int d0 = ((int)blockIdx.y * (8 / rw) + warp / rw) * 64, d = d0 + 8 * g;
  // H as the second operand of dW: b0 = tokens 2t, 2t + 1, b1 = 8 more, for
  // column 8 g + j of the chunk
  uint32_t hb[8][2];
  {
    uint4 r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int q = 2 * t + (i & 1) + 8 * (i >> 1);
      r[i] = ldg16(a.H + q * a.ldh + d, label[q] >= 0 && d < a.D);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      hb[j][0] = halves(r[0], r[1], j);
      hb[j][1] = halves(r[2], r[3], j);
    }
  }
  griddep_wait();
  {
    const int q = threadIdx.x & 15;
    // the maximum first, so that the exponentials do not wait for one another
    const float2* st = a.stats + q;
    float2 p = make_float2(-INFINITY, 0.0f);
#pragma unroll 4
    for (int i = threadIdx.x >> 4; i < a.n_stats; i += 16) p.x = fmaxf(p.x, st[i * kFewTokens].x);
#pragma unroll 4
    for (int i = threadIdx.x >> 4; i < a.n_stats; i += 16) {
      const float2 o = st[i * kFewTokens];
      p.y += o.x == -INFINITY ? 0.0f : o.y * expf(o.x - p.x);
    }
    combine_stats(p.x, p.y, __shfl_xor_sync(0xffffffffu, p.x, 16), __shfl_xor_sync(0xffffffffu, p.y, 16));
    if (lane < 16) joined[warp][q] = p;
    __syncthreads();
    if (threadIdx.x < kFewTokens) {
      p = joined[0][q];
#pragma unroll
      for (int i = 1; i < 8; ++i) combine_stats(p.x, p.y, joined[i][q].x, joined[i][q].y);
      lse[q] = p.x + logf(p.y);
      zy[q] = label[q] >= 0 ? a.label_logit[q] : 0.0f;
    }
    __syncthreads();
  }
  if (blockIdx.x == 0 && blockIdx.y == 0) {
    if (threadIdx.x < (unsigned)a.N && a.token_loss)
      a.token_loss[threadIdx.x] = label[threadIdx.x] >= 0 ? lse[threadIdx.x] - zy[threadIdx.x] : 0.0f;
    if (threadIdx.x == 0 && a.loss) {
      double sum = 0.0;
      for (int i = 0; i < kFewTokens; ++i)
        if (label[i] >= 0) sum += (double)(lse[i] - zy[i]);
      *a.loss = n ? (float)(sum / n) : 0.0f;
    }
  }
  const int64_t first = blockIdx.x * a.rows_part, end = min(a.V, first + a.rows_part);
  float acc[8][4] = {};
  for (int64_t base = first; base < end; base += kFewRows) {
    __syncthreads();      // the rows before have been used
    {
      const int r = threadIdx.x >> 1, q0 = 8 * (threadIdx.x & 1);
      const int64_t v = base + r;
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 8; i += 4) {
        const float4 z = v < end ? *reinterpret_cast<const float4*>(a.z + v * kFewTokens + q0 + i) : make_float4(0, 0, 0, 0);
        const float e[4] = {z.x, z.y, z.z, z.w};
        uint16_t b[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int q = q0 + i + k;
          const float x = e[k] - lse[q];
          const float p = v >= end || label[q] < 0 ? 0.0f : label[q] == v ? expm1f(x) : expf(x);
          b[k] = __bfloat16_as_ushort(__float2bfloat16_rn(p));
          gt[q][r] = b[k];
        }
        w[i / 2] = b[0] | (uint32_t)b[1] << 16;
        w[i / 2 + 1] = b[2] | (uint32_t)b[3] << 16;
      }
      *reinterpret_cast<uint4*>(&gr[r][q0]) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    __syncthreads();
    if (d0 >= a.D) continue;
#pragma unroll 2
    for (int r0 = 16 * set; r0 < kFewRows; r0 += 16 * rw) {
      const int64_t v0 = base + r0;
      if (v0 >= end) break;
      if (a.part) {
        uint4 r[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int64_t v = v0 + 2 * t + (i & 1) + 8 * (i >> 1);
          r[i] = ldg16(a.W + v * a.ldw + d, v < end && d < a.D);
        }
        const uint32_t a0 = *reinterpret_cast<const uint32_t*>(&gt[g][r0 + 2 * t]), a1 = *reinterpret_cast<const uint32_t*>(&gt[g + 8][r0 + 2 * t]);
        const uint32_t a2 = *reinterpret_cast<const uint32_t*>(&gt[g][r0 + 2 * t + 8]), a3 = *reinterpret_cast<const uint32_t*>(&gt[g + 8][r0 + 2 * t + 8]);
#pragma unroll
        for (int j = 0; j < 8; ++j) mma16(acc[j], a0, a1, a2, a3, halves(r[0], r[1], j), halves(r[2], r[3], j));
      }
      if (a.dW) {
        const uint32_t a0 = *reinterpret_cast<const uint32_t*>(&gr[r0 + g][2 * t]), a1 = *reinterpret_cast<const uint32_t*>(&gr[r0 + g + 8][2 * t]);
        const uint32_t a2 = *reinterpret_cast<const uint32_t*>(&gr[r0 + g][2 * t + 8]), a3 = *reinterpret_cast<const uint32_t*>(&gr[r0 + g + 8][2 * t + 8]);
        float c[8][4] = {};
#pragma unroll
        for (int j = 0; j < 8; ++j) mma16(c[j], a0, a1, a2, a3, hb[j][0], hb[j][1]);
        // c[0..7][i]: row g (i < 2) or g + 8, eight consecutive columns from 16 t (i even) or 16 t + 8 on
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int64_t v = v0 + g + (i < 2 ? 0 : 8);
          const int col = d0 + 16 * t + 8 * (i & 1);
          if (v >= end || col >= a.D) continue;
          if (a.dw_fp32) {
            float* p = static_cast<float*>(a.dW) + v * a.lddw + col;
            *reinterpret_cast<float4*>(p) = make_float4(f * c[0][i], f * c[1][i], f * c[2][i], f * c[3][i]);
            *reinterpret_cast<float4*>(p + 4) = make_float4(f * c[4][i], f * c[5][i], f * c[6][i], f * c[7][i]);
          } else {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) w[k] = bf16x2_rn(pack_f2(f * c[2 * k][i], f * c[2 * k + 1][i]));
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.dW) + v * a.lddw + col) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
    }
  }
  if (!a.part) return;
  if (rw > 1) {
    // warps of one column chunk: the others' sums onto the first one's, in order
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (set) sums[warp][i][lane] = acc[i >> 2][i & 3];
    __syncthreads();
    if (set) return;
    for (int w = warp + 1; w < warp + rw; ++w)
#pragma unroll
      for (int i = 0; i < 32; ++i) acc[i >> 2][i & 3] += sums[w][i][lane];
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int q = g + (i < 2 ? 0 : 8), col = d0 + 16 * t + 8 * (i & 1);
    if (q >= a.N || col >= a.D) continue;
    float* p = a.part + ((int64_t)blockIdx.x * a.N + q) * a.D + col;
    // an unlabelled token's sums are 0 times W, which a NaN or an infinity in W turns into NaN: exactly 0 instead
    const bool on = label[q] >= 0;
    float4 lo = make_float4(0.0f, 0.0f, 0.0f, 0.0f), hi = lo;
    if (on) {
      lo = make_float4(f * acc[0][i], f * acc[1][i], f * acc[2][i], f * acc[3][i]);
      hi = make_float4(f * acc[4][i], f * acc[5][i], f * acc[6][i], f * acc[7][i]);
    }
    *reinterpret_cast<float4*>(p) = lo;
    *reinterpret_cast<float4*>(p + 4) = hi;
  }
}

// Whether a call takes this form.  A rule on tokens and D alone: it gains most
// where W is small (24 us against 39, see above) and loses 1 % at the largest (16 x 4096 x
// 128256, 652 us against 645).
inline bool few_tokens(int64_t N, int64_t D) { return N <= kFewTokens && D % 8 == 0 && D <= 1 << 20; }

struct FewPlan {
  int n_stats, blocks;      // of the first kernel, and of the second (times its column blocks)
  int64_t rows_part;
  size_t off_stats, off_logit, off_part, bytes;
};

inline FewPlan plan_few(int64_t N, int64_t D, int64_t V) {
  constexpr int64_t kBlocks = 4 * kPairsGb300;      // two an SM
  FewPlan p;
  p.n_stats = (int)std::min<int64_t>(ceil_div<int64_t>(V, 32 * (8 / few_k_warps((int)D))), kBlocks);
  const int64_t columns = ceil_div<int64_t>(D, 512);
  const int64_t most = std::max<int64_t>(1, std::min<int64_t>(kBlocks / columns, ceil_div<int64_t>(V, 16 * few_row_warps((int)D))));
  p.rows_part = ceil_div<int64_t>(ceil_div<int64_t>(V, most), 16) * 16;
  p.blocks = (int)ceil_div<int64_t>(V, p.rows_part);
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = (off + bytes + 255) / 256 * 256;
    return o;
  };
  take((size_t)V * kFewTokens * 4);
  p.off_stats = take((size_t)p.n_stats * kFewTokens * 8);
  p.off_logit = take(kFewTokens * 4);
  p.off_part = take((size_t)p.blocks * N * D * 4);
  p.bytes = off;
  return p;
}

}  // namespace
}  // namespace sf
