// The layer for 1..16 tokens with 16-bit activations (W4A16): every weight is read once, decoded in
// registers and multiplied with all tokens.
//
//   Y[m, n] = bf16(alpha_w (sum_k xh[m, k] q[n, k] s[n, k / g] + sum_r T[m, r] L2[r, n] / alpha_w) + b[n])
//   xh = fp32(x inv_lam),  T = X L1'
//
// Bound by reading the weights (0.56 bytes each); the products run on mma.sync m16n8k16 (fp16
// inputs, fp32 sums) with 16 weight rows as the M side and the tokens as the N side, because a
// decoded weight then costs a fraction of an instruction per token instead of one each.
//
// Operands.  A NVFP4 weight q s has at most 6 significant bits between 2^-10 and 2688 and is exact
// in fp16; an INT4 code is exact, and its bf16 scale multiplies the group's fp32 sum.  An activation
// is scaled by a power of two per token (largest magnitude to [2^13, 2^14)) and split into two fp16
// columns, hi + lo: 22 significant bits, down to 2^-38 of the token's largest, so the inputs are
// not rounded further than fp32 sums are.  The first kernel lays these columns out in the order the
// second one's MMA fragments read them and computes T (bf16 inputs, exact products, fp32 sums).
//
// Order of k.  A contraction may run in any order, so a thread takes 16 consecutive bytes (32
// weights) of a row and feeds them to 8 MMA steps; the columns of X are laid out to match.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "rows.cuh"
#include "svdq_internal.h"

namespace svdq {
namespace {

using namespace dev;

constexpr int kMaxTokens = 16;
constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kStep = 128;        // weights of a row per warp step: 4 lanes x 32
constexpr int kUnitRows = 32;     // weight rows per CTA: two M = 16 tiles
constexpr int kTWarpK = 128;      // k per warp of the T kernel part
constexpr int kTSplit = kTWarpK * kWarps;

struct W4A16Params {
  const uint16_t* X;      // bf16 [M, K]
  const float* inv_lam;
  const uint16_t* L1t;    // bf16 [r_pad, K]
  const uint16_t* L2t;    // bf16 [N, r_pad], L2 / alpha_w
  const uint8_t* codes;   // [N, K/2]
  const void* sf;
  const float* bias;
  uint16_t* Y;
  uint4* frag;            // X as MMA fragments: [step][column tile][4][32] x 16 bytes
  float* pow2;            // [M] the tokens' scales
  float* T;               // [splits of K][M][r_pad]
  int M, N, K, r_pad, steps, tiles, t_splits;
  float alpha_w;
};

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t as_u32(__half2 h) { return *reinterpret_cast<const uint32_t*>(&h); }
__device__ __forceinline__ __half2 as_half2(uint32_t w) { return *reinterpret_cast<const __half2*>(&w); }

// Eight E2M1 codes of a word (low nibble first) as four fp16 pairs.
__device__ __forceinline__ void e2m1_pairs(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t"
      ".reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t"
      "}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

// Eight INT4 codes of a word (elements 0, 2, 4, 6 then 1, 3, 5, 7) as four fp16 pairs: 1024 + (q + 8)
// assembled from its bits, less 1032.
__device__ __forceinline__ void int4_pairs(uint32_t w, uint32_t (&h)[4]) {
  w ^= 0x88888888u;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    h[j] = as_u32(__hsub2(as_half2(((w >> (4 * j)) & 0x000F000Fu) | 0x64006400u), as_half2(0x64086408u)));
}

// Weight row of lane group g (0..7), slot b (0..3) of unit u: the rows whose scales a thread gets in
// one access.  NVFP4 scale atoms hold rows r, r + 32, r + 64, r + 96 side by side.
template <bool INT4>
__device__ __forceinline__ int unit_row(int u, int b, int g) {
  return INT4 ? u * kUnitRows + 4 * g + b : (u >> 2) * 128 + 32 * b + 8 * (u & 3) + g;
}

// CTAs 0..M-1: a token's columns and scale.  The others: 16 ranks of T over one split of K.
template <bool INT4>
__global__ void __launch_bounds__(kThreads) w4a16_prepare_kernel(W4A16Params p) {
  __shared__ float red[kWarps][16][16];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  if (static_cast<int>(blockIdx.x) < p.M) {
    const int m = blockIdx.x;
    const uint16_t* x = p.X + static_cast<size_t>(m) * p.K;
    auto chunk = [&](int c, float (&v)[8]) {  // xh of columns 8 c..8 c + 7, 0 beyond K
      if (c * 8 < p.K) {
        float f[8];
        unpack8(__ldg(reinterpret_cast<const uint4*>(x) + c), v, static_cast<const __nv_bfloat16*>(nullptr));
        load8(p.inv_lam + c * 8, f);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] *= f[j];
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = 0.0f;
      }
    };
    uint32_t top = 0;  // bits of the largest finite magnitude
    for (int c = threadIdx.x; c < p.K / 8; c += kThreads) {
      float v[8];
      chunk(c, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t a = abs_bits(v[j]);
        if (a < 0x7F800000u) top = max(top, a);
      }
    }
    top = __reduce_max_sync(0xffffffffu, top);
    uint32_t* r = reinterpret_cast<uint32_t*>(red);
    if (lane == 0) r[warp] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = max(top, r[w]);
    const int e = max(static_cast<int>(top >> 23) - 13, 1);  // biased: the scale is 2^(e - 127), a normal number
    const float inv = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
    if (threadIdx.x == 0) p.pow2[m] = __uint_as_float(static_cast<uint32_t>(e) << 23);
    for (int c = threadIdx.x; c < p.steps * (kStep / 8); c += kThreads) {
      float v[8];
      chunk(c, v);
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float a = v[2 * j] * inv, b = v[2 * j + 1] * inv;
        const __half2 h = __floats2half2_rn(a, b);
        const float2 f = __half22float2(h);
        // an infinity or a NaN stays in hi alone
        const float la = isfinite(a) ? a - f.x : 0.0f, lb = isfinite(b) ? b - f.y : 0.0f;
        hi[j] = as_u32(h);
        lo[j] = as_u32(__floats2half2_rn(la, lb));
      }
      const int w = c % 16;  // place in the 128-wide step
      const int q = INT4 ? (w >> 3) * 2 + (w & 1) : w & 3, ft = INT4 ? (w & 7) >> 1 : w >> 2;
      const int col = 2 * m;
      uint4* to = p.frag + ((static_cast<size_t>(c / 16) * p.tiles + col / 8) * 4 + q) * 32 + (col % 8) * 4 + ft;
      to[0] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      to[4] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
    return;
  }

  const int job = blockIdx.x - p.M, split = job % p.t_splits, r0 = job / p.t_splits * 16;
  float acc[2][4] = {};
  const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
  for (int i = 0; i < kTWarpK / 32; ++i) {
    const int k = split * kTSplit + warp * kTWarpK + i * 32 + t * 8;
    uint4 a = zero, b = zero, x[2] = {zero, zero};
    if (k < p.K) {
      a = __ldg(reinterpret_cast<const uint4*>(p.L1t + static_cast<size_t>(r0 + g) * p.K + k));
      b = __ldg(reinterpret_cast<const uint4*>(p.L1t + static_cast<size_t>(r0 + g + 8) * p.K + k));
#pragma unroll
      for (int j = 0; j < 2; ++j)
        if (j * 8 + g < p.M) x[j] = __ldg(reinterpret_cast<const uint4*>(p.X + static_cast<size_t>(j * 8 + g) * p.K + k));
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if (j * 8 >= p.M) break;
      mma_bf16(acc[j], a.x, b.x, a.y, b.y, x[j].x, x[j].y);
      mma_bf16(acc[j], a.z, b.z, a.w, b.w, x[j].z, x[j].w);
    }
  }
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) red[warp][g + 8 * (e >> 1)][j * 8 + 2 * t + (e & 1)] = acc[j][e];
  __syncthreads();
  const int r = threadIdx.x % 16, m = threadIdx.x / 16;
  if (m < p.M) {
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) s += red[w][r][m];
    p.T[(static_cast<size_t>(split) * p.M + m) * p.r_pad + r0 + r] = s;
  }
}

// One unit of 32 weight rows per CTA; its warps take the 128-wide steps of K in turn.
template <bool INT4, int NT>
__global__ void __launch_bounds__(kThreads) w4a16_kernel(W4A16Params p) {
  __shared__ float red[kWarps][NT * 4][kUnitRows + 1];
  __shared__ float s_t[kMaxTokens * 128];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int u = blockIdx.x;
  const size_t row_bytes = p.K / 2;
  const uint4 zero = make_uint4(0, 0, 0, 0);

  float acc[2][NT][4] = {};
  for (int s = warp; s < p.steps; s += kWarps) {
    uint4 w[4];
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const int n = unit_row<INT4>(u, b, g);
      const uint8_t* row = p.codes + n * row_bytes + s * (kStep / 2);
      w[b] = zero;
      if (n < p.N) {
        if (INT4) {  // 8 bytes of each 64-wide group
          const uint2 a = __ldg(reinterpret_cast<const uint2*>(row + t * 8));
          w[b].x = a.x, w[b].y = a.y;
          if (s * kStep + 64 < p.K) {
            const uint2 c = __ldg(reinterpret_cast<const uint2*>(row + 32 + t * 8));
            w[b].z = c.x, w[b].w = c.y;
          }
        } else if (s * kStep + t * 32 < p.K) {
          w[b] = __ldg(reinterpret_cast<const uint4*>(row + t * 16));
        }
      }
    }
    uint4 x[NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        x[j][q] = j * 8 + g < 2 * p.M ? __ldg(p.frag + ((static_cast<size_t>(s) * NT + j) * 4 + q) * 32 + lane) : zero;

    if (INT4) {
      const uint16_t* sf = static_cast<const uint16_t*>(p.sf) + u * kUnitRows + 4 * g;
      const size_t n_pad = static_cast<size_t>((p.N + 255) / 256) * 256;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        if (s * kStep + half * 64 >= p.K) break;
        const uint2 sc = __ldg(reinterpret_cast<const uint2*>(sf + (static_cast<size_t>(s) * 2 + half) * n_pad));
        const float f[4] = {pair_lo(sc.x), pair_hi(sc.x), pair_lo(sc.y), pair_hi(sc.y)};
#pragma unroll
        for (int tile = 0; tile < 2; ++tile) {
          float sum[NT][4] = {};
#pragma unroll
          for (int q = 2 * half; q < 2 * half + 2; ++q) {
            uint32_t a[4], b[4];
            int4_pairs((&w[2 * tile].x)[q], a);
            int4_pairs((&w[2 * tile + 1].x)[q], b);
#pragma unroll
            for (int j = 0; j < NT; ++j) {
              mma_f16(sum[j], a[0], b[0], a[1], b[1], x[j][q].x, x[j][q].y);
              mma_f16(sum[j], a[2], b[2], a[3], b[3], x[j][q].z, x[j][q].w);
            }
          }
#pragma unroll
          for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[tile][j][e] = __fmaf_rn(sum[j][e], f[2 * tile + (e >> 1)], acc[tile][j][e]);
        }
      }
    } else {
      // scales of rows b = 0..3 and columns 64 kb..64 kb + 63; this thread's 32 weights are two groups
      const int kb = 2 * s + (t >> 1);
      uint4 sc = zero;
      if (kb < p.K / 64)
        sc = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.sf) +
                                                  (static_cast<size_t>(u >> 2) * (p.K / 64) + kb) * 512) +
                   8 * (u & 3) + g);
      __half2 s01[4];
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        uint32_t h;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>((&sc.x)[b] >> (16 * (t & 1)))));
        s01[b] = as_half2(h);
      }
#pragma unroll
      for (int tile = 0; tile < 2; ++tile) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t a[4], b[4];
          e2m1_pairs((&w[2 * tile].x)[q], a);
          e2m1_pairs((&w[2 * tile + 1].x)[q], b);
          const __half2 sa = q < 2 ? __low2half2(s01[2 * tile]) : __high2half2(s01[2 * tile]);
          const __half2 sb = q < 2 ? __low2half2(s01[2 * tile + 1]) : __high2half2(s01[2 * tile + 1]);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            a[j] = as_u32(__hmul2(as_half2(a[j]), sa));
            b[j] = as_u32(__hmul2(as_half2(b[j]), sb));
          }
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            mma_f16(acc[tile][j], a[0], b[0], a[1], b[1], x[j][q].x, x[j][q].y);
            mma_f16(acc[tile][j], a[2], b[2], a[3], b[3], x[j][q].z, x[j][q].w);
          }
        }
      }
    }
  }

  // a thread holds a token's hi and lo columns side by side: their sum, then the sum over the warps
#pragma unroll
  for (int tile = 0; tile < 2; ++tile)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        red[warp][j * 4 + t][(2 * tile + h) * 8 + g] = acc[tile][j][2 * h] + acc[tile][j][2 * h + 1];
  for (int i = threadIdx.x; i < p.M * p.r_pad; i += kThreads) {
    float v = 0.0f;
    for (int j = 0; j < p.t_splits; ++j) v += p.T[static_cast<size_t>(j) * p.M * p.r_pad + i];
    s_t[i] = v * p.alpha_w;  // exact, and keeps the products with L2 / alpha_w in range
  }
  __syncthreads();
  for (int i = threadIdx.x; i < p.M * kUnitRows; i += kThreads) {
    const int m = i / kUnitRows, row = i % kUnitRows;
    const int n = unit_row<INT4>(u, row >> 3, row & 7);
    if (n >= p.N) continue;
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v += red[w][m][row];
    v *= p.pow2[m] * p.alpha_w;
    const uint4* l2 = reinterpret_cast<const uint4*>(p.L2t + static_cast<size_t>(n) * p.r_pad);
    float low = 0.0f;
    for (int r = 0; r < p.r_pad / 8; ++r) {
      float f[8];
      unpack8(__ldg(l2 + r), f, static_cast<const __nv_bfloat16*>(nullptr));
#pragma unroll
      for (int j = 0; j < 8; ++j) low = __fmaf_rn(s_t[m * p.r_pad + r * 8 + j], f[j], low);
    }
    const __nv_bfloat16 y = __float2bfloat16_rn(v + low + p.bias[n]);
    p.Y[static_cast<size_t>(m) * p.N + n] = *reinterpret_cast<const uint16_t*>(&y);
  }
}

inline size_t up256(size_t x) { return (x + 255) / 256 * 256; }
int column_tiles(int M) { return M <= 4 ? 1 : M <= 8 ? 2 : 4; }

template <bool INT4>
svdq_status launch(const W4A16Params& p, cudaStream_t stream) {
  w4a16_prepare_kernel<INT4><<<p.M + p.r_pad / 16 * p.t_splits, kThreads, 0, stream>>>(p);
  SVDQ_CUDA_TRY(cudaGetLastError());
  const int units = INT4 ? (p.N + kUnitRows - 1) / kUnitRows : (p.N + 127) / 128 * 4;
  switch (p.tiles) {
    case 1: w4a16_kernel<INT4, 1><<<units, kThreads, 0, stream>>>(p); break;
    case 2: w4a16_kernel<INT4, 2><<<units, kThreads, 0, stream>>>(p); break;
    default: w4a16_kernel<INT4, 4><<<units, kThreads, 0, stream>>>(p); break;
  }
  SVDQ_CUDA_TRY(cudaGetLastError());
  return SVDQ_OK;
}

}  // namespace

size_t w4a16_workspace(int M, int K, int r_pad) {
  const int steps = (K + kStep - 1) / kStep, splits = (K + kTSplit - 1) / kTSplit;
  return up256(static_cast<size_t>(steps) * column_tiles(M) * 4 * 32 * 16) + 256 +
         up256(static_cast<size_t>(splits) * M * r_pad * sizeof(float));
}

svdq_status launch_w4a16(const svdq_weights* w, const void* X, int M, void* Y, void* workspace, cudaStream_t stream) {
  W4A16Params p{};
  p.X = static_cast<const uint16_t*>(X);
  p.inv_lam = w->d_inv_lam;
  p.L1t = w->d_L1t;
  p.L2t = w->d_L2t;
  p.codes = w->d_wq;
  p.sf = w->d_wsf;
  p.bias = w->d_bias;
  p.Y = static_cast<uint16_t*>(Y);
  p.M = M;
  p.N = w->N;
  p.K = w->K;
  p.r_pad = w->r_pad;
  p.steps = (w->K + kStep - 1) / kStep;
  p.tiles = column_tiles(M);
  p.t_splits = (w->K + kTSplit - 1) / kTSplit;
  p.alpha_w = w->alpha_w;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.frag = reinterpret_cast<uint4*>(ws);
  ws += up256(static_cast<size_t>(p.steps) * p.tiles * 4 * 32 * 16);
  p.pow2 = reinterpret_cast<float*>(ws);
  p.T = reinterpret_cast<float*>(ws + 256);
  return w->format == SVDQ_FORMAT_INT4 ? launch<true>(p, stream) : launch<false>(p, stream);
}

}  // namespace svdq
