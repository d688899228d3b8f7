// Gradient of a low-rank factor: G[K, r] = X^T S over M tokens, X an activation (bf16, or its 8-bit
// checkpoint) and S [M, r] bf16.
//
// With y += (x A) B: dA = X^T (dY B^T) and dB^T = dY^T (X A), both this product.  X is the large
// operand (M K values against (M + K) r), so the kernel is bound by reading it once as long as the
// 2 M K r operations keep up; they run on the tensor cores (mma.sync m16n8k16, bf16 inputs, fp32
// sums).  X needs no copy or transpose: the contraction runs over rows, so each thread reads the
// same 8 consecutive columns of 4 rows and pairs the rows' values in registers.  Checkpoint values
// are q 2^e with at most 7 significant bits, exact in bf16.
//
// The tensor cores' additions truncate, which would add up over thousands of tokens, so a warp sums
// at most some 300 tokens in one accumulator; those sums are joined by ordinary fp32 additions, in
// a fixed order: over the CTA's warps in shared memory, over the CTAs by a second kernel.
#include <cuda_bf16.h>

#include "rows.cuh"
#include "svdq_internal.h"

namespace svdq {
namespace {

using namespace dev;

constexpr int kSMs = 148;
constexpr int kWarpCols = 64;                  // columns of X per warp: 8 lanes x 8
constexpr int kColWarps = 2, kRowWarps = 4;    // warps along the columns and along the rows
constexpr int kCtaCols = kWarpCols * kColWarps;
constexpr int kCtaRows = 16 * kRowWarps;       // rows per step of the CTA
constexpr int kThreads = 32 * kColWarps * kRowWarps;

struct WgradParams {
  const void* X;  // bf16 [M, K], or the codes
  const uint8_t* scales;
  const uint16_t* S;  // bf16 [M, r]
  float* out;         // G, or the partial sums [splits][K][r]
  int M, K, r, steps; // steps: row steps of kCtaRows per split
};

__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Pairs over two rows of 8 columns: w[j] holds (row a, row b) of column j.
template <int SRC>
__device__ __forceinline__ void pair_rows(const uint4& a, const uint4& b, float sa, float sb, uint32_t (&w)[8]) {
  if (SRC == 0) {
    const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      w[2 * j] = __byte_perm(x[j], y[j], 0x5410);
      w[2 * j + 1] = __byte_perm(x[j], y[j], 0x7632);
    }
  } else {
    constexpr int F = SRC == 1 ? SVDQ_CKPT8_INT8 : SVDQ_CKPT8_E4M3;
    float u[8], v[8];
    ckpt_values4<F>(a.x, sa, u);
    ckpt_values4<F>(a.y, sa, u + 4);
    ckpt_values4<F>(b.x, sb, v);
    ckpt_values4<F>(b.y, sb, v + 4);
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = bf16_pair(u[j], v[j]);
  }
}

// The raw 8 columns at (m, k) and their scale; zeros outside.
template <int SRC>
__device__ __forceinline__ void fetch(const WgradParams& p, int m, int k, uint4& v, uint32_t& scale) {
  v = make_uint4(0, 0, 0, 0);
  scale = 0;
  if (m >= p.M || k >= p.K) return;
  const size_t at = static_cast<size_t>(m) * p.K + k;
  if (SRC == 0) {
    v = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.X) + at));
  } else {
    const uint2 c = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(p.X) + at));
    v.x = c.x, v.y = c.y;
    scale = __ldg(p.scales + static_cast<size_t>(m) * ((p.K + kCkptGroup - 1) / kCkptGroup) + k / kCkptGroup);
  }
}

// NT: columns of S per CTA in tiles of 8.  blockIdx: x columns of X, y row split, z columns of S.
template <int SRC, int NT>
__global__ void __launch_bounds__(kThreads) wgrad_kernel(WgradParams p) {
  constexpr int kLd = NT * 8 + 8;  // bf16 per row of the S tile: rows fall into different banks
  // the S tiles of the loop, then the sums that the row warps join
  constexpr int kTileBytes = 2 * kCtaRows * kLd * 2, kSumBytes = kCtaCols * (NT * 8 + 1) * 4;
  __shared__ __align__(16) uint8_t smem[kTileBytes > kSumBytes ? kTileBytes : kSumBytes];
  auto* s_tile = reinterpret_cast<uint16_t(*)[kCtaRows][kLd]>(smem);
  auto* s_sum = reinterpret_cast<float(*)[NT * 8 + 1]>(smem);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int cw = warp % kColWarps, rw = warp / kColWarps;
  const int k = blockIdx.x * kCtaCols + cw * kWarpCols + g * 8;
  const int n0 = blockIdx.z * NT * 8;
  const int row0 = blockIdx.y * p.steps * kCtaRows;

  float acc[4][NT][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j][0] = acc[i][j][1] = acc[i][j][2] = acc[i][j][3] = 0.0f;

  uint4 x[4];
  uint32_t sc[4];
  auto fetch_rows = [&](int step) {
    const int m = row0 + step * kCtaRows + rw * 16 + 2 * t;
#pragma unroll
    for (int i = 0; i < 4; ++i) fetch<SRC>(p, step < p.steps ? m + (i & 1) + (i >> 1) * 8 : p.M, k, x[i], sc[i]);
  };
  auto stage_s = [&](int step, int buf) {
    const int m0 = row0 + step * kCtaRows;
    for (int i = threadIdx.x; i < kCtaRows * NT * 8; i += kThreads) {
      const int m = m0 + i / (NT * 8), n = n0 + i % (NT * 8);
      s_tile[buf][i / (NT * 8)][i % (NT * 8)] = m < p.M && n < p.r ? p.S[static_cast<size_t>(m) * p.r + n] : 0;
    }
  };

  fetch_rows(0);
  stage_s(0, 0);
  __syncthreads();
  for (int step = 0; step < p.steps; ++step) {
    uint32_t lo[8], hi[8];  // rows 2t, 2t+1 and 2t+8, 2t+9
    pair_rows<SRC>(x[0], x[1], ckpt_scale(sc[0]), ckpt_scale(sc[1]), lo);
    pair_rows<SRC>(x[2], x[3], ckpt_scale(sc[2]), ckpt_scale(sc[3]), hi);
    fetch_rows(step + 1);
    uint32_t b[NT][2];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const uint32_t at = static_cast<uint32_t>(
          __cvta_generic_to_shared(&s_tile[step & 1][rw * 16 + (lane & 15)][j * 8]));
      asm volatile("ldmatrix.sync.aligned.m8n8.x2.trans.shared.b16 {%0, %1}, [%2];"
                   : "=r"(b[j][0]), "=r"(b[j][1])
                   : "r"(at));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t a[4] = {lo[2 * i], lo[2 * i + 1], hi[2 * i], hi[2 * i + 1]};
#pragma unroll
      for (int j = 0; j < NT; ++j) mma_bf16(acc[i][j], a, b[j][0], b[j][1]);
    }
    if (step + 1 < p.steps) stage_s(step + 1, (step + 1) & 1);
    __syncthreads();
  }

  // the row warps add their sums in turn
  for (int w = 0; w < kRowWarps; ++w) {
    if (rw == w) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float* s = &s_sum[cw * kWarpCols + g * 8 + 2 * i + (e >> 1)][j * 8 + 2 * t + (e & 1)];
            *s = w ? *s + acc[i][j][e] : acc[i][j][e];
          }
    }
    __syncthreads();
  }
  float* out = p.out + static_cast<size_t>(blockIdx.y) * p.K * p.r;
  for (int i = threadIdx.x; i < kCtaCols * NT * 8; i += kThreads) {
    const int c = blockIdx.x * kCtaCols + i / (NT * 8), n = n0 + i % (NT * 8);
    if (c < p.K && n < p.r) out[static_cast<size_t>(c) * p.r + n] = s_sum[i / (NT * 8)][i % (NT * 8)];
  }
}

__global__ void __launch_bounds__(256) wgrad_sum_kernel(const float* __restrict__ partial, int splits, size_t n,
                                                     float* __restrict__ G) {
  const size_t i = static_cast<size_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= n) return;
  float s = partial[i];
  for (int j = 1; j < splits; ++j) s += partial[j * n + i];
  G[i] = s;
}

struct Plan {
  int nt, cols, zs, splits, steps;
};

Plan plan(int M, int K, int r) {
  Plan q{};
  const int tiles = (r + 7) / 8;
  q.nt = tiles <= 1 ? 1 : tiles <= 2 ? 2 : tiles <= 4 ? 4 : 8;
  q.zs = (tiles + q.nt - 1) / q.nt;
  q.cols = (K + kCtaCols - 1) / kCtaCols;
  const int all = (M + kCtaRows - 1) / kCtaRows;
  // two CTAs per SM, and no accumulator over more than 20 steps (320 tokens a warp)
  int splits = (2 * kSMs + q.cols * q.zs - 1) / (q.cols * q.zs);
  if (splits * 20 < all) splits = (all + 19) / 20;
  if (splits > all) splits = all;
  q.steps = (all + splits - 1) / splits;
  q.splits = (all + q.steps - 1) / q.steps;
  return q;
}

template <int SRC>
svdq_status launch(const WgradParams& p, const Plan& q, cudaStream_t stream) {
  const dim3 grid(q.cols, q.splits, q.zs);
  switch (q.nt) {
    case 1: wgrad_kernel<SRC, 1><<<grid, kThreads, 0, stream>>>(p); break;
    case 2: wgrad_kernel<SRC, 2><<<grid, kThreads, 0, stream>>>(p); break;
    case 4: wgrad_kernel<SRC, 4><<<grid, kThreads, 0, stream>>>(p); break;
    default: wgrad_kernel<SRC, 8><<<grid, kThreads, 0, stream>>>(p); break;
  }
  SVDQ_CUDA_TRY(cudaGetLastError());
  return SVDQ_OK;
}

}  // namespace

size_t lowrank_wgrad_workspace(int M, int K, int r) {
  const Plan q = plan(M, K, r);
  return q.splits > 1 ? static_cast<size_t>(q.splits) * K * r * sizeof(float) : 0;
}

svdq_status launch_lowrank_wgrad(const void* X, const uint8_t* scales, int src, const void* S, int M, int K, int r,
                                 float* G, void* workspace, cudaStream_t stream) {
  const Plan q = plan(M, K, r);
  WgradParams p{X, scales, static_cast<const uint16_t*>(S), q.splits > 1 ? static_cast<float*>(workspace) : G,
                M, K, r, q.steps};
  SVDQ_TRY(src == 0 ? launch<0>(p, q, stream) : src == 1 ? launch<1>(p, q, stream) : launch<2>(p, q, stream));
  if (q.splits > 1) {
    const size_t n = static_cast<size_t>(K) * r;
    wgrad_sum_kernel<<<static_cast<unsigned>((n + 255) / 256), 256, 0, stream>>>(p.out, q.splits, n, G);
    SVDQ_CUDA_TRY(cudaGetLastError());
  }
  return SVDQ_OK;
}

}  // namespace svdq
