// Layer norm with per-group scale and shift (adaLN: one pair of vectors per image), and its gradient.
//
//   xh = (z - mu) rstd,  y = xh m + c,  m = scale or 1 + scale
//   dz = rstd (g - mean_j(g) - xh mean_j(g xh)),  g = dy m
//   dscale_j = sum_rows dy xh,  dshift_j = sum_rows dy   (rows of one group)
//
// Both are bound by HBM: each reads its rows once and writes its result once.  A row is held in
// registers by a team of warps (rows.cuh), so the forward takes the mean and then the centred sum
// of squares without a second read and without the cancellation of E[z^2] - E[z]^2; all sums are
// fp32.  In the backward a thread keeps its columns over all rows that its CTA takes, so the column
// sums stay in registers too; CTAs that share a group leave partial sums in the workspace and a
// second kernel adds them in a fixed order (no atomics: equal calls give equal bits).
#include <initializer_list>

#include "rows.cuh"
#include "svdq_internal.h"

namespace svdq {
namespace {

using namespace dev;

constexpr int kTeamWarps = 8;  // warps of a CTA shared out to teams of up to that many

// Sums of a and b over a team of `warps` warps, the same in every thread.  `red` holds two buffers
// of 16 pairs per team, used in turn: the barrier of one call separates the reads of the call before
// from the writes of the call after.
__device__ __forceinline__ float2 team_sum2(float a, float b, int warps, int team, float2* red, int& turn) {
  a = warp_sum(a);
  b = warp_sum(b);
  if (warps == 1) return make_float2(a, b);
  float2* r = red + turn * 16;
  turn ^= 1;
  const int w = (threadIdx.x >> 5) - team * warps;
  if ((threadIdx.x & 31) == 0) r[w] = make_float2(a, b);
  asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "r"(warps * 32) : "memory");
  float2 s = r[0];
  for (int i = 1; i < warps; ++i) s.x += r[i].x, s.y += r[i].y;
  return s;
}

struct FwdParams {
  const void* Z;
  const void* scale;
  const void* shift;
  void* Y;
  float2* stats;
  uint8_t* codes;
  uint8_t* scales;
  int64_t ld_z, ld_y, ld_param;
  int M, K, rows, param_dtype, warps, ckpt;  // ckpt: -1 none, else svdq_ckpt8_format
  float eps, one;
};

template <typename T, int NV, bool VEC>
__global__ void __launch_bounds__(512) layer_norm_kernel(FwdParams p) {
  __shared__ float2 red[kTeamWarps][32];
  const int threads = p.warps * 32, team = threadIdx.x / threads, t = threadIdx.x % threads;
  const int m = blockIdx.x * (blockDim.x / threads) + team;
  if (m >= p.M) return;  // whole teams: a barrier has all of its team's warps
  int turn = 0;
  const T* z = static_cast<const T*>(p.Z) + m * p.ld_z;
  float v[NV][8];
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    load_chunk<T, VEC>(z, p.K, i, t, threads, 0.0f, v[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) sum += v[i][j];
  }
  if (p.ckpt >= 0) {
    uint8_t* codes = p.codes + static_cast<size_t>(m) * p.K;
    uint8_t* scales = p.scales + static_cast<size_t>(m) * ((p.K + kCkptGroup - 1) / kCkptGroup);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (p.ckpt == SVDQ_CKPT8_INT8)
        ckpt_store_chunk<SVDQ_CKPT8_INT8, VEC>(codes, scales, p.K, i, t, threads, v[i]);
      else
        ckpt_store_chunk<SVDQ_CKPT8_E4M3, VEC>(codes, scales, p.K, i, t, threads, v[i]);
    }
  }
  const float inv_k = 1.0f / static_cast<float>(p.K);
  const float mu = team_sum2(sum, 0.0f, p.warps, team, red[team], turn).x * inv_k;
  float sq = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[i][j] -= mu;
      if (row_column<VEC>(i, j, t, threads) < p.K) sq = __fmaf_rn(v[i][j], v[i][j], sq);
    }
  }
  const float var = team_sum2(sq, 0.0f, p.warps, team, red[team], turn).x * inv_k;
  const float rstd = __frcp_rn(__fsqrt_rn(__fadd_rn(var, p.eps)));
  if (p.stats && t == 0) p.stats[m] = make_float2(mu, rstd);
  const size_t group = static_cast<size_t>(m / p.rows) * p.ld_param;
  T* y = static_cast<T*>(p.Y) + m * p.ld_y;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    float a[8], c[8];
    if (p.scale) load_param_chunk<VEC>(p.scale, p.param_dtype, group, p.K, i, t, threads, 0.0f, a);
    if (p.shift) load_param_chunk<VEC>(p.shift, p.param_dtype, group, p.K, i, t, threads, 0.0f, c);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float xh = v[i][j] * rstd;
      v[i][j] = __fmaf_rn(xh, p.scale ? a[j] + p.one : 1.0f, p.shift ? c[j] : 0.0f);
    }
    store_chunk<T, VEC>(y, p.K, i, t, threads, v[i]);
  }
}

struct BwdParams {
  const void* dY;
  const void* Z;          // or codes and scales
  const uint8_t* codes;
  const uint8_t* scales;
  const float2* stats;
  const void* scale;
  void* dZ;
  float* dscale;
  float* dshift;
  float* partial;         // [groups][splits][2][K], or null with one split
  int64_t ld_z, ld_dy, ld_dz, ld_param;
  int M, K, rows, splits, param_dtype, warps;
  float one;
};

// SRC: 0 the values themselves, 1 an int8 checkpoint, 2 an E4M3 one.
template <typename T, int NV, bool VEC, int SRC>
__global__ void __launch_bounds__(512) layer_norm_backward_kernel(BwdParams p) {
  extern __shared__ float sums[];  // [2][K] where several teams share the CTA
  __shared__ float2 red[kTeamWarps][32];
  const int threads = p.warps * 32, teams = blockDim.x / threads;
  const int team = threadIdx.x / threads, t = threadIdx.x % threads;
  const int group = blockIdx.x / p.splits, split = blockIdx.x % p.splits;
  const int first = group * p.rows, last = min(p.M, first + p.rows);
  const float inv_k = 1.0f / static_cast<float>(p.K);
  int turn = 0;

  float mul[NV][8], da[NV][8], dc[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if (p.scale)
      load_param_chunk<VEC>(p.scale, p.param_dtype, static_cast<size_t>(group) * p.ld_param, p.K, i, t, threads, 0.0f,
                            mul[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      mul[i][j] = p.scale ? mul[i][j] + p.one : 1.0f;
      da[i][j] = dc[i][j] = 0.0f;
    }
  }

  for (int m = first + split * teams + team; m < last; m += p.splits * teams) {
    const float2 st = p.stats[m];
    float x[NV][8], dy[NV][8];
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      // beyond K: dy is 0, and so are its terms in every sum
      load_chunk<T, VEC>(static_cast<const T*>(p.dY) + m * p.ld_dy, p.K, i, t, threads, 0.0f, dy[i]);
      if (SRC == 0)
        load_chunk<T, VEC>(static_cast<const T*>(p.Z) + m * p.ld_z, p.K, i, t, threads, 0.0f, x[i]);
      else
        ckpt_load_chunk<SRC == 1 ? SVDQ_CKPT8_INT8 : SVDQ_CKPT8_E4M3, VEC>(
            p.codes + static_cast<size_t>(m) * p.K,
            p.scales + static_cast<size_t>(m) * ((p.K + kCkptGroup - 1) / kCkptGroup), p.K, i, t, threads, x[i]);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        // a row that is not finite gives NaN statistics: its padding must not reach the sums
        const bool in = row_column<VEC>(i, j, t, threads) < p.K;
        x[i][j] = in ? (x[i][j] - st.x) * st.y : 0.0f;
        da[i][j] = __fmaf_rn(dy[i][j], x[i][j], da[i][j]);
        dc[i][j] += dy[i][j];
        dy[i][j] *= in ? mul[i][j] : 0.0f;
        s1 += dy[i][j];
        s2 = __fmaf_rn(dy[i][j], x[i][j], s2);
      }
    }
    const float2 s = team_sum2(s1, s2, p.warps, team, red[team], turn);
    const float m1 = s.x * inv_k, m2 = s.y * inv_k;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
      for (int j = 0; j < 8; ++j) dy[i][j] = st.y * (dy[i][j] - m1 - x[i][j] * m2);
      store_chunk<T, VEC>(static_cast<T*>(p.dZ) + m * p.ld_dz, p.K, i, t, threads, dy[i]);
    }
  }

  float* out_a = p.partial ? p.partial + static_cast<size_t>(blockIdx.x) * 2 * p.K
                           : p.dscale ? p.dscale + static_cast<size_t>(group) * p.K : nullptr;
  float* out_c = p.partial ? out_a + p.K : p.dshift ? p.dshift + static_cast<size_t>(group) * p.K : nullptr;
  if (teams > 1) {  // the teams add their columns in turn
    for (int r = 0; r < teams; ++r) {
      if (team == r) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int c = row_column<VEC>(i, j, t, threads);
            if (c < p.K) {
              sums[c] = r ? sums[c] + da[i][j] : da[i][j];
              sums[p.K + c] = r ? sums[p.K + c] + dc[i][j] : dc[i][j];
            }
          }
        }
      }
      __syncthreads();
    }
    for (int c = threadIdx.x; c < p.K; c += blockDim.x) {
      if (out_a) out_a[c] = sums[c];
      if (out_c) out_c[c] = sums[p.K + c];
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (out_a) store_chunk<float, VEC>(out_a, p.K, i, t, threads, da[i]);
      if (out_c) store_chunk<float, VEC>(out_c, p.K, i, t, threads, dc[i]);
    }
  }
}

// dscale and dshift from the partial sums: 32 columns and 8 shares of the splits per CTA.
__global__ void __launch_bounds__(256) layer_norm_sum_kernel(const float* __restrict__ partial, int splits, int K,
                                                          float* dscale, float* dshift) {
  __shared__ float part[8][32];
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), share = threadIdx.x >> 5, group = blockIdx.y, which = blockIdx.z;
  float* out = which ? dshift : dscale;
  if (!out) return;
  float s = 0.0f;
  if (c < K)
    for (int i = share; i < splits; i += 8)
      s += partial[((static_cast<size_t>(group) * splits + i) * 2 + which) * K + c];
  part[share][threadIdx.x & 31] = s;
  __syncthreads();
  if (share == 0 && c < K) {
    for (int i = 1; i < 8; ++i) s += part[i][threadIdx.x];
    out[static_cast<size_t>(group) * K + c] = s;
  }
}

constexpr int kSMs = 148;

struct Shape {
  int nv, warps, teams;
};

// Forward: up to 5 chunks of 8 values a thread; one warp a row while that reaches (no barriers), else
// the chunk count that wastes the fewest threads, the larger one when they tie.
Shape forward_shape(int K) {
  const int nvec = (K + 7) / 8;
  Shape s{};
  if (nvec <= 160) {
    s.warps = 1;
    s.nv = (nvec + 31) / 32;
  } else {
    int best = 1 << 30;
    for (int nv = 4; nv >= 2; --nv) {
      const int warps = (nvec + 32 * nv - 1) / (32 * nv);
      if (warps <= 16 && warps * nv < best) best = warps * nv, s.nv = nv, s.warps = warps;
    }
  }
  s.teams = s.warps >= kTeamWarps ? 1 : kTeamWarps / s.warps;
  return s;
}

// Backward: 24 fp32 a chunk stay in registers over all rows, so as few chunks as 16 warps allow.
Shape backward_shape(int K) {
  const int nvec = (K + 7) / 8;
  Shape s{};
  s.nv = nvec <= 512 ? 1 : nvec <= 1024 ? 2 : 4;
  s.warps = (nvec + 32 * s.nv - 1) / (32 * s.nv);
  s.teams = s.warps >= kTeamWarps ? 1 : kTeamWarps / s.warps;
  return s;
}

// CTAs that share a group's rows: two per SM over all groups, four rows a team at least.
int backward_splits(int K, int rows, int groups) {
  const Shape s = backward_shape(K);
  const int want = (2 * kSMs + groups - 1) / groups;
  const int most = (rows + 4 * s.teams - 1) / (4 * s.teams);
  return want < most ? want : most;
}

template <typename T, int NV, bool VEC>
svdq_status run_forward(const FwdParams& p, const Shape& s, cudaStream_t stream) {
  const int blocks = (p.M + s.teams - 1) / s.teams;
  layer_norm_kernel<T, NV, VEC><<<blocks, s.teams * s.warps * 32, 0, stream>>>(p);
  SVDQ_CUDA_TRY(cudaGetLastError());
  return SVDQ_OK;
}

template <typename T, bool VEC>
svdq_status forward_nv(const FwdParams& p, const Shape& s, cudaStream_t stream) {
  switch (s.nv) {
    case 1: return run_forward<T, 1, VEC>(p, s, stream);
    case 2: return run_forward<T, 2, VEC>(p, s, stream);
    case 3: return run_forward<T, 3, VEC>(p, s, stream);
    case 4: return run_forward<T, 4, VEC>(p, s, stream);
    default: return run_forward<T, 5, VEC>(p, s, stream);
  }
}

template <typename T, int NV, bool VEC, int SRC>
svdq_status run_backward(const BwdParams& p, const Shape& s, int groups, cudaStream_t stream) {
  const size_t smem = s.teams > 1 ? static_cast<size_t>(p.K) * 8 : 0;  // teams > 1: K <= 4096, 32 KB at most
  layer_norm_backward_kernel<T, NV, VEC, SRC><<<groups * p.splits, s.teams * s.warps * 32, smem, stream>>>(p);
  SVDQ_CUDA_TRY(cudaGetLastError());
  return SVDQ_OK;
}

template <typename T, bool VEC, int SRC>
svdq_status backward_nv(const BwdParams& p, const Shape& s, int groups, cudaStream_t stream) {
  switch (s.nv) {
    case 1: return run_backward<T, 1, VEC, SRC>(p, s, groups, stream);
    case 2: return run_backward<T, 2, VEC, SRC>(p, s, groups, stream);
    default: return run_backward<T, 4, VEC, SRC>(p, s, groups, stream);
  }
}

template <typename T>
svdq_status backward_type(const BwdParams& p, const Shape& s, int groups, bool vec, int src, cudaStream_t stream) {
  switch (src) {
    case 0: return vec ? backward_nv<T, true, 0>(p, s, groups, stream) : backward_nv<T, false, 0>(p, s, groups, stream);
    case 1: return vec ? backward_nv<T, true, 1>(p, s, groups, stream) : backward_nv<T, false, 1>(p, s, groups, stream);
    default: return vec ? backward_nv<T, true, 2>(p, s, groups, stream) : backward_nv<T, false, 2>(p, s, groups, stream);
  }
}

// 16-byte accesses of 8 values are possible: 16-byte aligned addresses (null is) and strides of whole chunks
bool vector_rows(int K, std::initializer_list<const void*> ptrs, std::initializer_list<int64_t> lds) {
  if (K % 8) return false;
  for (const void* p : ptrs)
    if (!aligned16(p)) return false;
  for (int64_t ld : lds)
    if (ld % 8) return false;
  return true;
}

}  // namespace

size_t layer_norm_backward_workspace(int M, int K, int rows) {
  const int groups = (M + rows - 1) / rows;
  const int splits = backward_splits(K, rows, groups);
  return splits > 1 ? static_cast<size_t>(groups) * splits * 2 * K * sizeof(float) : 0;
}

svdq_status launch_layer_norm(const NormArgs& a, const void* Z, const void* scale, const void* shift, void* Y,
                              float* stats, uint8_t* codes, uint8_t* scales, int ckpt, cudaStream_t stream) {
  FwdParams p{Z, scale, shift, Y, reinterpret_cast<float2*>(stats), codes, scales, a.ld_z, a.ld_y, a.ld_param,
              a.M, a.K, a.rows, a.param_dtype, 0, codes ? ckpt : -1, a.eps, a.plus_one ? 1.0f : 0.0f};
  const Shape s = forward_shape(a.K);
  p.warps = s.warps;
  const bool vec = vector_rows(a.K, {Z, scale, shift, Y, codes}, {a.ld_z, a.ld_y, a.ld_param});
  switch (a.dtype) {
    case SVDQ_DTYPE_BF16:
      return vec ? forward_nv<__nv_bfloat16, true>(p, s, stream) : forward_nv<__nv_bfloat16, false>(p, s, stream);
    case SVDQ_DTYPE_FP16:
      return vec ? forward_nv<__half, true>(p, s, stream) : forward_nv<__half, false>(p, s, stream);
    default: return vec ? forward_nv<float, true>(p, s, stream) : forward_nv<float, false>(p, s, stream);
  }
}

svdq_status launch_layer_norm_backward(const NormArgs& a, const void* dY, const void* Z, const uint8_t* codes,
                                       const uint8_t* scales, int ckpt, const float* stats, const void* scale,
                                       void* dZ, float* dscale, float* dshift, void* workspace, cudaStream_t stream) {
  const int groups = (a.M + a.rows - 1) / a.rows;
  const Shape s = backward_shape(a.K);
  BwdParams p{dY, Z, codes, scales, reinterpret_cast<const float2*>(stats), scale, dZ, dscale, dshift, nullptr,
              a.ld_z, a.ld_dy, a.ld_dz, a.ld_param, a.M, a.K, a.rows, backward_splits(a.K, a.rows, groups),
              a.param_dtype, s.warps, a.plus_one ? 1.0f : 0.0f};
  if (p.splits > 1 && (dscale || dshift)) p.partial = static_cast<float*>(workspace);
  const bool vec = vector_rows(a.K, {dY, Z, codes, scale, dZ, p.partial ? nullptr : dscale, p.partial ? nullptr : dshift},
                               {a.ld_z, a.ld_dy, a.ld_dz, a.ld_param});
  const int src = !codes ? 0 : ckpt == SVDQ_CKPT8_INT8 ? 1 : 2;
  svdq_status st;
  switch (a.dtype) {
    case SVDQ_DTYPE_BF16: st = backward_type<__nv_bfloat16>(p, s, groups, vec, src, stream); break;
    case SVDQ_DTYPE_FP16: st = backward_type<__half>(p, s, groups, vec, src, stream); break;
    default: st = backward_type<float>(p, s, groups, vec, src, stream); break;
  }
  SVDQ_TRY(st);
  if (p.partial) {
    layer_norm_sum_kernel<<<dim3((a.K + 31) / 32, groups, 2), 256, 0, stream>>>(p.partial, p.splits, a.K, dscale, dshift);
    SVDQ_CUDA_TRY(cudaGetLastError());
  }
  return SVDQ_OK;
}

}  // namespace svdq
