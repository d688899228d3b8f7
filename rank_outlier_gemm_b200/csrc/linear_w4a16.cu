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
// second one's MMA fragments read them and computes T (bf16 inputs, exact products, fp32 sums), which enters
// its product with L2 as three bf16 parts, all of its 24 bits.
//
// Measured (one B200, device time in a graph): NVFP4 1 x 4096 -> 24576, rank 32: 17.3-17.8 us, 3.3 TB/s, half
// the copy rate.  Reading alone takes 14.3 us of it, the products alone 13.7, and 4.8 are in both (two
// launches, the first kernel, the join): registers for three CTAs per SM leave the two to overlap only in
// part, and 384 CTAs are three on 88 SMs and two on 60.  Smaller layers are that fixed part: INT4 5 x 1280 ->
// 10240 10.6 us, NVFP4 16 x 10240 -> 1280 11.9, 1 x 640 -> 640 5.5.  For more than 4 tokens
// 60 to 164 bytes a thread spill.
//
// Order of k.  A contraction may run in any order, so a thread takes 16 consecutive bytes (32
// weights) of a row and feeds them to 8 MMA steps; the columns of X are laid out to match.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "ptx.cuh"
#include "rows.cuh"
#include "svdq_internal.h"

namespace svdq {
namespace {

using namespace dev;

constexpr int kSMs = 148;
constexpr int kMaxSmem = 112 * 1024;  // two CTAs per SM at least
constexpr int kMaxTokens = 16;
constexpr int kPrepWarps = 16, kPrepThreads = 32 * kPrepWarps;
constexpr int kStep = 128;        // weights of a row per warp step: 4 lanes x 32
constexpr int kUnitRows = 32;     // weight rows per warp: two M = 16 tiles
constexpr int kSlices = 2, kGroups = 4, kWarps = kSlices * kGroups;  // of a CTA: units, and warps per unit
constexpr int kTWarpK = 64;       // k per warp in a split of T
constexpr int kTSplit = kTWarpK * kPrepWarps;

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
  int groups, cluster, blocks;  // of steps; CTAs that share an output; pairs of units
  int branch_exp;               // |T| max |L2 / alpha_w| over the token's scale stay finite while the scale's (biased)
                                // exponent is at least this and that of the largest |x| together
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

// The larger magnitudes of two bf16 pairs, with any sign; a NaN does not count.
__device__ __forceinline__ uint32_t larger_pair(uint32_t a, uint32_t b) {
  uint32_t m;
  asm("max.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(m) : "r"(a), "r"(b));
  return m;
}
// What rounding to `hi` left of v; nothing of an infinity or a NaN, which stays in hi alone.
__device__ __forceinline__ float rest(float v, float hi) { return isfinite(hi) ? v - hi : 0.0f; }

__device__ __forceinline__ uint4 lds128(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
  return v;
}

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
__global__ void __launch_bounds__(kPrepThreads) w4a16_prepare_kernel(W4A16Params p) {
  __shared__ float red[kPrepWarps][16][16];
  grid_dep_launch_dependents();  // the second kernel starts on the weights
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  if (static_cast<int>(blockIdx.x) < p.M) {
    const int m = blockIdx.x;
    const uint16_t* x = p.X + static_cast<size_t>(m) * p.K;
    // xh of columns 8 c..8 c + 7, 0 beyond K; the first kHeld chunks of a thread stay in registers
    constexpr int kHeld = 4;
    uint32_t raw = 0;  // the largest magnitudes of x at even and at odd places, of any sign
    auto chunk = [&](int c, float (&v)[8]) {
      uint4 w = make_uint4(0, 0, 0, 0);
      float f[8] = {};
      if (c * 8 < p.K) {
        w = __ldg(reinterpret_cast<const uint4*>(x) + c);
        load8(p.inv_lam + c * 8, f);
      }
      unpack8(w, v, static_cast<const __nv_bfloat16*>(nullptr));
      raw = larger_pair(larger_pair(raw, larger_pair(w.x, w.y)), larger_pair(w.z, w.w));
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] *= f[j];
    };
    const int chunks = p.steps * (kStep / 8);
    uint32_t top = 0;  // bits of the largest finite magnitude
    auto note = [&](const float (&v)[8]) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t a = abs_bits(v[j]);
        if (a < 0x7F800000u) top = max(top, a);
      }
    };
    float held[kHeld][8];
#pragma unroll
    for (int i = 0; i < kHeld; ++i) chunk(threadIdx.x + i * kPrepThreads, held[i]);
#pragma unroll
    for (int i = 0; i < kHeld; ++i) note(held[i]);
    for (int c = threadIdx.x + kHeld * kPrepThreads; c < chunks; c += kPrepThreads) {
      float v[8];
      chunk(c, v);
      note(v);
    }
    // the token's scale 2^(e - 127), a normal number: brings the largest xh to [2^13, 2^14), or is as large as the
    // branch needs it, where x inv_lam is a hundred binary orders below x
    const int ex = static_cast<int>(max(raw >> 7 & 0xFF, raw >> 23 & 0xFF));
    int e = max(max(static_cast<int>(top >> 23) - 13, ex + p.branch_exp), 1);
    e = __reduce_max_sync(0xffffffffu, e);
    int* r = reinterpret_cast<int*>(red);
    if (lane == 0) r[warp] = e;
    __syncthreads();
    e = min(__reduce_max_sync(0xffffffffu, lane < kPrepWarps ? r[lane] : 1), 253);
    const float inv = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
    if (threadIdx.x == 0) p.pow2[m] = __uint_as_float(static_cast<uint32_t>(e) << 23);
    auto place = [&](int c, const float (&v)[8]) {
      if (c >= chunks) return;
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float a = v[2 * j] * inv, b = v[2 * j + 1] * inv;
        const __half2 h = __floats2half2_rn(a, b);
        const float2 f = __half22float2(h);
        // an infinity or a NaN stays in hi alone
        const float la = rest(a, f.x), lb = rest(b, f.y);
        hi[j] = as_u32(h);
        lo[j] = as_u32(__floats2half2_rn(la, lb));
      }
      const int w = c % 16;  // place in the 128-wide step
      const int q = INT4 ? (w >> 3) * 2 + (w & 1) : w & 3, ft = INT4 ? (w & 7) >> 1 : w >> 2;
      const int column = 2 * m;
      uint4* to = p.frag + ((static_cast<size_t>(c / 16) * p.tiles + column / 8) * 4 + q) * 32 + (column % 8) * 4 + ft;
      to[0] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      to[4] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    };
#pragma unroll
    for (int i = 0; i < kHeld; ++i) place(threadIdx.x + i * kPrepThreads, held[i]);
    for (int c = threadIdx.x + kHeld * kPrepThreads; c < chunks; c += kPrepThreads) {
      float v[8];
      chunk(c, v);
      place(c, v);
    }
    return;
  }

  const int job = blockIdx.x - p.M, split = job % p.t_splits, r0 = job / p.t_splits * 16;
  float acc[2][4] = {};
  const uint4 zero = make_uint4(0, 0, 0, 0);
  constexpr int kIter = kTWarpK / 32;
  uint4 a[kIter], b[kIter], x[kIter][2];
#pragma unroll
  for (int i = 0; i < kIter; ++i) {
    const int k = split * kTSplit + warp * kTWarpK + i * 32 + t * 8;
    a[i] = b[i] = x[i][0] = x[i][1] = zero;
    if (k < p.K) {
      a[i] = __ldg(reinterpret_cast<const uint4*>(p.L1t + static_cast<size_t>(r0 + g) * p.K + k));
      b[i] = __ldg(reinterpret_cast<const uint4*>(p.L1t + static_cast<size_t>(r0 + g + 8) * p.K + k));
#pragma unroll
      for (int j = 0; j < 2; ++j)
        if (j * 8 + g < p.M)
          x[i][j] = __ldg(reinterpret_cast<const uint4*>(p.X + static_cast<size_t>(j * 8 + g) * p.K + k));
    }
  }
#pragma unroll
  for (int i = 0; i < kIter; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      mma_bf16(acc[j], a[i].x, b[i].x, a[i].y, b[i].y, x[i][j].x, x[i][j].y);
      mma_bf16(acc[j], a[i].z, b[i].z, a[i].w, b[i].w, x[i][j].z, x[i][j].w);
    }
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) red[warp][g + 8 * (e >> 1)][j * 8 + 2 * t + (e & 1)] = acc[j][e];
  __syncthreads();
  const int r = threadIdx.x % 16, m = threadIdx.x / 16;  // m up to 31
  if (m < p.M) {
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < kPrepWarps; ++w) s += red[w][r][m];
    p.T[(static_cast<size_t>(split) * p.M + m) * p.r_pad + r0 + r] = s;
  }
}

// What a thread needs of the weights for one step: 32 weights of each of its 4 rows and their scales.  It
// copies them to its own places of a ring in shared memory, [piece][lane] x 16 bytes per stage of a
// warp, and reads only those back.
struct Step {
  uint4 w[4];
  uint4 sc;
};
constexpr int kPieces = 5, kStageBytes = kPieces * 32 * 16, kStages = 3;

// 16 or 8 bytes to shared memory, zeros if !in (`src` is then not read)
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy8(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(in ? 8 : 0) : "memory");
}

// Where a thread finds its part of a unit: its first row's codes and its scales, at step 0.
struct Source {
  const uint8_t* codes;
  const uint8_t* sf;
  int rows;  // of its 4 rows, those below N (the first ones)
};
template <bool INT4>
__device__ __forceinline__ Source unit_source(const W4A16Params& p, int u, int g, int t) {
  Source v;
  const int n = unit_row<INT4>(u, 0, g);
  v.rows = INT4 ? min(4, max(0, p.N - n)) : n < p.N ? min(4, (p.N - n + 31) / 32) : 0;
  v.codes = p.codes + static_cast<size_t>(n < p.N ? n : 0) * (p.K / 2) + t * (INT4 ? 8 : 16);
  if (INT4)  // of rows b = 0..3, bf16
    v.sf = static_cast<const uint8_t*>(p.sf) + (u * kUnitRows + 4 * g) * 2;
  else  // of rows b = 0..3 (a word each) and 64 columns
    v.sf = static_cast<const uint8_t*>(p.sf) +
           (static_cast<size_t>(u >> 2) * (p.K / 64) + (t >> 1)) * 512 + (8 * (u & 3) + g) * 16;
  return v;
}

// Starts the copies of step s.
template <bool INT4>
__device__ __forceinline__ void fetch_step(const W4A16Params& p, const Source& from, int s, int t, uint32_t to) {
  const uint8_t* row = from.codes + s * (kStep / 2);
  const size_t next = static_cast<size_t>(INT4 ? 1 : 32) * (p.K / 2);
  const bool second = s * kStep + 64 < p.K;  // the step's second 64 columns exist
#pragma unroll
  for (int b = 0; b < 4; ++b, to += 512) {
    const bool in = b < from.rows;
    const uint8_t* at = in ? row + b * next : p.codes;
    if (INT4) {  // 8 bytes of each 64-wide group
      copy8(to, at, in);
      copy8(to + 8, second ? at + 32 : at, in && second);
    } else {
      const bool inside = in && (second || t < 2);
      copy16(to, inside ? at : p.codes, inside);
    }
  }
  if (INT4) {
    const size_t group = static_cast<size_t>((p.N + 255) / 256) * 256 * 2;
    const uint8_t* at = from.sf + 2 * s * group;
    copy8(to, at, true);
    copy8(to + 8, second ? at + group : at, second);
  } else {
    const bool inside = second || t < 2;
    copy16(to, inside ? from.sf + static_cast<size_t>(s) * 1024 : static_cast<const uint8_t*>(p.sf), inside);
  }
}

template <bool INT4, int NT>
__device__ __forceinline__ void multiply_step(const W4A16Params& p, int s, int g, int t, int lane, const Step& v,
                                              float (&acc)[2][NT][4]) {
  const uint4 zero = make_uint4(0, 0, 0, 0);
  const uint4* frag = p.frag + static_cast<size_t>(s) * NT * 128 + lane;
  __half2 s01[4];  // NVFP4: the scales of this thread's two groups, per row
  if (!INT4) {
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      uint32_t h;
      asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>((&v.sc.x)[b] >> (16 * (t & 1)))));
      s01[b] = as_half2(h);
    }
  }
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    uint4 x[NT][2];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int q = 0; q < 2; ++q) x[j][q] = j * 8 + g < 2 * p.M ? frag[(j * 4 + 2 * half + q) * 32] : zero;
#pragma unroll
    for (int tile = 0; tile < 2; ++tile) {
      float sum[NT][4] = {};  // INT4: of one group
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        uint32_t a[4], b[4];
        if (INT4) {
          int4_pairs((&v.w[2 * tile].x)[2 * half + q], a);
          int4_pairs((&v.w[2 * tile + 1].x)[2 * half + q], b);
        } else {
          e2m1_pairs((&v.w[2 * tile].x)[2 * half + q], a);
          e2m1_pairs((&v.w[2 * tile + 1].x)[2 * half + q], b);
          const __half2 sa = half ? __high2half2(s01[2 * tile]) : __low2half2(s01[2 * tile]);
          const __half2 sb = half ? __high2half2(s01[2 * tile + 1]) : __low2half2(s01[2 * tile + 1]);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            a[j] = as_u32(__hmul2(as_half2(a[j]), sa));
            b[j] = as_u32(__hmul2(as_half2(b[j]), sb));
          }
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          float(&to)[4] = INT4 ? sum[j] : acc[tile][j];
          mma_f16(to, a[0], b[0], a[1], b[1], x[j][q].x, x[j][q].y);
          mma_f16(to, a[2], b[2], a[3], b[3], x[j][q].z, x[j][q].w);
        }
      }
      if (INT4) {
        const uint32_t c = tile ? (half ? v.sc.w : v.sc.y) : (half ? v.sc.z : v.sc.x);  // rows 2 tile, 2 tile + 1
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            acc[tile][j][e] = __fmaf_rn(sum[j][e], e < 2 ? pair_lo(c) : pair_hi(c), acc[tile][j][e]);
      }
    }
  }
}

// The low-rank branch as MMA steps of 16 ranks: rows of L2 / alpha_w against the tokens' T over their
// scale, `s_t`, in three bf16 parts, which are all 24 bits of the fp32 sum.  Two parts are a token's columns, the
// third takes a second product.
template <bool INT4, int NT>
__device__ __forceinline__ void multiply_branch(const W4A16Params& p, const uint16_t* s_t, int u, int g, int t,
                                                float (&acc)[2][NT][4]) {
  constexpr int kAhead = 4;  // steps whose loads of L2 are in flight at once
  for (int r0 = 0; r0 < p.r_pad; r0 += 16 * kAhead) {
    uint2 l2[kAhead][4];
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const int n = unit_row<INT4>(u, b, g), r = r0 + 16 * i;
        l2[i][b] = n < p.N && r < p.r_pad
                       ? __ldg(reinterpret_cast<const uint2*>(p.L2t + static_cast<size_t>(n) * p.r_pad + r) + t)
                       : make_uint2(0, 0);
      }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int r = r0 + 16 * i;
      if (r >= p.r_pad) break;
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const int m = (j * 8 + g) >> 1;
        const uint16_t* parts = s_t + m * 3 * p.r_pad + r + 4 * t;  // an even column's are 0 and 2, an odd one's is 1
        uint2 first = make_uint2(0, 0), third = first;
        if (m < p.M) {
          first = *reinterpret_cast<const uint2*>(parts + (g & 1) * p.r_pad);
          if (!(g & 1)) third = *reinterpret_cast<const uint2*>(parts + 2 * p.r_pad);
        }
#pragma unroll
        for (int tile = 0; tile < 2; ++tile) {
          const uint2 even = l2[i][2 * tile], odd = l2[i][2 * tile + 1];
          mma_bf16(acc[tile][j], even.x, odd.x, even.y, odd.y, first.x, first.y);
          mma_bf16(acc[tile][j], even.x, odd.x, even.y, odd.y, third.x, third.y);
        }
      }
    }
  }
}

// A CTA takes two units of 32 weight rows at a time; its warps, four per unit, and those of the other
// CTAs of its cluster take the 128-wide steps of K in turn (p.groups in all).  Every warp leaves its
// sums in shared memory, where each CTA of the cluster adds up a share of the outputs: the CTA's four
// groups first, then the CTAs.  Copies of weights run two steps ahead of the products, over the ends of
// units and ahead of the wait for the first kernel's results; what that kernel wrote is read through
// L1, which the CTAs of an SM share.
template <bool INT4, int NT>
__global__ void __launch_bounds__(32 * kWarps, NT > 2 ? 2 : 3) w4a16_kernel(W4A16Params p) {
  constexpr int kRows = kSlices * kUnitRows, kPitch = kRows + 8;  // a warp's stores fall into different banks
  constexpr int kGroupFloats = NT * 4 * kPitch;
  extern __shared__ __align__(16) uint8_t smem[];  // the warps' rings, the groups' sums
                                                   // [kGroups][NT * 4 tokens][kPitch], T over the tokens' scales
                                                   // [M][3 parts][r_pad] in bf16
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int slice = warp % kSlices, kg = warp / kSlices;
  const int rank = blockIdx.x % p.cluster, block_step = gridDim.x / p.cluster;
  const int first = rank * kGroups + kg;  // this warp's first step of a unit
  const int jobs = p.M * kRows;
  const uint32_t ring = smem_u32(smem) + warp * kStages * kStageBytes + lane * 16;
  float* red = reinterpret_cast<float*>(smem + kWarps * kStages * kStageBytes);
  uint16_t* s_t = reinterpret_cast<uint16_t*>(red + kGroups * kGroupFloats);

  // this warp's steps, unit by unit, as they are fetched
  int next_block = first < p.steps ? static_cast<int>(blockIdx.x) / p.cluster : p.blocks, next_step = first;
  Source source = unit_source<INT4>(p, next_block * kSlices + slice, g, t);
  auto fetch = [&](int stage) {
    if (next_block < p.blocks) {
      fetch_step<INT4>(p, source, next_step, t, ring + stage * kStageBytes);
      next_step += p.groups;
      if (next_step >= p.steps) {
        next_step = first, next_block += block_step;
        source = unit_source<INT4>(p, next_block * kSlices + slice, g, t);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) fetch(i);
  grid_dep_wait();
  const bool branch = p.r_pad > 0 && rank == p.cluster - 1;  // has the last group of steps, which is the shortest
  if (branch) {
    const int n = p.M * p.r_pad;
    for (int i0 = threadIdx.x; i0 < n; i0 += 2 * blockDim.x) {
      float v[2] = {0.0f, 0.0f};
      for (int k = 0; k < p.t_splits; k += 6) {  // all loads of K <= 12288 at once, for two values
        float a[2][6];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int j = 0; j < 6; ++j) {
            const int i = i0 + h * blockDim.x;
            a[h][j] = k + j < p.t_splits && i < n ? p.T[static_cast<size_t>(k + j) * n + i] : 0.0f;
          }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int j = 0; j < 6; ++j) v[h] += a[h][j];
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int i = i0 + h * blockDim.x;
        if (i >= n) continue;
        const int m = i / p.r_pad;
        float left = v[h] * __frcp_rn(p.pow2[m]);  // exact: a power of two
        uint16_t* to = s_t + 2 * m * p.r_pad + i;
#pragma unroll
        for (int part = 0; part < 3; ++part) {
          const __nv_bfloat16 b = __float2bfloat16_rn(left);
          to[part * p.r_pad] = __bfloat16_as_ushort(b);
          left = rest(left, __bfloat162float(b));
        }
      }
    }
    __syncthreads();
  }

  int stage = 0;
  for (int block = blockIdx.x / p.cluster; block < p.blocks; block += block_step) {
    const int unit0 = block * kSlices, u = unit0 + slice;
    float acc[2][NT][4] = {};
    if (branch && kg == kGroups - 1) multiply_branch<INT4, NT>(p, s_t, u, g, t, acc);
    for (int s = first; s < p.steps; s += p.groups) {
      fetch(stage ? stage - 1 : kStages - 1);  // the stage read last
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
      Step v;
      const uint32_t from = ring + stage * kStageBytes;
#pragma unroll
      for (int b = 0; b < 4; ++b) v.w[b] = lds128(from + b * 512);
      v.sc = lds128(from + 4 * 512);
      multiply_step<INT4, NT>(p, s, g, t, lane, v, acc);
      if (++stage == kStages) stage = 0;
    }

    // a thread holds a token's hi and lo columns side by side: their sum
#pragma unroll
    for (int tile = 0; tile < 2; ++tile)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          red[kg * kGroupFloats + (j * 4 + t) * kPitch + slice * kUnitRows + (2 * tile + h) * 8 + g] =
              acc[tile][j][2 * h] + acc[tile][j][2 * h + 1];
    __syncthreads();
    auto four = [&](int at) {
      const float* r = red + at;
      return ((r[0] + r[kGroupFloats]) + r[2 * kGroupFloats]) + r[3 * kGroupFloats];
    };
    auto finish = [&](int i, float v) {
      const int m = i / kRows, row = i % kRows, n = unit_row<INT4>(unit0 + row / kUnitRows, (row >> 3) & 3, row & 7);
      if (n >= p.N) return;
      // the sum times alpha_w first: the product of the two powers of two may leave fp32's range where Y does not
      const __nv_bfloat16 y = __float2bfloat16_rn(__fmaf_rn(v * p.alpha_w, p.pow2[m], __ldg(p.bias + n)));
      p.Y[static_cast<size_t>(m) * p.N + n] = *reinterpret_cast<const uint16_t*>(&y);
    };
    if (p.cluster == 1) {
      for (int i = threadIdx.x; i < jobs; i += blockDim.x) finish(i, four(i / kRows * kPitch + i % kRows));
      __syncthreads();  // before the next units' sums
    } else {
      for (int i = threadIdx.x; i < jobs; i += blockDim.x) {
        const int at = i / kRows * kPitch + i % kRows;
        red[at] = four(at);
      }
      cluster_sync_all();
      const uint32_t mine = smem_u32(red);
      const int share = jobs / p.cluster;  // neighbouring outputs to neighbouring lanes: rows of 128 bytes
      for (int i = rank * share + threadIdx.x; i < (rank + 1) * share; i += blockDim.x) {
        const int at = i / kRows * kPitch + i % kRows;
        float fours[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) fours[c] = c < p.cluster ? ld_dsmem_f32(mapa_shared(mine, c) + at * 4) : 0.0f;
        float v = fours[0];
#pragma unroll
        for (int c = 1; c < 8; ++c) v += fours[c];
        finish(i, v);
      }
      cluster_sync_all();  // the others may still read this CTA's sums
    }
  }
}

inline size_t up256(size_t x) { return (x + 255) / 256 * 256; }
int column_tiles(int M) { return M <= 4 ? 1 : M <= 8 ? 2 : 4; }

// How the steps of K are shared out: to the 4 groups of one CTA, or to 8, 16 or 32 (a cluster of CTAs)
// while there are steps for them and the device still has fewer than two thousand warps.  The number
// depends on the layer alone, so a token's sums are the same for any M.
int step_groups(int N, int steps) {
  const int units = (N + kUnitRows - 1) / kUnitRows;
  int groups = kGroups;
  while (groups < 8 * kGroups && groups < steps && units * groups < 2048) groups *= 2;
  return groups;
}

template <bool INT4, int NT>
svdq_status launch_main(W4A16Params& p, cudaStream_t stream) {
  p.cluster = p.groups / kGroups;
  const int units = INT4 ? (p.N + kUnitRows - 1) / kUnitRows : (p.N + 127) / 128 * 4;
  p.blocks = (units + kSlices - 1) / kSlices;
  const size_t smem = static_cast<size_t>(kWarps) * kStages * kStageBytes +
                      static_cast<size_t>(kGroups) * NT * 4 * (kSlices * kUnitRows + 8) * sizeof(float) +
                      static_cast<size_t>(p.M) * p.r_pad * 3 * sizeof(uint16_t);
  // no more CTAs than the SMs hold at a time (dealt out evenly only where there are more pairs of units than that,
  // or no more than SMs)
  const int resident = kSMs * (NT > 2 ? 2 : 3);
  const int grid = p.cluster > 1 || p.blocks < resident ? p.blocks : resident;
  static std::atomic<uint64_t> allowed{0};
  SVDQ_TRY(allow_dynamic_smem(reinterpret_cast<const void*>(w4a16_kernel<INT4, NT>), kMaxSmem, allowed));
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = p.cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid * p.cluster);
  cfg.blockDim = dim3(32 * kWarps);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = p.cluster > 1 ? 2 : 1;
  SVDQ_CUDA_TRY(cudaLaunchKernelEx(&cfg, w4a16_kernel<INT4, NT>, p));
  return SVDQ_OK;
}

template <bool INT4>
svdq_status launch(W4A16Params& p, cudaStream_t stream) {
  w4a16_prepare_kernel<INT4><<<p.M + p.r_pad / 16 * p.t_splits, kPrepThreads, 0, stream>>>(p);
  SVDQ_CUDA_TRY(cudaGetLastError());
  switch (p.tiles) {
    case 1: return launch_main<INT4, 1>(p, stream);
    case 2: return launch_main<INT4, 2>(p, stream);
    default: return launch_main<INT4, 4>(p, stream);
  }
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
  p.groups = step_groups(w->N, p.steps);
  p.alpha_w = w->alpha_w;
  p.branch_exp = w->branch_exp - 124;  // |T L2 / alpha_w| <= 2^(ex - 126 + branch_exp), at most 2^125 over the scale
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.frag = reinterpret_cast<uint4*>(ws);
  ws += up256(static_cast<size_t>(p.steps) * p.tiles * 4 * 32 * 16);
  p.pow2 = reinterpret_cast<float*>(ws);
  p.T = reinterpret_cast<float*>(ws + 256);
  return w->format == SVDQ_FORMAT_INT4 ? launch<true>(p, stream) : launch<false>(p, stream);
}

}  // namespace svdq
