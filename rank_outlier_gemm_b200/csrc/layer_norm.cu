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
//
// Measured (one B200, device time in a graph; the copy rate would take the time in brackets): forward
// bf16 8192 x 4096 43.5 us (20.5), fp32 53.4 (40.9), bf16 4096 x 1152 with an int8 checkpoint 10.3 (3.6), fp16
// 8192 x 1280 17 (6.4); gradient bf16 8192 x 4096 38.6 (30.7), 4608 x 12288 70.7 (51.8), 4500 x 4096 from an int8
// checkpoint 27.3 (14.2), 8192 x 640 13.5 (4.8).  The 16-bit forward and decoding issue for half of their time, and
// the rest is a row's chain of two reductions with 32 warps per SM to cover it.  The fp16 forward spills at three
// to five chunks a thread (up to 108 bytes a thread at K = 1032 to 1280), the gradient at four (36 to 104 bytes).
#include <algorithm>
#include <initializer_list>
#include <type_traits>

#include "ptx.cuh"
#include "rows.cuh"
#include "svdq_internal.h"

namespace svdq {
namespace {

using namespace dev;

// Warps of a CTA, shared out to teams (a team may have more: it is alone then).  The backward takes one CTA
// of 16 warps per SM, which halves the partial sums that two of 8 would leave.
constexpr int kForwardWarps = 8, kBackwardWarps = 16;
constexpr int kSMs = 148;

// Sums over a team of `warps` warps, the same in every thread.  `red` holds two buffers of 2 x 16
// values per team, used in turn: the barrier of one call separates the reads of the call before from
// the writes of the call after.  Each warp adds the warps' values by shuffles, one value a lane.
__device__ __forceinline__ void team_barrier(int team, int warps) {
  asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "r"(warps * 32) : "memory");
}
// Of a and b: lanes 0-15 of the result hold the first sum, lanes 16-31 the second.  `flag`, if given, is read
// behind the barrier into `seen`.
__device__ __forceinline__ float team_sum_halves(float a, float b, int warps, int team, float* red, int& turn,
                                                 const volatile int* flag = nullptr, int* seen = nullptr) {
  float v = warp_sum2_halves(a, b);
  if (warps == 1) return v;
  const int lane = threadIdx.x & 31;
  float* r = red + turn * 32;
  turn ^= 1;
  if ((lane & 15) == 0) r[lane + (threadIdx.x >> 5) - team * warps] = v;
  team_barrier(team, warps);
  if (flag) *seen = *flag;
  v = (lane & 15) < warps ? r[lane] : 0.0f;
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float2 team_sum2(float a, float b, int warps, int team, float* red, int& turn,
                                            const volatile int* flag = nullptr, int* seen = nullptr) {
  const float v = team_sum_halves(a, b, warps, team, red, turn, flag, seen);
  const float o = __shfl_xor_sync(0xffffffffu, v, 16);
  return (threadIdx.x & 16) ? make_float2(o, v) : make_float2(v, o);
}
__device__ __forceinline__ float team_sum(float a, int warps, int team, float* red, int& turn) {
  if (warps == 1) return warp_sum(a);
  return __shfl_sync(0xffffffffu, team_sum_halves(a, 0.0f, warps, team, red, turn), 0);
}

// sum / count.  The product with the rounded reciprocal alone is off by a step at many counts (896 and 3584 among
// them), which is not 0 on a row of one value; what it leaves of the sum is exact in one FMA, and added back gives
// the quotient itself where that is a value of fp32.  (IEEE division instead: bf16 4608 x 12288 67 -> 72 us.)
__device__ __forceinline__ float mean_of(float sum, float count, float inv_count) {
  const float q = sum * inv_count;
  return isfinite(q) ? __fmaf_rn(__fmaf_rn(-q, count, sum), inv_count, q) : q;
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
  int ahead;                                 // rows ahead that are brought into L2, 0: none
  float eps, one;
};

// A chunk of the per-group vectors.  P: their type where it is known (vector layout), void where it is not.
template <typename P, bool VEC>
__device__ __forceinline__ void param_chunk(const void* p, int dtype, size_t offset, int K, int i, int t, int threads,
                                            float (&v)[8]) {
  if constexpr (std::is_void<P>::value)
    load_param_chunk<VEC>(p, dtype, offset, K, i, t, threads, 0.0f, v);
  else
    load8(static_cast<const P*>(p) + offset + chunk_column(i, t, threads), v);
}

template <typename T, typename P, int NV, bool VEC>
__global__ void __launch_bounds__(512, VEC && sizeof(T) == 2 ? 2 : 0) layer_norm_kernel(FwdParams p) {
  __shared__ float red[kForwardWarps][64];
  const int threads = p.warps * 32, team = threadIdx.x / threads, t = threadIdx.x % threads;
  const int m = blockIdx.x * (blockDim.x / threads) + team;
  if (m >= p.M) return;  // whole teams: a barrier has all of its team's warps
  int turn = 0;
  const T* z = static_cast<const T*>(p.Z) + m * p.ld_z;
  if (VEC && p.ahead && t == 0 && m + p.ahead < p.M) bulk_prefetch(z + p.ahead * p.ld_z, p.K * sizeof(T));
  Held<T, VEC> held[NV];
  auto inside = [&](int i) { return chunk_column(i, t, threads) < p.K; };
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if constexpr (VEC) {
      held[i].clear();
      if (inside(i)) held[i].load(z + chunk_column(i, t, threads));
    } else {
      load_chunk<T, false>(z, p.K, i, t, threads, 0.0f, held[i].f);
    }
  }
  F2 sum = f2(0.0f, 0.0f);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    float v[8];
    held[i].values(v);
#pragma unroll
    for (int j = 0; j < 4; ++j) sum = add2(sum, f2(v[2 * j], v[2 * j + 1]));
  }
  float s0, s1;
  unpack2(sum, s0, s1);
  const float count = static_cast<float>(p.K), inv_k = 1.0f / count;
  const float mu = mean_of(team_sum(s0 + s1, p.warps, team, red[team], turn), count, inv_k);
  F2 sq = f2(0.0f, 0.0f);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if (!inside(i)) continue;
    float v[8];
    held[i].values(v);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (!VEC && chunk_column(i, t, threads) + j >= p.K) v[j] = mu;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const F2 d = add2(f2(v[2 * j], v[2 * j + 1]), f2(-mu, -mu));
      sq = fma2(d, d, sq);
    }
  }
  unpack2(sq, s0, s1);
  const float var = team_sum(s0 + s1, p.warps, team, red[team], turn) * inv_k;
  const float rstd = __frcp_rn(__fsqrt_rn(__fadd_rn(var, p.eps)));
  if (p.stats && t == 0) p.stats[m] = make_float2(mu, rstd);
  const size_t group = static_cast<size_t>(m / p.rows) * p.ld_param;
  T* y = static_cast<T*>(p.Y) + m * p.ld_y;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    float v[8], a[8], c[8];
    held[i].values(v);
    // one chunk's parameters at a time: all at once would take the registers of half the warps
    if (VEC && sizeof(T) == 2) asm volatile("" ::: "memory");
    const bool in = inside(i);
    if (p.scale && in) param_chunk<P, VEC>(p.scale, p.param_dtype, group, p.K, i, t, threads, a);
    if (p.shift && in) param_chunk<P, VEC>(p.shift, p.param_dtype, group, p.K, i, t, threads, c);
    if (p.ckpt >= 0) {
      uint8_t* codes = p.codes + static_cast<size_t>(m) * p.K;
      uint8_t* scales = p.scales + static_cast<size_t>(m) * ((p.K + kCkptGroup - 1) / kCkptGroup);
      const uint32_t top = held[i].largest();
      if (p.ckpt == SVDQ_CKPT8_INT8)
        ckpt_store_chunk<SVDQ_CKPT8_INT8, VEC>(codes, scales, p.K, i, t, threads, top, v);
      else
        ckpt_store_chunk<SVDQ_CKPT8_E4M3, VEC>(codes, scales, p.K, i, t, threads, top, v);
    }
    if (!in) continue;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      // (z - mu) rstd in two steps: a value that is the mean gives an exact zero
      F2 r = mul2(add2(f2(v[2 * j], v[2 * j + 1]), f2(-mu, -mu)), f2(rstd, rstd));
      if (p.scale) r = mul2(r, add2(f2(a[2 * j], a[2 * j + 1]), f2(p.one, p.one)));
      if (p.shift) r = add2(r, f2(c[2 * j], c[2 * j + 1]));
      unpack2(r, v[2 * j], v[2 * j + 1]);
    }
    store_chunk<T, VEC>(y, p.K, i, t, threads, v);
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
  int M, K, rows, splits, param_dtype, warps, teams, stages, packed;
  float one;
  int* err;
  uint64_t wait_ns;
  int stall;              // test hook: one arrival more than the ring's stages get
};

constexpr int kMaxStages = 4;

// A barrier of the CTA's `workers` threads (the copying warp is not among them).
__device__ __forceinline__ void workers_barrier(int workers) { asm volatile("bar.sync 15, %0;" ::"r"(workers) : "memory"); }

// Floats of the multipliers in shared memory: K, eight zeros, and 16-byte alignment behind them.
__host__ __device__ constexpr int mul_floats(int K) { return (K + 8 + 3) / 4 * 4; }

// A stage of the ring of the vector layout: one row for each of the CTA's teams, side by side (dY, then Z
// or its codes), then the 4-byte aligned words that hold their scale bytes, then their statistics.
template <typename T, int SRC>
struct Stage {
  int z, scales, stats, bytes;
  __host__ __device__ Stage(int K, int teams)
      : z(teams * K * static_cast<int>(sizeof(T))),
        scales(z + teams * K * (SRC ? 1 : static_cast<int>(sizeof(T)))),
        stats(scales + (SRC ? (teams * ((K + kCkptGroup - 1) / kCkptGroup) + 3 + 15) / 16 * 16 : 0)),
        bytes(stats + (teams * 8 + 15) / 16 * 16) {}
};

// SRC: 0 the values themselves, 1 an int8 checkpoint, 2 an E4M3 one.
// In the vector layout one more warp copies the teams' next rows, which are consecutive, into a ring of
// `stages` stages in shared memory by bulk copies, so that memory stays busy across the rows'
// reductions and the teams issue nothing for it.
template <typename T, int NV, bool VEC, int SRC>
__global__ void __launch_bounds__(32 * (kBackwardWarps + 1)) layer_norm_backward_kernel(BwdParams p) {
  // the multipliers, then the ring; at the end the teams' [2][K] sums where several share the CTA
  extern __shared__ __align__(16) float smem[];
  __shared__ float red[kBackwardWarps][64];
  __shared__ uint64_t full[kMaxStages], empty[kMaxStages];
  __shared__ int s_abort;
  constexpr int kFmt = SRC == 2 ? SVDQ_CKPT8_E4M3 : SVDQ_CKPT8_INT8;
  // chunks of a row held across its reduction; with more than two the row is read again (in place: dZ may be
  // dY, and without the ring the row is held whole)
  constexpr int kHeld = NV <= 2 || !VEC ? NV : 1;
  // Three or four chunks a thread: more than 1024 of them in the row, which takes the whole CTA (11 warps at least).
  // Saying so saves the registers of teams, without which a third and fourth chunk's sums spill (bf16 2048 x 16384
  // 62 us against 129, 4608 x 12288 70.7 against 76.5).
  constexpr bool kAlone = NV >= 3;
  const int threads = p.warps * 32, teams = kAlone ? 1 : p.teams, workers = teams * threads;
  const int team = kAlone ? 0 : threadIdx.x / threads, t = kAlone ? threadIdx.x : threadIdx.x % threads;
  const int lane = threadIdx.x & 31;
  const Stage<T, SRC> at(p.K, teams);
  const int group = blockIdx.x / p.splits, split = blockIdx.x % p.splits;
  const int first = group * p.rows, last = min(p.M, first + p.rows);
  const int scale_row = (p.K + kCkptGroup - 1) / kCkptGroup;
  const float inv_k = 1.0f / static_cast<float>(p.K);
  // the CTA's rows: `teams` consecutive ones from m0, m0 + step, ...
  const int step = p.splits * teams, m0 = first + split * teams;
  const WaitCtl ctl{p.err, p.wait_ns, &s_abort};
  uint8_t* ring = reinterpret_cast<uint8_t*>(smem + mul_floats(p.K));
  int turn = 0;

  if (VEC) {
    if (threadIdx.x == 0) {
      s_abort = 0;
      for (int s = 0; s < p.stages; ++s) {
        mbar_init(&full[s], 33 + p.stall);
        mbar_init(&empty[s], workers / 32);
      }
      fence_barrier_init();
    }
    __syncthreads();
    if (static_cast<int>(threadIdx.x) >= workers) {
      uint32_t parity = 1;  // of the stage's release; the first pass finds every stage free
      int stage = 0;
      for (int m = m0; m < last; m += step) {
        if (!wait_warp(&empty[stage], parity, ctl)) break;
        const int n = min(teams, last - m);
        uint64_t* bar = &full[stage];
        uint8_t* to = ring + stage * at.bytes;
        const uint32_t dy = p.K * sizeof(T), z = SRC ? p.K : p.K * sizeof(T);
        if (lane == 0) mbar_arrive_expect_tx(bar, n * (dy + z));
        __syncwarp();
        if (p.packed) {
          if (lane == 0) bulk_load(to, static_cast<const T*>(p.dY) + m * p.ld_dy, n * dy, bar);
          if (lane == 1)
            bulk_load(to + at.z, SRC ? static_cast<const void*>(p.codes + static_cast<size_t>(m) * p.K)
                                     : static_cast<const T*>(p.Z) + m * p.ld_z, n * z, bar);
        } else if (lane < n) {
          bulk_load(to + lane * dy, static_cast<const T*>(p.dY) + (m + lane) * p.ld_dy, dy, bar);
          bulk_load(to + at.z + lane * z, SRC ? static_cast<const void*>(p.codes + static_cast<size_t>(m + lane) * p.K)
                                              : static_cast<const T*>(p.Z) + (m + lane) * p.ld_z, z, bar);
        }
        if (lane < n) copy8_async(to + at.stats + lane * 8, p.stats + m + lane);
        if (SRC) {
          const uint8_t* from = p.scales + static_cast<size_t>(m) * scale_row;
          const uint8_t* base = from - (reinterpret_cast<uintptr_t>(from) & 3);
          const uint8_t* end = p.scales + static_cast<size_t>(p.M) * scale_row;
          const int words = static_cast<int>(from + n * scale_row - base + 3) / 4;
          for (int i = lane; i < words; i += 32) {
            const uint8_t* word = base + 4 * i;
            if (word >= p.scales && word + 4 <= end) {
              copy4_async(to + at.scales + 4 * i, word);
            } else {  // the array's first or last bytes
              for (int b = 0; b < 4; ++b)
                if (word + b >= p.scales && word + b < end) to[at.scales + 4 * i + b] = word[b];
              __threadfence_block();
            }
          }
        }
        copies_arrive(bar);
        if (++stage == p.stages) stage = 0, parity ^= 1;
      }
      // None of these copies may land after the CTA has ended, which the teams alone do not see to once a wait ran
      // out.  The stages below `stage` were filled in this pass, the others in the one before (or not at all).
      WaitCtl drain = ctl;
      int none = 0;
      drain.abort = &none;
      for (int s = 0; s < p.stages; ++s) wait_warp(&full[s], s < stage ? parity ^ 1 : parity, drain);
      return;
    }
  }

  float* mul = smem;
  if (team == 0) {
    float w[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
      for (int j = 0; j < 8; ++j) w[i][j] = 1.0f - p.one;
      if (p.scale)
        load_param_chunk<VEC>(p.scale, p.param_dtype, static_cast<size_t>(group) * p.ld_param, p.K, i, t, threads, 0.0f,
                              w[i]);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
      for (int j = 0; j < 8; ++j) w[i][j] += p.one;
      store_chunk<float, VEC>(mul, p.K, i, t, threads, w[i]);
    }
    if (t < 8) mul[p.K + t] = 0.0f;
  }
  workers_barrier(workers);

  F2 da[NV][4], dc[NV][4];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) da[i][j] = dc[i][j] = f2(0.0f, 0.0f);

  // a chunk beyond K works on column 0 with multipliers 0: it adds nothing to the row's sums and its own are dropped
  int col[NV], mcol[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c0 = chunk_column(i, t, threads);
    const bool in = (kAlone && i + 1 < NV) || c0 < p.K;  // a long row's last chunks alone may be beyond
    col[i] = in ? c0 : 0;
    mcol[i] = in ? c0 : p.K;
  }
  uint32_t parity = 0;
  int stage = 0;
  // False once a wait ran out (the error word says so) or the CTA gave up: the teams then go through their rows
  // without freeing stages or storing, so that their barriers still match.
  bool alive = true;
  for (int m = m0 + team, block = m0; block < last; block += step, m += step) {
    const uint8_t* here = ring + stage * at.bytes;
    if (VEC) alive = wait_warp(&full[stage], parity, ctl) && alive;
    if (m < last) {
      F2 x[kHeld][4], g[kHeld][4];
      F2 s1 = f2(0.0f, 0.0f), s2 = s1;
      const float2 st = VEC ? *reinterpret_cast<const float2*>(here + at.stats + team * 8) : __ldg(p.stats + m);
      const T* row_dy = reinterpret_cast<const T*>(here) + team * p.K;
      const uint8_t* row_z = here + at.z + team * p.K * (SRC ? 1 : sizeof(T));
      const uint8_t* row_s = here + at.scales + team * scale_row +
                             ((static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p.scales)) +
                               static_cast<uint32_t>(block) * static_cast<uint32_t>(scale_row)) & 3);
      const float rstd = st.y;
      // chunk i: dy, xh and the multipliers
      auto read = [&](int i, F2(&d)[4], F2(&xh)[4], F2(&w)[4]) {
        float scale = 1.0f;  // of a checkpoint's group
        if (VEC) {
          const int c0 = col[i];
          load8_pairs(row_dy + c0, d);
          if (SRC) {
            ckpt_codes8_pairs<kFmt>(*reinterpret_cast<const uint2*>(row_z + c0), xh);
            scale = ckpt_scale(row_s[static_cast<uint32_t>(c0) / kCkptGroup]);
          } else {
            load8_pairs(reinterpret_cast<const T*>(row_z) + c0, xh);
          }
          load8_pairs(mul + mcol[i], w);
        } else {
          float a[8], b[8], c[8];
          load_chunk<T, false>(static_cast<const T*>(p.dY) + m * p.ld_dy, p.K, i, t, threads, 0.0f, a);
          if (SRC == 0)
            load_chunk<T, false>(static_cast<const T*>(p.Z) + m * p.ld_z, p.K, i, t, threads, st.x, b);
          else
            ckpt_load_chunk<kFmt, false>(p.codes + static_cast<size_t>(m) * p.K,
                                         p.scales + static_cast<size_t>(m) * scale_row, p.K, i, t, threads, b, st.x);
          load_chunk<float, false>(mul, p.K, i, t, threads, 0.0f, c);  // columns beyond K: z = mu and g = 0
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            d[j] = f2(a[2 * j], a[2 * j + 1]);
            xh[j] = f2(b[2 * j], b[2 * j + 1]);
            w[j] = f2(c[2 * j], c[2 * j + 1]);
          }
        }
        // (z - mu) rstd as the forward has it, not z rstd - mu rstd: that would round at the size of mu rstd.
        // A checkpoint's code times its scale, a power of two, is exact.
        const F2 off = f2(-st.x, -st.x), by = f2(scale, scale), rs = f2(rstd, rstd);
#pragma unroll
        for (int j = 0; j < 4; ++j) xh[j] = mul2(VEC && SRC ? fma2(xh[j], by, off) : add2(xh[j], off), rs);
      };
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        F2(&xh)[4] = x[kHeld == NV ? i : 0];
        F2(&gi)[4] = g[kHeld == NV ? i : 0];
        F2 w[4];
        read(i, gi, xh, w);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          da[i][j] = fma2(gi[j], xh[j], da[i][j]);
          dc[i][j] = add2(dc[i][j], gi[j]);
          gi[j] = mul2(gi[j], w[j]);
          s1 = add2(s1, gi[j]);
          s2 = fma2(gi[j], xh[j], s2);
        }
      }
      float a1, b1, a2, b2;
      unpack2(s1, a1, b1);
      unpack2(s2, a2, b2);
      if (VEC && kHeld == NV) {  // the row is in registers
        __syncwarp();
        if (lane == 0 && alive) mbar_arrive(&empty[stage]);
      }
      int aborted = VEC && !alive;  // or any other warp of the team
      const float2 s = team_sum2(a1 + b1, a2 + b2, p.warps, team, red[team], turn, VEC ? &s_abort : nullptr, &aborted);
      const F2 m1 = f2(-s.x * inv_k, -s.x * inv_k), m2 = f2(-s.y * inv_k, -s.y * inv_k), rs = f2(rstd, rstd);
      T* dz = static_cast<T*>(p.dZ) + m * p.ld_dz;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        F2(&xh)[4] = x[kHeld == NV ? i : 0];
        F2(&gi)[4] = g[kHeld == NV ? i : 0];
        if (kHeld != NV) {
          F2 w[4];
          read(i, gi, xh, w);
#pragma unroll
          for (int j = 0; j < 4; ++j) gi[j] = mul2(gi[j], w[j]);
        }
        float v[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) unpack2(mul2(rs, fma2(xh[j], m2, add2(gi[j], m1))), v[2 * j], v[2 * j + 1]);
        if (!aborted) store_chunk<T, VEC>(dz, p.K, i, t, threads, v);
      }
      if (VEC && kHeld != NV) {
        __syncwarp();
        if (lane == 0 && alive) mbar_arrive(&empty[stage]);
      }
    } else if (VEC && lane == 0 && alive) {
      mbar_arrive(&empty[stage]);
    }
    if (++stage == p.stages) stage = 0, parity ^= 1;
  }
  float fa[NV][8], fc[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      unpack2(da[i][j], fa[i][2 * j], fa[i][2 * j + 1]);
      unpack2(dc[i][j], fc[i][2 * j], fc[i][2 * j + 1]);
    }
  grid_dep_launch_dependents();  // the joining kernel may be put in place
  float* out_a = p.partial ? p.partial + static_cast<size_t>(blockIdx.x) * 2 * p.K
                           : p.dscale ? p.dscale + static_cast<size_t>(group) * p.K : nullptr;
  float* out_c = p.partial ? out_a + p.K : p.dshift ? p.dshift + static_cast<size_t>(group) * p.K : nullptr;
  if (VEC && *static_cast<volatile int*>(&s_abort)) out_a = out_c = nullptr;
  if (teams > 1) {  // the teams' sums side by side, then added in order
    float* sums = smem;  // [teams][2][K]
    workers_barrier(workers);  // the multipliers and the ring are done with
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      store_chunk<float, VEC>(sums + team * 2 * p.K, p.K, i, t, threads, fa[i]);
      store_chunk<float, VEC>(sums + (team * 2 + 1) * p.K, p.K, i, t, threads, fc[i]);
    }
    workers_barrier(workers);
    constexpr int kWide = VEC ? 4 : 1;
    for (int c = threadIdx.x * kWide; c < 2 * p.K; c += workers * kWide) {
      float s[kWide];
#pragma unroll
      for (int j = 0; j < kWide; ++j) s[j] = sums[c + j];
      for (int r = 1; r < teams; ++r)
#pragma unroll
        for (int j = 0; j < kWide; ++j) s[j] += sums[r * 2 * p.K + c + j];
      float* out = c < p.K ? out_a + c : out_c + (c - p.K);
      if (c < p.K ? out_a : out_c)
#pragma unroll
        for (int j = 0; j < kWide; ++j) out[j] = s[j];
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (out_a) store_chunk<float, VEC>(out_a, p.K, i, t, threads, fa[i]);
      if (out_c) store_chunk<float, VEC>(out_c, p.K, i, t, threads, fc[i]);
    }
  }
}

// dscale and dshift from the partial sums: 32 columns per CTA, its warps share the splits out.
// Launched while the first kernel still runs; the wait is for its results.
__global__ void __launch_bounds__(1024) layer_norm_sum_kernel(const float* partial, int splits, int K, float* dscale,
                                                           float* dshift) {
  __shared__ float part[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int c = blockIdx.x * 32 + lane, group = blockIdx.y, which = blockIdx.z;
  float* out = which ? dshift : dscale;
  grid_dep_wait();
  if (!out) return;
  const size_t pitch = static_cast<size_t>(2) * K;
  const float* from = partial + static_cast<size_t>(group) * splits * pitch + static_cast<size_t>(which) * K + c;
  float s = 0.0f;
  if (c < K) {
    for (int i = warp; i < splits; i += 5 * warps) {  // five loads in flight
      float v[5];
#pragma unroll
      for (int j = 0; j < 5; ++j) v[j] = i + j * warps < splits ? ld_after_wait(from + (i + j * warps) * pitch) : 0.0f;
#pragma unroll
      for (int j = 0; j < 5; ++j) s += v[j];
    }
  }
  part[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < K) {
    for (int i = 1; i < warps; ++i) s += part[i][lane];
    out[static_cast<size_t>(group) * K + c] = s;
  }
}

constexpr int kMaxSmem = 220 * 1024;

struct Shape {
  int nv, warps, teams;
};

// Forward: one warp a row while 5 chunks of 8 values a thread reach (no barriers), else the chunk count that
// wastes the fewest threads; when they tie the smaller one for 16-bit rows (more warps: 4608 x 12288 bf16
// 108 -> 72 us then) and the larger one for fp32 (8192 x 4096: 53 against 65 us).  A ring of rows as the backward
// has it was slower (8192 x 4096 bf16 63 against 46 us).
Shape forward_shape(int K, bool narrow) {
  const int nvec = (K + 7) / 8;
  Shape s{};
  if (nvec <= 160) {
    s.warps = 1;
    s.nv = (nvec + 31) / 32;
  } else {
    int best = 1 << 30;
    for (int i = 0; i < 3; ++i) {
      const int nv = narrow ? 2 + i : 4 - i, warps = (nvec + 32 * nv - 1) / (32 * nv);
      if (warps <= 16 && warps * nv < best) best = warps * nv, s.nv = nv, s.warps = warps;
    }
  }
  s.teams = s.warps >= kForwardWarps ? 1 : kForwardWarps / s.warps;
  return s;
}

// Backward: 16 sums a chunk stay in registers over all rows and 16 more values across a row's reduction:
// two chunks a thread while 16 warps reach, then three or four.
Shape backward_shape(int K, int rows) {
  const int nvec = (K + 7) / 8;
  Shape s{};
  s.nv = nvec <= 32 ? 1 : nvec <= 1024 ? 2 : nvec <= 1536 ? 3 : 4;
  s.warps = (nvec + 32 * s.nv - 1) / (32 * s.nv);
  s.teams = s.warps >= kBackwardWarps ? 1 : kBackwardWarps / s.warps;
  if (s.teams > rows) s.teams = rows;  // smaller CTAs, more of them per SM, for groups of a few rows
  return s;
}

// CTAs that share a group's rows: one per SM over all groups, four rows a team at least.
int backward_splits(int K, int rows, int groups) {
  const Shape s = backward_shape(K, rows);
  const int want = (kSMs + groups - 1) / groups;
  const int most = (rows + 4 * s.teams - 1) / (4 * s.teams);
  return want < most ? want : most;
}

template <typename T, typename P, int NV, bool VEC>
svdq_status run_forward(const FwdParams& p, const Shape& s, cudaStream_t stream) {
  const int blocks = (p.M + s.teams - 1) / s.teams;
  layer_norm_kernel<T, P, NV, VEC><<<blocks, s.teams * s.warps * 32, 0, stream>>>(p);
  SVDQ_CUDA_TRY(cudaGetLastError());
  return SVDQ_OK;
}

template <typename T, typename P, bool VEC>
svdq_status forward_nv(const FwdParams& p, const Shape& s, cudaStream_t stream) {
  switch (s.nv) {
    case 1: return run_forward<T, P, 1, VEC>(p, s, stream);
    case 2: return run_forward<T, P, 2, VEC>(p, s, stream);
    case 3: return run_forward<T, P, 3, VEC>(p, s, stream);
    case 4: return run_forward<T, P, 4, VEC>(p, s, stream);
    default: return run_forward<T, P, 5, VEC>(p, s, stream);
  }
}

// The parameters' type is compiled in where it is the rows' own or fp32.
template <typename T>
svdq_status forward_type(const FwdParams& p, const Shape& s, bool vec, int dtype, cudaStream_t stream) {
  if (!vec) return forward_nv<T, void, false>(p, s, stream);
  if (p.param_dtype == SVDQ_DTYPE_FP32) return forward_nv<T, float, true>(p, s, stream);
  if (p.param_dtype == dtype) return forward_nv<T, T, true>(p, s, stream);
  return forward_nv<T, void, true>(p, s, stream);
}

template <typename T, int NV, bool VEC, int SRC>
svdq_status run_backward(BwdParams p, const Shape& s, int groups, cudaStream_t stream) {
  const size_t mul = mul_floats(p.K) * sizeof(float);
  const size_t sums = s.teams > 1 ? static_cast<size_t>(s.teams) * p.K * 8 : 0;  // 16 KB a warp at most
  const size_t stage = Stage<T, SRC>(p.K, s.teams).bytes;
  size_t smem = mul;
  if (VEC) {  // up to four rows in flight per team
    p.packed = p.ld_dy == p.K && (SRC || p.ld_z == p.K);
    p.stages = kMaxStages;
    while (p.stages > 1 && mul + p.stages * stage > kMaxSmem) --p.stages;
    smem += p.stages * stage;
  }
  if (smem < sums) smem = sums;
  p.err = device_error_word();
  if (!p.err) return fail(SVDQ_ERR_CUDA, "device error word unavailable");
  p.wait_ns = wait_limit_ns();
  auto* kernel = layer_norm_backward_kernel<T, NV, VEC, SRC>;
  static std::atomic<uint64_t> allowed{0};
  SVDQ_TRY(allow_dynamic_smem(reinterpret_cast<const void*>(kernel), kMaxSmem, allowed));
  kernel<<<groups * p.splits, (s.teams * s.warps + (VEC ? 1 : 0)) * 32, smem, stream>>>(p);
  SVDQ_CUDA_TRY(cudaGetLastError());
  return SVDQ_OK;
}

template <typename T, bool VEC, int SRC>
svdq_status backward_nv(const BwdParams& p, const Shape& s, int groups, cudaStream_t stream) {
  switch (s.nv) {
    case 1: return run_backward<T, 1, VEC, SRC>(p, s, groups, stream);
    case 2: return run_backward<T, 2, VEC, SRC>(p, s, groups, stream);
    case 3: return run_backward<T, 3, VEC, SRC>(p, s, groups, stream);
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
              a.M, a.K, a.rows, a.param_dtype, 0, codes ? ckpt : -1, 0, a.eps, a.plus_one ? 1.0f : 0.0f};
  const Shape s = forward_shape(a.K, a.dtype != SVDQ_DTYPE_FP32);
  p.warps = s.warps;
  // 8 warps' rows per SM ahead, a quarter of those at work: 4608 x 12288 bf16 71.5 -> 67 us, 8192 x 4096 46 -> 43
  // (half and all of them the same, twice as many slower); no gain for a row per warp or in fp32.
  if (s.warps > 1 && a.dtype != SVDQ_DTYPE_FP32) p.ahead = (kSMs * 8 + s.warps - 1) / s.warps;
  const bool vec = vector_rows(a.K, {Z, scale, shift, Y, codes}, {a.ld_z, a.ld_y, a.ld_param});
  switch (a.dtype) {
    case SVDQ_DTYPE_BF16: return forward_type<__nv_bfloat16>(p, s, vec, a.dtype, stream);
    case SVDQ_DTYPE_FP16: return forward_type<__half>(p, s, vec, a.dtype, stream);
    default: return forward_type<float>(p, s, vec, a.dtype, stream);
  }
}

svdq_status launch_layer_norm_backward(const NormArgs& a, const void* dY, const void* Z, const uint8_t* codes,
                                       const uint8_t* scales, int ckpt, const float* stats, const void* scale,
                                       void* dZ, float* dscale, float* dshift, void* workspace, cudaStream_t stream) {
  const int groups = (a.M + a.rows - 1) / a.rows;
  const Shape s = backward_shape(a.K, a.rows);
  BwdParams p{dY, Z, codes, scales, reinterpret_cast<const float2*>(stats), scale, dZ, dscale, dshift, nullptr,
              a.ld_z, a.ld_dy, a.ld_dz, a.ld_param, a.M, a.K, a.rows, backward_splits(a.K, a.rows, groups),
              a.param_dtype, s.warps, s.teams, 0, 0, a.plus_one ? 1.0f : 0.0f, nullptr, 0, a.stall};
  if (p.splits > 1 && (dscale || dshift)) p.partial = static_cast<float*>(workspace);
  const bool vec = vector_rows(a.K, {dY, Z, codes, scale, dZ, p.partial ? nullptr : dscale, p.partial ? nullptr : dshift},
                               {a.ld_z, a.ld_dy, a.ld_dz, a.ld_param}) &&
                   (!codes || a.K % 16 == 0);  // bulk copies of whole rows of codes
  if (a.stall && !vec) return fail(SVDQ_ERR_INVALID_ARG, "rows of this layout are read without a wait");
  const int src = !codes ? 0 : ckpt == SVDQ_CKPT8_INT8 ? 1 : 2;
  svdq_status st;
  switch (a.dtype) {
    case SVDQ_DTYPE_BF16: st = backward_type<__nv_bfloat16>(p, s, groups, vec, src, stream); break;
    case SVDQ_DTYPE_FP16: st = backward_type<__half>(p, s, groups, vec, src, stream); break;
    default: st = backward_type<float>(p, s, groups, vec, src, stream); break;
  }
  SVDQ_TRY(st);
  if (p.partial) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((a.K + 31) / 32, groups, 2);
    cfg.blockDim = dim3(32 * std::min(32, std::max(1, (p.splits + 4) / 5)));  // five splits a warp
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    SVDQ_CUDA_TRY(cudaLaunchKernelEx(&cfg, layer_norm_sum_kernel, static_cast<const float*>(p.partial), p.splits, a.K,
                                     dscale, dshift));
  }
  return SVDQ_OK;
}

}  // namespace svdq
