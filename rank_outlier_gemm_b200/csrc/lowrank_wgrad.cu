// Gradient of a low-rank factor: G[K, r] = X^T S over M tokens, X an activation (bf16, or its 8-bit
// checkpoint) and S [M, r] bf16.
//
// With y += (x A) B: dA = X^T (dY B^T) and dB^T = dY^T (X A), both this product.  X is the large
// operand (M K values against (M + K) r), so the kernel is bound by reading it once as long as the
// 2 M K r operations keep up; they run on the tensor cores (mma.sync m16n8k16, bf16 inputs, fp32
// sums), the columns of X as the M side.  The contraction runs over rows, so a thread takes the same
// columns of 4 rows and pairs the rows' values in registers: X is never transposed or stored again.
//
// A checkpoint's codes are exact in bf16, and so are its values, code times a power of two, from 2^-126 on.  The
// scales multiply the codes and not the fragments of S: S times a scale leaves bf16's range where the values do
// not, and a code of 0 times an infinity is NaN.  (On the fragments: int8 4608 x 12288 20.4, 29.7 and 55.6 us at
// r = 8, 32 and 64 against 20.2, 28.3 and 53.8 on the codes, E4M3 at r = 16 22.0 against 23.5.)
//
// Measured (one B200, device time in a graph): int8 4608 x 12288, r = 32: 28.0 us against 9.2 for one pass
// over the bytes, bf16 27.4 against 17.6.  About 8 us are fixed (first copies, joins, second kernel), 13 the
// decoding and products alone; the scale bytes, a sector each per row and 64 columns, cost 5.  bf16 4099 x 1152,
// r = 16: 7.0 us.  r = 64 and 128 take two and four passes (54 and 106 us from int8).
//
// A CTA holds its rows of S in shared memory; each warp copies its 16 x 64 tiles of X ahead through a
// ring of its own, so the main loop has no CTA barrier.  Sums are joined by ordinary fp32 additions in
// a fixed order: the CTA's row warps in shared memory, then the CTAs that share the rows by a second kernel
// over partial results.  (Clusters in its place left SMs idle: at one CTA of 16 warps per SM 45 clusters of 3
// or 15 of 8 are resident, not 49 or 18.)
#include <cuda_bf16.h>

#include <algorithm>

#include "ptx.cuh"
#include "rows.cuh"
#include "svdq_internal.h"

namespace svdq {
namespace {

using namespace dev;

constexpr int kSMs = 148;
constexpr int kTileCols = 64;          // of X per warp step, 16 rows (bf16) or 32
constexpr int kWarps = 16, kThreads = 32 * kWarps;
constexpr int kSBytes = 96 * 1024;    // of S in shared memory at a time
constexpr int kMaxY = 65535;          // of a grid's y
constexpr int kMaxRows = 512;         // of one warp between two joins

struct WgradParams {
  const uint8_t* X;       // bf16 [M, K], or the codes
  const uint8_t* scales;
  const uint16_t* S;      // bf16 [M, r]
  float* out;             // G, or the partial sums [parts][K][r]
  int M, K, r;
  int col_warps;          // 1, 2 or 4; the others of the 16 warps share out the rows
  int rows;               // per CTA, a multiple of a step's rows
  int parts, zs;          // of the rows, of the columns of S
};

__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// 16 bytes to shared memory, zeros if !in
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ uint32_t lds32(uint32_t at) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(at));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t at) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at));
  return v;
}
__device__ __forceinline__ uint32_t lds8(uint32_t at) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(at));
  return v;
}
// (v & mask) | bits; `bits` from a register, so that it is one instruction
__device__ __forceinline__ uint32_t mask_or(uint32_t v, uint32_t mask, uint32_t bits) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(v), "r"(mask), "r"(bits));
  return r;
}
__device__ __forceinline__ uint32_t opaque(uint32_t constant) {
  uint32_t r;
  asm volatile("mov.u32 %0, %1;" : "=r"(r) : "r"(constant));
  return r;
}
__device__ __forceinline__ uint32_t scale_pair(uint32_t values, uint32_t pow2) {
  const __nv_bfloat162 v = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&values),
                                   *reinterpret_cast<const __nv_bfloat162*>(&pow2));
  return *reinterpret_cast<const uint32_t*>(&v);
}

// A stage of a warp's ring: 16-byte pieces of 64 values of each row, placed so that the four rows a warp
// reads at a time fall into different banks, then 8 bytes per row around its two scale bytes.  A step
// of codes takes 32 rows, which halves what the copies and the scales cost a value.
template <int SRC>
struct Tile {
  static constexpr int rows = SRC ? 32 : 16, stages = SRC ? 3 : 4;
  static constexpr int piece_values = SRC ? 16 : 8;
  static constexpr int pieces = kTileCols / piece_values;  // per row
  static constexpr int scales = rows * pieces * 16;
  static constexpr int bytes = scales + (SRC ? rows * 8 : 0);
  __device__ static uint32_t at(int row, int piece) {
    return SRC ? (row >> 1) * 128 + ((((row & 1) << 2 | piece) ^ (((row >> 1) & 3) << 1)) << 4)
               : row * 128 + ((piece ^ (((row >> 1) & 1) << 2)) << 4);
  }
};

// Where piece `j` (8 columns) of row `row` of S lies: NT pieces a row, spread over the banks.
template <int NT>
__device__ __forceinline__ uint32_t s_place(int row, int j) {
  return (row * NT + (j ^ ((row / (8 / NT)) & (NT - 1)))) * 16;
}

// Pairs over two rows of four columns of a tile: the words at `a` (one row) and `b` (the next).
template <int SRC>
__device__ __forceinline__ void pair_rows(uint32_t at_a, uint32_t at_b, uint32_t bf16_128, uint32_t (&w)[4]) {
  if (SRC == 0) {
    const uint2 a = lds64(at_a), b = lds64(at_b);
    w[0] = __byte_perm(a.x, b.x, 0x5410), w[1] = __byte_perm(a.x, b.x, 0x7632);
    w[2] = __byte_perm(a.y, b.y, 0x5410), w[3] = __byte_perm(a.y, b.y, 0x7632);
  } else if (SRC == 1) {
    // q = u7 - 128 s in two's complement; bf16 has 7 mantissa bits: (128 + u7) - (128 + 128 s), exact, both rows
    // at once
    const uint32_t a = lds32(at_a), b = lds32(at_b);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t v = __byte_perm(a, b, 0x4400 + 0x1111 * j);  // bytes j of a, -, j of b, -
      const uint32_t u = mask_or(v, 0x007F007Fu, bf16_128), c = mask_or(v, 0x00800080u, bf16_128);
      const __nv_bfloat162 h = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&u), *reinterpret_cast<const __nv_bfloat162*>(&c));
      w[j] = *reinterpret_cast<const uint32_t*>(&h);
    }
  } else {
    float x[4], y[4];
    ckpt_values4<SVDQ_CKPT8_E4M3>(lds32(at_a), 1.0f, x);
    ckpt_values4<SVDQ_CKPT8_E4M3>(lds32(at_b), 1.0f, y);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x[j], y[j]);
      w[j] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
}

// NT: columns of S per CTA in tiles of 8.  blockIdx: x columns of X, y part of the rows, z columns of S (and once
// more for each kMaxY parts that tall X have).
template <int SRC, int NT>
__global__ void __launch_bounds__(kThreads, 1) wgrad_kernel(WgradParams p) {
  extern __shared__ __align__(128) uint8_t smem[];  // S, then the rings; at the end the warps' sums
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int cw = warp % p.col_warps, rw = warp / p.col_warps, row_warps = kWarps / p.col_warps;
  int part = blockIdx.y, z = blockIdx.z;
  while (z >= p.zs) z -= p.zs, part += kMaxY;  // seldom: no division
  if (part >= p.parts) return;
  const int k0 = (blockIdx.x * p.col_warps + cw) * kTileCols;
  const int n0 = z * NT * 8;
  const int row0 = part * p.rows, row_end = min(p.M, row0 + p.rows);
  const int groups = (p.K + kCkptGroup - 1) / kCkptGroup;
  const uint32_t s_tile = smem_u32(smem);
  const uint32_t ring = s_tile + kSBytes + warp * Tile<SRC>::stages * Tile<SRC>::bytes;
  const int block_rows = row_warps * Tile<SRC>::rows;                      // of one step of the CTA
  const int s_steps = kSBytes / (NT * 16) / block_rows;              // steps whose rows of S fit

  float acc[4][NT][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j][0] = acc[i][j][1] = acc[i][j][2] = acc[i][j][3] = 0.0f;

  // this lane's part of the warp's next tile: 16-byte pieces of rows `fetch_row`, + 8 or + 4, ...
  using Tl = Tile<SRC>;
  constexpr int kTileRows = Tl::rows, kStages = Tl::stages;
  constexpr int kRowsAtOnce = 32 / Tl::pieces;
  const int piece = lane % Tl::pieces, piece_k = k0 + piece * Tl::piece_values, fetch_row = lane / Tl::pieces;
  const size_t row_bytes = static_cast<size_t>(p.K) * (SRC ? 1 : 2), row_jump = kRowsAtOnce * row_bytes,
               block_bytes = block_rows * row_bytes;
  const uint8_t* next_x = p.X + (row0 + rw * kTileRows + fetch_row) * row_bytes + static_cast<size_t>(piece_k) * (SRC ? 1 : 2);
  const uint8_t* next_s = SRC ? p.scales + static_cast<size_t>(row0 + rw * kTileRows + lane) * groups + k0 / kCkptGroup
                              : nullptr;
  const uint8_t* scales_end = SRC ? p.scales + static_cast<size_t>(p.M) * groups : nullptr;
  const uint32_t fetch_at = Tl::at(fetch_row, piece);  // kRowsAtOnce rows on: 512 bytes on
  int fetch_left = piece_k < p.K ? row_end - row0 - rw * kTileRows : 0;  // rows from the tile's first to the end
  int scale_left = k0 < p.K ? row_end - row0 - rw * kTileRows - lane : 0;
  // the rows whose aligned words (3 bytes before their first scale to 8 behind) lie inside the array
  int scale_row = row0 + rw * kTileRows + lane;
  const int scale_first = (3 + groups - 1) / groups, scale_last = p.M - (8 + k0 / kCkptGroup + groups - 1) / groups;
  auto fetch = [&](int stage) {
    const uint32_t to = ring + stage * Tl::bytes, at = to + fetch_at;
    if (fetch_left >= kTileRows) {
      const uint8_t* from = next_x;
#pragma unroll
      for (int i = 0; i < kTileRows / kRowsAtOnce; ++i, from += row_jump)
        copy16(at + i * 512, from, true);
    } else {
#pragma unroll
      for (int i = 0; i < kTileRows / kRowsAtOnce; ++i) {
        const bool in = i * kRowsAtOnce + fetch_row < fetch_left;
        copy16(at + i * 512, in ? next_x + i * row_jump : p.X, in);
      }
    }
    if (SRC && scale_left > 0) {  // the aligned words around a row's scale bytes
      const uint32_t skip = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(next_s)) & 3;
      const uint8_t* word = next_s - skip;
      uint8_t* here = smem + (to + Tl::scales + lane * 8 - s_tile);
      if (scale_row >= scale_first && scale_row < scale_last) {
        copy4_async(here, word);
        if (skip == 3) copy4_async(here + 4, word + 4);  // each costs a sector of its own
      } else {  // words that may reach over the array's ends
        for (int b = 0; b < 8; ++b)
          if (word + b >= p.scales && word + b < scales_end) here[b] = word[b];
      }
    }
    next_x += block_bytes;
    fetch_left -= block_rows;
    if (SRC) next_s += static_cast<size_t>(block_rows) * groups, scale_left -= block_rows, scale_row += block_rows;
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  // where this lane finds rows 2 t (and, by other bits of the address, 2 t + 1, + 8, the second 32 columns)
  const uint32_t x_at = SRC ? t * 128 + (((g >> 2) ^ (t << 1)) << 4) + (g & 3) * 4
                            : t * 256 + (((g >> 1) ^ ((t & 1) << 2)) << 4) + (g & 1) * 8;
  // the scale bytes of row `lane` of a tile
  const uint32_t my_byte0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p.scales)) + k0 / kCkptGroup;
  const bool second = k0 + 32 < p.K;  // the columns' second group exists
  const uint32_t bf16_128 = opaque(0x43004300u);  // two bf16 of 128
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) fetch(i);

  int stage = 0;
  for (int row = row0; row < row_end; row += s_steps * block_rows) {
    const int n_rows = min(s_steps * block_rows, row_end - row);
    const int n_steps = (n_rows + block_rows - 1) / block_rows;
    __syncthreads();  // the rows of S before these are done with
    constexpr int kAtOnce = kThreads / NT;  // rows; a multiple of the placement's period
    const int j = threadIdx.x % NT, n = n0 + j * 8;
    const uint16_t* from = p.S + static_cast<size_t>(row + threadIdx.x / NT) * p.r + n;
    uint32_t to = s_tile + s_place<NT>(threadIdx.x / NT, j);
    for (int m = threadIdx.x / NT; m < n_steps * block_rows; m += kAtOnce, from += kAtOnce * p.r, to += kAtOnce * NT * 16) {
      const bool in = m < n_rows && n < p.r;
      if (p.r % 8 == 0) {
        copy16(to, in ? from : p.S, in);
      } else {
        uint16_t* v = reinterpret_cast<uint16_t*>(smem + (to - s_tile));
        for (int e = 0; e < 8; ++e) v[e] = in && n + e < p.r ? from[e] : 0;
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();

    for (int step = 0; step < n_steps; ++step) {
      __syncwarp();
      fetch(stage ? stage - 1 : kStages - 1);  // the stage that every lane read last
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
      __syncwarp();
      const uint32_t tile = ring + stage * Tile<SRC>::bytes;
      const int local = step * block_rows + rw * kTileRows, m0 = row + local;
      if (++stage == kStages) stage = 0;
      if (m0 >= row_end) continue;  // the warp's last tiles; k0 >= K reads what no one reads back

      // 2^(byte - 127) as bf16 of rows (lane, lane + 1), for both groups; rows beyond M: 0
      uint32_t pow2[2] = {0, 0};
      if (SRC) {
        const int m = m0 + lane;
        const uint32_t at = tile + Tl::scales + lane * 8 +
                            ((my_byte0 + static_cast<uint32_t>(m) * static_cast<uint32_t>(groups)) & 3);
        const uint32_t first = lds8(at), other = lds8(at + 1);
        uint32_t both = (first ? first << 7 : 0x40u) | (other ? other << 7 : 0x40u) << 16;
        if (!second) both &= 0xFFFFu;
        if (m >= row_end) both = 0;
        const uint32_t next = __shfl_down_sync(0xffffffffu, both, 1);
        pow2[0] = __byte_perm(both, next, 0x5410);
        pow2[1] = __byte_perm(both, next, 0x7632);
      }
#pragma unroll
      for (int sub = 0; sub < kTileRows / 16; ++sub) {
        uint32_t b[NT][2];
        const uint32_t s_at = s_tile + (local + 16 * sub) * NT * 16 + s_place<NT>(lane & 15, NT == 1 ? 0 : lane >> 4);
        if (NT == 1) {
          asm volatile("ldmatrix.sync.aligned.m8n8.x2.trans.shared.b16 {%0, %1}, [%2];"
                       : "=r"(b[0][0]), "=r"(b[0][1])
                       : "r"(s_at));
        } else {
#pragma unroll
          for (int j = 0; j + 1 < NT; j += 2)
            asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                         : "=r"(b[j][0]), "=r"(b[j][1]), "=r"(b[j + 1][0]), "=r"(b[j + 1][1])
                         : "r"(s_at ^ (j * 16)));
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {  // the two scale groups: columns 32 half + 4 g..4 g + 3
          uint32_t lo[4], hi[4];
          const uint32_t at = (tile + x_at) ^ (SRC ? 32 * half : 64 * half);
          constexpr uint32_t kNext = SRC ? 0 : 128, kEight = SRC ? 512 : 1024;
          const uint32_t odd = SRC ? at ^ 64 : at;
          pair_rows<SRC>(at + 2 * sub * kEight, odd + kNext + 2 * sub * kEight, bf16_128, lo);
          pair_rows<SRC>(at + (2 * sub + 1) * kEight, odd + kNext + (2 * sub + 1) * kEight, bf16_128, hi);
          if (SRC) {  // the pairs are two rows, as the scales are
            const uint32_t p0 = __shfl_sync(0xffffffffu, pow2[half], 16 * sub + 2 * t);
            const uint32_t p1 = __shfl_sync(0xffffffffu, pow2[half], 16 * sub + 8 + 2 * t);
#pragma unroll
            for (int j = 0; j < 4; ++j) lo[j] = scale_pair(lo[j], p0), hi[j] = scale_pair(hi[j], p1);
          }
#pragma unroll
          for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint32_t a[4] = {lo[2 * i], lo[2 * i + 1], hi[2 * i], hi[2 * i + 1]};
              mma_bf16(acc[2 * half + i][j], a, b[j][0], b[j][1]);
            }
        }
      }
    }
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  grid_dep_launch_dependents();

  // the row warps' sums: [row warps][columns of X][kPitch]; the pitch spreads a warp's stores over the banks
  constexpr int kPitch = NT * 8 + 2;
  const int cols = p.col_warps * kTileCols;
  float* sums = reinterpret_cast<float*>(smem);
  float* out = p.out + static_cast<size_t>(part) * p.K * p.r;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int col = cw * kTileCols + (i >> 1) * 32 + 4 * g + 2 * (i & 1) + h;
        *reinterpret_cast<float2*>(sums + (rw * cols + col) * kPitch + j * 8 + 2 * t) =
            make_float2(acc[i][j][2 * h], acc[i][j][2 * h + 1]);
      }
  __syncthreads();
  for (int i = threadIdx.x; i < cols * NT * 8; i += kThreads) {
    const int col = i / (NT * 8), n = i % (NT * 8);
    const float* s = sums + col * kPitch + n;
    float v = s[0];
#pragma unroll 4
    for (int w = 1; w < row_warps; ++w) v += s[w * cols * kPitch];
    const int k = blockIdx.x * cols + col;
    if (k < p.K && n0 + n < p.r) out[static_cast<size_t>(k) * p.r + n0 + n] = v;
  }
}

__global__ void __launch_bounds__(256) wgrad_sum_kernel(const float* partial, int parts, size_t n, float* G) {
  const size_t i = static_cast<size_t>(blockIdx.x) * 256 + threadIdx.x;
  grid_dep_wait();
  if (i >= n) return;
  float s = 0.0f;
  for (int j = 0; j < parts; j += 8) {  // eight loads in flight
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = j + e < parts ? ld_after_wait(partial + (j + e) * n + i) : 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) s += v[e];
  }
  G[i] = s;
}

struct Plan {
  int nt, col_warps, blocks, zs, parts, rows;
};

// One CTA of 16 warps per SM.  The column warps are as many as leave 18 column blocks, which 8 CTAs along the
// rows make the whole device; the rows are split into as many parts as the device has room for, but no
// warp sums more than kMaxRows into one accumulator.
Plan plan(int M, int K, int r, int tile_rows) {
  Plan q{};
  const int tiles = (r + 7) / 8;
  q.nt = tiles <= 1 ? 1 : tiles <= 2 ? 2 : 4;  // 8 would spill: at r = 64 102 us against 54 for two passes (4608 x 12288, int8)
  q.zs = (tiles + q.nt - 1) / q.nt;
  q.col_warps = K >= 17 * 256 + 1 ? 4 : K >= 17 * 128 + 1 ? 2 : 1;
  q.blocks = (K + q.col_warps * kTileCols - 1) / (q.col_warps * kTileCols);
  const int block_rows = kWarps / q.col_warps * tile_rows, max_steps = kMaxRows / tile_rows;
  const int steps = (M + block_rows - 1) / block_rows;
  const int parts = std::max({1, std::min(kSMs / (q.blocks * q.zs), steps), (steps + max_steps - 1) / max_steps});
  const int per_cta = (steps + parts - 1) / parts;
  q.parts = (steps + per_cta - 1) / per_cta;
  q.rows = per_cta * block_rows;
  return q;
}

template <int SRC, int NT>
svdq_status launch(const WgradParams& p, const Plan& q, cudaStream_t stream) {
  const size_t loop = kSBytes + static_cast<size_t>(kWarps) * Tile<SRC>::stages * Tile<SRC>::bytes;
  const size_t join = static_cast<size_t>(kWarps) * kTileCols * (NT * 8 + 2) * sizeof(float);
  const size_t smem = std::max(loop, join);
  static std::atomic<uint64_t> allowed{0};
  SVDQ_TRY(allow_dynamic_smem(reinterpret_cast<const void*>(wgrad_kernel<SRC, NT>), static_cast<int>(smem), allowed));
  wgrad_kernel<SRC, NT><<<dim3(q.blocks, std::min(q.parts, kMaxY), q.zs * ((q.parts + kMaxY - 1) / kMaxY)), kThreads, smem, stream>>>(p);
  SVDQ_CUDA_TRY(cudaGetLastError());
  return SVDQ_OK;
}

template <int SRC>
svdq_status launch_nt(const WgradParams& p, const Plan& q, cudaStream_t stream) {
  switch (q.nt) {
    case 1: return launch<SRC, 1>(p, q, stream);
    case 2: return launch<SRC, 2>(p, q, stream);
    default: return launch<SRC, 4>(p, q, stream);
  }
}

}  // namespace

size_t lowrank_wgrad_workspace(int M, int K, int r) {
  const int parts = std::max(plan(M, K, r, Tile<0>::rows).parts, plan(M, K, r, Tile<1>::rows).parts);
  return parts > 1 ? static_cast<size_t>(parts) * K * r * sizeof(float) : 0;
}

svdq_status launch_lowrank_wgrad(const void* X, const uint8_t* scales, int src, const void* S, int M, int K, int r,
                                 float* G, void* workspace, cudaStream_t stream) {
  const Plan q = plan(M, K, r, src ? Tile<1>::rows : Tile<0>::rows);
  WgradParams p{static_cast<const uint8_t*>(X), scales, static_cast<const uint16_t*>(S),
                q.parts > 1 ? static_cast<float*>(workspace) : G, M, K, r, q.col_warps, q.rows, q.parts, q.zs};
  SVDQ_TRY(src == 0 ? launch_nt<0>(p, q, stream) : src == 1 ? launch_nt<1>(p, q, stream) : launch_nt<2>(p, q, stream));
  if (q.parts > 1) {
    const size_t n = static_cast<size_t>(K) * r;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>((n + 255) / 256));
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    SVDQ_CUDA_TRY(cudaLaunchKernelEx(&cfg, wgrad_sum_kernel, static_cast<const float*>(p.out), q.parts, n, G));
  }
  return SVDQ_OK;
}

}  // namespace svdq
