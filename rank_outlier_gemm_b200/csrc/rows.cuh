// Row operands of the layer norm and checkpoint kernels: eight values at a time as fp32, and the
// 8-bit checkpoint codec.
//
// A team of `threads` (a multiple of 32) threads covers a row of K columns in chunks of 8: thread t owns
// columns 8 (i threads + t) + j, j < 8.  Where K, the row strides and the addresses allow it (VEC) a
// chunk is one 16-byte access (two for fp32); else each row takes the widest accesses that its own
// address allows (16, 4 or an element's bytes), and the chunk that K cuts takes its elements one by one.
// A checkpoint group (32 consecutive columns) is 4 neighbouring threads' chunks, so its largest
// magnitude is two shuffles away.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>
#include <string.h>

#include "svdq.h"

namespace svdq {
namespace dev {

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// One bf16 pair as fp32 (a bf16 is the top half of an fp32).
__device__ __forceinline__ float pair_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float pair_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Eight consecutive values (16-byte aligned for 16-bit types, two aligned halves for fp32).
__device__ __forceinline__ void unpack8(const uint4& a, float (&v)[8], const __nv_bfloat16*) {
  v[0] = pair_lo(a.x), v[1] = pair_hi(a.x), v[2] = pair_lo(a.y), v[3] = pair_hi(a.y);
  v[4] = pair_lo(a.z), v[5] = pair_hi(a.z), v[6] = pair_lo(a.w), v[7] = pair_hi(a.w);
}
__device__ __forceinline__ void unpack8(const uint4& a, float (&v)[8], const __half*) {
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
    v[2 * j] = f.x, v[2 * j + 1] = f.y;
  }
}
__device__ __forceinline__ void unpack8(const uint4&, float (&)[8], const float*) {}  // no 16-bit words
template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&v)[8]) {
  unpack8(*reinterpret_cast<const uint4*>(p), v, p);
}
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
  uint4 a;
  uint32_t* w = &a.x;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
    w[j] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = a;
}
__device__ __forceinline__ void store8(__half* p, const float (&v)[8]) {
  uint4 a;
  uint32_t* w = &a.x;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const __half2 h = __floats2half2_rn(v[2 * j], v[2 * j + 1]);
    w[j] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = a;
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}

// Two fp32 side by side.  (The packed add, mul and fma .f32x2 gained nothing here: what they save in issue
// slots goes into moves between pairs.)
struct F2 {
  float x, y;
};
__device__ __forceinline__ F2 f2(float a, float b) { return F2{a, b}; }
__device__ __forceinline__ void unpack2(F2 a, float& x, float& y) { x = a.x, y = a.y; }
__device__ __forceinline__ F2 add2(F2 a, F2 b) { return F2{__fadd_rn(a.x, b.x), __fadd_rn(a.y, b.y)}; }
__device__ __forceinline__ F2 mul2(F2 a, F2 b) { return F2{__fmul_rn(a.x, b.x), __fmul_rn(a.y, b.y)}; }
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) { return F2{__fmaf_rn(a.x, b.x, c.x), __fmaf_rn(a.y, b.y, c.y)}; }

// Eight values in shared or global memory as four pairs.
template <typename T>
__device__ __forceinline__ void load8_pairs(const T* p, F2 (&v)[4]) {
  float f[8];
  load8(p, f);
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = f2(f[2 * j], f[2 * j + 1]);
}

// The first column of chunk i of thread t.
__device__ __forceinline__ int chunk_column(int i, int t, int threads) { return (i * threads + t) * 8; }

// The first n of 8 values at any address that is aligned to its elements; `fill` for the others.
template <typename T>
__device__ __forceinline__ void load_any(const T* p, int n, float fill, float (&v)[8]) {
  const uint32_t low = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p));
  if (n == 8 && low % 16 == 0) {
    load8(p, v);
  } else if (n == 8 && sizeof(T) == 2 && low % 4 == 0) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(p);
    unpack8(make_uint4(w[0], w[1], w[2], w[3]), v, p);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = j < n ? to_f32(p[j]) : fill;
  }
}
template <typename T>
__device__ __forceinline__ void store_any(T* p, int n, const float (&v)[8]) {
  const uint32_t low = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p));
  if (n == 8 && low % 16 == 0) {
    store8(p, v);
  } else if (n == 8 && sizeof(T) == 2 && low % 4 == 0) {
    T h[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) h[j] = from_f32<T>(v[j]);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint16_t a, b;
      memcpy(&a, &h[2 * j], 2);
      memcpy(&b, &h[2 * j + 1], 2);
      reinterpret_cast<uint32_t*>(p)[j] = a | static_cast<uint32_t>(b) << 16;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) p[j] = from_f32<T>(v[j]);
  }
}

// Chunk i of a row: columns beyond K give `fill`.
template <typename T, bool VEC>
__device__ __forceinline__ void load_chunk(const T* row, int K, int i, int t, int threads, float fill, float (&v)[8]) {
  const int c = chunk_column(i, t, threads);
  if (c < K) {
    if (VEC)
      load8(row + c, v);
    else
      load_any(row + c, min(8, K - c), fill, v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = fill;
  }
}
template <typename T, bool VEC>
__device__ __forceinline__ void store_chunk(T* row, int K, int i, int t, int threads, const float (&v)[8]) {
  const int c = chunk_column(i, t, threads);
  if (c >= K) return;
  if (VEC)
    store8(row + c, v);
  else
    store_any(row + c, min(8, K - c), v);
}

// A vector whose type is known at run time (svdq_dtype).
template <bool VEC>
__device__ __forceinline__ void load_param_chunk(const void* p, int dtype, size_t offset, int K, int i, int t,
                                                 int threads, float fill, float (&v)[8]) {
  if (dtype == SVDQ_DTYPE_BF16)
    load_chunk<__nv_bfloat16, VEC>(static_cast<const __nv_bfloat16*>(p) + offset, K, i, t, threads, fill, v);
  else if (dtype == SVDQ_DTYPE_FP16)
    load_chunk<__half, VEC>(static_cast<const __half*>(p) + offset, K, i, t, threads, fill, v);
  else
    load_chunk<float, VEC>(static_cast<const float*>(p) + offset, K, i, t, threads, fill, v);
}

// ------------------------------------------------------------- 8-bit checkpoint
constexpr int kCkptGroup = 32;

// The scale byte (exponent + 127) of a group from the bits of its largest magnitude: the smallest
// power of two at which that magnitude does not leave the codes (int8: < 127.5, which rounds to
// 127; E4M3: <= 448).  amax = m 2^k, so e = k - 6 (or k - 8), one more where m is at least
// 127.5 / 64 (or above 448 / 256); e is at least -127 and, lest the largest code decode to an
// infinity, at most that of k = 127.  0xFF for an infinity or a NaN.
template <int FMT>
__device__ __forceinline__ uint32_t ckpt_scale_byte(uint32_t amax_bits) {
  if (amax_bits >= 0x7F800000u) return 0xFFu;
  const int k = static_cast<int>(amax_bits >> 23);
  const uint32_t m = amax_bits & 0x7FFFFFu;
  const int b = FMT == SVDQ_CKPT8_INT8 ? k - 6 + (m >= 0x7F0000u) : k - 8 + (m > 0x600000u);
  return static_cast<uint32_t>(min(max(b, 0), FMT == SVDQ_CKPT8_INT8 ? 248 : 246));
}
// 2^(byte - 127), exact (2^-127 is subnormal); NaN for 0xFF
__device__ __forceinline__ float ckpt_scale(uint32_t byte) {
  return byte == 0xFFu ? __uint_as_float(0x7FC00000u) : __uint_as_float(byte ? byte << 23 : 0x00400000u);
}

// Four codes of four values whose group has scale byte `byte`.  The product of an fp32 and a power
// of two is exact here (where it is subnormal the code is 0 either way), so the code is the value
// rounded once, ties to even.
template <int FMT>
__device__ __forceinline__ uint32_t ckpt_codes4(float a, float b, float c, float d, uint32_t byte) {
  if (byte == 0xFFu) return 0u;  // a NaN or an infinity in the group
  const float inv = __uint_as_float((254u - byte) << 23);
  if (FMT == SVDQ_CKPT8_INT8) {
    if (byte == 248u) {  // the largest scale: magnitudes up to 128
      const float top = 127.0f / inv;
      a = fminf(fmaxf(a, -top), top), b = fminf(fmaxf(b, -top), top);
      c = fminf(fmaxf(c, -top), top), d = fminf(fmaxf(d, -top), top);
    }
    // + 1.5 2^23: the rounded integer is in the low mantissa bits, as two's complement
    constexpr float kMagic = 12582912.0f;
    const uint32_t lo = __byte_perm(__float_as_uint(__fmaf_rn(a, inv, kMagic)), __float_as_uint(__fmaf_rn(b, inv, kMagic)), 0x0040);
    const uint32_t hi = __byte_perm(__float_as_uint(__fmaf_rn(c, inv, kMagic)), __float_as_uint(__fmaf_rn(d, inv, kMagic)), 0x0040);
    return __byte_perm(lo, hi, 0x5410);
  }
  a *= inv, b *= inv, c *= inv, d *= inv;
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return static_cast<uint32_t>(lo) | static_cast<uint32_t>(hi) << 16;
}

// Four codes as fp32, times their group's scale (exact).
template <int FMT>
__device__ __forceinline__ void ckpt_values4(uint32_t w, float scale, float* v) {
  if (FMT == SVDQ_CKPT8_INT8) {
#pragma unroll
    // q + 128 in the low mantissa bits of 2^23, less 2^23 + 128: exact, and no conversion instruction
    for (int j = 0; j < 4; ++j)
      v[j] = (__uint_as_float(__byte_perm(w ^ 0x80808080u, 0x4B000000u, 0x7540 + j)) - 8388736.0f) * scale;
  } else {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      uint32_t h;
      asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(w >> (16 * j))));
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
      v[2 * j] = f.x * scale, v[2 * j + 1] = f.y * scale;
    }
  }
}

// Eight codes as four pairs, not yet times their group's scale (exact).
template <int FMT>
__device__ __forceinline__ void ckpt_codes8_pairs(uint2 q, F2 (&v)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t w = j < 2 ? q.x : q.y;
    if (FMT == SVDQ_CKPT8_INT8) {
      const uint32_t u = w ^ 0x80808080u;
      const F2 b = f2(__uint_as_float(__byte_perm(u, 0x4B000000u, 0x7540 + 2 * (j & 1))),
                      __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7541 + 2 * (j & 1))));
      v[j] = add2(b, f2(-8388736.0f, -8388736.0f));
    } else {
      uint32_t h;
      asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(w >> (16 * (j & 1)))));
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
      v[j] = f2(f.x, f.y);
    }
  }
}

__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

// The bits, as fp32, of the largest magnitude of eight values; a NaN counts as the largest.
__device__ __forceinline__ uint32_t largest8(const float (&v)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = max(m, abs_bits(v[j]));
  return m;
}
__device__ __forceinline__ uint32_t largest8(const uint4& w, const __nv_bfloat16*) {
  uint32_t m = w.x & 0x7FFF7FFFu;
  const uint32_t r[3] = {w.y & 0x7FFF7FFFu, w.z & 0x7FFF7FFFu, w.w & 0x7FFF7FFFu};
#pragma unroll
  for (int j = 0; j < 3; ++j) asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(r[j]));
  return max(m << 16, m & 0xFFFF0000u);  // a NaN's bits are above an infinity's
}
__device__ __forceinline__ uint32_t largest8(const uint4& w, const __half*) {
  uint32_t m = w.x & 0x7FFF7FFFu;
  const uint32_t r[3] = {w.y & 0x7FFF7FFFu, w.z & 0x7FFF7FFFu, w.w & 0x7FFF7FFFu};
#pragma unroll
  for (int j = 0; j < 3; ++j) asm("max.NaN.f16x2 %0, %0, %1;" : "+r"(m) : "r"(r[j]));
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&m));
  return max(abs_bits(f.x), abs_bits(f.y));
}

// Eight raw values of the vector layout.
template <typename T>
struct Raw8 {
  uint4 w;
  __device__ __forceinline__ void clear() { w = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void load(const T* p) { w = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ uint32_t largest() const { return largest8(w, static_cast<const T*>(nullptr)); }
  __device__ __forceinline__ void values(float (&v)[8]) const { unpack8(w, v, static_cast<const T*>(nullptr)); }
};
template <>
struct Raw8<float> {
  float f[8];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = 0.0f;
  }
  __device__ __forceinline__ void load(const float* p) { load8(p, f); }
  __device__ __forceinline__ uint32_t largest() const { return largest8(f); }
  __device__ __forceinline__ void values(float (&v)[8]) const {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = f[j];
  }
};

// A chunk of a row as it was read: packed where the vector layout reads it so.
template <typename T, bool VEC>
struct Held : Raw8<T> {};
template <typename T>
struct Held<T, false> : Raw8<float> {};

// The codes of a chunk, at any address, and its group's scale byte.
template <int FMT, bool VEC>
__device__ __forceinline__ void ckpt_store_codes(uint8_t* codes, uint8_t* scales, int c, int K, uint32_t byte,
                                                 const float (&v)[8]) {
  const uint2 q = make_uint2(ckpt_codes4<FMT>(v[0], v[1], v[2], v[3], byte), ckpt_codes4<FMT>(v[4], v[5], v[6], v[7], byte));
  if (VEC || (c + 8 <= K && reinterpret_cast<uintptr_t>(codes + c) % 8 == 0)) {
    *reinterpret_cast<uint2*>(codes + c) = q;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (c + j < K) codes[c + j] = static_cast<uint8_t>((j < 4 ? q.x : q.y) >> (8 * (j & 3)));
  }
  if (c % kCkptGroup == 0) scales[c / kCkptGroup] = static_cast<uint8_t>(byte);
}

// Writes chunk i of a row's checkpoint: codes (K bytes) and scales (ceil(K / 32) bytes).  Every lane
// of the warp calls it, with its chunk's largest magnitude; columns beyond K hold 0.
template <int FMT, bool VEC>
__device__ __forceinline__ void ckpt_store_chunk(uint8_t* codes, uint8_t* scales, int K, int i, int t, int threads,
                                                 uint32_t top, const float (&v)[8]) {
  uint32_t m = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
  const int c = chunk_column(i, t, threads);
  if (c < K) ckpt_store_codes<FMT, VEC>(codes, scales, c, K, ckpt_scale_byte<FMT>(m), v);
}

// Chunk i of a row from its checkpoint; columns beyond K give `fill` (a chunk of the vector layout has none).
template <int FMT, bool VEC>
__device__ __forceinline__ void ckpt_load_chunk(const uint8_t* codes, const uint8_t* scales, int K, int i, int t,
                                                int threads, float (&v)[8], float fill = 0.0f) {
  const int c = chunk_column(i, t, threads);
  uint2 w = make_uint2(0, 0);
  float s = 0.0f;
  if (c < K) {
    if (VEC || (c + 8 <= K && reinterpret_cast<uintptr_t>(codes + c) % 8 == 0)) {
      w = *reinterpret_cast<const uint2*>(codes + c);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (c + j < K) (j < 4 ? w.x : w.y) |= static_cast<uint32_t>(codes[c + j]) << (8 * (j & 3));
    }
    s = ckpt_scale(scales[c / kCkptGroup]);
  }
  ckpt_values4<FMT>(w.x, s, v);
  ckpt_values4<FMT>(w.y, s, v + 4);
  if (!VEC) {  // 0 times a group's NaN is none of the row's padding
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = c + j < K ? v[j] : fill;
  }
}

// Sums of a and b over the warp with 5 + 1 shuffles instead of 10: the halves take one value each.
// Lanes 0-15 get the first, lanes 16-31 the second.
__device__ __forceinline__ float warp_sum2_halves(float a, float b) {
  const bool upper = threadIdx.x & 16;
  const float other = __shfl_xor_sync(0xffffffffu, upper ? a : b, 16);
  float v = (upper ? b : a) + other;
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

}  // namespace dev
}  // namespace svdq
