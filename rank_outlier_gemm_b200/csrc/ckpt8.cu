// 8-bit activation checkpoints: codes (int8 or E4M3) with one power-of-two scale per 32 consecutive
// values of a row, written once in the forward pass and read in the backward pass.
//
// The scale is a power of two, so x / s, q s and the choice of s are exact: the only rounding is the
// code's, and a checkpoint decodes to the same bf16 (or fp32) values everywhere.  8.25 bits a value
// against 16: an int8 code is off by at most 2^-7 of the group's largest magnitude (half a step), an
// E4M3 code by 2^-4 of the value.  Both directions are bound by HBM and read and write every byte once.
#include "rows.cuh"
#include "svdq_internal.h"

namespace svdq {
namespace {

using namespace dev;

constexpr int kThreads = 256;

// Row and position of item `idx` where each row has `per_row` items.
__device__ __forceinline__ void split_index(uint64_t idx, uint64_t total, uint32_t per_row, uint64_t& row, uint32_t& at) {
  if (total < (1ull << 32)) {
    const uint32_t i = static_cast<uint32_t>(idx);
    row = i / per_row;
    at = i - static_cast<uint32_t>(row) * per_row;
  } else {
    row = idx / per_row;
    at = static_cast<uint32_t>(idx - row * per_row);
  }
}

// Vector layout: kUnroll chunks of 8 values per thread, a group is 4 neighbouring threads' chunks; their
// loads are all in flight before the first is used.  Element layout: a value per thread, a group is a warp.
constexpr int kUnroll = 4;
template <typename T, int FMT>
__global__ void __launch_bounds__(kThreads) ckpt_encode_kernel(const T* __restrict__ X, int64_t ld, uint64_t total,
                                                            uint32_t per_row, int K, uint8_t* __restrict__ codes,
                                                            uint8_t* __restrict__ scales) {
  const int groups = (K + kCkptGroup - 1) / kCkptGroup;
  Raw8<T> raw[kUnroll];
  uint64_t row[kUnroll];
  uint32_t at[kUnroll];
  bool in[kUnroll];
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    const uint64_t idx = (static_cast<uint64_t>(blockIdx.x) * kUnroll + i) * kThreads + threadIdx.x;
    split_index(idx < total ? idx : total - 1, total, per_row, row[i], at[i]);
    in[i] = idx < total && at[i] * 8 < static_cast<uint32_t>(K);
    if (in[i]) raw[i].load(X + row[i] * ld + at[i] * 8);
  }
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    uint32_t m = in[i] ? raw[i].largest() : 0u;
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    const uint32_t b = ckpt_scale_byte<FMT>(m);
    if (in[i]) {
      float v[8];
      raw[i].values(v);
      *reinterpret_cast<uint2*>(codes + row[i] * K + at[i] * 8) =
          make_uint2(ckpt_codes4<FMT>(v[0], v[1], v[2], v[3], b), ckpt_codes4<FMT>(v[4], v[5], v[6], v[7], b));
      if (at[i] % 4 == 0) scales[row[i] * groups + at[i] / 4] = static_cast<uint8_t>(b);
    }
  }
}

template <typename T, int FMT>
__global__ void __launch_bounds__(kThreads) ckpt_encode_element_kernel(const T* __restrict__ X, int64_t ld, uint64_t total,
                                                                    uint32_t per_row, int K, uint8_t* __restrict__ codes,
                                                                    uint8_t* __restrict__ scales) {
  const uint64_t idx = static_cast<uint64_t>(blockIdx.x) * kThreads + threadIdx.x;
  uint64_t row = 0;
  uint32_t at = 0;
  split_index(idx < total ? idx : total - 1, total, per_row, row, at);
  const bool in = idx < total && at < static_cast<uint32_t>(K);
  const float v = in ? to_f32(X[row * ld + at]) : 0.0f;
  const uint32_t b = ckpt_scale_byte<FMT>(__reduce_max_sync(0xffffffffu, abs_bits(v)));
  if (in) {
    codes[row * K + at] = static_cast<uint8_t>(ckpt_codes4<FMT>(v, 0.0f, 0.0f, 0.0f, b) & 0xFFu);
    if (at % kCkptGroup == 0)
      scales[row * ((K + kCkptGroup - 1) / kCkptGroup) + at / kCkptGroup] = static_cast<uint8_t>(b);
  }
}

template <typename T, int FMT, bool VEC>
__global__ void __launch_bounds__(kThreads) ckpt_decode_kernel(const uint8_t* __restrict__ codes,
                                                            const uint8_t* __restrict__ scales, uint64_t total,
                                                            uint32_t per_row, int K, T* __restrict__ X, int64_t ld) {
  const uint64_t idx = static_cast<uint64_t>(blockIdx.x) * kThreads + threadIdx.x;
  if (idx >= total) return;
  uint64_t row = 0;
  uint32_t at = 0;
  split_index(idx, total, per_row, row, at);
  const int groups = (K + kCkptGroup - 1) / kCkptGroup;
  const uint8_t* q = codes + row * K;
  const uint8_t* s = scales + row * groups;
  float v[8];
  if (VEC) {
    ckpt_load_chunk<FMT, true>(q, s, K, 0, static_cast<int>(at), 0, v);
    store8(X + row * ld + at * 8, v);
  } else {
    ckpt_values4<FMT>(q[at], ckpt_scale(s[at / kCkptGroup]), v);
    X[row * ld + at] = from_f32<T>(v[0]);
  }
}

struct Grid {
  uint64_t total;
  uint32_t per_row;
  unsigned blocks;
};

// Items of M rows, each row's padded to whole groups for the encoder (`pad` items), `per_thread` a thread.
svdq_status item_grid(int M, int items, int pad, int per_thread, Grid* g) {
  g->per_row = static_cast<uint32_t>(round_up(items, pad));
  g->total = static_cast<uint64_t>(M) * g->per_row;
  const uint64_t blocks = (g->total + kThreads * per_thread - 1) / (kThreads * per_thread);
  if (blocks > 0x7FFFFFFFull) return fail(SVDQ_ERR_INVALID_ARG, "M=%d rows are too many", M);
  g->blocks = static_cast<unsigned>(blocks);
  return SVDQ_OK;
}

template <typename T, int FMT>
svdq_status encode(const void* X, int64_t ld, int M, int K, uint8_t* codes, uint8_t* scales, cudaStream_t stream) {
  Grid g;
  const T* x = static_cast<const T*>(X);
  if (K % 8 == 0 && ld % 8 == 0 && aligned16(X) && aligned16(codes)) {
    SVDQ_TRY(item_grid(M, K / 8, 4, kUnroll, &g));
    ckpt_encode_kernel<T, FMT><<<g.blocks, kThreads, 0, stream>>>(x, ld, g.total, g.per_row, K, codes, scales);
  } else {
    SVDQ_TRY(item_grid(M, K, kCkptGroup, 1, &g));
    ckpt_encode_element_kernel<T, FMT><<<g.blocks, kThreads, 0, stream>>>(x, ld, g.total, g.per_row, K, codes, scales);
  }
  SVDQ_CUDA_TRY(cudaGetLastError());
  return SVDQ_OK;
}

template <typename T, int FMT>
svdq_status decode(const uint8_t* codes, const uint8_t* scales, int M, int K, void* X, int64_t ld, cudaStream_t stream) {
  Grid g;
  T* x = static_cast<T*>(X);
  if (K % 8 == 0 && ld % 8 == 0 && aligned16(X) && aligned16(codes)) {
    SVDQ_TRY(item_grid(M, K / 8, 1, 1, &g));
    ckpt_decode_kernel<T, FMT, true><<<g.blocks, kThreads, 0, stream>>>(codes, scales, g.total, g.per_row, K, x, ld);
  } else {
    SVDQ_TRY(item_grid(M, K, 1, 1, &g));
    ckpt_decode_kernel<T, FMT, false><<<g.blocks, kThreads, 0, stream>>>(codes, scales, g.total, g.per_row, K, x, ld);
  }
  SVDQ_CUDA_TRY(cudaGetLastError());
  return SVDQ_OK;
}

}  // namespace

svdq_status launch_ckpt8_encode(const void* X, int dtype, int M, int K, int64_t ld, int format, uint8_t* codes,
                                uint8_t* scales, cudaStream_t stream) {
  const bool i8 = format == SVDQ_CKPT8_INT8;
  switch (dtype) {
    case SVDQ_DTYPE_BF16:
      return i8 ? encode<__nv_bfloat16, SVDQ_CKPT8_INT8>(X, ld, M, K, codes, scales, stream)
                : encode<__nv_bfloat16, SVDQ_CKPT8_E4M3>(X, ld, M, K, codes, scales, stream);
    case SVDQ_DTYPE_FP16:
      return i8 ? encode<__half, SVDQ_CKPT8_INT8>(X, ld, M, K, codes, scales, stream)
                : encode<__half, SVDQ_CKPT8_E4M3>(X, ld, M, K, codes, scales, stream);
    default:
      return i8 ? encode<float, SVDQ_CKPT8_INT8>(X, ld, M, K, codes, scales, stream)
                : encode<float, SVDQ_CKPT8_E4M3>(X, ld, M, K, codes, scales, stream);
  }
}

svdq_status launch_ckpt8_decode(const uint8_t* codes, const uint8_t* scales, int M, int K, int format, void* X,
                                int dtype, int64_t ld, cudaStream_t stream) {
  const bool i8 = format == SVDQ_CKPT8_INT8;
  switch (dtype) {
    case SVDQ_DTYPE_BF16:
      return i8 ? decode<__nv_bfloat16, SVDQ_CKPT8_INT8>(codes, scales, M, K, X, ld, stream)
                : decode<__nv_bfloat16, SVDQ_CKPT8_E4M3>(codes, scales, M, K, X, ld, stream);
    case SVDQ_DTYPE_FP16:
      return i8 ? decode<__half, SVDQ_CKPT8_INT8>(codes, scales, M, K, X, ld, stream)
                : decode<__half, SVDQ_CKPT8_E4M3>(codes, scales, M, K, X, ld, stream);
    default:
      return i8 ? decode<float, SVDQ_CKPT8_INT8>(codes, scales, M, K, X, ld, stream)
                : decode<float, SVDQ_CKPT8_E4M3>(codes, scales, M, K, X, ld, stream);
  }
}

}  // namespace svdq
