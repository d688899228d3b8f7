// 8-bit activation checkpoints: codes (int8 or E4M3) with one power-of-two scale per 32 consecutive
// values of a row, written once in the forward pass and read in the backward pass.
//
// The scale is a power of two, so x / s, q s and the choice of s are exact: the only rounding is the
// code's, and a checkpoint decodes to the same bf16 (or fp32) values everywhere.  8.25 bits a value
// against 16: an int8 code is off by at most 2^-7 of the group's largest magnitude (half a step), an
// E4M3 code by 2^-4 of the value.  Both directions are bound by HBM and read and write every byte once:
// 4608 x 12288 bf16 to int8 takes 27.4 us, 95 % of the copy rate; 2048 x 1280 E4M3 to fp16 2.3 us (from L2).
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

// How rows are addressed: packed rows of whole groups are one long row (the index arithmetic of the others
// took a fifth of the time: 33.3 against 27.4 us at 4608 x 12288, bf16 to int8).
enum Layout { kPacked, kVector, kAny };

// kUnroll chunks of 8 values per thread, a group is 4 neighbouring threads' chunks; the chunks' loads are all
// in flight before the first is used.
constexpr int kUnroll = 4;
template <typename T, int FMT, Layout L>
__global__ void __launch_bounds__(kThreads) ckpt_encode_kernel(const T* __restrict__ X, int64_t ld, uint64_t total,
                                                            uint32_t per_row, int K, uint8_t* __restrict__ codes,
                                                            uint8_t* __restrict__ scales) {
  const int groups = (K + kCkptGroup - 1) / kCkptGroup;
  Held<T, L != kAny> held[kUnroll];
  uint64_t row[kUnroll];  // packed: the chunk's first value instead
  uint32_t at[kUnroll];
  bool in[kUnroll];
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    const uint64_t idx = (static_cast<uint64_t>(blockIdx.x) * kUnroll + i) * kThreads + threadIdx.x;
    held[i].clear();
    if constexpr (L == kPacked) {
      in[i] = idx < total;
      row[i] = idx * 8;
      if (in[i]) held[i].load(X + row[i]);
      continue;
    }
    split_index(idx < total ? idx : total - 1, total, per_row, row[i], at[i]);
    at[i] *= 8;  // column
    in[i] = idx < total && at[i] < static_cast<uint32_t>(K);
    if (in[i]) {
      const T* x = X + row[i] * ld + at[i];
      if constexpr (L == kVector)
        held[i].load(x);
      else if constexpr (L == kAny)
        load_any(x, min(8, K - static_cast<int>(at[i])), 0.0f, held[i].f);
    }
  }
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    uint32_t m = in[i] ? held[i].largest() : 0u;
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    if (in[i]) {
      float v[8];
      held[i].values(v);
      const uint32_t byte = ckpt_scale_byte<FMT>(m);
      if constexpr (L == kPacked)  // the places of a row of one group
        ckpt_store_codes<FMT, true>(codes + row[i] / kCkptGroup * kCkptGroup, scales + row[i] / kCkptGroup,
                                    static_cast<int>(row[i] % kCkptGroup), kCkptGroup, byte, v);
      else
        ckpt_store_codes<FMT, L == kVector>(codes + row[i] * K, scales + row[i] * groups, static_cast<int>(at[i]), K,
                                            byte, v);
    }
  }
}

template <typename T, int FMT, Layout L>
__global__ void __launch_bounds__(kThreads) ckpt_decode_kernel(const uint8_t* __restrict__ codes,
                                                            const uint8_t* __restrict__ scales, uint64_t total,
                                                            uint32_t per_row, int K, T* __restrict__ X, int64_t ld) {
  const uint64_t idx = static_cast<uint64_t>(blockIdx.x) * kThreads + threadIdx.x;
  if (idx >= total) return;
  float v[8];
  if (L == kPacked) {
    const uint64_t group = idx / 4;
    const int at = static_cast<int>(idx % 4);
    ckpt_load_chunk<FMT, true>(codes + group * kCkptGroup, scales + group, kCkptGroup, 0, at, 0, v);
    store8(X + idx * 8, v);
    return;
  }
  uint64_t row = 0;
  uint32_t at = 0;
  split_index(idx, total, per_row, row, at);
  ckpt_load_chunk<FMT, L == kVector>(codes + row * K, scales + row * ((K + kCkptGroup - 1) / kCkptGroup), K, 0,
                                     static_cast<int>(at), 0, v);
  store_chunk<T, L == kVector>(X + row * ld, K, 0, static_cast<int>(at), 0, v);
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

Layout layout(const void* X, int K, int64_t ld) {
  if (K % 8 || ld % 8 || !aligned16(X)) return kAny;
  return K % kCkptGroup == 0 && ld == K ? kPacked : kVector;
}

template <typename T, int FMT>
svdq_status encode(const void* X, int64_t ld, int M, int K, uint8_t* codes, uint8_t* scales, cudaStream_t stream) {
  Grid g;
  const T* x = static_cast<const T*>(X);
  SVDQ_TRY(item_grid(M, (K + 7) / 8, 4, kUnroll, &g));
  switch (layout(X, K, ld)) {
    case kPacked:
      ckpt_encode_kernel<T, FMT, kPacked><<<g.blocks, kThreads, 0, stream>>>(x, ld, g.total, g.per_row, K, codes, scales);
      break;
    case kVector:
      ckpt_encode_kernel<T, FMT, kVector><<<g.blocks, kThreads, 0, stream>>>(x, ld, g.total, g.per_row, K, codes, scales);
      break;
    default:
      ckpt_encode_kernel<T, FMT, kAny><<<g.blocks, kThreads, 0, stream>>>(x, ld, g.total, g.per_row, K, codes, scales);
  }
  SVDQ_CUDA_TRY(cudaGetLastError());
  return SVDQ_OK;
}

template <typename T, int FMT>
svdq_status decode(const uint8_t* codes, const uint8_t* scales, int M, int K, void* X, int64_t ld, cudaStream_t stream) {
  Grid g;
  T* x = static_cast<T*>(X);
  SVDQ_TRY(item_grid(M, (K + 7) / 8, 1, 1, &g));
  switch (layout(X, K, ld)) {
    case kPacked:
      ckpt_decode_kernel<T, FMT, kPacked><<<g.blocks, kThreads, 0, stream>>>(codes, scales, g.total, g.per_row, K, x, ld);
      break;
    case kVector:
      ckpt_decode_kernel<T, FMT, kVector><<<g.blocks, kThreads, 0, stream>>>(codes, scales, g.total, g.per_row, K, x, ld);
      break;
    default:
      ckpt_decode_kernel<T, FMT, kAny><<<g.blocks, kThreads, 0, stream>>>(codes, scales, g.total, g.per_row, K, x, ld);
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
