// The packed layout of an int8 weight matrix with a scale per output channel, and
// the last step of its product.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "llama_q8.h"

namespace lq8 {

// Rows in tiles of 32 (padded with zero rows), k in chunks of 16 (padded with
// zero codes): the 32 rows' 16-byte pieces of a chunk lie next to each other, so a
// warp-wide 16-byte load (lane = row) reads 512 contiguous bytes and the chunks of
// a tile are one contiguous run:
//   byte offset(n, kk) = ((n / 32) * chunks + kk / 16) * 512 + (n % 32) * 16 + kk % 16
// The f32 scales of all padded rows follow, 256-byte aligned, and then for each tile
// the largest norm (root of the sum of squared codes, rounded up) of its rows.
struct I8Weights {
    const int8_t* codes;
    const float* scale;
    const float* norm;
    int64_t rows, rows_pad;
    int64_t chunks;  // k / 16, rounded up
};

__host__ __device__ inline int64_t i8_codes_bytes(int64_t rows, int64_t k) {
    return (rows + 31) / 32 * 32 * ((k + 15) / 16 * 16);
}
__host__ __device__ inline int64_t i8_scale_offset(int64_t rows, int64_t k) {
    return (i8_codes_bytes(rows, k) + 255) / 256 * 256;
}
__host__ __device__ inline int64_t i8_packed_total(int64_t rows, int64_t k) {
    return i8_scale_offset(rows, k) + (rows + 31) / 32 * 33 * 4;
}
inline I8Weights i8_view(const void* packed, int64_t rows, int64_t k) {
    const uint8_t* base = reinterpret_cast<const uint8_t*>(packed);
    const int64_t pad = (rows + 31) / 32 * 32;
    const float* scale = reinterpret_cast<const float*>(base + i8_scale_offset(rows, k));
    return {reinterpret_cast<const int8_t*>(base), scale, scale + pad, rows, pad, (k + 15) / 16};
}

// A sum (an integer, or f32 that holds one) times the token's and the channel's
// scale, rounded to the output type.
template <typename T> __device__ __forceinline__ T i8_round(float v);
template <> __device__ __forceinline__ float i8_round<float>(float v) { return v; }
template <> __device__ __forceinline__ __half i8_round<__half>(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 i8_round<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <typename T, typename S> __device__ __forceinline__ T i8_scaled(S sum, float sa, float sw) {
    return i8_round<T>((float)sum * sa * sw);
}

// i8_gemm.cu: any number of tokens on the tensor cores, in a workspace of i8_gemm_workspace bytes (LQ8_ERR_ARG if it is
// smaller)
size_t i8_gemm_workspace(int64_t k, int64_t m);
template <typename T>
llama_q8_status launch_i8_gemm(const I8Weights& W, int64_t k, const int8_t* a, const float* sa, int64_t m, T* y,
                               int64_t y_stride, void* workspace, size_t workspace_bytes, int32_t* err, cudaStream_t s);

}  // namespace lq8
