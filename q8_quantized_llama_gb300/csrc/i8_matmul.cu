// Products of int8 matrices with a scale per token and per channel:
//   y[t][n] = (sum_k a[t][k] W[n][k]) sa[t] sw[n]
// The sum is an exact integer; the two scales are applied in f32.
#include "i8.cuh"
#include "kernels.cuh"
#include "llama_q8.h"

namespace lq8 {

// ---------------------------------------------------------------------------
// Regroup row-major codes into the packed layout of i8.cuh: one thread per 16
// codes of a (padded) row.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(256) i8_pack_kernel(const uint4* __restrict__ codes, const float* __restrict__ scale,
                                                      int64_t rows, int64_t chunks, uint4* __restrict__ out,
                                                      float* __restrict__ out_scale, float* __restrict__ out_norm) {
    __shared__ uint32_t part[8][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t tile = blockIdx.x, n = tile * 32 + lane;
    int sum = 0;
    for (int64_t c = warp; c < chunks; c += 8) {
        const uint4 q = n < rows ? codes[n * chunks + c] : make_uint4(0, 0, 0, 0);
        out[(tile * chunks + c) * 32 + lane] = q;
        sum = __dp4a((int)q.x, (int)q.x, sum);
        sum = __dp4a((int)q.y, (int)q.y, sum);
        sum = __dp4a((int)q.z, (int)q.z, sum);
        sum = __dp4a((int)q.w, (int)q.w, sum);
    }
    part[warp][lane] = (uint32_t)sum;
    __syncthreads();
    if (warp == 0) {
        uint32_t all = 0;
#pragma unroll
        for (int w = 0; w < 8; ++w) all += part[w][lane];  // at most 131056 * 2^14 < 2^31
        out_scale[n] = n < rows ? scale[n] : 0.0f;
        const float norm = warp_max(__fsqrt_ru(__uint2float_ru(all)));
        if (lane == 0) out_norm[tile] = norm;
    }
}

// ---------------------------------------------------------------------------
// Few tokens: a CTA takes one 32-row tile (lane = row) for MT tokens, its 8
// warps every eighth 16-code chunk; four codes of both sides go through one
// integer dot product. The warps' sums meet in shared memory.
// ---------------------------------------------------------------------------
template <int MT, typename T>
__global__ void __launch_bounds__(256) i8_rows_kernel(const I8Weights W, const int8_t* __restrict__ a,
                                                      const float* __restrict__ sa, int64_t m, T* __restrict__ y,
                                                      int64_t y_stride) {
    __shared__ int part[8][MT][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t tile = blockIdx.x, t0 = (int64_t)blockIdx.y * MT;
    const uint4* w = reinterpret_cast<const uint4*>(W.codes) + tile * W.chunks * 32 + lane;
    int acc[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) acc[t] = 0;
#pragma unroll 4
    for (int c = warp; c < W.chunks; c += 8) {
        const uint4 q = ld_stream_u4(w + (int64_t)c * 32);
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            const int64_t row = t0 + t < m ? t0 + t : m - 1;
            const uint4 x = __ldg(reinterpret_cast<const uint4*>(a) + row * W.chunks + c);
            acc[t] = __dp4a((int)q.x, (int)x.x, acc[t]);
            acc[t] = __dp4a((int)q.y, (int)x.y, acc[t]);
            acc[t] = __dp4a((int)q.z, (int)x.z, acc[t]);
            acc[t] = __dp4a((int)q.w, (int)x.w, acc[t]);
        }
    }
#pragma unroll
    for (int t = 0; t < MT; ++t) part[warp][t][lane] = acc[t];
    __syncthreads();
    const int64_t n = tile * 32 + lane;
    for (int t = warp; t < MT; t += 8) {
        int s = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) s += part[i][t][lane];
        if (t0 + t < m && n < W.rows) y[(t0 + t) * y_stride + n] = i8_scaled<T>(s, sa[t0 + t], W.scale[n]);
    }
}

template <typename T>
static cudaError_t launch_i8_matmul(const I8Weights& W, int64_t k, const int8_t* a, const float* sa, int64_t m, T* y,
                                    int64_t y_stride, void* workspace, int32_t* err, cudaStream_t s) {
    if (m >= kI8GemmMin) {
        const cudaError_t e = ensure_kernel_attributes();
        return e != cudaSuccess ? e : launch_i8_gemm<T>(W, k, a, sa, m, y, y_stride, workspace, err, s);
    }
    const unsigned tiles = (unsigned)(W.rows_pad / 32);
    auto go = [&](auto kernel, int mt) {
        return launch_ex(kernel, dim3(tiles, (unsigned)((m + mt - 1) / mt)), dim3(256), 0, s, false, W, a, sa, m, y, y_stride);
    };
    if (m == 1) return go(i8_rows_kernel<1, T>, 1);
    if (m == 2) return go(i8_rows_kernel<2, T>, 2);
    if (m <= 4) return go(i8_rows_kernel<4, T>, 4);
    return go(i8_rows_kernel<8, T>, 8);
}

static bool i8_sizes_ok(int64_t rows, int64_t k) {
    return rows > 0 && k > 0 && rows <= (1ll << 30) && k <= LLAMA_Q8_I8_MAX_K;
}

}  // namespace lq8

using namespace lq8;

extern "C" {

size_t llama_q8_i8_packed_bytes(int64_t rows, int64_t k) {
    return i8_sizes_ok(rows, k) ? (size_t)i8_packed_total(rows, k) : 0;
}

llama_q8_status llama_q8_i8_pack(const int8_t* codes, const float* scale, int64_t rows, int64_t k, void* packed,
                                 void* stream) {
    if (!codes || !scale || !packed || rows < 0 || k <= 0) return LQ8_ERR_ARG;
    if (((uintptr_t)codes | (uintptr_t)packed) & 15 || ((uintptr_t)scale & 3)) return LQ8_ERR_ARG;
    if (rows > (1ll << 30) || k > LLAMA_Q8_I8_MAX_K) return LQ8_ERR_UNSUPPORTED;
    if (rows == 0) return LQ8_OK;
    const I8Weights w = i8_view(packed, rows, k);
    const cudaError_t e =
        launch_ex(i8_pack_kernel, dim3((unsigned)(w.rows_pad / 32)), dim3(256), 0, (cudaStream_t)stream, false,
                  reinterpret_cast<const uint4*>(codes), scale, rows, w.chunks,
                  reinterpret_cast<uint4*>(const_cast<int8_t*>(w.codes)), const_cast<float*>(w.scale),
                  const_cast<float*>(w.norm));
    return e == cudaSuccess ? LQ8_OK : LQ8_ERR_CUDA;
}

size_t llama_q8_i8_matmul_workspace_bytes(int64_t rows, int64_t k, int64_t m) {
    return !i8_sizes_ok(rows, k) || m < kI8GemmMin || m > (1ll << 30) ? 0 : i8_gemm_workspace(rows, k, m);
}

llama_q8_status llama_q8_i8_matmul(const void* packed, int64_t rows, int64_t k, const int8_t* codes,
                                   const float* scale, int64_t m, int32_t type, void* y, int64_t y_stride,
                                   void* workspace, size_t workspace_bytes, int32_t* err, void* stream) {
    if (!packed || !codes || !scale || !y || rows <= 0 || k <= 0 || m < 0 || y_stride < rows) return LQ8_ERR_ARG;
    if (type != LLAMA_Q8_GGUF_F32 && type != LLAMA_Q8_GGUF_F16 && type != LLAMA_Q8_GGUF_BF16)
        return LQ8_ERR_UNSUPPORTED;
    if (((uintptr_t)packed | (uintptr_t)codes | (uintptr_t)workspace) & 15) return LQ8_ERR_ARG;
    if (((uintptr_t)scale | (uintptr_t)err) & 3 || ((uintptr_t)y & (type == LLAMA_Q8_GGUF_F32 ? 3 : 1)))
        return LQ8_ERR_ARG;
    if (!i8_sizes_ok(rows, k) || m > (1ll << 30)) return LQ8_ERR_UNSUPPORTED;
    const size_t need = llama_q8_i8_matmul_workspace_bytes(rows, k, m);
    if (workspace_bytes < need || (need && !workspace)) return LQ8_ERR_ARG;
    if (m == 0) return LQ8_OK;
    const I8Weights w = i8_view(packed, rows, k);
    cudaStream_t s = (cudaStream_t)stream;
    cudaError_t e;
    if (type == LLAMA_Q8_GGUF_F32) e = launch_i8_matmul(w, k, codes, scale, m, (float*)y, y_stride, workspace, err, s);
    else if (type == LLAMA_Q8_GGUF_F16) e = launch_i8_matmul(w, k, codes, scale, m, (__half*)y, y_stride, workspace, err, s);
    else e = launch_i8_matmul(w, k, codes, scale, m, (__nv_bfloat16*)y, y_stride, workspace, err, s);
    return e == cudaSuccess ? LQ8_OK : LQ8_ERR_CUDA;
}

}  // extern "C"
