// Products of int8 matrices with a scale per token and per channel:
//   y[t][n] = (sum_k a[t][k] W[n][k]) sa[t] sw[n]
// The sum is an exact integer; the two scales are applied in f32.
#include "i8.cuh"
#include "kernels.cuh"
#include "llama_q8.h"
#include "ptx.cuh"
#include "tc.cuh"

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
// Few tokens: the weights' bytes are what counts, so warps read them straight into
// registers, 16 bytes a lane. The warps that share a 32-row tile take parts of k; their
// sums are integers and meet in shared memory, across a cluster where the tiles alone
// would leave SMs idle.
// ---------------------------------------------------------------------------
// The CTA's sums mine[token][32] of a cluster's tile are added up and stored, the tokens dealt over the CTAs.
template <typename T>
__device__ __forceinline__ void few_cluster_store(const I8Weights& W, const int (*mine)[33], int m, int64_t tile,
                                                  const float* __restrict__ sa, T* __restrict__ y, int64_t y_stride) {
    cluster_sync();
    const int64_t channel = tile * 32 + (threadIdx.x & 31);
    for (int tok = blockIdx.y + (threadIdx.x >> 5) * gridDim.y; tok < m; tok += (blockDim.x >> 5) * gridDim.y) {
        int s = 0;
        for (int i = 0; i < (int)gridDim.y; ++i)
            s += __float_as_int(ld_dsmem_f32(reinterpret_cast<const float*>(&mine[tok][threadIdx.x & 31]), (uint32_t)i));
        if (channel < W.rows) y[tok * y_stride + channel] = i8_scaled<T>(s, __ldca(sa + tok), W.scale[channel]);
    }
    cluster_sync();  // nobody leaves while its sums are read
}

// One token: lane = row, four codes of both sides through one integer dot product (its rate, 16 lanes a clock and SM,
// would be too low for four tokens: 28672 x 4096 34 us; one 18.8), each of the cluster's warps a chunk in turn.
constexpr int kRowWarps = 8;
template <typename T>
__global__ void __launch_bounds__(kRowWarps * 32, 6)
    i8_row_kernel(const I8Weights W, const int8_t* __restrict__ a, const float* __restrict__ sa, T* __restrict__ y,
                  int64_t y_stride) {
    __shared__ int part[kRowWarps][33];
    pdl_wait();
    pdl_launch_dependents();  // behind the wait: what is launched next may rely on everything before this kernel
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t tile = blockIdx.x, channel = tile * 32 + lane;
    const int chunks = (int)W.chunks, step = kRowWarps * gridDim.y;
    const uint4* w = reinterpret_cast<const uint4*>(W.codes) + tile * chunks * 32 + lane;
    const uint4* x = reinterpret_cast<const uint4*>(a);
    int acc = 0;
#pragma unroll 4
    for (int c = blockIdx.y * kRowWarps + warp; c < chunks; c += step) {
        const uint4 q = ld_stream_u4(w + (int64_t)c * 32), v = __ldca(x + c);
        acc = __dp4a((int)q.x, (int)v.x, acc);
        acc = __dp4a((int)q.y, (int)v.y, acc);
        acc = __dp4a((int)q.z, (int)v.z, acc);
        acc = __dp4a((int)q.w, (int)v.w, acc);
    }
    part[warp][lane] = acc;
    __syncthreads();
    if (warp == 0) {
        int s = 0;
#pragma unroll
        for (int i = 0; i < kRowWarps; ++i) s += part[i][lane];
        if (gridDim.y > 1) part[0][lane] = s;
        else if (channel < W.rows) y[channel] = i8_scaled<T>(s, __ldca(sa), W.scale[channel]);
    }
    if (gridDim.y > 1) few_cluster_store(W, part, 1, tile, sa, y, y_stride);
}

// Two to sixteen tokens, and more with small matrices: a warp multiplies 32 channels with 8 NT tokens by f16 matrix
// instructions (m16n8k16; codes are exact in f16, and sums of 1024 products in f32).
//
// A block is 64 k. Lane 4 g + t holds chunk t (16 codes) of rows g, g + 8, g + 16
// and g + 24 and of token g: the word w of each is the lane's part of step w, whose
// 16 k are words w of the four chunks (any order of k serves, if it is the same for
// both operands). Two blocks' loads are in flight, one with 16 tokens, as the
// registers of 24 warps an SM allow (28672 x 4096, 8 tokens: 21.6 us, 22.1 with four
// blocks and 12 warps, 23.4 with one and 40; 16 tokens: 23.8 us, 29.0 with two and 16).
constexpr int kFewWarps = 4;
template <int NT> constexpr int kFewDeep = NT == 1 ? 2 : 1;

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// S warps per tile, of a CTA (which then has kFewWarps / S tiles) or, S = kFewWarps, of each CTA of a cluster.
template <int NT, typename T>
__global__ void __launch_bounds__(kFewWarps * 32, NT <= 2 ? 6 : 4)
    i8_few_kernel(const I8Weights W, const int8_t* __restrict__ a, const float* __restrict__ sa, int m, int S,
                  T* __restrict__ y, int64_t y_stride) {
    pdl_wait();
    // tokens in groups of 8 NT along grid.z
    a += (int64_t)blockIdx.z * 8 * NT * W.chunks * 16, sa += blockIdx.z * 8 * NT, y += blockIdx.z * 8 * NT * y_stride;
    m = min(m - (int)blockIdx.z * 8 * NT, 8 * NT);
    constexpr int D = kFewDeep<NT>;
    __shared__ int part[kFewWarps][8 * NT][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int own = warp / S, share = blockIdx.y * S + warp % S, shares = gridDim.y * S;
    const int64_t tile = (int64_t)blockIdx.x * (kFewWarps / S) + own;
    const int chunks = (int)W.chunks, blocks = (chunks + 3) / 4;
    const int b0 = (int)((int64_t)blocks * share / shares);
    const int n = tile < W.rows_pad / 32 ? (int)((int64_t)blocks * (share + 1) / shares) - b0 : 0;
    const uint4* w = reinterpret_cast<const uint4*>(W.codes) + ((tile * chunks + 4 * b0 + t) * 32 + g);
    const uint4* x = reinterpret_cast<const uint4*>(a) + 4 * b0 + t;
    const int last = chunks - 4 * b0 - t;  // this lane's chunks are those with 4 b < last

    uint4 q[D][4], p[D][NT];
    auto load = [&](int u, int b) {
        const bool in = b < n && 4 * b < last;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            q[u][i] = in ? ld_stream_u4(w + (int64_t)b * 128 + i * 8) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int j = 0; j < NT; ++j)
            p[u][j] = in && j * 8 + g < m ? __ldca(x + (int64_t)(j * 8 + g) * chunks + 4 * b) : make_uint4(0, 0, 0, 0);
    };
#pragma unroll
    for (int u = 0; u < D; ++u) load(u, u);
    float d[2][NT][4];
    int sum[2][NT][4];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) d[i][j][e] = 0.0f, sum[i][j][e] = 0;
    for (int b = 0; b < n; b += D) {
#pragma unroll
        for (int u = 0; u < D; ++u) {  // blocks past the last are zeros
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                auto word = [&](const uint4& v) { return s == 0 ? v.x : s == 1 ? v.y : s == 2 ? v.z : v.w; };
                uint32_t f[4][2];
#pragma unroll
                for (int i = 0; i < 4; ++i) codes_to_f16x2(word(q[u][i]), f[i][0], f[i][1]);
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    uint32_t lo, hi;
                    codes_to_f16x2(word(p[u][j]), lo, hi);
                    mma_f16(d[0][j], f[0][0], f[1][0], f[0][1], f[1][1], lo, hi);
                    mma_f16(d[1][j], f[2][0], f[3][0], f[2][1], f[3][1], lo, hi);
                }
            }
            load(u, b + u + D);
        }
        if ((b + D) % 16 == 0 || b + D >= n) {  // 1024 products of at most 2^14: exact in f32 so far
            static_assert(16 % D == 0, "the sums are taken every 16 blocks");
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) sum[i][j][e] += __float2int_rn(d[i][j][e]), d[i][j][e] = 0.0f;
        }
    }
    // d[i][j]: channels 16 i + g (elements 0, 1) and 16 i + g + 8 (2, 3), tokens 8 j + 2 t and the next
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) part[warp][8 * j + 2 * t + (e & 1)][16 * i + 8 * (e >> 1) + g] = sum[i][j][e];
    __syncthreads();
    if (gridDim.y > 1) {
        for (int tok = warp; tok < m; tok += kFewWarps) {
            int s = 0;
#pragma unroll
            for (int i = 0; i < kFewWarps; ++i) s += part[i][tok][lane];
            part[0][tok][lane] = s;
        }
        few_cluster_store(W, part[0], m, tile, sa, y, y_stride);
        return;
    }
    // every warp takes tokens of its tile
    const int64_t channel = tile * 32 + lane;
    if (channel >= W.rows) return;
    for (int tok = share; tok < m; tok += S) {
        int s = 0;
        for (int i = 0; i < S; ++i) s += part[own * S + i][tok][lane];
        y[tok * y_stride + channel] = i8_scaled<T>(s, __ldca(sa + tok), W.scale[channel]);
    }
}

// grid.x CTAs in clusters of `size` along y, and z of those. The launch may overlap the end of the kernel before, whose
// outputs are read behind pdl_wait, and not by read-only loads. i8_row_kernel lets the next launch overlap all of its own
// (28672 x 4096 19.2 -> 18.7 us, 960 x 576 2.1 -> 1.8); after i8_few_kernel its CTAs would take the places that come free
// first, and leave SMs with too many and too few (8 tokens over 4096 x 14336 14.3 us, so 16.4).
template <typename... KArgs, typename... Args>
static cudaError_t launch_few(void (*kernel)(KArgs...), int64_t x, int64_t size, int64_t z, int threads, cudaStream_t s,
                              Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)x, (unsigned)size, (unsigned)z);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (size > 1) {
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = 1;
        attr[1].val.clusterDim.y = (unsigned)size;
        attr[1].val.clusterDim.z = 1;
        cfg.numAttrs = 2;
    }
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <typename T>
static cudaError_t launch_i8_few(const I8Weights& W, const int8_t* a, const float* sa, int m, T* y, int64_t y_stride,
                                 cudaStream_t s) {
    const int64_t tiles = W.rows_pad / 32, blocks = (W.chunks + 3) / 4;
    // A cluster per tile where the tiles leave SMs empty, of CTAs enough for four per SM, with at least `least` blocks of
    // k for each warp (4096 x 14336, one token: 42 us without clusters, 12.8 us with 4 CTAs, 17.9 with 8).
    auto cluster = [&](int warps, int64_t least) {
        const int64_t fit = 152 * 4 / tiles, k = blocks / (least * warps), c = fit < k ? fit : k;
        return c < 1 ? 1 : c > 8 ? 8 : c;
    };
    if (m == 1) return launch_few(i8_row_kernel<T>, tiles, cluster(kRowWarps, 1), 1, kRowWarps * 32, s, W, a, sa, y, y_stride);
    // warps of a CTA on one tile: two blocks each while the SMs are not full, else eight
    int S = 1;
    while (S < kFewWarps && blocks >= (tiles * 2 * S > 152 * 24 ? 8 : 2) * S) S *= 2;
    const int64_t c = S == kFewWarps ? cluster(kFewWarps, 2) : 1, x = (tiles * S + kFewWarps - 1) / kFewWarps;
    auto go = [&](auto kernel, int each) {
        return launch_few(kernel, x, c, (m + each - 1) / each, kFewWarps * 32, s, W, a, sa, m, S, y, y_stride);
    };
    return m <= 8 ? go(i8_few_kernel<1, T>, 8) : m <= 16 ? go(i8_few_kernel<2, T>, 16) : go(i8_few_kernel<4, T>, 32);
}

// Whether a product goes to the tensor cores' matrix kernel (i8_gemm.cu). Up to 16 tokens the kernels above are as fast or
// faster; with small matrices, which the groups of 32 tokens read again from L2, further on, as they take no launch, ring
// and tensor memory to set up (matrix kernel / these, in us: 32 tokens over 4096 x 2048, 4096 blocks of 32 channels x 64 k,
// 8.3 / 7.7, over 4096 x 4096 10.2 / 10.5; 64 over 2048 x 2048 7.9 / 7.7, over 4096 x 2048 9.1 / 14.4; 128 over 576 x 1536,
// 432 blocks, 7.8 / 6.5, over 2048 x 2048 9.7 / 14.4).
static bool i8_on_gemm(int64_t rows, int64_t k, int64_t m) {
    const int64_t blocks = (rows + 31) / 32 * ((k + 63) / 64);
    return m > 16 && (m > 32 ? m > 128 || (m + 31) / 32 * blocks > 4096 : blocks >= 8192);
}

template <typename T>
static llama_q8_status launch_i8_matmul(const I8Weights& W, int64_t k, const int8_t* a, const float* sa, int64_t m, void* y,
                                        int64_t y_stride, void* workspace, size_t workspace_bytes, int32_t* err,
                                        cudaStream_t s) {
    if (i8_on_gemm(W.rows, k, m))
        return launch_i8_gemm(W, k, a, sa, m, reinterpret_cast<T*>(y), y_stride, workspace, workspace_bytes, err, s);
    return launch_i8_few(W, a, sa, (int)m, reinterpret_cast<T*>(y), y_stride, s) == cudaSuccess ? LQ8_OK : LQ8_ERR_CUDA;
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
    return !i8_sizes_ok(rows, k) || m > (1ll << 30) || !i8_on_gemm(rows, k, m) ? 0 : i8_gemm_workspace(k, m);
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
    if (m == 0) return LQ8_OK;
    const I8Weights w = i8_view(packed, rows, k);
    cudaStream_t s = (cudaStream_t)stream;
    if (type == LLAMA_Q8_GGUF_F32)
        return launch_i8_matmul<float>(w, k, codes, scale, m, y, y_stride, workspace, workspace_bytes, err, s);
    if (type == LLAMA_Q8_GGUF_F16)
        return launch_i8_matmul<__half>(w, k, codes, scale, m, y, y_stride, workspace, workspace_bytes, err, s);
    return launch_i8_matmul<__nv_bfloat16>(w, k, codes, scale, m, y, y_stride, workspace, workspace_bytes, err, s);
}

}  // extern "C"
