// Grouped-query attention of single tokens over the pages of a KV cache.
//
// For a row and KV head: s_j = scale q . k_j over the visible positions, m =
// max s, l = sum exp(s_j - m), out = sum exp(s_j - m) v_j / l, lse = m + ln l.
// One CTA per (KV head, row) goes through the positions in tiles of 32 with a
// running maximum and sum.
#include "kernels.cuh"
#include "paged.cuh"

namespace lq8 {
namespace {

constexpr int kTile = 32, kThreads = 128, kMaxG = 8;

struct AttnArgs {
    const float* q;
    const int32_t* pos;
    const int32_t* seq;
    int n_head;
    float scale;
    int window;
    float* out;
    float* lse;
    int32_t* err;
};

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }

template <typename T, int HD>
__global__ void __launch_bounds__(kThreads) attention_paged_kernel(AttnArgs a, PageView<T> pg, TableView tb) {
    __shared__ float ks[kTile][HD + 1], vs[kTile][HD], qs[kMaxG][HD], ps[kMaxG][kTile];
    __shared__ float sm[kMaxG], sl[kMaxG], sc[kMaxG];
    __shared__ int ok[kTile];
    const int kh = blockIdx.x, row = blockIdx.y, tid = threadIdx.x, G = a.n_head / pg.n_kv;
    const int p = a.pos[row], sq = a.seq ? a.seq[row] : row;
    int64_t end = p < 0 ? 0 : (int64_t)p + 1;
    if (end > 0 && (sq < 0 || sq >= tb.n_seq)) {
        if (tid == 0) report(a.err, LQ8_ERR_ARG);
        end = 0;
    }
    const int lo = (int)(a.window > 0 && end > a.window ? end - a.window : 0);
    const int64_t cap = (int64_t)tb.stride << pg.page_shift;
    if (end > cap && tid == 0) report(a.err, LQ8_ERR_CTX);
    const int hi = (int)min(end, cap);
    const int64_t ob = ((int64_t)row * a.n_head + kh * G) * HD;
    for (int i = tid; i < G * HD; i += kThreads) qs[i / HD][i % HD] = a.q[ob + i] * a.scale;
    if (tid < kMaxG) { sm[tid] = -INFINITY; sl[tid] = 0.0f; }
    float acc[kMaxG][HD / 128 ? HD / 128 : 1] = {};
    __syncthreads();
    for (int j0 = lo; j0 < hi; j0 += kTile) {
        const int n = min(kTile, hi - j0);
        for (int i = tid; i < kTile * HD; i += kThreads) {
            const int r = i / HD, d = i % HD;
            float kv = 0.0f, vv = 0.0f;
            bool good = false;
            if (r < n) {
                const int j = j0 + r, page = page_of(tb, sq, j >> pg.page_shift, pg.n_pages);
                if (page >= 0) {
                    const int64_t o = page * pg.page_elems +
                                      (((int64_t)kh << pg.page_shift) + (j & ((1 << pg.page_shift) - 1))) * HD + d;
                    kv = to_f32(pg.k[o]);
                    vv = to_f32(pg.v[o]);
                    good = true;
                } else if (d == 0 && tb.table[(int64_t)sq * tb.stride + (j >> pg.page_shift)] >= pg.n_pages) {
                    report(a.err, LQ8_ERR_ARG);
                }
            }
            ks[r][d] = kv;
            vs[r][d] = vv;
            if (d == 0) ok[r] = good;
        }
        __syncthreads();
        for (int i = tid; i < G * kTile; i += kThreads) {
            const int g = i / kTile, r = i % kTile;
            float s = 0.0f;
            for (int d = 0; d < HD; ++d) s = fmaf(qs[g][d], ks[r][d], s);
            ps[g][r] = ok[r] ? s : -INFINITY;
        }
        __syncthreads();
        const int warp = tid >> 5, lane = tid & 31;
        for (int g = warp; g < G; g += kThreads / 32) {
            const float s = ps[g][lane], m0 = sm[g];
            const float m1 = fmaxf(m0, warp_max(s));
            const float e = m1 == -INFINITY ? 0.0f : expf(s - m1);
            const float c = m1 == -INFINITY ? 0.0f : expf(m0 - m1);
            const float t = warp_sum(e);
            ps[g][lane] = e;
            __syncwarp();
            if (lane == 0) { sm[g] = m1; sl[g] = sl[g] * c + t; sc[g] = c; }
        }
        __syncthreads();
        for (int g = 0; g < G; ++g)
            for (int u = 0; u * kThreads + tid < HD; ++u) {
                float x = acc[g][u] * sc[g];
                for (int r = 0; r < kTile; ++r) x = fmaf(ps[g][r], vs[r][u * kThreads + tid], x);
                acc[g][u] = x;
            }
        __syncthreads();
    }
    for (int g = 0; g < G; ++g) {
        for (int u = 0; u * kThreads + tid < HD; ++u)
            a.out[ob + g * HD + u * kThreads + tid] = sl[g] > 0.0f ? acc[g][u] / sl[g] : 0.0f;
        if (a.lse && tid == 0)
            a.lse[(int64_t)row * a.n_head + kh * G + g] = sl[g] > 0.0f ? sm[g] + logf(sl[g]) : -INFINITY;
    }
}

template <typename T>
cudaError_t launch_attention(const AttnArgs& a, const llama_q8_pages* p, int layer, const TableView& tb, int rows,
                             cudaStream_t s) {
    const dim3 grid(p->n_head_kv, rows);
    if (p->head_dim == 64)
        return launch_ex(attention_paged_kernel<T, 64>, grid, dim3(kThreads), 0, s, false, a, page_view<T>(p, layer), tb);
    return launch_ex(attention_paged_kernel<T, 128>, grid, dim3(kThreads), 0, s, false, a, page_view<T>(p, layer), tb);
}

}  // namespace
}  // namespace lq8

using namespace lq8;

extern "C" {

size_t llama_q8_attention_paged_workspace_bytes(int32_t rows, int32_t n_head, int32_t n_head_kv, int32_t head_dim) {
    if (rows < 0 || n_head <= 0 || n_head_kv <= 0 || n_head % n_head_kv || head_dim <= 0) return 0;
    return 256;
}

llama_q8_status llama_q8_attention_paged(const llama_q8_pages* pages, int32_t layer, const float* q, int32_t rows,
                                         const int32_t* pos, const int32_t* seq, int32_t n_head, float scale,
                                         int32_t window, const int32_t* table, int32_t n_seq, int32_t table_stride,
                                         float* out, float* lse, void* workspace, size_t workspace_bytes, int32_t* err,
                                         void* stream) {
    const llama_q8_status st = check_pages(pages);
    if (st != LQ8_OK) return st;
    if (!q || !pos || !table || !out || !workspace || rows < 0 || n_head <= 0 || n_seq <= 0 || table_stride <= 0 ||
        layer < 0 || layer >= pages->n_layer || n_head % pages->n_head_kv || window < 0)
        return LQ8_ERR_ARG;
    if (!seq && rows > n_seq) return LQ8_ERR_ARG;
    if (!(scale >= 0.0f) || !std::isfinite(scale)) return LQ8_ERR_ARG;
    if (n_head / pages->n_head_kv > kMaxG) return LQ8_ERR_UNSUPPORTED;
    if ((int64_t)rows * pages->n_head_kv >= (1 << 24)) return LQ8_ERR_UNSUPPORTED;
    if (((uintptr_t)q | (uintptr_t)out | (uintptr_t)workspace) & 15) return LQ8_ERR_ARG;
    if (((uintptr_t)pos | (uintptr_t)seq | (uintptr_t)table | (uintptr_t)lse | (uintptr_t)err) & 3) return LQ8_ERR_ARG;
    if (workspace_bytes < llama_q8_attention_paged_workspace_bytes(rows, n_head, pages->n_head_kv, pages->head_dim))
        return LQ8_ERR_ARG;
    if (rows == 0) return LQ8_OK;
    AttnArgs a{q, pos, seq, n_head, scale > 0.0f ? scale : 1.0f / sqrtf((float)pages->head_dim), window, out, lse, err};
    const TableView tb{table, n_seq, table_stride};
    cudaStream_t s = (cudaStream_t)stream;
    cudaError_t e = pages->type == LLAMA_Q8_GGUF_F32   ? launch_attention<float>(a, pages, layer, tb, rows, s)
                    : pages->type == LLAMA_Q8_GGUF_F16 ? launch_attention<__half>(a, pages, layer, tb, rows, s)
                                                       : launch_attention<__nv_bfloat16>(a, pages, layer, tb, rows, s);
    return e == cudaSuccess ? LQ8_OK : LQ8_ERR_CUDA;
}

}  // extern "C"
