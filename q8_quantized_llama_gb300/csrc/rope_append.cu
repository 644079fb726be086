// Rotary positions and the append of keys and values to the pages of a cache,
// one kernel for all rows of a step or a prompt.
//
// A row is [q heads | k heads | v heads] * head_dim floats. Value pairs (x, y)
// of the leading rot_dim values of a q or k head become (x c - y s, x s + y c)
// with c, s = magnitude * cos, sin of pos * freq_i. The product is taken in
// double and reduced to a fraction of a turn there (a position of 2^20 leaves
// an f32 product no digits of the angle); cos and sin of the fraction are f32.
// They are computed once per row and pair into shared memory and used by all
// heads.
//
// Bound: memory. Each thread moves items of 8 values (two 16-byte loads, one or
// two stores): the two halves of 4 pairs for the half layout, so that no value
// is read twice; the loads are issued before the angles are computed, whose
// latency (double multiply, sincospif) they cover. One CTA per row or per eight
// narrow rows, 6 or 5 of them resident per SM (registers). Wide rows of a prompt:
// 8195 of 32/8 heads of 128 into bf16 59.5 us, 6.2 TB/s (with 3, 4, 6 items ahead
// 60.6, 61.5, 83.6). Narrow rows are CTAs of 128 threads or fewer that live for one
// memory latency and a few KB, or, eight in a CTA, for two, as only two of a
// thread's four items are asked for before the barrier: 8195 of 9/3 heads of 64
// into f32 15.4 us in a captured graph, 9.4 for the bytes.
#include <algorithm>

#include "kernels.cuh"
#include "paged.cuh"

namespace lq8 {
namespace {

struct RopeArgs {
    const float* qkv;
    int64_t qkv_stride;
    const int32_t* pos;
    const int32_t* seq;
    int rows, n_head;
    const double* freq;
    int rot_dim, style;
    float magnitude;
    float* q_out;
    int32_t* err;
};

__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void store4(__half* p, float4 v) {
    __half2 h[2] = {__floats2half2_rn(v.x, v.y), __floats2half2_rn(v.z, v.w)};
    *reinterpret_cast<uint2*>(p) = *reinterpret_cast<uint2*>(h);
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 v) {
    __nv_bfloat162 h[2] = {__floats2bfloat162_rn(v.x, v.y), __floats2bfloat162_rn(v.z, v.w)};
    *reinterpret_cast<uint2*>(p) = *reinterpret_cast<uint2*>(h);
}

constexpr int kRopeThreads = 256;
constexpr int kRopeItems = 2;  // items loaded ahead per thread
constexpr int kRopeRows = 8;   // rows per CTA at most

// RC rows per CTA, from row RC * blockIdx.x on.
template <typename T, int HD, int RC>
__global__ void __launch_bounds__(kRopeThreads) rope_append_kernel(RopeArgs a, PageView<T> pg, TableView tb) {
    __shared__ float2 cs_all[RC][HD / 2];
    __shared__ int s_pos[RC], s_page[RC];
    constexpr int IPH = HD / 8;  // items per head
    const int row0 = blockIdx.x * RC, tid = threadIdx.x, threads = blockDim.x;
    const int rows = RC == 1 ? 1 : min(RC, a.rows - row0);
    const int half = a.rot_dim >> 1, rot_items = a.rot_dim >> 3;
    const int heads = a.n_head + 2 * pg.n_kv, per_row = heads * IPH, items = rows * per_row;
    const float* x = a.qkv + row0 * a.qkv_stride;

    // where the first and second four values of item `it` of a head lie
    auto first = [&](int it, bool rot) { return (rot && a.style) ? 4 * it : 8 * it; };
    auto second = [&](int it, bool rot) { return (rot && a.style) ? 4 * it + half : 8 * it + 4; };
    float4 u[kRopeItems], w[kRopeItems];
    auto load = [&](int i0) {
#pragma unroll
        for (int j = 0; j < kRopeItems; ++j) {
            const int i = i0 + j * threads;
            if (i < items) {
                const int r = RC == 1 ? 0 : i / per_row, h = (i - r * per_row) / IPH, it = i % IPH;
                const bool rot = h < a.n_head + pg.n_kv && it < rot_items;
                const float* v = x + r * a.qkv_stride + h * HD;
                u[j] = __ldcs(reinterpret_cast<const float4*>(v + first(it, rot)));
                w[j] = __ldcs(reinterpret_cast<const float4*>(v + second(it, rot)));
            }
        }
    };
    // the position before the row's values: what depends on it does not wait behind their loads
    int p1 = RC == 1 ? a.pos[row0] : 0, page1 = 0;
    if (RC == 1 && p1 < 0) return;  // a padding row
    load(tid);
    auto angle = [&](int r, int k, int p) {
        // in turns: the product and its reduction in double
        const double turns = (double)p * (a.freq[k] * 0.15915494309189533577);  // 1 / 2 pi
        float s, c;
        sincospif(2.0f * (float)(turns - rint(turns)), &s, &c);
        cs_all[r][k] = make_float2(c * a.magnitude, s * a.magnitude);
    };
    if (RC == 1) {
        if (tid < half) angle(0, tid, p1);
    } else {
        for (int i = tid; i < rows * half; i += threads) angle(i / half, i % half, a.pos[row0 + i / half]);
    }
    // the page of a row's position, -1: no append
    auto find_page = [&](int row, int p, bool tell) {
        if (p < 0) return -1;
        const int sq = a.seq ? a.seq[row] : row, block = p >> pg.page_shift;
        int page = -1, status = LQ8_ERR_ARG;
        if (sq >= 0 && sq < tb.n_seq) {
            if (block < tb.stride)
                page = page_of(tb, sq, block, pg.n_pages);
            else
                status = LQ8_ERR_CTX;
        }
        if (page < 0 && tell) report(a.err, status);
        return page;
    };
    if (RC == 1) {
        page1 = find_page(row0, p1, tid == 0);
    } else if (tid < rows) {
        s_pos[tid] = p1 = a.pos[row0 + tid];
        s_page[tid] = find_page(row0 + tid, p1, true);
    }
    __syncthreads();

    for (int i0 = tid; i0 < items;) {
#pragma unroll
        for (int j = 0; j < kRopeItems; ++j) {
            const int i = i0 + j * threads;
            if (i >= items) break;
            const int r = RC == 1 ? 0 : i / per_row, h = (i - r * per_row) / IPH, it = i % IPH;
            const int p = RC == 1 ? p1 : s_pos[r], page = RC == 1 ? page1 : s_page[r];
            if (p < 0) continue;
            const float2* cs = cs_all[r];
            const bool rot = h < a.n_head + pg.n_kv && it < rot_items;
            float4 y = u[j], z = w[j];
            if (rot && a.style) {  // y holds values 4 it .. + 3, z their partners
                const float2 c0 = cs[4 * it], c1 = cs[4 * it + 1], c2 = cs[4 * it + 2], c3 = cs[4 * it + 3];
                y = make_float4(u[j].x * c0.x - w[j].x * c0.y, u[j].y * c1.x - w[j].y * c1.y,
                                u[j].z * c2.x - w[j].z * c2.y, u[j].w * c3.x - w[j].w * c3.y);
                z = make_float4(u[j].x * c0.y + w[j].x * c0.x, u[j].y * c1.y + w[j].y * c1.x,
                                u[j].z * c2.y + w[j].z * c2.x, u[j].w * c3.y + w[j].w * c3.x);
            } else if (rot) {  // pairs side by side
                const float2 c0 = cs[4 * it], c1 = cs[4 * it + 1], c2 = cs[4 * it + 2], c3 = cs[4 * it + 3];
                y = make_float4(u[j].x * c0.x - u[j].y * c0.y, u[j].x * c0.y + u[j].y * c0.x,
                                u[j].z * c1.x - u[j].w * c1.y, u[j].z * c1.y + u[j].w * c1.x);
                z = make_float4(w[j].x * c2.x - w[j].y * c2.y, w[j].x * c2.y + w[j].y * c2.x,
                                w[j].z * c3.x - w[j].w * c3.y, w[j].z * c3.y + w[j].w * c3.x);
            }
            const int o1 = first(it, rot), o2 = second(it, rot);
            if (h < a.n_head) {
                float* q = a.q_out + ((int64_t)(row0 + r) * a.n_head + h) * HD;
                store4(q + o1, y);
                store4(q + o2, z);
            } else if (page >= 0) {
                const int kh = h - a.n_head, slot = p & ((1 << pg.page_shift) - 1);
                const bool is_v = kh >= pg.n_kv;
                T* dst = (is_v ? pg.v : pg.k) + page * pg.page_elems +
                         ((int64_t)((is_v ? kh - pg.n_kv : kh) << pg.page_shift) + slot) * HD;
                store4(dst + o1, y);
                store4(dst + o2, z);
            }
        }
        i0 += kRopeItems * threads;
        load(i0);
    }
}

template <typename T, int HD>
cudaError_t launch_rope_hd(const RopeArgs& a, const llama_q8_pages* p, int layer, const TableView& tb, cudaStream_t s) {
    const int items = (a.n_head + 2 * p->n_head_kv) * (HD / 8);
    const PageView<T> pg = page_view<T>(p, layer);
    // One row per CTA, as many warps as one pass over its items needs (at least those that compute the angles): the
    // shortest call, and the better one while its CTAs are few waves. Rows too narrow to fill a CTA, in longer calls:
    // eight per CTA, from where that is three waves of CTAs (six for heads of 128, whose angles cost more). One
    // and eight, into f32: 14000 rows of 9/3 heads of 64 23.0 and 23.0 us, 8195 15.4 and 16.0, 27000 41.7 and 38.9;
    // 40000 of 4/1 heads of 128 47.6 and 47.8, 20000 25.9 and 27.3, 100000 113 and 110. Rows of 64 items and less fill
    // neither: 100000 of 6/1 heads of 64 77 and 81.
    if (items <= kRopeThreads / 2 && items > kRopeThreads / 4 && a.rows >= 152 * 16 * kRopeRows * (HD / 64))
        return launch_ex(rope_append_kernel<T, HD, kRopeRows>, dim3((a.rows + kRopeRows - 1) / kRopeRows),
                         dim3(kRopeThreads), 0, s, false, a, pg, tb);
    const int threads = std::min(kRopeThreads, std::max((items + 31) / 32 * 32, HD / 2));
    return launch_ex(rope_append_kernel<T, HD, 1>, dim3(a.rows), dim3(threads), 0, s, false, a, pg, tb);
}
template <typename T>
cudaError_t launch_rope(const RopeArgs& a, const llama_q8_pages* p, int layer, const TableView& tb, cudaStream_t s) {
    return p->head_dim == 64 ? launch_rope_hd<T, 64>(a, p, layer, tb, s) : launch_rope_hd<T, 128>(a, p, layer, tb, s);
}

}  // namespace
}  // namespace lq8

using namespace lq8;

extern "C" {

llama_q8_status llama_q8_rope_frequencies(int32_t rot_dim, double theta, const llama_q8_rope_scaling* sc, double* freq,
                                          float* magnitude) {
    if (!sc || !freq || !magnitude || rot_dim < 2 || rot_dim % 2 || !(theta > 0) || !std::isfinite(theta))
        return LQ8_ERR_ARG;
    if (sc->kind < LQ8_ROPE_NONE || sc->kind > LQ8_ROPE_RAMP_M) return LQ8_ERR_ARG;
    const bool ramp = sc->kind == LQ8_ROPE_RAMP || sc->kind == LQ8_ROPE_RAMP_M;
    if (sc->kind != LQ8_ROPE_NONE && !(sc->factor >= 1 && std::isfinite(sc->factor))) return LQ8_ERR_ARG;
    if (sc->kind == LQ8_ROPE_BASE && rot_dim == 2) return LQ8_ERR_ARG;
    if (ramp && !(sc->trained_ctx > 0 && sc->low >= 0 && sc->high > sc->low && std::isfinite(sc->high)))
        return LQ8_ERR_ARG;
    if (sc->kind == LQ8_ROPE_BASE) theta *= std::pow(sc->factor, (double)rot_dim / (rot_dim - 2));
    for (int i = 0; i < rot_dim / 2; ++i) {
        double f = std::pow(theta, -2.0 * i / rot_dim);
        if (sc->kind == LQ8_ROPE_LINEAR) f /= sc->factor;
        if (ramp) {
            const double turns = sc->trained_ctx * f / 6.283185307179586477;
            const double t = (turns - sc->low) / (sc->high - sc->low);
            const double keep = t < 0 ? 0 : t > 1 ? 1 : t;
            f = f * keep + f / sc->factor * (1 - keep);
        }
        freq[i] = f;
    }
    *magnitude = sc->kind == LQ8_ROPE_RAMP_M ? (float)(0.1 * std::log(sc->factor) + 1.0) : 1.0f;
    return LQ8_OK;
}

llama_q8_status llama_q8_rope_append(const llama_q8_pages* pages, int32_t layer, const float* qkv, int64_t qkv_stride,
                                     int32_t rows, const int32_t* pos, const int32_t* seq, int32_t n_head,
                                     const llama_q8_rope* rope, const int32_t* table, int32_t n_seq,
                                     int32_t table_stride, float* q_out, int32_t* err, void* stream) {
    const llama_q8_status st = check_pages(pages);
    if (st != LQ8_OK) return st;
    if (!rope || !rope->freq || !qkv || !pos || !table || !q_out || rows < 0 || n_head <= 0 || n_seq <= 0 ||
        table_stride <= 0 || layer < 0 || layer >= pages->n_layer || n_head % pages->n_head_kv)
        return LQ8_ERR_ARG;
    if (!seq && rows > n_seq) return LQ8_ERR_ARG;
    if (rope->style != 0 && rope->style != 1) return LQ8_ERR_ARG;
    if (!std::isfinite(rope->magnitude)) return LQ8_ERR_ARG;
    if (rope->rot_dim <= 0 || rope->rot_dim % 8 || rope->rot_dim > pages->head_dim) return LQ8_ERR_UNSUPPORTED;
    const int64_t width = ((int64_t)n_head + 2 * (int64_t)pages->n_head_kv) * pages->head_dim;
    if (width > INT32_MAX) return LQ8_ERR_UNSUPPORTED;
    if (qkv_stride < width || qkv_stride % 4) return LQ8_ERR_ARG;
    // rows move in 16-byte pieces
    if (((uintptr_t)qkv | (uintptr_t)q_out) & 15) return LQ8_ERR_ARG;
    if (((uintptr_t)rope->freq & 7) || (((uintptr_t)pos | (uintptr_t)seq | (uintptr_t)table | (uintptr_t)err) & 3))
        return LQ8_ERR_ARG;
    if (rows == 0) return LQ8_OK;
    RopeArgs a{qkv, qkv_stride, pos, seq, rows, n_head, rope->freq, rope->rot_dim, rope->style, rope->magnitude, q_out, err};
    const TableView tb{table, n_seq, table_stride};
    cudaStream_t s = (cudaStream_t)stream;
    cudaError_t e = pages->type == LLAMA_Q8_GGUF_F32   ? launch_rope<float>(a, pages, layer, tb, s)
                    : pages->type == LLAMA_Q8_GGUF_F16 ? launch_rope<__half>(a, pages, layer, tb, s)
                                                       : launch_rope<__nv_bfloat16>(a, pages, layer, tb, s);
    return e == cudaSuccess ? LQ8_OK : LQ8_ERR_CUDA;
}

}  // extern "C"
