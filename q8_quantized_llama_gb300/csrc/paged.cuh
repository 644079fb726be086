// The paged KV cache as the kernels see it: one layer of a pool, element types
// and the checks shared by the entry points.
#pragma once

#include <cmath>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "llama_q8.h"

namespace lq8 {

constexpr int kPageMin = 8, kPageMax = 256;

// Every workspace starts with the completion counters, in an area of one size,
// so that no call's data lie where another call (of other sizes, or of another
// operator) has its counters.
constexpr int kMaxCounters = 65536;
constexpr size_t kCounterBytes = 4 * (size_t)kMaxCounters;

inline int page_type_bytes(int type) {
    return type == LLAMA_Q8_GGUF_F32 ? 4 : (type == LLAMA_Q8_GGUF_F16 || type == LLAMA_Q8_GGUF_BF16) ? 2 : 0;
}

// One layer of a pool. page_elems = n_kv * page * head_dim values per page.
template <typename T>
struct PageView {
    T* k;
    T* v;
    int n_pages, page_shift, n_kv;
    int64_t page_elems;
};

// Page table of the sequences; entries outside [0, n_pages) are holes.
struct TableView {
    const int32_t* table;
    int n_seq, stride;
};

inline int log2_of(int x) {
    int s = 0;
    while ((1 << s) < x) ++s;
    return s;
}

// LQ8_OK, or what is wrong with a pool's description.
inline llama_q8_status check_pages(const llama_q8_pages* p) {
    if (!p || !p->k || !p->v || p->n_layer <= 0 || p->n_pages <= 0 || p->n_head_kv <= 0) return LQ8_ERR_ARG;
    if (!page_type_bytes(p->type)) return LQ8_ERR_UNSUPPORTED;
    if (p->page < kPageMin || p->page > kPageMax || (p->page & (p->page - 1))) return LQ8_ERR_UNSUPPORTED;
    if (p->head_dim != 64 && p->head_dim != 128) return LQ8_ERR_UNSUPPORTED;
    if (((uintptr_t)p->k | (uintptr_t)p->v) & 15) return LQ8_ERR_ARG;
    return LQ8_OK;
}

template <typename T>
inline PageView<T> page_view(const llama_q8_pages* p, int layer) {
    PageView<T> w;
    w.page_elems = (int64_t)p->n_head_kv * p->page * p->head_dim;
    const int64_t off = (int64_t)layer * p->n_pages * w.page_elems;
    w.k = reinterpret_cast<T*>(p->k) + off;
    w.v = reinterpret_cast<T*>(p->v) + off;
    w.n_pages = p->n_pages;
    w.page_shift = log2_of(p->page);
    w.n_kv = p->n_head_kv;
    return w;
}

// Arrival at a counter: the caller's CTA has written its part (and passed a CTA
// barrier); the CTA that gets the last number sees every other's part.
__device__ __forceinline__ unsigned take_ticket(unsigned int* counter, unsigned n = 1) {
    unsigned old;
    asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], %2;" : "=r"(old) : "l"(counter), "r"(n) : "memory");
    return old;
}

// Report a status found on the device: the largest one stays.
__device__ __forceinline__ void report(int32_t* err, int status) {
    if (err) atomicMax(err, status);
}

__device__ __forceinline__ int page_of(const TableView& t, int seq, int block, int n_pages) {
    const int p = t.table[(int64_t)seq * t.stride + block];
    return p < n_pages ? p : -1;
}

}  // namespace lq8
