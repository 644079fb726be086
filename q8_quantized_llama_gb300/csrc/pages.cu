// Bookkeeping of a page pool on the device: forking (with extension and
// freeing) and compaction. Two launches each.
//
// A plan kernel of one CTA decides everything that depends on everything: how
// many pages each child needs (a scan over the children in order), which free
// pages they get, or which page moves where (a scan over the counts in order;
// ballots turn 32 coalesced loads per lane into a rank per page, 32768 pages
// per pass). Order makes the result a function of the inputs alone: no atomic
// decides a page number. The second kernel, launched to start as the plan ends,
// does what is independent per entry: table rows, counts and the page copies,
// spread over the GPU by warps.
//
// Bound: the plan's chain of dependent loads and the hand-over (about 8 us), then
// the copies at the memory's rate; where few pages are copied, the first alone.
// 36 rows of a pool of 8x128, 32 layers, compacted: 120 us (721 MB, 6.0 TB/s); 24
// rows of 3x64, 30 layers: 26 us (108 MB). Fork of 16 groups of 4 beams on the
// first pool: 51 us, its copies 42 (children of one parent read their page from
// L2); of 4 x 4 on the second: 10 us, 7.8 of them on the GPU.
// Not built: small pools in one launch, each CTA making the plan for itself (the
// plan depends only on arrays that the call does not write).
#include <algorithm>

#include "kernels.cuh"
#include "paged.cuh"
#include "ptx.cuh"

namespace lq8 {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanChunk = kPlanThreads * 32;  // counts ranked per pass at most
constexpr int kMoveThreads = 256;
constexpr int kMoveCtas = 152 * 4;
constexpr int kMaxForkRows = 65536;

// Exclusive scan of v over the CTA's 1024 threads; *total gets the sum.
__device__ __forceinline__ int block_scan(int v, int* warp_sums, int* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();  // warp_sums of an earlier scan are no longer read
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    int w = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += y;
    }
    *total = __shfl_sync(0xffffffffu, w, 31);
    const int before = __shfl_sync(0xffffffffu, w, (warp + 31) & 31);
    return (warp ? before : 0) + x - v;
}

// One page copy of a fork: n_rows valid positions of page src to page dst.
struct ForkCopy {
    int32_t src, dst, n_rows;
};
struct PlanHeader {
    int32_t ok, n_copies;
};

struct ForkArgs {
    int rows_in, rows_out, width, page_shift, n_pages, reserve;
    const int32_t *len_in, *table_in, *refs_in, *parent;
    int32_t *len_out, *table_out, *refs_out, *err;
    // workspace
    PlanHeader* head;
    int32_t *first, *kids;  // [rows_in]: lowest child, number of children
    int32_t* base;          // [rows_out]: the child's first entry of `fresh`
    ForkCopy* copies;       // [rows_out]
    int32_t* fresh;         // free pages in the order they are given out
};

size_t fork_workspace(int rows_in, int rows_out, int width, ForkArgs* a, void* ws) {
    size_t o = kCounterBytes;
    auto take = [&](size_t bytes) {
        const size_t at = o;
        o += (bytes + 255) / 256 * 256;
        return at;
    };
    const size_t h = take(sizeof(PlanHeader)), f = take(4 * (size_t)rows_in), k = take(4 * (size_t)rows_in),
                 b = take(4 * (size_t)rows_out), c = take(sizeof(ForkCopy) * (size_t)rows_out),
                 g = take(4 * (size_t)rows_out * width);
    if (a) {
        uint8_t* w = reinterpret_cast<uint8_t*>(ws);
        a->head = reinterpret_cast<PlanHeader*>(w + h);
        a->first = reinterpret_cast<int32_t*>(w + f);
        a->kids = reinterpret_cast<int32_t*>(w + k);
        a->base = reinterpret_cast<int32_t*>(w + b);
        a->copies = reinterpret_cast<ForkCopy*>(w + c);
        a->fresh = reinterpret_cast<int32_t*>(w + g);
    }
    return o;
}

// The page of entry b of a parent's row, -1 for a hole or a number out of range.
__device__ __forceinline__ int held_page(const ForkArgs& a, int row, int b) {
    const int t = a.table_in[(int64_t)row * a.width + b];
    return t < a.n_pages ? (t < 0 ? -1 : t) : -1;
}

// Counts per lane and pass: a warp has 32 * j_n consecutive pages, w0 + j * 32 + lane.
__device__ __forceinline__ int counts_per_lane(int n_pages) {
    return min(32, (n_pages + kPlanThreads - 1) / kPlanThreads);
}
__device__ __forceinline__ void load_counts(int (&v)[32], const int32_t* refs, int w0, int j_n, int n_pages, int lane) {
#pragma unroll
    for (int j = 0; j < 32; ++j) {
        if (j >= j_n) break;
        const int p = w0 + j * 32 + lane;
        v[j] = p < n_pages ? refs[p] : -1;
    }
}

// The chains of dependent loads are what this kernel waits for: the counts of
// the first pass are asked for before anything else, the children are counted
// in shared memory (for up to kSharedRows parents), and copies learn their page
// from a list there.
constexpr int kSharedRows = 2048, kSharedFresh = 2048;

__global__ void __launch_bounds__(kPlanThreads) fork_plan_kernel(ForkArgs a) {
    __shared__ int warp_sums[32];
    __shared__ int s_bad, s_first[kSharedRows], s_kids[kSharedRows], s_fresh[kSharedFresh];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_launch_dependents();  // the second kernel's CTAs take their places and wait
    const int j_n = counts_per_lane(a.n_pages);
    int v[32];
    load_counts(v, a.refs_in, warp * 32 * j_n, j_n, a.n_pages, lane);
    const int p0 = tid < a.rows_out ? a.parent[tid] : -1;  // of the first 1024 children
    if (tid == 0) s_bad = 0;
    int* first = a.rows_in <= kSharedRows ? s_first : a.first;
    int* kids = a.rows_in <= kSharedRows ? s_kids : a.kids;
    for (int p = tid; p < a.rows_in; p += kPlanThreads) {
        first[p] = INT32_MAX;
        kids[p] = 0;
    }
    __syncthreads();
    for (int i = tid; i < a.rows_out; i += kPlanThreads) {
        const int p = i == tid ? p0 : a.parent[i];
        if (p < -1 || p >= a.rows_in) {
            atomicMax(&s_bad, (int)LQ8_ERR_ARG);
        } else if (p >= 0) {
            atomicMin(first + p, i);
            atomicAdd(kids + p, 1);
        }
    }
    __syncthreads();
    if (first == s_first) {
        for (int p = tid; p < a.rows_in; p += kPlanThreads) {
            a.first[p] = s_first[p];
            a.kids[p] = s_kids[p];
        }
    }
    // pages each child needs, in the children's order
    int need_all = 0, n_copies = 0;
    for (int i0 = 0; i0 < a.rows_out; i0 += kPlanThreads) {
        const int i = i0 + tid;
        int fresh = 0, src = -1, part = 0;
        if (i < a.rows_out) {
            const int p = i0 == 0 ? p0 : a.parent[i];
            int n = 0;
            if (p >= 0 && p < a.rows_in) {
                n = a.len_in[p];
                const int64_t top = (int64_t)a.width << a.page_shift;
                if (n < 0 || (int64_t)n + a.reserve > top) {
                    atomicMax(&s_bad, (int)LQ8_ERR_CTX);
                } else {
                    const int page = 1 << a.page_shift, full = n >> a.page_shift;
                    const int need = (int)(((int64_t)n + a.reserve + page - 1) >> a.page_shift);
                    part = n & (page - 1);
                    // (atomics on global memory leave older values in L1)
                    if ((first == s_first ? s_first[p] : __ldcg(a.first + p)) == i) {
                        for (int b = full; b < need; ++b) {
                            const int t = held_page(a, p, b);
                            if (t >= 0 && a.refs_in[t] == 1) continue;
                            if (b == full && part > 0) src = t;
                            ++fresh;
                        }
                    } else {
                        fresh = max(0, need - full);
                        if (fresh > 0 && part > 0) src = held_page(a, p, full);
                    }
                }
            }
            a.len_out[i] = n;
        }
        int total, copies;
        const int at = need_all + block_scan(fresh, warp_sums, &total);
        const int c = n_copies + block_scan(src >= 0, warp_sums, &copies);
        if (i < a.rows_out) a.base[i] = at;
        if (src >= 0) a.copies[c] = ForkCopy{src, at, part};  // dst: its place in `fresh` for now
        need_all += total;
        n_copies += copies;
        // each of at most rows_out * width < 2^31 entries asks for one page
    }
    // the lowest free pages, and the counts as they were
    int found = 0;
    for (int c0 = 0; c0 < a.n_pages; c0 += kPlanThreads * j_n) {
        const int w0 = c0 + warp * 32 * j_n;
        if (c0 > 0) load_counts(v, a.refs_in, w0, j_n, a.n_pages, lane);
        unsigned mine = 0;
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            if (j >= j_n) break;
            const int p = w0 + j * 32 + lane;
            if (p < a.n_pages) a.refs_out[p] = v[j];
            const unsigned m = __ballot_sync(0xffffffffu, v[j] == 0);
            if (lane == j) mine = m;
        }
        int total;
        int at = found + block_scan(__popc(mine), warp_sums, &total);
        for (; mine && at < need_all; mine &= mine - 1, ++at) {
            const int p = w0 + lane * 32 + __ffs(mine) - 1;
            a.fresh[at] = p;
            if (at < kSharedFresh) s_fresh[at] = p;
        }
        found += total;
    }
    __syncthreads();
    if (found < need_all && tid == 0) atomicMax(&s_bad, (int)LQ8_ERR_OOM);
    __syncthreads();
    if (tid == 0) {
        a.head->ok = s_bad == 0;
        a.head->n_copies = n_copies;
        if (s_bad) report(a.err, s_bad);
    }
    if (s_bad) return;
    for (int c = tid; c < n_copies; c += kPlanThreads) {
        const int at = a.copies[c].dst;
        a.copies[c].dst = at < kSharedFresh ? s_fresh[at] : a.fresh[at];
    }
}

// Bytes [0, n) (a multiple of 16) from src to dst by one warp, eight 16-byte pieces in flight per lane.
__device__ __forceinline__ void warp_copy(uint8_t* dst, const uint8_t* src, int n, int lane) {
    const uint4* s = reinterpret_cast<const uint4*>(src);
    uint4* d = reinterpret_cast<uint4*>(dst);
    const int m = n >> 4;
    for (int i0 = lane; i0 < m; i0 += 8 * 32) {
        uint4 v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (i0 + j * 32 < m) v[j] = ld_stream_u4(s + i0 + j * 32);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (i0 + j * 32 < m) __stcs(d + i0 + j * 32, v[j]);
    }
}

struct PoolBytes {
    uint8_t *k, *v;
    int n_layer, n_kv;
    int64_t page_bytes, layer_bytes;
    int row_bytes, head_bytes;  // one position, one head of a page
};

__global__ void __launch_bounds__(kMoveThreads) fork_apply_kernel(ForkArgs a, PoolBytes pool) {
    pdl_wait();
    if (!a.head->ok) return;
    const int lane = threadIdx.x & 31, warps = kMoveThreads / 32;
    // warps spread over the CTAs first
    const int warp = (threadIdx.x >> 5) * gridDim.x + blockIdx.x;
    const int n_warps = gridDim.x * warps;
    // one warp per child: its table row; one per parent: the counts of its pages
    for (int job = warp; job < a.rows_out + a.rows_in; job += n_warps) {
        if (job < a.rows_out) {
            const int p = a.parent[job];
            const int n = p >= 0 ? a.len_in[p] : 0;
            const int full = n >> a.page_shift;
            const int need = p >= 0 ? (int)(((int64_t)n + a.reserve + (1 << a.page_shift) - 1) >> a.page_shift) : 0;
            const bool first = p >= 0 && a.first[p] == job;
            int next = a.base[job];
            int32_t* to = a.table_out + (int64_t)job * a.width;
            for (int b0 = 0; b0 < a.width; b0 += 8 * 32) {
                int t[8], c[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int b = b0 + j * 32 + lane;
                    t[j] = p >= 0 && b < a.width ? held_page(a, p, b) : -1;
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int b = b0 + j * 32 + lane;
                    c[j] = first && b >= full && t[j] >= 0 ? a.refs_in[t[j]] : 0;
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int b = b0 + j * 32 + lane;
                    const bool kept = b < full || c[j] == 1;
                    const bool fresh = !kept && b < need;
                    const unsigned m = __ballot_sync(0xffffffffu, fresh);
                    int e = kept ? t[j] : -1;
                    if (fresh) {
                        e = a.fresh[next + __popc(m & ((1u << lane) - 1))];
                        a.refs_out[e] = 1;
                    }
                    if (b < a.width) to[b] = e;
                    next += __popc(m);
                }
            }
        } else {
            const int p = job - a.rows_out, kids = a.kids[p], n = a.len_in[p];
            const int full = kids > 0 ? n >> a.page_shift : a.width;
            for (int b0 = 0; b0 < a.width; b0 += 32) {
                const int b = b0 + lane;
                if (b >= a.width) continue;
                const int raw = a.table_in[(int64_t)p * a.width + b];
                if (raw >= a.n_pages) report(a.err, LQ8_ERR_ARG);
                if (raw < 0 || raw >= a.n_pages) continue;
                // shared blocks: one count per child instead of the parent's; from `full` on the first child
                // has taken the count over where it is the only one
                const int d = b < full ? kids - 1 : (a.refs_in[raw] == 1 ? 0 : -1);
                if (d) atomicAdd(a.refs_out + raw, d);
            }
        }
    }
    const int per_copy = pool.n_layer * 2 * pool.n_kv;
    const int64_t units = (int64_t)a.head->n_copies * per_copy;
    // from the warps that had no job on
    const int jobs = min(n_warps - 1, a.rows_out + a.rows_in);
    for (int64_t u = warp < jobs ? warp + n_warps - jobs : warp - jobs; u < units; u += n_warps) {
        const int c = (int)(u / per_copy);
        int r = (int)(u % per_copy);
        const int h = r % pool.n_kv;
        r /= pool.n_kv;
        const ForkCopy cp = a.copies[c];
        uint8_t* base = ((r & 1) ? pool.v : pool.k) + (r >> 1) * pool.layer_bytes + (int64_t)h * pool.head_bytes;
        warp_copy(base + cp.dst * pool.page_bytes, base + cp.src * pool.page_bytes, cp.n_rows * pool.row_bytes, lane);
    }
}

// ---------------------------------------------------------------------------

struct CompactArgs {
    int rows, width, n_pages;
    const int32_t *table_in, *refs_in;
    int32_t *table_out, *refs_out, *n_used, *err;
    // workspace
    int32_t* n_moves;
    int32_t *to;           // [n_pages] new number, -1: free
    int32_t *from, *hole;  // [n_pages / 2 + 1]
};

size_t compact_workspace(int n_pages, CompactArgs* a, void* ws) {
    const size_t all = (4 * (size_t)n_pages + 255) / 256 * 256, part = (4 * ((size_t)n_pages / 2 + 1) + 255) / 256 * 256;
    if (a) {
        uint8_t* w = reinterpret_cast<uint8_t*>(ws) + kCounterBytes;
        a->n_moves = reinterpret_cast<int32_t*>(w);
        a->to = reinterpret_cast<int32_t*>(w + 256);
        a->from = reinterpret_cast<int32_t*>(w + 256 + all);
        a->hole = reinterpret_cast<int32_t*>(w + 256 + all + part);
    }
    return kCounterBytes + 256 + all + 2 * part;
}

__global__ void __launch_bounds__(kPlanThreads) compact_plan_kernel(CompactArgs a) {
    __shared__ int warp_sums[32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_launch_dependents();
    const int j_n = counts_per_lane(a.n_pages), step = kPlanThreads * j_n;
    int v[32];
    // bit b of lane l's word: page w0 + l * 32 + b is in use
    auto words = [&](int w0) {
        load_counts(v, a.refs_in, w0, j_n, a.n_pages, lane);
        unsigned mine = 0;
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            if (j >= j_n) break;
            const unsigned m = __ballot_sync(0xffffffffu, v[j] > 0);
            if (lane == j) mine = m;
        }
        return mine;
    };
    unsigned word = 0;
    int n = 0, used;
    for (int c0 = 0; c0 < a.n_pages; c0 += step) {
        word = words(c0 + warp * 32 * j_n);
        n += __popc(word);
    }
    block_scan(n, warp_sums, &used);
    // holes below `used`, pages in use from there on: as many of one as of the other
    int moves = 0, holes = 0;
    for (int c0 = 0; c0 < a.n_pages; c0 += step) {
        const int w0 = c0 + warp * 32 * j_n;
        if (a.n_pages > kPlanChunk) word = words(w0);  // of one pass the word is still there
        const int below = lane < j_n ? min(32, max(0, used - (w0 + lane * 32))) : 0;
        const unsigned low = below == 32 ? ~0u : (1u << below) - 1;
        unsigned hole = ~word & low, from = word & ~low;
        int total;
        int at = holes + block_scan(__popc(hole), warp_sums, &total);
        holes += total;
        for (; hole; hole &= hole - 1) a.hole[at++] = w0 + lane * 32 + __ffs(hole) - 1;
        at = moves + block_scan(__popc(from), warp_sums, &total);
        moves += total;
        for (; from; from &= from - 1) a.from[at++] = w0 + lane * 32 + __ffs(from) - 1;
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            if (j >= j_n) break;
            const int p = w0 + j * 32 + lane;
            if (p < a.n_pages) {
                const bool in = v[j] > 0, stays = in && p < used;
                if (!in || stays) a.to[p] = stays ? p : -1;
                if (stays || p >= used) a.refs_out[p] = stays ? v[j] : 0;
            }
        }
    }
    __syncthreads();
    for (int m = tid; m < moves; m += kPlanThreads) {
        const int f = a.from[m], h = a.hole[m];
        a.to[f] = h;
        a.refs_out[h] = a.refs_in[f];
    }
    if (tid == 0) {
        *a.n_moves = moves;
        *a.n_used = used;
    }
}

constexpr int kMovePiece = 8192;

__global__ void __launch_bounds__(kMoveThreads) compact_apply_kernel(CompactArgs a, PoolBytes pool) {
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int warp = (threadIdx.x >> 5) * gridDim.x + blockIdx.x, n_warps = gridDim.x * (kMoveThreads / 32);
    const int64_t entries = (int64_t)a.rows * a.width;
    for (int64_t e = (int64_t)blockIdx.x * kMoveThreads + threadIdx.x; e < entries;
         e += (int64_t)gridDim.x * kMoveThreads) {
        const int t = a.table_in[e];
        int to = -1;
        if (t >= 0) {
            if (t < a.n_pages) to = a.to[t];
            if (to < 0) report(a.err, LQ8_ERR_ARG);
        }
        a.table_out[e] = to;
    }
    const int pieces = (int)((pool.page_bytes + kMovePiece - 1) / kMovePiece);
    const int per_move = pool.n_layer * 2 * pieces;
    const int64_t units = (int64_t)*a.n_moves * per_move;
    for (int64_t u = warp; u < units; u += n_warps) {
        const int m = (int)(u / per_move);
        int r = (int)(u % per_move);
        const int64_t off = (int64_t)(r % pieces) * kMovePiece;
        r /= pieces;
        uint8_t* base = ((r & 1) ? pool.v : pool.k) + (r >> 1) * pool.layer_bytes + off;
        warp_copy(base + a.hole[m] * pool.page_bytes, base + a.from[m] * pool.page_bytes,
                  (int)min((int64_t)kMovePiece, pool.page_bytes - off), lane);
    }
}

PoolBytes pool_bytes(const llama_q8_pages* p) {
    PoolBytes b;
    b.k = reinterpret_cast<uint8_t*>(p->k);
    b.v = reinterpret_cast<uint8_t*>(p->v);
    b.n_layer = p->n_layer;
    b.n_kv = p->n_head_kv;
    b.row_bytes = p->head_dim * page_type_bytes(p->type);
    b.head_bytes = b.row_bytes * p->page;
    b.page_bytes = (int64_t)b.head_bytes * p->n_head_kv;
    b.layer_bytes = b.page_bytes * p->n_pages;
    return b;
}

bool misaligned(const void* p) { return ((uintptr_t)p & 3) != 0; }

// Units of copy work are counted in 32 bits per page: layers * 2 * heads (or pieces). The plans' passes over the counts
// step past n_pages in 32 bits.
bool pool_too_large(const llama_q8_pages* p) {
    return p->n_pages > (1 << 30) || (int64_t)p->n_layer * p->n_head_kv > (1 << 24) ||
           (int64_t)p->n_head_kv * p->page * p->head_dim * 4 > (int64_t)1 << 36;
}

}  // namespace
}  // namespace lq8

using namespace lq8;

extern "C" {

size_t llama_q8_pages_fork_workspace_bytes(int32_t rows_in, int32_t rows_out, int32_t table_stride) {
    if (rows_in <= 0 || rows_out <= 0 || table_stride <= 0) return 0;
    return fork_workspace(rows_in, rows_out, table_stride, nullptr, nullptr);
}

llama_q8_status llama_q8_pages_fork(const llama_q8_pages* pages, int32_t rows_in, const int32_t* len_in,
                                    const int32_t* table_in, int32_t table_stride, const int32_t* refs_in,
                                    int32_t rows_out, const int32_t* parent, int32_t reserve, int32_t* len_out,
                                    int32_t* table_out, int32_t* refs_out, void* workspace, size_t workspace_bytes,
                                    int32_t* err, void* stream) {
    const llama_q8_status st = check_pages(pages);
    if (st != LQ8_OK) return st;
    if (!len_in || !table_in || !refs_in || !parent || !len_out || !table_out || !refs_out || !workspace || !err ||
        rows_in <= 0 || rows_out <= 0 || table_stride <= 0 || reserve < 0)
        return LQ8_ERR_ARG;
    if (len_in == len_out || table_in == table_out || refs_in == refs_out) return LQ8_ERR_ARG;
    if (misaligned(len_in) || misaligned(table_in) || misaligned(refs_in) || misaligned(parent) ||
        misaligned(len_out) || misaligned(table_out) || misaligned(refs_out) || misaligned(err) ||
        ((uintptr_t)workspace & 15))
        return LQ8_ERR_ARG;
    if (rows_in > kMaxForkRows || rows_out > kMaxForkRows || pool_too_large(pages) ||
        (int64_t)rows_out * table_stride > INT32_MAX || (int64_t)rows_in * table_stride > INT32_MAX)
        return LQ8_ERR_UNSUPPORTED;
    ForkArgs a{};
    if (workspace_bytes < fork_workspace(rows_in, rows_out, table_stride, &a, workspace)) return LQ8_ERR_ARG;
    a.rows_in = rows_in, a.rows_out = rows_out, a.width = table_stride, a.page_shift = log2_of(pages->page);
    a.n_pages = pages->n_pages, a.reserve = reserve;
    a.len_in = len_in, a.table_in = table_in, a.refs_in = refs_in, a.parent = parent;
    a.len_out = len_out, a.table_out = table_out, a.refs_out = refs_out, a.err = err;
    cudaStream_t s = (cudaStream_t)stream;
    if (launch_ex(fork_plan_kernel, dim3(1), dim3(kPlanThreads), 0, s, false, a) != cudaSuccess) return LQ8_ERR_CUDA;
    return launch_ex(fork_apply_kernel, dim3(kMoveCtas), dim3(kMoveThreads), 0, s, true, a, pool_bytes(pages)) ==
                   cudaSuccess
               ? LQ8_OK
               : LQ8_ERR_CUDA;
}

size_t llama_q8_pages_compact_workspace_bytes(int32_t n_pages) {
    return n_pages > 0 ? compact_workspace(n_pages, nullptr, nullptr) : 0;
}

llama_q8_status llama_q8_pages_compact(const llama_q8_pages* pages, int32_t rows, const int32_t* table_in,
                                       int32_t table_stride, const int32_t* refs_in, int32_t* table_out,
                                       int32_t* refs_out, int32_t* n_used, void* workspace, size_t workspace_bytes,
                                       int32_t* err, void* stream) {
    const llama_q8_status st = check_pages(pages);
    if (st != LQ8_OK) return st;
    if (!refs_in || !refs_out || !n_used || !workspace || !err || rows < 0 || refs_in == refs_out) return LQ8_ERR_ARG;
    if (rows > 0 && (!table_in || !table_out || table_stride <= 0 || table_in == table_out)) return LQ8_ERR_ARG;
    if (misaligned(table_in) || misaligned(refs_in) || misaligned(table_out) || misaligned(refs_out) ||
        misaligned(n_used) || misaligned(err) || ((uintptr_t)workspace & 15))
        return LQ8_ERR_ARG;
    if (pool_too_large(pages)) return LQ8_ERR_UNSUPPORTED;
    CompactArgs a{};
    if (workspace_bytes < compact_workspace(pages->n_pages, &a, workspace)) return LQ8_ERR_ARG;
    a.rows = rows, a.width = table_stride, a.n_pages = pages->n_pages;
    a.table_in = table_in, a.refs_in = refs_in, a.table_out = table_out, a.refs_out = refs_out;
    a.n_used = n_used, a.err = err;
    cudaStream_t s = (cudaStream_t)stream;
    if (launch_ex(compact_plan_kernel, dim3(1), dim3(kPlanThreads), 0, s, false, a) != cudaSuccess)
        return LQ8_ERR_CUDA;
    return launch_ex(compact_apply_kernel, dim3(kMoveCtas), dim3(kMoveThreads), 0, s, true, a, pool_bytes(pages)) ==
                   cudaSuccess
               ? LQ8_OK
               : LQ8_ERR_CUDA;
}

}  // extern "C"
