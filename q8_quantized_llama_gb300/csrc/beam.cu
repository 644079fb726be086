// Beam search's selection: the n_out best continuations of each group of beams
// over beams x vocabulary, in one kernel that reads the logits once.
//
// total(beam, token) = score[beam] + logit - lse[beam], lse = ln sum exp(logit).
// A CTA takes one chunk of one row's logits into registers and gets from them
// the chunk's maximum, its sum of exponentials and its n_out largest logits:
// within a row totals rise with logits, so no other value of the chunk can be
// chosen. The last CTA of a group to finish (a counter in the workspace) joins
// the chunks' sums in double and picks the n_out largest totals.
//
// Largest of many by a bound: lanes form groups (32, 64 or 128 per CTA, at
// least twice n_out); n_out groups reach the n_out-th largest of the groups'
// maxima, so at least n_out values do, and only a few more. Those few are
// ranked by counting the larger ones, as keys (value, lowest index) that all
// differ. Where equal values leave too many of them (a row of one value, say),
// the bound is taken again over the threads' keys, which leaves at most IT per
// chosen thread.
//
// Bound: memory (each logit read once); issue slots are next: about 8 per value
// (load, maximum, subtract, scale, ex2 and add, packed in pairs where there is
// a packed form, and one comparison).
#include "kernels.cuh"
#include "paged.cuh"

namespace lq8 {
namespace {

constexpr int kBeamThreads = 256;
constexpr int kBeamMax = 64;   // beams per group, results per group
constexpr int kPickItems = 4;  // candidates per thread and pass of the final choice

struct ChunkStat {
    float m, s;  // largest logit and sum of exp(logit - m); NaN s: a NaN or +inf among them
};
struct ChunkCand {
    float logit;
    int32_t token;  // -1: fewer than n_out values in the chunk
};

struct BeamArgs {
    const float* logits;
    int64_t stride;
    const float* scores;
    int beams, n_vocab, n_out, chunks;
    float* out_scores;
    int32_t *out_parent, *out_token;
    unsigned int* counters;  // [groups], zero between launches
    ChunkStat* stat;         // [groups * beams][chunks]
    ChunkCand* cand;         // [groups * beams][chunks][n_out]
};

// Few rows: short chunks, so that more SMs have one. Long chunks otherwise:
// fewer candidates to join.
inline int beam_items(int64_t rows, int n_vocab) {
    const int64_t ctas = rows * (((int64_t)n_vocab + kBeamThreads * 32 - 1) / (kBeamThreads * 32));
    return ctas >= 2 * 152 ? 32 : 8;
}

size_t beam_workspace(int groups, int beams, int n_vocab, int n_out, BeamArgs* a, void* ws) {
    const int64_t rows = (int64_t)groups * beams;
    const int per = kBeamThreads * beam_items(rows, n_vocab);
    const int64_t chunks = ((int64_t)n_vocab + per - 1) / per;
    size_t o = 0;
    auto take = [&](size_t bytes) {
        const size_t at = o;
        o += (bytes + 255) / 256 * 256;
        return at;
    };
    const size_t c = take(kCounterBytes), t = take(sizeof(ChunkStat) * (size_t)(rows * chunks)),
                 d = take(sizeof(ChunkCand) * (size_t)(rows * chunks) * n_out);
    if (a) {
        uint8_t* w = reinterpret_cast<uint8_t*>(ws);
        a->counters = reinterpret_cast<unsigned int*>(w + c);
        a->stat = reinterpret_cast<ChunkStat*>(w + t);
        a->cand = reinterpret_cast<ChunkCand*>(w + d);
        a->chunks = (int)chunks;
    }
    return o;
}

__device__ __forceinline__ float key_value(unsigned long long key) {
    const uint32_t u = (uint32_t)(key >> 32);
    return __uint_as_float((u & 0x80000000u) ? (u & 0x7fffffffu) : ~u);
}

// A total and its place as a pair that compares like (total, lowest place).
struct Pick {
    unsigned long long hi, lo;  // order-preserving bits of the total; ~(beam << 32 | token)
};
__device__ __forceinline__ bool above(const Pick& a, const Pick& b) {
    return a.hi > b.hi || (a.hi == b.hi && a.lo > b.lo);
}
__device__ __forceinline__ unsigned long long f64_order_key(double v) {
    const unsigned long long u = (unsigned long long)__double_as_longlong(v);
    return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}
__device__ __forceinline__ double f64_of_key(unsigned long long k) {
    return __longlong_as_double((long long)((k >> 63) ? (k & 0x7fffffffffffffffull) : ~k));
}

// Lanes per group: 32, 64 or 128 groups of the CTA's 256 threads.
__device__ __forceinline__ int group_lanes(int n_out) { return n_out <= 16 ? 8 : n_out <= 32 ? 4 : 2; }

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint64_t mul_f2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t add_f2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

template <int IT>
__global__ void __launch_bounds__(kBeamThreads) beam_select_kernel(BeamArgs a) {
    constexpr int kCand = kBeamMax * IT;
    constexpr int kFew = 256;                          // candidates the first bound may leave
    constexpr int kFinal = 16 * 8 * kPickItems;        // n_out groups of group_lanes threads: 16 x 8, 32 x 4, 64 x 2
    // the chunk's part and the group's part use the memory one after the other
    __shared__ __align__(16) union {
        struct {
            unsigned long long best[kBeamThreads], cand[kCand];
        } c;
        struct {
            Pick best[kBeamThreads / 2], cand[kFinal], keep[kBeamMax];
            double lse[kBeamMax];
        } g;
    } sm;
    __shared__ float red_m[kBeamThreads / 32], red_s[kBeamThreads / 32], s_top[kBeamThreads / 2];
    __shared__ unsigned long long s_bound;
    __shared__ float s_floor;
    __shared__ Pick s_pick;
    __shared__ int s_n, s_last;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int chunk = blockIdx.x, group = blockIdx.y / a.beams;
    const int64_t row = blockIdx.y;
    const int64_t base = (int64_t)chunk * kBeamThreads * IT;
    const int n = (int)min((int64_t)kBeamThreads * IT, a.n_vocab - base);
    const float* x = a.logits + row * a.stride + base;
    const int gl = group_lanes(a.n_out), groups = kBeamThreads / gl;

    float v[IT];
    if (n == kBeamThreads * IT) {
#pragma unroll
        for (int j = 0; j < IT; ++j) v[j] = __ldcs(x + j * kBeamThreads + tid);
    } else {
#pragma unroll
        for (int j = 0; j < IT; ++j) v[j] = j * kBeamThreads + tid < n ? __ldcs(x + j * kBeamThreads + tid) : -INFINITY;
    }
    float m = v[0];
#pragma unroll
    for (int j = 1; j < IT; ++j) m = fmaxf(m, v[j]);  // of the numbers; -inf if there is none
    if (m != m) m = -INFINITY;
    // exponentials of the differences; a NaN or +inf makes the sum NaN
    const float ref = m > -INFINITY ? m : 0.0f;
    uint64_t sum2 = 0;
    const uint64_t ref2 = pack_f2(ref, ref), log2e = pack_f2(1.4426950408889634f, 1.4426950408889634f);
#pragma unroll
    for (int j = 0; j < IT; j += 2) {
        const uint64_t t = mul_f2(sub_f2(pack_f2(v[j], v[j + 1]), ref2), log2e);
        sum2 = add_f2(sum2, pack_f2(ex2(f2_lo(t)), ex2(f2_hi(t))));
    }
    const float s = f2_lo(sum2) + f2_hi(sum2);
    // the groups' maxima, the chunk's maximum and sum
    float gm = m;
    for (int o = 1; o < gl; o <<= 1) gm = fmaxf(gm, __shfl_xor_sync(0xffffffffu, gm, o));
    if (tid % gl == 0) s_top[tid / gl] = gm;
    {
        const float wm = warp_max(gm);
        const float ws = warp_sum(m > -INFINITY ? s * expf(m - wm) : s);
        if (lane == 0) { red_m[warp] = wm; red_s[warp] = ws; }
    }
    if (tid == 0) s_n = 0;
    __syncthreads();
    if (tid < groups) {
        const float mine = s_top[tid];
        int over = 0, same = 0;
#pragma unroll 8
        for (int t = 0; t < groups; ++t) {
            over += s_top[t] > mine;
            same += s_top[t] == mine;
        }
        // the same value from every group that has it
        if (over < a.n_out && over + same >= a.n_out) s_floor = mine;
    }
    if (warp == kBeamThreads / 32 - 1) {
        const float wm0 = lane < kBeamThreads / 32 ? red_m[lane] : -INFINITY;
        const float ws0 = lane < kBeamThreads / 32 ? red_s[lane] : 0.0f;
        const float wm = warp_max(wm0);
        const float ws = warp_sum(wm0 > -INFINITY ? ws0 * expf(wm0 - wm) : ws0);
        if (lane == 0) a.stat[row * a.chunks + chunk] = ChunkStat{wm, ws};
    }
    __syncthreads();
    const float floor = s_floor;
    if (m >= floor) {
#pragma unroll
        for (int j = 0; j < IT; ++j) {
            const int i = j * kBeamThreads + tid;
            if (v[j] >= floor && i < n) {
                const int at = atomicAdd(&s_n, 1);
                if (at < kFew) sm.c.cand[at] = argmax_key(v[j] + 0.0f, i);  // -0 and 0 are one value
            }
        }
    }
    __syncthreads();
    int nc = s_n;
    if (nc > kFew) {
        // many equal values: the n_out-th largest of the threads' keys (m and its first place)
        int at = -1;
#pragma unroll
        for (int j = IT - 1; j >= 0; --j) {
            if (v[j] != v[j]) v[j] = -INFINITY;
            if (v[j] == m && j * kBeamThreads + tid < n) at = j * kBeamThreads + tid;
        }
        const unsigned long long mine = at >= 0 ? argmax_key(m + 0.0f, at) : 0ull;
        sm.c.best[tid] = mine;
        __syncthreads();
        if (tid == 0) { s_bound = 0; s_n = 0; }
        __syncthreads();
        if (mine) {
            int above_me = 0;
            for (int t = 0; t < kBeamThreads; ++t) above_me += sm.c.best[t] > mine;
            if (above_me == a.n_out - 1) s_bound = mine;
        }
        __syncthreads();
        const unsigned long long bound = s_bound;
        if (mine && mine >= bound) {
#pragma unroll
            for (int j = 0; j < IT; ++j) {
                const int i = j * kBeamThreads + tid;
                const unsigned long long key = argmax_key(v[j] + 0.0f, i);
                if (i < n && key >= bound) sm.c.cand[atomicAdd(&s_n, 1)] = key;
            }
        }
        __syncthreads();
        nc = s_n;
    }
    ChunkCand* out = a.cand + (row * a.chunks + chunk) * a.n_out;
    for (int c = tid; c < nc; c += kBeamThreads) {
        const unsigned long long key = sm.c.cand[c];
        int r = 0;
        for (int t = 0; t < nc; ++t) r += sm.c.cand[t] > key;
        if (r < a.n_out) out[r] = ChunkCand{key_value(key), (int32_t)base + argmax_key_index(key)};
    }
    // fewer values than n_out (NaN are none: their row is not chosen from)
    for (int r = nc + tid; r < a.n_out; r += kBeamThreads) out[r] = ChunkCand{-INFINITY, -1};

    __threadfence();
    __syncthreads();
    if (tid == 0) {
        const unsigned int ticket = atomicAdd(a.counters + group, 1u);
        s_last = ticket == (unsigned)(a.beams * a.chunks - 1);
    }
    __syncthreads();
    if (!s_last) return;
    __threadfence();
    if (tid == 0) a.counters[group] = 0;

    // ---- the group: log sums of its rows, then the best totals -----------------------
    const int64_t row0 = (int64_t)group * a.beams;
    for (int b = warp; b < a.beams; b += kBeamThreads / 32) {
        const ChunkStat* st = a.stat + (row0 + b) * a.chunks;
        float top = -INFINITY;
        for (int c = lane; c < a.chunks; c += 32) top = fmaxf(top, __ldcg(&st[c].m));
        top = warp_max(top);
        double sum = 0.0;
        for (int c = lane; c < a.chunks; c += 32) {
            const float cm = __ldcg(&st[c].m);
            const double cs = (double)__ldcg(&st[c].s);
            sum += cm > -INFINITY ? cs * (double)expf(cm - top) : cs;  // a chunk of NaN alone: cs is NaN
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        const float sc = a.scores[row0 + b];
        // +inf marks a beam whose totals are all -inf
        if (lane == 0) {
            const double lse = (double)top + log(sum);
            sm.g.lse[b] = isfinite(lse) && isfinite(sc) ? lse : (double)INFINITY;
        }
    }
    __syncthreads();
    const int per_row = a.chunks * a.n_out;
    const int64_t all = (int64_t)a.beams * per_row;
    int kept = 0;
    for (int64_t i0 = 0; i0 < all;) {
        const int fresh = kBeamThreads * kPickItems - kept;
        Pick p[kPickItems];
        Pick best{0, 0};
#pragma unroll
        for (int j = 0; j < kPickItems; ++j) {
            p[j] = Pick{0, 0};
            const int slot = j * kBeamThreads + tid;
            const int64_t i = i0 + slot - kept;
            if (slot < kept) {
                p[j] = sm.g.keep[slot];
            } else if (i < all) {
                const int b = (int)(i / per_row), r = (int)(i % per_row);
                const int token = __ldcg(&a.cand[row0 * per_row + i].token);
                const float logit = __ldcg(&a.cand[row0 * per_row + i].logit);
                const double lse = sm.g.lse[b];
                if (lse < (double)INFINITY) {
                    if (token >= 0)
                        p[j] = Pick{f64_order_key((double)a.scores[row0 + b] + ((double)logit - lse)),
                                    ~(((unsigned long long)b << 32) | (unsigned)token)};
                } else if (r < a.n_out && r < a.n_vocab) {  // its lowest tokens, all -inf
                    p[j] = Pick{f64_order_key(-(double)INFINITY), ~(((unsigned long long)b << 32) | (unsigned)r)};
                }
            }
            if (above(p[j], best)) best = p[j];
        }
        i0 += fresh;
        for (int o = 1; o < gl; o <<= 1) {
            const Pick y{__shfl_xor_sync(0xffffffffu, best.hi, o), __shfl_xor_sync(0xffffffffu, best.lo, o)};
            if (above(y, best)) best = y;
        }
        __syncthreads();
        if (tid % gl == 0) sm.g.best[tid / gl] = best;
        if (tid == 0) { s_pick = Pick{0, 0}; s_n = 0; }
        __syncthreads();
        if (tid < groups) {
            const Pick mine = sm.g.best[tid];
            int above_me = 0;
#pragma unroll 8
            for (int t = 0; t < groups; ++t) above_me += above(sm.g.best[t], mine);
            if (mine.lo && above_me == a.n_out - 1) s_pick = mine;
        }
        __syncthreads();
        const Pick bnd = s_pick;
#pragma unroll
        for (int j = 0; j < kPickItems; ++j)
            if (p[j].lo && !above(bnd, p[j])) sm.g.cand[atomicAdd(&s_n, 1)] = p[j];
        __syncthreads();
        const int np = s_n;
        for (int c = tid; c < np; c += kBeamThreads) {
            const Pick k = sm.g.cand[c];
            int r = 0;
            for (int t = 0; t < np; ++t) r += above(sm.g.cand[t], k);
            if (r < a.n_out) sm.g.keep[r] = k;
        }
        kept = min(np, a.n_out);
        __syncthreads();
    }
    if (tid < kept) {
        const Pick k = sm.g.keep[tid];
        const unsigned long long place = ~k.lo;
        const int64_t o = (int64_t)group * a.n_out + tid;
        a.out_scores[o] = (float)f64_of_key(k.hi);
        a.out_parent[o] = (int32_t)(row0 + (int64_t)(place >> 32));
        a.out_token[o] = (int32_t)(place & 0xffffffffull);
    }
}

}  // namespace
}  // namespace lq8

using namespace lq8;

extern "C" {

static bool beam_sizes_ok(int32_t groups, int32_t beams, int32_t n_vocab, int32_t n_out) {
    return groups >= 0 && beams > 0 && n_vocab > 0 && n_out > 0 && n_out <= (int64_t)beams * n_vocab;
}
static bool beam_sizes_supported(int32_t groups, int32_t beams, int32_t n_out) {
    return beams <= kBeamMax && n_out <= kBeamMax && (int64_t)groups * beams < kMaxCounters;
}

size_t llama_q8_beam_select_workspace_bytes(int32_t groups, int32_t beams, int32_t n_vocab, int32_t n_out) {
    if (!beam_sizes_ok(groups, beams, n_vocab, n_out) || !beam_sizes_supported(groups, beams, n_out)) return 0;
    return beam_workspace(groups, beams, n_vocab, n_out, nullptr, nullptr);
}

llama_q8_status llama_q8_beam_select(const float* logits, int64_t logits_stride, int32_t groups, int32_t beams,
                                     int32_t n_vocab, const float* scores, int32_t n_out, float* out_scores,
                                     int32_t* out_parent, int32_t* out_token, void* workspace, size_t workspace_bytes,
                                     void* stream) {
    if (!logits || !scores || !out_scores || !out_parent || !out_token || !workspace ||
        !beam_sizes_ok(groups, beams, n_vocab, n_out) || logits_stride < n_vocab)
        return LQ8_ERR_ARG;
    if (!beam_sizes_supported(groups, beams, n_out)) return LQ8_ERR_UNSUPPORTED;
    if ((((uintptr_t)logits | (uintptr_t)scores | (uintptr_t)out_scores | (uintptr_t)out_parent |
          (uintptr_t)out_token) & 3) || ((uintptr_t)workspace & 15))
        return LQ8_ERR_ARG;
    BeamArgs a{};
    if (workspace_bytes < beam_workspace(groups, beams, n_vocab, n_out, &a, workspace)) return LQ8_ERR_ARG;
    if (groups == 0) return LQ8_OK;
    a.logits = logits, a.stride = logits_stride, a.scores = scores, a.beams = beams, a.n_vocab = n_vocab;
    a.n_out = n_out, a.out_scores = out_scores, a.out_parent = out_parent, a.out_token = out_token;
    const dim3 grid(a.chunks, groups * beams);
    const cudaError_t e =
        beam_items((int64_t)groups * beams, n_vocab) == 32
            ? launch_ex(beam_select_kernel<32>, grid, dim3(kBeamThreads), 0, (cudaStream_t)stream, false, a)
            : launch_ex(beam_select_kernel<8>, grid, dim3(kBeamThreads), 0, (cudaStream_t)stream, false, a);
    return e == cudaSuccess ? LQ8_OK : LQ8_ERR_CUDA;
}

}  // extern "C"
