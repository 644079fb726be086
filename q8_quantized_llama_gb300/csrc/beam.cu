// Beam search's selection: the n_out best continuations of each group of beams
// over beams x vocabulary, in one kernel that reads the logits once and a few
// blocks of them a second time.
//
// total(beam, token) = score[beam] + logit - lse[beam], lse = ln sum exp(logit).
// Rows are cut into blocks of 512 (or 256) values, one warp per block and no
// CTA barrier between blocks: a block gives its largest logit and its sum of
// exponentials. The CTA that finishes a group last (a counter in the workspace)
// adds up the rows' sums, takes the n_out blocks with the largest totals, reads
// those again and ranks their values.
//
// Why n_out blocks are enough: order blocks by (largest total, lowest place
// first). A value of a block that is not among the first n_out has n_out blocks
// before it, each with a value at least as large, and where equal, at a lower
// place. So ties, also rows of one value, need no more blocks.
//
// A block's sums are added in the same order wherever it lies: equal rows get
// equal log sums, and equal totals of different beams are found equal.
//
// Bound: memory for large calls (each logit read once; about 6 issue slots per
// value: load, maximum, subtract, scale, ex2, add, packed in pairs where there is
// a packed form) up to the end, where the last groups' choices, chains of a few
// thousand cycles each (sums, blocks, values, ranks), pass alone: 8 of the 28 us
// of 240 rows of 100003 (14 for the bytes), and most of a small call's 10.
// Not kept: candidate lists with a rising bound during the one pass (34 to 46
// us, most of it for the lists); a pass that looks up the values of the threads
// whose maximum reaches a bound in every piece (53 us); a ring of 4-byte cp.async
// stages (41 us).
#include <algorithm>

#include "kernels.cuh"
#include "paged.cuh"

namespace lq8 {
namespace {

constexpr int kBeamThreads = 256, kBeamWarps = kBeamThreads / 32;
constexpr int kBeamMax = 64;         // beams per group, results per group
constexpr int kBeamVocab = 1 << 24;  // longest row: places of a group (64 rows of whole blocks) stay below 2^31
constexpr int kBeamWave = 152 * 4;   // CTAs resident at once on a GB300's 152 SMs
constexpr int kPickItems = 4;        // blocks per thread that the final choice holds in registers

struct BlockStat {
    float m, s;  // largest logit and sum of exp(logit - m); NaN s: a NaN or +inf among them
};

struct BeamArgs {
    const float* logits;
    int64_t stride;
    const float* scores;
    int beams, n_vocab, n_out;
    int blocks, ctas, share;  // blocks per row, CTAs per group, blocks per CTA
    float* out_scores;
    int32_t *out_parent, *out_token;
    unsigned int* counters;  // [groups], zero between launches
    BlockStat* stat;         // [groups * beams][blocks]
};

// A group's blocks of 512 values are dealt evenly to `ctas` CTAs of its own (a CTA
// that chooses for its group keeps no other group waiting), together one wave of
// them (28 us for 240 rows of 100003; one and a half and two waves: 31 and 29).
// Where blocks of 512 would leave warps idle, blocks of 256, one per warp: more
// SMs take part, and less is read again.
struct BeamCut {
    int vpl;  // values per lane
    int blocks, ctas, share;
};
inline BeamCut beam_cut(int groups, int beams, int n_vocab) {
    const bool few = (int64_t)groups * beams * (((int64_t)n_vocab + 511) / 512) < kBeamWave * kBeamWarps / 4;
    const int size = few ? 256 : 512, blocks = (n_vocab + size - 1) / size, all = beams * blocks;
    const int most = (all + kBeamWarps - 1) / kBeamWarps, ctas = std::max(1, std::min(most, kBeamWave / std::max(groups, 1)));
    const int share = (all + ctas - 1) / ctas;
    return BeamCut{size / 32, blocks, (all + share - 1) / share, share};
}

size_t beam_workspace(int groups, int beams, int n_vocab, BeamArgs* a, void* ws) {
    const int64_t rows = (int64_t)groups * beams;
    const BeamCut cut = beam_cut(groups, beams, n_vocab);
    if (a) {
        a->counters = reinterpret_cast<unsigned int*>(ws);
        a->stat = reinterpret_cast<BlockStat*>(reinterpret_cast<uint8_t*>(ws) + kCounterBytes);
        a->blocks = cut.blocks, a->ctas = cut.ctas, a->share = cut.share;
    }
    return kCounterBytes + sizeof(BlockStat) * (size_t)(rows * cut.blocks);
}

// A total and its place: beam * blocks * block size + token for a value, beam * blocks + block for a block.
struct Pick {
    unsigned long long key;  // order-preserving bits of the total, 0: none
    unsigned place;
};
__device__ __forceinline__ bool above(const Pick& a, const Pick& b) {
    // no short circuits: as branches they made the counting loops wait 100 cycles and more per entry
    return (a.key > b.key) | ((a.key == b.key) & (a.place < b.place));
}
// Totals are unevaluated sums hi + lo of two f32 numbers (about 48 bits): double
// arithmetic runs at a small fraction of f32's rate here. So are the sums of a
// row's blocks; the exponentials and a block's sum of them are f32, and the log
// sum is as good as those (2^-19 at most, a few 2^-24 as a rule).
struct Sum2 {
    float hi, lo;
};
// a + b exactly: the rounded sum and what the rounding dropped (Knuth's two-sum)
__device__ __forceinline__ Sum2 two_sum(float a, float b) {
    const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
    return Sum2{s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
__device__ __forceinline__ Sum2 add2(Sum2 x, float y) {
    const Sum2 s = two_sum(x.hi, y);
    return two_sum(s.hi, __fadd_rn(s.lo, x.lo));
}
// The key of score - lse + logit; -inf for a beam that cannot be chosen from, and for NaN.
__device__ __forceinline__ unsigned long long total_key(Sum2 add, float logit) {
    Sum2 t = add2(add, logit + 0.0f);
    if (!(t.hi > -INFINITY) || !isfinite(add.hi)) t = Sum2{-INFINITY, 0.0f};  // two_sum of an infinity leaves NaN in lo
    return ((unsigned long long)f32_order_key(t.hi + 0.0f) << 32) | f32_order_key(t.lo + 0.0f);
}
__device__ __forceinline__ float key_total(unsigned long long key) {
    const uint32_t u = (uint32_t)(key >> 32);
    return __uint_as_float((u & 0x80000000u) ? (u & 0x7fffffffu) : ~u);
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

constexpr int kList = 1280;  // values kept for ranking; a block adds at most 512 to at most 256
struct ChooseShared {
    Pick best[kBeamThreads / 2], list[kList], sel[kBeamMax], bound;
    Sum2 add[kBeamMax];  // score - lse of each beam; not finite: its totals are all -inf
    int sel_beam[kBeamMax], n;
};

// How many of the first n entries are above p.
__device__ __forceinline__ int rank(const Pick* list, int n, const Pick& p) {
    int r = 0;
#pragma unroll 8
    for (int t = 0; t < n; ++t) r += above(list[t], p);
    return r;
}

// A group whose blocks are all known. All threads of a CTA.
template <int VPL>
__device__ __noinline__ void choose(const BeamArgs& a, ChooseShared& sm, int group) {
    constexpr int kBlock = VPL * 32;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // 32, 64 or 128 groups of threads, at least twice n_out
    const int gl = a.n_out <= 16 ? 8 : a.n_out <= 32 ? 4 : 2, groups = kBeamThreads / gl;
    const int row0 = group * a.beams, all = a.beams * a.blocks, n_sel = min(a.n_out, all);
    const BlockStat* stat = a.stat + (int64_t)row0 * a.blocks;
    // the thread's first blocks, asked for before the sums
    float ahead[kPickItems];
#pragma unroll
    for (int j = 0; j < kPickItems; ++j) {
        const int i = j * kBeamThreads + tid;
        ahead[j] = i < all ? __ldcg(&stat[i].m) : 0.0f;
    }
    for (int b = warp; b < a.beams; b += kBeamWarps) {
        const BlockStat* st = stat + (int64_t)b * a.blocks;
        const float sc = a.scores[row0 + b];
        // The lane's blocks, eight at a time: eight in f32, those of a lane in two parts (in one f32 sum the 1024 blocks
        // per lane of a row of 2^24 were off by 1e-5). The exponentials' reference follows the maximum only in steps of
        // 8 or more, as every change of it rounds.
        float top = -INFINITY;
        Sum2 sum{0.0f, 0.0f};
        for (int c0 = lane; c0 < a.blocks; c0 += 256) {
            float2 x[8];
            float m1 = -INFINITY, y[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                x[j] = c0 + j * 32 < a.blocks ? __ldcg(reinterpret_cast<const float2*>(st + c0 + j * 32))
                                              : make_float2(-INFINITY, 0.0f);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) m1 = fmaxf(m1, x[j].x);
            if (m1 > top + 8.0f) {
                const float f = top > -INFINITY ? expf(top - m1) : 1.0f;
                sum = Sum2{sum.hi * f, sum.lo * f};
                top = m1;
            }
            const float ref = top > -INFINITY ? top : 0.0f;
            // a block of -inf alone adds 0, one with NaN NaN
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = x[j].y * (x[j].x > -INFINITY ? expf(x[j].x - ref) : 1.0f);
            sum = add2(sum, ((y[0] + y[1]) + (y[2] + y[3])) + ((y[4] + y[5]) + (y[6] + y[7])));
        }
        const float all_top = warp_max(top);
        const float f1 = top > -INFINITY ? expf(top - all_top) : 1.0f;
        sum = Sum2{sum.hi * f1, sum.lo * f1};
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const float y = __shfl_xor_sync(0xffffffffu, sum.hi, o), z = __shfl_xor_sync(0xffffffffu, sum.lo, o);
            sum = add2(add2(sum, y), z);
        }
        if (lane == 0) {
            // ln of 2^e f, f in [1/2, 1): e ln 2 in two parts, the first with few enough bits to be exact, and the
            // logarithm of f, off by 2^-25 where that of the sum itself would be by 2^-21
            int e = 0;
            const float f = frexpf(sum.hi, &e);
            Sum2 t = two_sum(sc, -all_top);
            t = add2(t, -0.69140625f * e);  // 177 / 256
            t = add2(t, -fmaf(1.7409305599453e-3f, (float)e, logf(f)));
            t = add2(t, -sum.lo / sum.hi);
            if (!(isfinite(sc) && isfinite(all_top) && isfinite(sum.hi))) t.hi = INFINITY;
            sm.add[b] = t;
        }
    }
    if (tid == 0) {
        sm.bound = Pick{0, ~0u};
        sm.n = 0;
    }
    __syncthreads();

    // ---- the n_out first blocks, in order, to sel ----------------------------------------
    auto block_pick = [&](int i, float m) { return Pick{total_key(sm.add[(unsigned)i / (unsigned)a.blocks], m), (unsigned)i}; };
    auto block_of = [&](int i) { return block_pick(i, __ldcg(&stat[i].m)); };
    Pick mine[kPickItems], best{0, ~0u};
#pragma unroll
    for (int j = 0; j < kPickItems; ++j) {
        const int i = j * kBeamThreads + tid;
        mine[j] = i < all ? block_pick(i, ahead[j]) : Pick{0, ~0u};
        if (above(mine[j], best)) best = mine[j];
    }
    // those from the n_out-th largest of the thread groups' best on
    bool chosen = false;
    {
        for (int i = kPickItems * kBeamThreads + tid; i < all; i += kBeamThreads) {
            const Pick p = block_of(i);
            if (above(p, best)) best = p;
        }
        for (int o = 1; o < gl; o <<= 1) {
            const Pick y{__shfl_xor_sync(0xffffffffu, best.key, o), __shfl_xor_sync(0xffffffffu, best.place, o)};
            if (above(y, best)) best = y;
        }
        if (tid % gl == 0) sm.best[tid / gl] = best;
        __syncthreads();
        // each lane of a group counts its part of the larger ones
        int over = 0;
#pragma unroll 4
        for (int t = tid % gl; t < groups; t += gl) over += above(sm.best[t], best);
        for (int o = 1; o < gl; o <<= 1) over += __shfl_xor_sync(0xffffffffu, over, o);
        if (tid % gl == 0 && best.key && over == a.n_out - 1) sm.bound = best;
        __syncthreads();
        const Pick bound = sm.bound;
        auto keep = [&](const Pick& p) {
            if (!p.key || above(bound, p)) return;
            const int at = atomicAdd(&sm.n, 1);
            if (at < kList) sm.list[at] = p;
        };
#pragma unroll
        for (int j = 0; j < kPickItems; ++j) keep(mine[j]);
        for (int i = kPickItems * kBeamThreads + tid; i < all; i += kBeamThreads) keep(block_of(i));
        __syncthreads();
        const int n = sm.n;
        if (n <= kList) {
            for (int c = tid; c < n; c += kBeamThreads) {
                const Pick p = sm.list[c];
                const int r = rank(sm.list, n, p);
                if (r < n_sel) sm.sel[r] = p;
            }
            chosen = true;
        }
    }
    __syncthreads();
    if (!chosen) {  // too many in few groups: 1024 at a time beside the best so far
        int kept = 0;
        for (int at = 0; at < all;) {
            const int fresh = min(all - at, kBeamThreads * kPickItems - kept);
            for (int c = tid; c < kept + fresh; c += kBeamThreads)
                sm.list[c] = c < kept ? sm.sel[c] : block_of(at + c - kept);
            __syncthreads();
            for (int c = tid; c < kept + fresh; c += kBeamThreads) {
                const Pick p = sm.list[c];
                const int r = rank(sm.list, kept + fresh, p);
                if (r < n_sel) sm.sel[r] = p;
            }
            kept = min(n_sel, kept + fresh);
            at += fresh;
            __syncthreads();
        }
    }

    // ---- their values: those that reach the last block's total, ranked ---------------------
    const int values = n_sel * kBlock;
    Pick least = n_sel == a.n_out ? Pick{sm.sel[n_sel - 1].key, ~0u} : Pick{0, ~0u};
    if (tid < n_sel) sm.sel_beam[tid] = (int)sm.sel[tid].place / a.blocks;
    if (tid == 0) sm.n = 0;
    __syncthreads();
    auto consider = [&](float y, int b, unsigned block, int i) {  // value i of a block of beam b
        const Pick p{total_key(sm.add[b], y), block * kBlock + i};
        if (above(least, p)) return;
        const int at = atomicAdd(&sm.n, 1);
        if (at < kList) sm.list[at] = p;
    };
    auto token0 = [&](unsigned block, int b) { return ((int)block - b * a.blocks) * kBlock; };  // the block's first
    const float least_total = least.key ? key_total(least.key) : -INFINITY;
    for (int c = warp; c < n_sel; c += kBeamWarps) {
        const unsigned block = sm.sel[c].place;
        const int b = sm.sel_beam[c], t0 = token0(block, b), left = a.n_vocab - t0 - lane;
        const float* x = a.logits + (int64_t)(row0 + b) * a.stride + t0 + lane;
        float y[VPL];
#pragma unroll
        for (int j = 0; j < VPL; ++j) y[j] = j * 32 < left ? x[j * 32] : 0.0f;
        // a total in one f32 addition is off by less than a millionth part of itself and of score - lse
        const float add = sm.add[b].hi, sure = least_total - 1e-6f * (fabsf(least_total) + fabsf(add));
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
            const float t = y[j] + add;
            if (j * 32 < left && !(t < sure - 1e-6f * fabsf(t))) consider(y[j], b, block, j * 32 + lane);
        }
    }
    __syncthreads();
    if (sm.n > kList) {
        // many equal or rising values: block by block, the list cut to its best whenever it has grown
        __syncthreads();
        if (tid == 0) sm.n = 0;
        __syncthreads();
        for (int i0 = 0; i0 < values; i0 += kBlock) {
            const unsigned block = sm.sel[i0 / kBlock].place;
            const int b = sm.sel_beam[i0 / kBlock], t0 = token0(block, b);
            for (int i = tid; i < kBlock && t0 + i < a.n_vocab; i += kBeamThreads)
                consider(a.logits[(int64_t)(row0 + b) * a.stride + t0 + i], b, block, i);
            __syncthreads();
            const int n = sm.n;
            if (n > kBeamThreads) {
                Pick p[(kList + kBeamThreads - 1) / kBeamThreads];
                int r[(kList + kBeamThreads - 1) / kBeamThreads];
#pragma unroll
                for (int k = 0; k < (kList + kBeamThreads - 1) / kBeamThreads; ++k) {
                    const int c = k * kBeamThreads + tid;
                    p[k] = c < n ? sm.list[c] : Pick{0, ~0u};
                    r[k] = c < n ? rank(sm.list, n, p[k]) : kBeamMax;
                }
                __syncthreads();
#pragma unroll
                for (int k = 0; k < (kList + kBeamThreads - 1) / kBeamThreads; ++k)
                    if (r[k] < a.n_out) sm.list[r[k]] = p[k];
                if (tid == 0) sm.n = a.n_out;
                __syncthreads();
                least = sm.list[a.n_out - 1];
            }
            __syncthreads();
        }
    }
    const int n = sm.n;
    for (int c = tid; c < n; c += kBeamThreads) {
        const Pick p = sm.list[c];
        const int r = rank(sm.list, n, p);
        if (r >= a.n_out) continue;
        const int b = p.place / (unsigned)(a.blocks * kBlock);
        const int64_t o = (int64_t)group * a.n_out + r;
        a.out_scores[o] = key_total(p.key);
        a.out_parent[o] = row0 + b;
        a.out_token[o] = (int32_t)(p.place - (unsigned)b * (unsigned)(a.blocks * kBlock));
    }
}

// QUAD: all rows start at 16-byte boundaries, a lane's values lie in groups of four, otherwise 32 apart.
template <int VPL, bool QUAD>
__global__ void __launch_bounds__(kBeamThreads, 4) beam_select_kernel(BeamArgs a) {
    constexpr int kBlock = VPL * 32;
    __shared__ ChooseShared sm;
    __shared__ int s_last;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int group = blockIdx.x / a.ctas, row0 = group * a.beams, all = a.beams * a.blocks;
    const int u0 = (blockIdx.x - group * a.ctas) * a.share, u1 = min(all, u0 + a.share);
    for (int u = u0 + warp; u < u1; u += kBeamWarps) {
        const int b = (unsigned)u / (unsigned)a.blocks, at = (u - b * a.blocks) * kBlock, left = a.n_vocab - at;
        const float* x = a.logits + (int64_t)(row0 + b) * a.stride + at;
        float v[VPL];
        if (left >= kBlock) {
#pragma unroll
            for (int j = 0; j < VPL; j += QUAD ? 4 : 1) {
                if (QUAD) {
                    const float4 y = __ldcs(reinterpret_cast<const float4*>(x) + j * 8 + lane);
                    v[j] = y.x; v[j + 1] = y.y; v[j + 2] = y.z; v[j + 3] = y.w;
                } else {
                    v[j] = __ldcs(x + j * 32 + lane);
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < VPL; ++j) {
                const int i = QUAD ? ((j >> 2) * 32 + lane) * 4 + (j & 3) : j * 32 + lane;
                v[j] = i < left ? x[i] : -INFINITY;
            }
        }
        float m = v[0];
#pragma unroll
        for (int j = 1; j < VPL; ++j) m = fmaxf(m, v[j]);  // of the numbers
        if (m != m) m = -INFINITY;
        m = warp_max(m);
        // a NaN or +inf makes the sum NaN
        const float ref = m > -INFINITY ? m : 0.0f;
        const uint64_t ref2 = pack_f2(ref, ref), log2e = pack_f2(1.4426950408889634f, 1.4426950408889634f);
        uint64_t sum2 = 0;
#pragma unroll
        for (int j = 0; j < VPL; j += 2) {
            const uint64_t t = mul_f2(sub_f2(pack_f2(v[j], v[j + 1]), ref2), log2e);
            sum2 = add_f2(sum2, pack_f2(ex2(f2_lo(t)), ex2(f2_hi(t))));
        }
        const float s = warp_sum(f2_lo(sum2) + f2_hi(sum2));
        if (lane == 0) a.stat[(int64_t)row0 * a.blocks + u] = BlockStat{m, s};
    }
    __syncthreads();
    if (tid == 0) {
        s_last = take_ticket(a.counters + group) == (unsigned)(a.ctas - 1);
        if (s_last) a.counters[group] = 0;
    }
    __syncthreads();
    if (s_last) choose<VPL>(a, sm, group);
}

}  // namespace
}  // namespace lq8

using namespace lq8;

extern "C" {

static bool beam_sizes_ok(int32_t groups, int32_t beams, int32_t n_vocab, int32_t n_out) {
    return groups >= 0 && beams > 0 && n_vocab > 0 && n_out > 0 && n_out <= (int64_t)beams * n_vocab;
}
static bool beam_sizes_supported(int32_t groups, int32_t beams, int32_t n_vocab, int32_t n_out) {
    return beams <= kBeamMax && n_out <= kBeamMax && (int64_t)groups * beams < kMaxCounters && n_vocab <= kBeamVocab &&
           // blocks are counted in 31 bits, a CTA's share past the last one included
           (int64_t)groups * beams * (n_vocab / 512 + 1) < INT32_MAX / 2;
}

size_t llama_q8_beam_select_workspace_bytes(int32_t groups, int32_t beams, int32_t n_vocab, int32_t n_out) {
    if (!beam_sizes_ok(groups, beams, n_vocab, n_out) || !beam_sizes_supported(groups, beams, n_vocab, n_out)) return 0;
    return beam_workspace(groups, beams, n_vocab, nullptr, nullptr);
}

llama_q8_status llama_q8_beam_select(const float* logits, int64_t logits_stride, int32_t groups, int32_t beams,
                                     int32_t n_vocab, const float* scores, int32_t n_out, float* out_scores,
                                     int32_t* out_parent, int32_t* out_token, void* workspace, size_t workspace_bytes,
                                     void* stream) {
    if (!logits || !scores || !out_scores || !out_parent || !out_token || !workspace ||
        !beam_sizes_ok(groups, beams, n_vocab, n_out) || logits_stride < n_vocab)
        return LQ8_ERR_ARG;
    if (!beam_sizes_supported(groups, beams, n_vocab, n_out)) return LQ8_ERR_UNSUPPORTED;
    if ((((uintptr_t)logits | (uintptr_t)scores | (uintptr_t)out_scores | (uintptr_t)out_parent |
          (uintptr_t)out_token) & 3) || ((uintptr_t)workspace & 15))
        return LQ8_ERR_ARG;
    BeamArgs a{};
    if (workspace_bytes < beam_workspace(groups, beams, n_vocab, &a, workspace)) return LQ8_ERR_ARG;
    if (groups == 0) return LQ8_OK;
    a.logits = logits, a.stride = logits_stride, a.scores = scores, a.beams = beams, a.n_vocab = n_vocab;
    a.n_out = n_out, a.out_scores = out_scores, a.out_parent = out_parent, a.out_token = out_token;
    const BeamCut cut = beam_cut(groups, beams, n_vocab);
    const dim3 grid((unsigned)(groups * cut.ctas)), block(kBeamThreads);
    cudaStream_t st = (cudaStream_t)stream;
    const bool quad = ((uintptr_t)logits & 15) == 0 && logits_stride % 4 == 0;
    const cudaError_t e =
        cut.vpl == 16
            ? (quad ? launch_ex(beam_select_kernel<16, true>, grid, block, 0, st, false, a)
                    : launch_ex(beam_select_kernel<16, false>, grid, block, 0, st, false, a))
            : (quad ? launch_ex(beam_select_kernel<8, true>, grid, block, 0, st, false, a)
                    : launch_ex(beam_select_kernel<8, false>, grid, block, 0, st, false, a));
    return e == cudaSuccess ? LQ8_OK : LQ8_ERR_CUDA;
}

}  // extern "C"
