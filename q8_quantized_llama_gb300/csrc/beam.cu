// Beam search's selection: the n_out best continuations of each group of beams
// over beams x vocabulary, in one kernel that reads the logits once.
//
// total(beam, token) = score[beam] + logit - lse[beam], lse = ln sum exp(logit).
// A CTA goes through its piece of a row, a block of values per thread at a time,
// with the next block's loads in flight, and gets the sums of exponentials (a
// running maximum and sum per thread, given out per segment) and its n_out
// largest logits: within a row totals rise with logits, so no other value of the
// piece can be chosen. The last CTA of a group to finish (a counter in the
// workspace) joins the sums and picks the n_out largest totals.
//
// Rows are cut into segments at the same places, and a segment's sums are added
// in the same order, wherever it lies: equal rows get equal log sums, so that
// equal totals of different beams are found equal. Pieces are whole segments.
//
// Largest of many by a bound: in the first block lanes form groups (32, 64 or
// 128 per CTA, at least twice n_out); n_out groups reach the n_out-th largest of
// the groups' maxima, so at least n_out values do, and only a few more. They
// are kept, and of the later blocks the values above the bound: an equal one
// there has a higher index and loses. When the list has grown by 16 or half it is
// cut to its n_out best, and the bound rises: keys (value, lowest index), which
// all differ, are ranked by counting the larger ones. The list is looked at every
// fourth block; where it overflows in between (rising values, a row of one
// value), the piece's list is made again 1024 values at a time.
//
// Bound: the steps that end a piece and a group, and issue slots, more than
// memory: 240 rows of 100003 take 36 us, 14 of them for the bytes; the final
// choice alone is 4 to 5.
// Not kept: one CTA per 8192 values without a list (46 us: barriers and fences);
// a pass of maxima and sums alone, then a second look at the threads that reach
// the bound (53 us: what they look up again has left L2); a ring of 4-byte
// cp.async stages (41 us); pieces cut anywhere, the sums with them (34 us, but
// equal rows got log sums that differed in the last bits).
#include <algorithm>

#include "kernels.cuh"
#include "paged.cuh"

namespace lq8 {
namespace {

constexpr int kBeamThreads = 256;
constexpr int kBeamMax = 64;   // beams per group, results per group
constexpr int kPickItems = 4;  // candidates per thread and pass of the final choice
constexpr int kBeamVocab = 1 << 28;  // longest row: 64 beams x 64 results x its chunks stay below 2^31 - 1024

struct SegmentStat {
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
    int beams, n_vocab, n_out;
    int chunks, segs;     // pieces per row at most, segments per row
    int share, units;     // segments per CTA, of all rows
    float* out_scores;
    int32_t *out_parent, *out_token;
    unsigned int* counters;  // [groups], zero between launches
    SegmentStat* stat;       // [groups * beams][segs]
    ChunkCand* cand;         // [groups * beams][chunks][n_out], by the CTA's place among the row's
};

// How the work is cut: rows in segments of four blocks of 4096 values, the
// segments of all rows dealt evenly to one wave of CTAs, `share` each, so that a
// row is in pieces of up to `chunks` CTAs and a CTA may hold pieces of several
// rows. Where that would leave most SMs without one: segments of one block of
// 2048, one per CTA.
struct BeamCut {
    int j, segs, chunks;
    int share, ctas;
};
constexpr int kBeamCtas = 4;  // per SM
constexpr int kBeamWave = 152 * kBeamCtas;
template <int J>
constexpr int kSegBlocks = J == 4 ? 4 : 1;
inline BeamCut beam_cut(int64_t rows, int n_vocab) {
    const bool few = rows * (((int64_t)n_vocab + 4095) / 4096) <= 152 * 2;
    const int seg = few ? 2048 : 4 * 4096;
    const int64_t segs = ((int64_t)n_vocab + seg - 1) / seg;
    const int64_t share = few ? 1 : (rows * segs + kBeamWave - 1) / kBeamWave;
    return BeamCut{few ? 2 : 4, (int)segs, (int)((segs - 1 + share - 1) / share + 1), (int)share,
                   (int)((rows * segs + share - 1) / share)};
}

size_t beam_workspace(int groups, int beams, int n_vocab, int n_out, BeamArgs* a, void* ws) {
    const int64_t rows = (int64_t)groups * beams;
    const BeamCut cut = beam_cut(std::max<int64_t>(rows, 1), n_vocab);
    const int64_t chunks = cut.chunks;
    size_t o = 0;
    auto take = [&](size_t bytes) {
        const size_t at = o;
        o += (bytes + 255) / 256 * 256;
        return at;
    };
    const size_t c = take(kCounterBytes), t = take(sizeof(SegmentStat) * (size_t)(rows * cut.segs)),
                 d = take(sizeof(ChunkCand) * (size_t)(rows * chunks) * n_out);
    if (a) {
        uint8_t* w = reinterpret_cast<uint8_t*>(ws);
        a->counters = reinterpret_cast<unsigned int*>(w + c);
        a->stat = reinterpret_cast<SegmentStat*>(w + t);
        a->cand = reinterpret_cast<ChunkCand*>(w + d);
        a->chunks = cut.chunks;
        a->segs = cut.segs;
        a->share = cut.share;
        a->units = (int)(rows * cut.segs);
    }
    return o;
}

__device__ __forceinline__ float key_value(unsigned long long key) {
    const uint32_t u = (uint32_t)(key >> 32);
    return __uint_as_float((u & 0x80000000u) ? (u & 0x7fffffffu) : ~u);
}

// A total and its slot among the group's candidates (beam, chunk, place in the
// chunk's falling list). Of equal totals the lowest slot is the lowest (beam,
// token): a chunk's equal values are listed by index.
struct Pick {
    unsigned long long key;  // order-preserving bits of the total, 0: none
    unsigned slot;
};
__device__ __forceinline__ bool above(const Pick& a, const Pick& b) {
    // no short circuits: as branches they made the counting loops wait 100 cycles and more per entry
    return (a.key > b.key) | ((a.key == b.key) & (a.slot < b.slot));
}
// Totals and log sums are unevaluated sums hi + lo of two f32 numbers (about 48
// bits): double arithmetic runs at a small fraction of f32's rate here.
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
__device__ __forceinline__ unsigned long long total_key(Sum2 t) {
    if (!(t.hi > -INFINITY)) t = Sum2{-INFINITY, 0.0f};  // two_sum of an infinity leaves NaN in lo
    return ((unsigned long long)f32_order_key(t.hi + 0.0f) << 32) | f32_order_key(t.lo + 0.0f);
}

// Lanes per group: 32, 64 or 128 groups of the CTA's 256 threads.
__device__ __forceinline__ int group_lanes(int n_out) { return n_out <= 16 ? 8 : n_out <= 32 ? 4 : 2; }

// CTAs that hold a row's pieces: from first_cta on, row_pieces of them.
__device__ __forceinline__ int first_cta(const BeamArgs& a, int row) { return row * a.segs / a.share; }
__device__ __forceinline__ int row_pieces(const BeamArgs& a, int row) {
    return ((row + 1) * a.segs - 1) / a.share - first_cta(a, row) + 1;
}

constexpr int kFinal = 16 * 8 * kPickItems;  // n_out groups of group_lanes threads: 16 x 8, 32 x 4, 64 x 2
struct ChooseShared {
    Pick best[kBeamThreads], cand[kFinal], keep[kBeamMax], bound;
    Sum2 add[kBeamMax];  // score - lse of each beam; not finite: its totals are all -inf
    int pieces[kBeamMax], n;
};

// A group whose pieces are all written: the log sums of its rows, then the best totals. All threads of a CTA.
__device__ __noinline__ void choose(const BeamArgs& a, ChooseShared& sm, int group) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int gl = group_lanes(a.n_out), groups = kBeamThreads / gl;
    const int64_t row0 = (int64_t)group * a.beams;
    const int lists = a.beams * a.chunks, all = lists * a.n_out;  // below 2^31 (kBeamVocab)
    const ChunkCand* cand = a.cand + row0 * a.chunks * (int64_t)a.n_out;
    auto fetch = [&](int i) {
        const float2 x = __ldcg(reinterpret_cast<const float2*>(cand + i));
        return ChunkCand{x.x, __float_as_int(x.y)};
    };
    auto pick = [&](const ChunkCand& c, int i) {
        const int list = i / a.n_out, b = list / a.chunks, piece = list - b * a.chunks;
        const Sum2 add = sm.add[b];
        Pick p{0ull, (unsigned)i};
        if (!isfinite(add.hi)) {  // the lowest tokens of the beam
            if (piece == 0 && i - list * a.n_out < a.n_vocab) p.key = total_key(Sum2{-INFINITY, 0.0f});
        } else if (piece < sm.pieces[b] && c.token >= 0) {
            p.key = total_key(add2(add, c.logit));
        }
        return p;
    };
    auto put = [&](const Pick& p, int r) {
        const int list = (int)p.slot / a.n_out, b = list / a.chunks;
        const int64_t o = (int64_t)group * a.n_out + r;
        a.out_scores[o] = key_value(p.key);
        a.out_parent[o] = (int32_t)(row0 + b);
        a.out_token[o] = isfinite(sm.add[b].hi) ? fetch((int)p.slot).token : (int)p.slot - list * a.n_out;
    };
    // a candidate asked for before the sums: one per thread, or the first of the thread's first list
    const bool direct = all <= kBeamThreads;
    const int i0 = direct ? tid : tid * a.n_out;
    const ChunkCand c0 = i0 < all ? fetch(i0) : ChunkCand{-INFINITY, -1};
    for (int b = warp; b < a.beams; b += kBeamThreads / 32) {
        const SegmentStat* st = a.stat + (row0 + b) * a.segs;
        const int pieces = row_pieces(a, (int)row0 + b);
        const float sc = a.scores[row0 + b];
        float top = -INFINITY, part = 0.0f;  // the lane's segments
        for (int c = lane; c < a.segs; c += 32) {
            const float2 x = __ldcg(reinterpret_cast<const float2*>(st + c));
            const float m1 = fmaxf(top, x.x);
            // -inf alone adds 0, NaN alone NaN
            part = (top > -INFINITY ? part * expf(top - m1) : part) + (x.x > -INFINITY ? x.y * expf(x.x - m1) : x.y);
            top = m1;
        }
        const float all_top = warp_max(top);
        Sum2 sum{top > -INFINITY ? part * expf(top - all_top) : part, 0.0f};
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
            sm.pieces[b] = pieces;
        }
    }
    if (tid == 0) {
        sm.bound = Pick{0, ~0u};
        sm.n = 0;
    }
    __syncthreads();
    // rank of p among the first n entries
    auto rank = [](const Pick* list, int n, const Pick& p) {
        int r = 0;
#pragma unroll 8
        for (int t = 0; t < n; ++t) r += above(list[t], p);
        return r;
    };
    if (direct) {
        const Pick p = i0 < all ? pick(c0, i0) : Pick{0, ~0u};
        sm.cand[tid] = p;
        __syncthreads();
        const int r = p.key ? rank(sm.cand, all, p) : a.n_out;
        if (r < a.n_out) put(p, r);
        return;
    }
    if (lists >= a.n_out) {
        // the n_out-th largest of the threads' best first entries is a bound; each list is read down to it
        Pick head{0, ~0u};
        for (int l = tid; l < lists; l += kBeamThreads) {
            const Pick p = pick(l == tid ? c0 : fetch(l * a.n_out), l * a.n_out);
            if (above(p, head)) head = p;
        }
        sm.best[tid] = head;
        __syncthreads();
        if (head.key && rank(sm.best, min(lists, kBeamThreads), head) == a.n_out - 1) sm.bound = head;
        __syncthreads();
        const Pick bound = sm.bound;
        auto take = [&](const Pick& p) {
            if (!p.key || above(bound, p)) return false;
            const int at = atomicAdd(&sm.n, 1);
            if (at < kFinal) sm.cand[at] = p;
            return true;
        };
        if (all <= 16 * kBeamThreads) {  // a few loads per thread, none waiting for another
#pragma unroll 4
            for (int i = tid; i < all; i += kBeamThreads) take(pick(fetch(i), i));
        } else {
            for (int l = tid; l < lists; l += kBeamThreads)
                for (int r = 0; r < a.n_out; ++r)
                    if (!take(pick(fetch(l * a.n_out + r), l * a.n_out + r))) break;  // the list falls
        }
        __syncthreads();
        const int n = sm.n;
        if (n <= kFinal) {
            for (int c = tid; c < n; c += kBeamThreads) {
                const Pick p = sm.cand[c];
                const int r = rank(sm.cand, n, p);
                if (r < a.n_out) put(p, r);
            }
            return;
        }
    }
    // a few long lists, or many equal values: all candidates, 1024 at a time beside the best so far, by a bound from groups of
    // lanes as in the chunks
    int kept = 0;
    for (int at = 0; at < all;) {
        Pick p[kPickItems], best{0, ~0u};
#pragma unroll
        for (int j = 0; j < kPickItems; ++j) {
            const int slot = j * kBeamThreads + tid, i = at + slot - kept;
            p[j] = slot < kept ? sm.keep[slot] : i < all ? pick(fetch(i), i) : Pick{0, ~0u};
            if (above(p[j], best)) best = p[j];
        }
        at += kBeamThreads * kPickItems - kept;
        for (int o = 1; o < gl; o <<= 1) {
            const Pick y{__shfl_xor_sync(0xffffffffu, best.key, o), __shfl_xor_sync(0xffffffffu, best.slot, o)};
            if (above(y, best)) best = y;
        }
        __syncthreads();
        if (tid % gl == 0) sm.best[tid / gl] = best;
        if (tid == 0) {
            sm.bound = Pick{0, ~0u};
            sm.n = 0;
        }
        __syncthreads();
        if (tid < groups) {
            const Pick mine = sm.best[tid];
            if (mine.key && rank(sm.best, groups, mine) == a.n_out - 1) sm.bound = mine;
        }
        __syncthreads();
        const Pick bound = sm.bound;
#pragma unroll
        for (int j = 0; j < kPickItems; ++j)
            if (p[j].key && !above(bound, p[j])) sm.cand[atomicAdd(&sm.n, 1)] = p[j];
        __syncthreads();
        const int n = sm.n;
        for (int c = tid; c < n; c += kBeamThreads) {
            const Pick k = sm.cand[c];
            const int r = rank(sm.cand, n, k);
            if (r < a.n_out) sm.keep[r] = k;
        }
        kept = min(n, a.n_out);
        __syncthreads();
    }
    if (tid < kept) put(sm.keep[tid], tid);
}

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

// How many of the first n keys are larger.
__device__ __forceinline__ int key_rank(const unsigned long long* list, int n, unsigned long long key) {
    int r = 0;
#pragma unroll 8
    for (int t = 0; t < n; ++t) r += list[t] > key;
    return r;
}

constexpr int kList = 1280;  // keys the list holds; a step of the careful form adds at most 1024 to at most 96
constexpr int kCut = kBeamMax * (kList / kBeamThreads);
// QUAD: all rows start at 16-byte boundaries; a thread's values lie in groups of four, otherwise 256 apart.
template <int J, bool QUAD>
__global__ void __launch_bounds__(kBeamThreads, kBeamCtas) beam_select_kernel(BeamArgs a) {
    constexpr int IT = 4 * J, kBlock = kBeamThreads * IT, kSeg = kSegBlocks<J>;
    // the pieces' part and the groups' part use the memory one after the other
    __shared__ __align__(16) union {
        struct {
            unsigned long long best[kBeamThreads], list[kList], cut[kCut];
        } c;
        ChooseShared g;
    } sm;
    __shared__ float s_top[kBeamThreads / 2];
    __shared__ unsigned long long s_bound;
    __shared__ float s_floor;
    __shared__ int s_n, s_cut, s_last;
    __shared__ float red_m[2][kBeamThreads / 32], red_s[2][kBeamThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int gl = group_lanes(a.n_out), groups = kBeamThreads / gl;
    const int few = a.n_out + max(16, a.n_out / 2);  // keys a step may find in the list: at most 96
    int unit = blockIdx.x * a.share;
    const int unit1 = min(a.units - unit, a.share) + unit;
    while (unit < unit1) {
        const int row = unit / a.segs, seg0 = unit % a.segs, n_segs = min(a.segs - seg0, unit1 - unit);
        unit += n_segs;
        const int group = row / a.beams, chunk = blockIdx.x - first_cta(a, row);
        const int64_t base = (int64_t)seg0 * (kSeg * kBlock);
        const int n = (int)min((int64_t)n_segs * (kSeg * kBlock), a.n_vocab - base);
        const float* x = a.logits + (int64_t)row * a.stride + base;
        const int blocks = (n + kBlock - 1) / kBlock;

        // place in the piece of the thread's value j of block b
        auto index = [&](int b, int j) {
            return QUAD ? b * kBlock + ((j >> 2) * kBeamThreads + tid) * 4 + (j & 3) : b * kBlock + j * kBeamThreads + tid;
        };
        const float* xt = x + index(0, 0);
        float v[IT], next[IT] = {};
        auto load = [&](float (&to)[IT], int b) {
            const float* from = xt + b * kBlock;
            const int left = n - index(b, 0);  // values from the thread's first on
            if (QUAD) {
#pragma unroll
                for (int j = 0; j < IT; j += 4) {
                    const float4 y = j * kBeamThreads + 3 < left ? __ldcs(reinterpret_cast<const float4*>(from + j * kBeamThreads))
                                                                 : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
                    to[j] = y.x; to[j + 1] = y.y; to[j + 2] = y.z; to[j + 3] = y.w;
                }
                if (left < IT * kBeamThreads && (n & 3)) {  // a row's last one to three values
#pragma unroll
                    for (int j = 0; j < IT; j += 4)
#pragma unroll
                        for (int k = 0; k < 3; ++k)
                            if (j * kBeamThreads + k < left && j * kBeamThreads + 3 >= left) to[j + k] = from[j * kBeamThreads + k];
                }
            } else if (n - b * kBlock >= kBlock) {
#pragma unroll
                for (int j = 0; j < IT; ++j) to[j] = __ldcs(from + j * kBeamThreads);
            } else {
#pragma unroll
                for (int j = 0; j < IT; ++j) to[j] = j * kBeamThreads < left ? __ldcs(from + j * kBeamThreads) : -INFINITY;
            }
        };
        load(v, 0);

        float m = -INFINITY, s = 0.0f;  // running maximum and sum; a NaN or +inf makes the sum NaN
        auto take_block = [&]() {       // largest number of the block's values
            float top = v[0];
#pragma unroll
            for (int j = 1; j < IT; ++j) top = fmaxf(top, v[j]);
            if (top != top) top = -INFINITY;
            const float m1 = fmaxf(m, top), ref = m1 > -INFINITY ? m1 : 0.0f;
            const uint64_t ref2 = pack_f2(ref, ref), log2e = pack_f2(1.4426950408889634f, 1.4426950408889634f);
            uint64_t sum2 = pack_f2(m > -INFINITY ? s * ex2((m - ref) * 1.4426950408889634f) : s, 0.0f);
#pragma unroll
            for (int j = 0; j < IT; j += 2) {
                const uint64_t t = mul_f2(sub_f2(pack_f2(v[j], v[j + 1]), ref2), log2e);
                sum2 = add_f2(sum2, pack_f2(ex2(f2_lo(t)), ex2(f2_hi(t))));
            }
            s = f2_lo(sum2) + f2_hi(sum2);
            m = m1;
            return top;
        };
        // the CTA's sum of segment seg (two sets of warp sums in turn: the next segment's are written while these are read)
        auto give_segment = [&](int seg) {
            const float wm = warp_max(m);
            const float ws = warp_sum(m > -INFINITY ? s * expf(m - wm) : s);
            if (lane == 0) {
                red_m[seg & 1][warp] = wm;
                red_s[seg & 1][warp] = ws;
            }
            m = -INFINITY;
            s = 0.0f;
            __syncthreads();
            if (warp == kBeamThreads / 32 - 1) {
                const float m0 = lane < kBeamThreads / 32 ? red_m[seg & 1][lane] : -INFINITY;
                const float s0 = lane < kBeamThreads / 32 ? red_s[seg & 1][lane] : 0.0f;
                const float m1 = warp_max(m0), s1 = warp_sum(m0 > -INFINITY ? s0 * expf(m0 - m1) : s0);
                if (lane == 0) a.stat[(int64_t)row * a.segs + seg] = SegmentStat{m1, s1};
            }
        };
        // s_floor: the n_out-th largest of the lane groups' values of `top`
        auto find_floor = [&](float top) {
            for (int o = 1; o < gl; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            if (tid % gl == 0) s_top[tid / gl] = top;
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
            __syncthreads();
        };
        auto push = [&](float y, int i) {
            const int at = atomicAdd(&s_n, 1);
            if (at < kList) sm.c.list[at] = argmax_key(y + 0.0f, i);  // -0 and 0 are one value
        };
        // the list's n_out best to its front, in order; s_floor: the smallest of them (all threads; the list is complete
        // and has n_out keys or more)
        auto cut_list = [&](int count) {
            if (count <= kBeamThreads) {  // one key per thread
                const unsigned long long key = tid < count ? sm.c.list[tid] : 0ull;
                const int r = tid < count ? key_rank(sm.c.list, count, key) : kBeamThreads;
                __syncthreads();  // all have read the list
                if (r < a.n_out) sm.c.list[r] = key;
                if (r == a.n_out - 1) s_floor = key_value(key);
            } else {  // first those from the n_out-th largest of the threads' own largest keys on
                unsigned long long mine = 0;
                for (int c = tid; c < count; c += kBeamThreads) mine = max(mine, sm.c.list[c]);
                sm.c.best[tid] = mine;
                if (tid == 0) s_cut = 0;
                __syncthreads();
                if (key_rank(sm.c.best, kBeamThreads, mine) == a.n_out - 1) s_bound = mine;
                __syncthreads();
                const unsigned long long bound = s_bound;
                if (mine >= bound)
                    for (int c = tid; c < count; c += kBeamThreads)
                        if (sm.c.list[c] >= bound) sm.c.cut[atomicAdd(&s_cut, 1)] = sm.c.list[c];
                __syncthreads();
                const int kept = s_cut;
                for (int c = tid; c < kept; c += kBeamThreads) {
                    const unsigned long long key = sm.c.cut[c];
                    const int r = key_rank(sm.c.cut, kept, key);
                    if (r < a.n_out) sm.c.list[r] = key;
                    if (r == a.n_out - 1) s_floor = key_value(key);
                }
            }
            if (tid == 0) s_n = a.n_out;
            __syncthreads();
        };

        if (tid == 0) s_n = 0;
        float floor = -INFINITY;
        bool full = false;
        for (int b = 0; b < blocks; ++b) {
            if (b + 1 < blocks) load(next, b + 1);
            const float top = take_block();
            if ((b + 1) % kSeg == 0 || b + 1 == blocks) give_segment(seg0 + b / kSeg);
            if (b == 0) {
                find_floor(top);
                floor = s_floor;
            }
            // a later value has to be above the bound, one of the first block at it
            if (!full && (b == 0 ? top >= floor : top > floor)) {
                // one bit per value, the last in bit 0: the sign of bound - value (of value - bound in the first block;
                // a bound of 0 gets the sign with which -0 and 0 leave no sign)
                const float fl = floor == 0.0f ? (b == 0 ? -0.0f : 0.0f) : floor;
                const uint64_t fl2 = pack_f2(fl, fl);
                unsigned hit = 0;
#pragma unroll
                for (int j = 0; j < IT; j += 2) {
                    const uint64_t x2 = pack_f2(v[j], v[j + 1]);
                    const uint64_t d = b == 0 ? sub_f2(x2, fl2) : sub_f2(fl2, x2);
                    hit = __funnelshift_l((uint32_t)d, hit, 1);
                    hit = __funnelshift_l((uint32_t)(d >> 32), hit, 1);
                }
                if (b == 0) hit = ~hit & ((1u << IT) - 1);
                while (hit) {
                    const int bit = 31 - __clz(hit), j = IT - 1 - bit, i = index(b, j);
                    hit ^= 1u << bit;
                    float y[IT];  // y[0] becomes v[j]
#pragma unroll
                    for (int t = 0; t < IT; ++t) y[t] = v[t];
#pragma unroll
                    for (int w = IT / 2; w > 0; w >>= 1)
#pragma unroll
                        for (int t = 0; t < w; ++t) y[t] = (j & w) ? y[t + w] : y[t];
                    if (i < n) push(y[0], i);
                }
            }
            if (!full && ((b & 3) == 3 || b + 1 == blocks)) {
                __syncthreads();
                const int count = s_n;
                __syncthreads();  // s_n has been read before anyone adds to it
                full = count > kList;
                if (!full && count > few) {
                    cut_list(count);
                    floor = s_floor;
                }
            }
#pragma unroll
            for (int j = 0; j < IT; ++j) v[j] = next[j];
        }
        if (full) {  // 1024 values at a time, the list looked at after each
            if (tid == 0) s_n = 0;
            for (int i0 = tid; i0 - tid < n; i0 += 4 * kBeamThreads) {
                float y[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) y[k] = i0 + k * kBeamThreads < n ? x[i0 + k * kBeamThreads] : -INFINITY;
                if (i0 == tid) {
                    const float top = fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3]));
                    find_floor(top == top ? top : -INFINITY);
                    floor = s_floor;
                }
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (i0 + k * kBeamThreads < n && (i0 == tid ? y[k] >= floor : y[k] > floor))
                        push(y[k], i0 + k * kBeamThreads);
                __syncthreads();
                const int count = s_n;
                __syncthreads();
                if (count > few) {
                    cut_list(count);
                    floor = s_floor;
                }
            }
        }
        ChunkCand* out = a.cand + ((int64_t)row * a.chunks + chunk) * a.n_out;
        const int nc = s_n;
        for (int c = tid; c < nc; c += kBeamThreads) {
            const unsigned long long key = sm.c.list[c];
            const int r = key_rank(sm.c.list, nc, key);
            if (r < a.n_out) out[r] = ChunkCand{key_value(key), (int32_t)base + argmax_key_index(key)};
        }
        // fewer values than n_out (NaN are none: their row is not chosen from)
        for (int r = nc + tid; r < a.n_out; r += kBeamThreads) out[r] = ChunkCand{-INFINITY, -1};

        __syncthreads();
        if (warp == 0) {
            int all_pieces = 0;
            for (int b = lane; b < a.beams; b += 32) all_pieces += row_pieces(a, group * a.beams + b);
            all_pieces = __reduce_add_sync(0xffffffffu, all_pieces);
            if (lane == 0) s_last = take_ticket(a.counters + group) == (unsigned)(all_pieces - 1);
        }
        __syncthreads();
        if (!s_last) continue;  // the same in every thread; what the next piece writes first is behind a barrier
        if (tid == 0) a.counters[group] = 0;
        choose(a, sm.g, group);
        __syncthreads();  // the shared memory is the next piece's
    }
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
           // blocks are counted in 32 bits
           (int64_t)groups * beams * (n_vocab / 2048 + 1) < INT32_MAX - kBeamVocab;
}

size_t llama_q8_beam_select_workspace_bytes(int32_t groups, int32_t beams, int32_t n_vocab, int32_t n_out) {
    if (!beam_sizes_ok(groups, beams, n_vocab, n_out) || !beam_sizes_supported(groups, beams, n_vocab, n_out)) return 0;
    return beam_workspace(groups, beams, n_vocab, n_out, nullptr, nullptr);
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
    if (workspace_bytes < beam_workspace(groups, beams, n_vocab, n_out, &a, workspace)) return LQ8_ERR_ARG;
    if (groups == 0) return LQ8_OK;
    a.logits = logits, a.stride = logits_stride, a.scores = scores, a.beams = beams, a.n_vocab = n_vocab;
    a.n_out = n_out, a.out_scores = out_scores, a.out_parent = out_parent, a.out_token = out_token;
    const BeamCut cut = beam_cut((int64_t)groups * beams, n_vocab);
    const dim3 grid((unsigned)cut.ctas), block(kBeamThreads);
    cudaStream_t st = (cudaStream_t)stream;
    const bool quad = ((uintptr_t)logits & 15) == 0 && logits_stride % 4 == 0;
    const cudaError_t e =
        cut.j == 4 ? (quad ? launch_ex(beam_select_kernel<4, true>, grid, block, 0, st, false, a)
                           : launch_ex(beam_select_kernel<4, false>, grid, block, 0, st, false, a))
                   : (quad ? launch_ex(beam_select_kernel<2, true>, grid, block, 0, st, false, a)
                           : launch_ex(beam_select_kernel<2, false>, grid, block, 0, st, false, a));
    return e == cudaSuccess ? LQ8_OK : LQ8_ERR_CUDA;
}

}  // extern "C"
