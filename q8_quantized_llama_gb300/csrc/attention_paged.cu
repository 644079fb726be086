// Grouped-query attention of single tokens over the pages of a KV cache.
//
// For a row and KV head: s_j = scale q . k_j over the visible positions, m =
// max s, l = sum exp(s_j - m), out = sum exp(s_j - m) v_j / l, lse = m + ln l,
// in one pass with a running m and l (in units of log2: q is multiplied by
// scale * log2 e once).
//
// Bound: memory; each visible K and V row is read once, for all query heads of
// its group.
//
// Split. The visible positions of all (row, KV head) pairs are laid end to end
// in units of a few tiles and dealt evenly to the CTAs, whatever the lengths:
// every CTA adds up the rows' units itself (positions live on the device) and
// takes the same share. Pairs that lie in one CTA's share are finished there;
// the parts of the others go to the workspace and the CTA that finishes last
// (a counter per pair) joins them in the order of the positions.
//
// Inside a CTA each of four warps takes one tile of every unit through a ring
// of its own (cp.async, zero-filled outside the visible range, 16-byte pieces
// XOR-swizzled by row), keeps its own m, l and output in registers and needs no
// CTA barrier until the end of the pair. Page numbers are fetched 32 at a time,
// one per lane; a piece's successor is begun before the piece is joined.
//
// 16-bit pages: mma.sync m16n8k16. A group has at most 8 query heads, so rows
// 0-7 of the A operand carry the high part of q (or of the probabilities) and
// rows 8-15 the rest: one product gives both, and their sum is two registers of
// one thread. tcgen05 (128 rows) would idle 15/16 of its rows and pass the
// probabilities through tensor memory; the kernel is bound by memory without.
//  - f16: q is scaled per head by a power of two (largest value into [2^14,
//    2^15)) and split in two: 22 bits; the probabilities by 2^14.
//  - bf16: q and the probabilities in three parts, 24 bits. Groups of up to 4
//    heads have the three parts in rows 0-3, 4-7 and 8-11 of one product; larger
//    ones the third in a second product.
// Long sums are kept in two levels: o and l of up to kFold tiles, added to o_all
// and l_all. In one chain a warp's share of 131071 positions was off by up to
// 1.2e-4 (f32, equal probabilities, whose roundings all go one way), and by 3.5e-5
// on average in the tensor cores, which cut digits off; in two levels 1.4e-6 and
// less (64 rows 150 -> 151 us, one row of 131071 90.3 -> 91).
// f32 pages: f32 products. Scores: a few lanes per key over the dimensions,
// q from shared memory; output: a few dimensions per lane.
//
// Measured (bytes of the visible rows per time, of 6.7 TB/s that a copy reaches):
// 64 rows up to 8191 positions, f16, 32/8 heads of 128: 151 us, 6.4 TB/s; one
// row of 131071, bf16: 91 us, 5.9; 48 rows up to 4096, f32, 9/3 heads of 64: 32
// us, 4.3. Where the bytes are few, the fixed chain is what takes the time:
// positions (1.3 us), page numbers, first tiles, join, ticket and parts, about 7
// us in all. f32 groups of 5-8 heads are bound by their arithmetic instead (2900
// cycles per tile and warp: 16/2 heads of 128, 32 rows: 45 us, 20 for the bytes).
#include <algorithm>
#include <type_traits>

#include "kernels.cuh"
#include "paged.cuh"
#include "ptx.cuh"

namespace lq8 {
namespace {

constexpr int kWarps = 4, kThreads = kWarps * 32, kMaxG = 8;
constexpr int kMaxCtas = 2 * 152;      // two per SM: one joins while the other streams
constexpr int kRingBytes = 24 * 1024;  // per warp
constexpr int kMinShare = 2;           // units a CTA takes at least
constexpr int kJoin = 16;              // parts joined at once where a pair has more than twice as many
static_assert((kMaxCtas + kJoin - 1) / kJoin <= 32, "one lane per part or group");

// The running reference m of the exponentials follows the maximum when that is more than kLag (units of log2) above it:
// every change rounds all sums so far, and one per tile, as under rising scores, put 1.2e-4 on lse over 131071
// positions; this way what a change rounds counts half after the next. Probabilities are 2^kLag at most, which times
// kUpF16 f16 holds.
constexpr float kLag = 1.0f, kUpF16 = 16384.0f;

struct AttnArgs {
    const float* q;
    const int32_t* pos;
    const int32_t* seq;
    int rows, n_head;
    float scale_log2;
    int window;
    float* out;
    float* lse;
    int32_t* err;
    // workspace
    unsigned int* counters;  // zero between launches: [2 * kMaxCtas] by the first part's slot, [kMaxCtas] by the first CTA
    float2* part_ml;         // [2 * kMaxCtas][G]
    float* part_o;           // [2 * kMaxCtas][G][HD]
};

size_t attn_paged_workspace(int n_head, int n_kv, int hd, AttnArgs* a, void* ws) {
    const int G = n_head / n_kv;
    const size_t c = kCounterBytes;
    const size_t ml = (sizeof(float2) * 2 * kMaxCtas * G + 255) / 256 * 256;
    if (a) {
        uint8_t* w = reinterpret_cast<uint8_t*>(ws);
        a->counters = reinterpret_cast<unsigned int*>(w);
        a->part_ml = reinterpret_cast<float2*>(w + c);
        a->part_o = reinterpret_cast<float*>(w + c + ml);
    }
    return c + ml + sizeof(float) * 2 * kMaxCtas * (size_t)G * hd;
}

template <typename T, int HD>
struct Shape {
    static constexpr int kTile = 4096 / (HD * (int)sizeof(T));     // keys per warp and step: 4 KB of K, 4 KB of V
    static constexpr int kRowBytes = HD * (int)sizeof(T);
    static constexpr int kUnit = kWarps * kTile;                   // positions
    static constexpr int kChunks = kRowBytes / 16;
    static constexpr int kFold = sizeof(T) == 4 ? 16 : 32;         // tiles per partial sum
};
constexpr int kTileBytes = 4096;                                   // of K or of V
constexpr int kStages = kRingBytes / (2 * kTileBytes);
constexpr int kSmemQ = kWarps * kRingBytes;                        // [2][8][HD] q of this piece and the next
constexpr int kSmemP = kSmemQ + 2 * kMaxG * 128 * 4;               // f32: [warp][tile][8] probabilities, each twice
constexpr int kSmemMl = kSmemP + kWarps * 16 * kMaxG * 8;          // [warp][8] m, l
constexpr int kSmemBytes = kSmemMl + kWarps * kMaxG * 8;
static_assert(kMaxG * 128 * 4 <= kTileBytes, "a warp's output waits in one tile of its ring");

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void mma16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, __half) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, __nv_bfloat16) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// (x, y) rounded to the type; x, y left with what the rounding dropped
__device__ __forceinline__ uint32_t take_part(float& x, float& y, __half) {
    const __half2 h = __floats2half2_rn(x, y);
    const float2 f = __half22float2(h);
    x -= f.x;
    y -= f.y;
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t take_part(float& x, float& y, __nv_bfloat16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    const float2 f = __bfloat1622float2(h);
    x -= f.x;
    y -= f.y;
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ int order_int(float x) {
    const int b = __float_as_int(x);
    return b >= 0 ? b : b ^ 0x7fffffff;
}
__device__ __forceinline__ float order_float(int b) { return __int_as_float(b >= 0 ? b : b ^ 0x7fffffff); }

// Visible positions [lo, hi) of a row; status: what is wrong with it.
struct Range {
    int lo, hi, seq, status;
};
__device__ __forceinline__ Range row_range(const AttnArgs& a, const TableView& tb, int shift, int row) {
    Range g{0, 0, 0, 0};
    const int p = a.pos[row];
    g.seq = a.seq ? a.seq[row] : row;
    if (p < 0) return g;
    if (g.seq < 0 || g.seq >= tb.n_seq) {
        g.status = LQ8_ERR_ARG;
        return g;
    }
    const int64_t end = (int64_t)p + 1, cap = min((int64_t)tb.stride << shift, (int64_t)INT32_MAX - 1023);
    if (end > cap) g.status = LQ8_ERR_CTX;
    const int64_t lo = a.window > 0 && end > a.window ? end - a.window : 0;
    g.hi = (int)min(end, cap);
    g.lo = (int)min(lo, (int64_t)g.hi);
    return g;
}
template <int UNIT>
__device__ __forceinline__ int range_units(const Range& g) {
    return g.hi > g.lo ? (g.hi + UNIT - 1) / UNIT - g.lo / UNIT : 0;
}

__device__ constexpr int log2_ceil(int x) { return x <= 1 ? 0 : 1 + log2_ceil((x + 1) / 2); }

// One warp's running state over one (row, KV head). A lane's accumulators belong to rows lane / 4 and lane / 4 + 8.
template <typename T, int HD, int GP>
struct State16 {
    static constexpr bool kHalf = std::is_same<T, __half>::value;
    static constexpr bool kOne = !kHalf && GP == 4;  // three parts in one product: lanes of rows 4-7 have the second
    static constexpr bool kTwo = !kHalf && GP == 8;  // the third part in a second product
    uint32_t q[HD / 16][4];
    uint32_t q3[kTwo ? HD / 16 : 1][2];
    uint64_t o[HD / 8], o_all[HD / 8];  // pairs of dimensions
    float m, l, l_all, q_inv;
};
// (x, y) as the two words of an A operand for a row's parts: rows lane / 4 and lane / 4 + 8, and the third part apart.
template <typename St, typename T>
__device__ __forceinline__ void split_parts(float x, float y, uint32_t& top, uint32_t& low, uint32_t& third, int lane, T tag) {
    top = take_part(x, y, tag);
    low = take_part(x, y, tag);
    if (St::kTwo) third = take_part(x, y, tag);
    if (St::kOne) {
        const bool second = lane >= 16;  // rows 4-7
        top = second ? low : top;
        low = second ? 0u : take_part(x, y, tag);
    }
}
template <int HD>
struct State32 {
    uint64_t o[kMaxG][HD / 64], o_all[kMaxG][HD / 64];  // pairs of dimensions
    float m[kMaxG], l[kMaxG], l_all[kMaxG];  // m the same in every lane, l a part per lane
};

// q [G][HD] in shared memory
template <typename T, int HD, int GP>
__device__ __forceinline__ void state_init(State16<T, HD, GP>& s, const float* q, int G, float scale, int lane) {
    using St = State16<T, HD, GP>;
    const int g = St::kOne ? (lane >> 2) & 3 : lane >> 2, t = lane & 3;
    const T tag{};
    float v[HD / 16][4];
    float mx = 0.0f;
#pragma unroll
    for (int k = 0; k < HD / 16; ++k) {
        float2 x = make_float2(0.f, 0.f), y = x;
        if (g < G) {
            x = *reinterpret_cast<const float2*>(q + g * HD + k * 16 + 2 * t);
            y = *reinterpret_cast<const float2*>(q + g * HD + k * 16 + 8 + 2 * t);
        }
        v[k][0] = x.x * scale; v[k][1] = x.y * scale;
        v[k][2] = y.x * scale; v[k][3] = y.y * scale;
#pragma unroll
        for (int j = 0; j < 4; ++j) mx = fmaxf(mx, fabsf(v[k][j]));
    }
    float up = 1.0f;
    s.q_inv = 1.0f;
    if (St::kHalf) {
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const int sh = row_shift(mx);
        up = pow2f(sh);
        s.q_inv = pow2f(-sh);
    }
#pragma unroll
    for (int k = 0; k < HD / 16; ++k) {
        uint32_t* third = s.q3[St::kTwo ? k : 0];
        split_parts<St>(v[k][0] * up, v[k][1] * up, s.q[k][0], s.q[k][1], third[0], lane, tag);
        split_parts<St>(v[k][2] * up, v[k][3] * up, s.q[k][2], s.q[k][3], third[1], lane, tag);
    }
#pragma unroll
    for (int d = 0; d < HD / 8; ++d) s.o[d] = s.o_all[d] = 0;
    s.m = -INFINITY;
    s.l = s.l_all = 0.0f;
}

// A tile of 2048 / HD keys: K at ks, V at vs (shared addresses); key j of the tile counts if bit j of see is set.
template <typename T, int HD, int GP>
__device__ __forceinline__ void state_tile(State16<T, HD, GP>& s, uint32_t ks, uint32_t vs, unsigned see, int lane) {
    using St = State16<T, HD, GP>;
    constexpr int RB = HD * 2, NT = 2048 / HD / 8;  // blocks of 8 keys
    const T tag{};
    const int l8 = lane & 7, mi = lane >> 3, t = lane & 3;
    // short chains: even and odd steps, and the third part of q, each in sums of their own (the tensor cores cut
    // digits off at every addition to a sum, in proportion to the sum)
    float x[2 * NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        float c[2][4] = {}, c3[4] = {};
#pragma unroll
        for (int k = 0; k < HD / 32; ++k) {
            uint32_t b[4];
            ldsm4(b, ks + (n * 8 + l8) * RB + (((k * 4 + mi) ^ l8) << 4));
            mma16(c[0], s.q[2 * k], b[0], b[1], tag);
            mma16(c[1], s.q[2 * k + 1], b[2], b[3], tag);
            if constexpr (St::kTwo) {
                const uint32_t a0[4] = {s.q3[2 * k][0], 0, s.q3[2 * k][1], 0};
                const uint32_t a1[4] = {s.q3[2 * k + 1][0], 0, s.q3[2 * k + 1][1], 0};
                mma16(c3, a0, b[0], b[1], tag);
                mma16(c3, a1, b[2], b[3], tag);
            }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float y = (c[0][i] + c[1][i]) + (c[0][i + 2] + c[1][i + 2] + c3[i]);
            if (St::kOne) y += __shfl_xor_sync(0xffffffffu, y, 16);  // the first and third part, and the second
            if (St::kHalf) y *= s.q_inv;
            x[2 * n + i] = (see >> (n * 8 + 2 * t + i)) & 1 ? y : -INFINITY;
        }
    }
    float mx = x[0];
#pragma unroll
    for (int j = 1; j < 2 * NT; ++j) mx = fmaxf(mx, x[j]);
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    // finite: a tile in which nothing counts is not given to this function
    const float m = mx - s.m > kLag ? mx : s.m;
    if (__any_sync(0xffffffffu, m > s.m)) {
        const float f = ex2(s.m - m);
        s.m = m;
        s.l *= f;
        s.l_all *= f;
        const uint64_t f2 = pack_f2(f, f);
#pragma unroll
        for (int d = 0; d < HD / 8; ++d) {
            s.o[d] = mul_f2(s.o[d], f2);
            s.o_all[d] = mul_f2(s.o_all[d], f2);
        }
    }
    uint32_t a[NT / 2][4], a3[NT / 2][4] = {};
#pragma unroll
    for (int j = 0; j < 2 * NT; ++j) {
        x[j] = ex2(x[j] - m);
        // f16: times 2^14, so that the second part of a small one is not lost below f16's range. Not as m - 14 in the
        // exponent: far from zero that rounds, up to where the largest probability leaves f16's range.
        if (St::kHalf) x[j] *= kUpF16;
    }
#pragma unroll
    for (int h = 0; h < NT / 2; ++h) {
        split_parts<St>(x[4 * h], x[4 * h + 1], a[h][0], a[h][1], a3[h][0], lane, tag);
        split_parts<St>(x[4 * h + 2], x[4 * h + 3], a[h][2], a[h][3], a3[h][2], lane, tag);
    }
#pragma unroll
    for (int w = NT; w > 0; w >>= 1)
#pragma unroll
        for (int j = 0; j < w; ++j) x[j] += x[j + w];
    s.l += x[0];
    // the tile's products in sums of their own, added to the running ones with rounding
#pragma unroll
    for (int d = 0; d < HD / 16; ++d) {
        float c[2][4] = {};
#pragma unroll
        for (int h = 0; h < NT / 2; ++h) {
            uint32_t b[4];
            ldsm4_t(b, vs + (h * 16 + (mi & 1) * 8 + l8) * RB + (((2 * d + (mi >> 1)) ^ l8) << 4));
            mma16(c[0], a[h], b[0], b[1], tag);
            mma16(c[1], a[h], b[2], b[3], tag);
            if constexpr (St::kTwo) {
                mma16(c[0], a3[h], b[0], b[1], tag);
                mma16(c[1], a3[h], b[2], b[3], tag);
            }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
            s.o[2 * d + i] = add_f2(s.o[2 * d + i], add_f2(pack_f2(c[i][0], c[i][1]), pack_f2(c[i][2], c[i][3])));
    }
}
template <typename T, int HD, int GP>
__device__ __forceinline__ void state_fold(State16<T, HD, GP>& s) {
#pragma unroll
    for (int d = 0; d < HD / 8; ++d) {
        s.o_all[d] = add_f2(s.o_all[d], s.o[d]);
        s.o[d] = 0;
    }
    s.l_all += s.l;
    s.l = 0.0f;
}

// The warp's part: output [8][HD] to ob, m and l of its heads to ml (l of f16 pages carries kUpF16).
template <typename T, int HD, int GP>
__device__ __forceinline__ void state_store(State16<T, HD, GP>& s, float* ob, float2* ml, int lane) {
    constexpr bool kOne = State16<T, HD, GP>::kOne;
    const int g = lane >> 2, t = lane & 3;
    float l = s.l_all + s.l;
    l += __shfl_xor_sync(0xffffffffu, l, 1);
    l += __shfl_xor_sync(0xffffffffu, l, 2);
    if (t == 0) ml[g] = make_float2(s.m, l);
#pragma unroll
    for (int d = 0; d < HD / 8; ++d) {
        const uint64_t o = add_f2(s.o_all[d], s.o[d]);
        float x = f2_lo(o), y = f2_hi(o);
        if (kOne) {
            x += __shfl_xor_sync(0xffffffffu, x, 16);
            y += __shfl_xor_sync(0xffffffffu, y, 16);
        }
        if (!kOne || g < 4) *reinterpret_cast<float2*>(ob + g * HD + d * 8 + 2 * t) = make_float2(x, y);
    }
}

template <int HD, int GP>
__device__ __forceinline__ void state_init(State32<HD>& s) {
#pragma unroll
    for (int g = 0; g < GP; ++g) {
#pragma unroll
        for (int d = 0; d < HD / 64; ++d) s.o[g][d] = s.o_all[g][d] = 0;
        s.m[g] = -INFINITY;
        s.l[g] = s.l_all[g] = 0.0f;
    }
}

// A tile of 1024 / HD keys; q [GP][HD] and the warp's probabilities [tile][8], each twice, in shared memory.
template <int HD, int GP>
__device__ __forceinline__ void state_tile(State32<HD>& s, const uint8_t* ks, const uint8_t* vs, const float* q,
                                           float* pb, float scale, unsigned see, int lane) {
    constexpr int TK = 1024 / HD, LPK = 32 / TK, CPL = HD / 4 / LPK;  // keys, lanes per key, 16-byte pieces per lane
    constexpr int RB = HD * 4;
    const int key = lane % TK, part = lane / TK;
    uint64_t acc[GP];
#pragma unroll
    for (int g = 0; g < GP; ++g) acc[g] = 0;
#pragma unroll
    for (int i = 0; i < CPL; ++i) {
        const int ch = part * CPL + i;
        const ulonglong2 kv = *reinterpret_cast<const ulonglong2*>(ks + key * RB + ((ch ^ (key & 7)) << 4));
#pragma unroll
        for (int g = 0; g < GP; ++g) {
            const ulonglong2 qv = *reinterpret_cast<const ulonglong2*>(q + g * HD + ch * 4);
            acc[g] = fma_f2(kv.x, qv.x, acc[g]);
            acc[g] = fma_f2(kv.y, qv.y, acc[g]);
        }
    }
    const bool in = (see >> key) & 1;
    float p[GP], m[GP];
    bool grew = false;
#pragma unroll
    for (int g = 0; g < GP; ++g) {
        float x = (f2_lo(acc[g]) + f2_hi(acc[g])) * scale;
#pragma unroll
        for (int o = TK; o < 32; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
        if (!in) x = -INFINITY;
        const float mx = order_float(__reduce_max_sync(0xffffffffu, order_int(x)));
        m[g] = mx - s.m[g] > kLag ? mx : s.m[g];
        grew |= m[g] > s.m[g];
        p[g] = ex2(x - m[g]);
    }
    if (grew) {  // the same in every lane
#pragma unroll
        for (int g = 0; g < GP; ++g) {
            const float f = ex2(s.m[g] - m[g]);
            s.m[g] = m[g];
            s.l[g] *= f;
            s.l_all[g] *= f;
            const uint64_t f2 = pack_f2(f, f);
#pragma unroll
            for (int d = 0; d < HD / 64; ++d) {
                s.o[g][d] = mul_f2(s.o[g][d], f2);
                s.o_all[g][d] = mul_f2(s.o_all[g][d], f2);
            }
        }
    }
    __syncwarp();  // the last tile's probabilities have been read
    if (part == 0) {
#pragma unroll
        for (int g = 0; g < GP; ++g) s.l[g] += p[g];
#pragma unroll
        for (int g = 0; g < GP; g += 2)
            *reinterpret_cast<float4*>(pb + (key * kMaxG + g) * 2) = make_float4(p[g], p[g], p[g + 1], p[g + 1]);
    }
    __syncwarp();
#pragma unroll
    for (int j = 0; j < TK; ++j) {
        uint64_t v[HD / 64];
        if constexpr (HD == 128) {
            const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(vs + j * RB + ((lane ^ (j & 7)) << 4));
            v[0] = x.x;
            v[1] = x.y;
        } else {
            v[0] = *reinterpret_cast<const uint64_t*>(vs + j * RB + (((lane >> 1) ^ (j & 7)) << 4) + (lane & 1) * 8);
        }
#pragma unroll
        for (int g = 0; g < GP; g += 2) {
            const ulonglong2 w = *reinterpret_cast<const ulonglong2*>(pb + (j * kMaxG + g) * 2);
#pragma unroll
            for (int d = 0; d < HD / 64; ++d) {
                s.o[g][d] = fma_f2(w.x, v[d], s.o[g][d]);
                s.o[g + 1][d] = fma_f2(w.y, v[d], s.o[g + 1][d]);
            }
        }
    }
}

template <int HD, int GP>
__device__ __forceinline__ void state_fold(State32<HD>& s) {
#pragma unroll
    for (int g = 0; g < GP; ++g) {
#pragma unroll
        for (int d = 0; d < HD / 64; ++d) {
            s.o_all[g][d] = add_f2(s.o_all[g][d], s.o[g][d]);
            s.o[g][d] = 0;
        }
        s.l_all[g] += s.l[g];
        s.l[g] = 0.0f;
    }
}

template <int HD, int GP>
__device__ __forceinline__ void state_store(State32<HD>& s, float* ob, float2* ml, int lane) {
#pragma unroll
    for (int g = 0; g < GP; ++g) {
        const float l = warp_sum(s.l_all[g] + s.l[g]);
        if (lane == 0) ml[g] = make_float2(s.m[g], l);
#pragma unroll
        for (int d = 0; d < HD / 64; ++d)
            *reinterpret_cast<uint64_t*>(ob + g * HD + lane * (HD / 32) + 2 * d) = add_f2(s.o_all[g][d], s.o[g][d]);
    }
}

// GP: query heads the f32 and bf16 forms carry (4 or 8); f16 has room for 8 in any case.
template <typename T, int HD, int GP>
__global__ void __launch_bounds__(kThreads, 2) attention_paged_kernel(AttnArgs a, PageView<T> pg, TableView tb) {
    using S = Shape<T, HD>;
    constexpr bool kF32 = sizeof(T) == 4;
    constexpr bool kHalf = std::is_same<T, __half>::value;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int s_scan[kWarps], s_base, s_row, s_last;
    __shared__ Range s_range;
    __shared__ unsigned s_see[kWarps][kStages];  // keys that count in each stage's tile
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int G = a.n_head / pg.n_kv, shift = pg.page_shift;
    uint8_t* ring = smem + warp * kRingBytes;
    float* pb = reinterpret_cast<float*>(smem + kSmemP) + warp * 16 * kMaxG * 2;
    float2* ml = reinterpret_cast<float2*>(smem + kSmemMl);
    if constexpr (kF32) {  // heads behind the group stay zero
        for (int i = G * HD + tid; i < GP * HD; i += kThreads) {
            reinterpret_cast<float*>(smem + kSmemQ)[i] = 0.0f;
            reinterpret_cast<float*>(smem + kSmemQ)[kMaxG * HD + i] = 0.0f;
        }
    }

    // ---- this CTA's share of the units of all rows -------------------------------------
    const int per = (a.rows + kThreads - 1) / kThreads;
    int mine = 0;
    Range own{0, 0, 0, 0};
    for (int i = 0; i < per; ++i) {
        const int r = tid * per + i;
        if (r < a.rows) {
            own = row_range(a, tb, shift, r);
            mine += range_units<S::kUnit>(own);
        }
    }
    int before = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += y;
    }
    if (lane == 31) s_scan[warp] = before;
    __syncthreads();
    int total = 0;
    before -= mine;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += s_scan[w];
        total += s_scan[w];
    }
    total *= pg.n_kv;
    const int share = max(kMinShare, (int)(((unsigned)total + gridDim.x - 1) / gridDim.x));
    int w0 = min(total, share * (int)blockIdx.x);  // units of all rows are counted in 31 bits (checked by the host)
    const int w1 = min(total - w0, share) + w0;
    if (w0 < w1 && before * pg.n_kv <= w0 && w0 < (before + mine) * pg.n_kv) {
        for (int r = tid * per;; ++r) {
            const Range g = per == 1 ? own : row_range(a, tb, shift, r);
            const int u = range_units<S::kUnit>(g);
            if (w0 < (before + u) * pg.n_kv) {
                s_row = r;
                s_range = g;
                s_base = before * pg.n_kv;
                break;
            }
            before += u;
        }
    }
    __syncthreads();
    // ---- the share's pieces: the part of a (row, KV head) pair that lies in it -------------
    // The next piece's page numbers and q are asked for during a piece, and its first tiles before the piece is
    // joined, so that only the first waits for the memory.
    struct Piece {
        Range rg;
        int row, kh, units, u, n;  // of the pair's `units` units, n from u on
        int base;                  // units before the row
        int tile0;                 // the warp's first tile
    };
    auto place = [&](Piece& p, int row, Range rg, int base, int w) {  // the piece that starts at unit w
        int units = range_units<S::kUnit>(rg);
        while (w - base >= units * pg.n_kv) {
            base += units * pg.n_kv;
            rg = row_range(a, tb, shift, ++row);
            units = range_units<S::kUnit>(rg);
        }
        const unsigned at = (unsigned)(w - base);
        p.rg = rg;
        p.row = row;
        p.base = base;
        p.units = units;
        p.kh = (int)(at / (unsigned)units);
        p.u = (int)(at % (unsigned)units);
        p.n = min(units - p.u, w1 - w);
        p.tile0 = (rg.lo / S::kUnit + p.u) * kWarps + warp;
    };
    // Page numbers, one per lane: entry e is part e % parts of tile e / parts (a tile can lie in 2 or 4 pages)
    const int part_shift = max(0, log2_ceil(S::kTile) - shift);
    auto entry = [&](const Piece& p, int e) {
        const int64_t pos = (int64_t)(p.tile0 + (e >> part_shift) * kWarps) * S::kTile +
                            ((e & ((1 << part_shift) - 1)) << shift);
        if ((e >> part_shift) >= p.n || pos >= p.rg.hi || pos + min(S::kTile, 1 << shift) <= p.rg.lo) return -1;
        return tb.table[(int64_t)p.rg.seq * tb.stride + (pos >> shift)];
    };
    auto ask_q = [&](const Piece& p, int buf) {
        const float* q = a.q + ((int64_t)p.row * a.n_head + p.kh * G) * HD;
        float* qs = reinterpret_cast<float*>(smem + kSmemQ) + buf * kMaxG * HD;
        for (int i = tid; i < G * (HD / 4); i += kThreads) cp_async16(qs + 4 * i, q + 4 * i, 16);
    };
    // The warp's tile j of p to stage st; ent: the entries of tiles from (j * parts) & ~31 on.
    auto issue = [&](const Piece& p, int j, int st, int ent) {
        const int pos = (p.tile0 + j * kWarps) * S::kTile;
        unsigned bits = S::kTile == 32 ? ~0u : (1u << S::kTile) - 1;
        if (pos + S::kTile > p.rg.hi) bits &= (1u << max(0, p.rg.hi - pos)) - 1;
        if (pos < p.rg.lo) bits &= p.rg.lo - pos >= S::kTile ? 0u : ~0u << (p.rg.lo - pos);
        constexpr int RPI = 32 / S::kChunks >= 1 ? 32 / S::kChunks : 1;  // rows per warp-wide copy
        const int ch = lane % S::kChunks, r0 = lane / S::kChunks;
        uint8_t* dst = ring + st * 2 * kTileBytes + r0 * S::kRowBytes;
        const int64_t lane_off = r0 * HD + ch * (16 / (int)sizeof(T)) + (((int64_t)p.kh << shift) * HD);
        int64_t off = 0;
#pragma unroll
        for (int g8 = 0; g8 < S::kTile / 8; ++g8) {  // 8 rows lie in one page
            const int part = (g8 * 8) >> shift;
            if (g8 == 0 || (part_shift && ((g8 * 8) & ((1 << shift) - 1)) == 0)) {
                int e = __shfl_sync(0xffffffffu, ent, ((j << part_shift) + part) & 31);
                if (e >= pg.n_pages) {
                    if (lane == 0) report(a.err, LQ8_ERR_ARG);
                    e = -1;
                }
                if (e < 0) bits &= ~(part_shift ? ((1u << (1 << shift)) - 1) << (part << shift) : ~0u);
                off = max(e, 0) * pg.page_elems + ((pos + g8 * 8) & ((1 << shift) - 1)) * HD + lane_off;
            }
#pragma unroll
            for (int i = 0; i < 8 / RPI; ++i) {
                const int r = i * RPI;  // + r0: the row of the block
                const uint32_t bytes = (bits >> (g8 * 8 + r + r0)) & 1 ? 16u : 0u;
                uint8_t* d = dst + (g8 * 8 + r) * S::kRowBytes + ((ch ^ (r + r0)) << 4);
                const int64_t o = off + (int64_t)r * HD;
                cp_async16(d, pg.k + o, bytes);
                cp_async16(d + kTileBytes, pg.v + o, bytes);
            }
            off += 8 * HD;
        }
        if (lane == 0) s_see[warp][st] = bits;
    };

    Piece cur, nxt;
    int ent = -1, ent_more = -1;  // of the current piece: the entries in use, and the 32 after them
    const int ent_tiles = 32 >> part_shift;
    if (w0 < w1) {
        place(cur, s_row, s_range, s_base, w0);
        ent = entry(cur, lane);
        ask_q(cur, 0);
        cp_async_commit();
        ent_more = entry(cur, 32 + lane);
#pragma unroll
        for (int j = 0; j < kStages - 1; ++j) {
            if (j < cur.n) issue(cur, j, j, ent);
            cp_async_commit();
        }
        cp_async_wait<kStages - 1>();
        __syncthreads();  // q of all threads' copies
    }
    int buf = 0, st0 = 0;  // q buffer, stage of the piece's first tile
    bool first = true;     // of this CTA's pieces
    while (w0 < w1) {
        const bool more = w0 + cur.n < w1;
        int nxt_ent = -1, nxt_more = -1;
        if (more) {
            place(nxt, cur.row, cur.rg, cur.base, w0 + cur.n);
            nxt_ent = entry(nxt, lane);
            nxt_more = entry(nxt, 32 + lane);
            ask_q(nxt, buf ^ 1);  // arrives with the next tile asked for
        }
        const float* qs = reinterpret_cast<const float*>(smem + kSmemQ) + buf * kMaxG * HD;
        std::conditional_t<kF32, State32<HD>, State16<std::conditional_t<kF32, __half, T>, HD, GP>> state;
        if constexpr (kF32)
            state_init<HD, GP>(state);
        else
            state_init(state, qs, G, a.scale_log2, lane);
        int st = st0;
        for (int j = 0; j < cur.n; ++j) {
            cp_async_wait<kStages - 2>();
            __syncwarp();  // every lane's pieces of tile j have arrived, and tile j - 1 has been read
            const unsigned bits = s_see[warp][st];
            const int ja = j + kStages - 1, sta = st == 0 ? kStages - 1 : st - 1;
            if (ja < cur.n) {
                if ((ja & (ent_tiles - 1)) == 0) {
                    ent = ent_more;
                    ent_more = entry(cur, (ja << part_shift) + 32 + lane);
                }
                issue(cur, ja, sta, ent);
            }
            cp_async_commit();
            if (bits) {
                const uint8_t* t = ring + st * 2 * kTileBytes;
                if constexpr (kF32)
                    state_tile<HD, GP>(state, t, t + kTileBytes, qs, pb, a.scale_log2, bits, lane);
                else
                    state_tile(state, smem_u32(t), smem_u32(t + kTileBytes), bits, lane);
            }
            if (j % S::kFold == S::kFold - 1) {
                if constexpr (kF32)
                    state_fold<HD, GP>(state);
                else
                    state_fold(state);
            }
            st = st == kStages - 1 ? 0 : st + 1;
        }
        // stages st and the one after it are free for the next piece's first tiles; the output waits in the last one's
        const int stl = st == 0 ? kStages - 1 : st - 1;
        __syncwarp();
        if (more) {
            int sj = st;
#pragma unroll
            for (int j = 0; j < kStages - 1; ++j) {
                if (j < nxt.n) issue(nxt, j, sj, nxt_ent);
                cp_async_commit();
                sj = sj == kStages - 1 ? 0 : sj + 1;
            }
            cp_async_wait<kStages - 1>();  // q of the next piece
        }
        float* ob = reinterpret_cast<float*>(ring + stl * 2 * kTileBytes);
        if constexpr (kF32)
            state_store<HD, GP>(state, ob, ml + warp * kMaxG, lane);
        else
            state_store(state, ob, ml + warp * kMaxG, lane);
        __syncthreads();

        // ---- join the warps: the result, or a part of it -----------------------------------
        const bool whole = cur.n == cur.units;
        const int slot = 2 * blockIdx.x + (first ? 0 : 1);
        const int64_t orow = (int64_t)cur.row * a.n_head + cur.kh * G;  // first head of the pair
        const uint8_t* parts_of_warps = smem + stl * 2 * kTileBytes;
        auto finish = [&](int e, float4 o, float m, float l) {  // value e of the pair from its sums
            const int g = e / (HD / 4);
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;
            reinterpret_cast<float4*>(a.out + orow * HD)[e] = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
            if (a.lse && e % (HD / 4) == 0)
                a.lse[orow + g] = l == 0.0f ? -INFINITY : m * 0.69314718055994531f + logf(kHalf ? l * (1.0f / kUpF16) : l);
        };
        for (int e = tid; e < G * (HD / 4); e += kThreads) {
            const int g = e / (HD / 4);
            float m = -INFINITY, l = 0.0f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) m = fmaxf(m, ml[w * kMaxG + g].x);
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float2 x = ml[w * kMaxG + g];
                const float f = x.x > -INFINITY ? ex2(x.x - m) : 0.0f;
                const float4 y = reinterpret_cast<const float4*>(parts_of_warps + w * kRingBytes)[e];
                l = fmaf(f, x.y, l);
                o.x = fmaf(f, y.x, o.x); o.y = fmaf(f, y.y, o.y);
                o.z = fmaf(f, y.z, o.z); o.w = fmaf(f, y.w, o.w);
            }
            if (whole) {
                finish(e, o, m, l);
            } else {
                reinterpret_cast<float4*>(a.part_o + (int64_t)slot * G * HD)[e] = o;
                if (e % (HD / 4) == 0) a.part_ml[slot * G + g] = make_float2(m, l);
            }
        }
        if (!whole) {
            // ---- the parts of a pair: many of them in groups of kJoin, each group and then the groups' results by
            // the CTA that finishes last, in the order of the positions -----------------------------
            const int seg0 = cur.base + cur.kh * cur.units;
            const int c0 = seg0 / share, c1 = (seg0 + cur.units - 1) / share, parts = c1 - c0 + 1;
            // the pair starts inside the first CTA's share unless it starts it
            const int slot0 = 2 * c0 + (seg0 == c0 * share ? 0 : 1);
            auto slot_of = [&](int i) { return i == 0 ? slot0 : 2 * (c0 + i); };
            auto arrive = [&](unsigned int* counter, int all) {
                __syncthreads();
                if (tid == 0) {
                    s_last = take_ticket(counter) == (unsigned)(all - 1);
                    if (s_last) *counter = 0;
                }
                __syncthreads();
                return s_last != 0;
            };
            float* wgt = reinterpret_cast<float*>(smem + stl * 2 * kTileBytes + kTileBytes);  // [count][G]
            float4* sums = reinterpret_cast<float4*>(smem + kRingBytes + stl * 2 * kTileBytes + kTileBytes);
            // parts i0, i0 + step, .. (count of them) to the result, or to the place of part i0
            auto join = [&](int i0, int step, int count, bool last) {
                for (int g = warp; g < G; g += kWarps) {
                    float m = -INFINITY, l = 0.0f;
                    const float2 x = lane < count ? __ldcg(&a.part_ml[slot_of(i0 + lane * step) * G + g])
                                                  : make_float2(-INFINITY, 0.0f);
                    m = warp_max(x.x);
                    const float f = x.x > -INFINITY ? ex2(x.x - m) : 0.0f;
                    if (lane < count) wgt[lane * G + g] = f;
                    l = warp_sum(f * x.y);
                    if (lane == 0) ml[g] = make_float2(m, l);
                }
                __syncthreads();
                // few heads: several groups of threads share the parts
                const int vecs = G * (HD / 4), groups = max(1, kThreads / vecs);
                const int chunk = (count + groups - 1) / groups;
                for (int e0 = tid; e0 < vecs * groups; e0 += kThreads) {
                    const int e = e0 % vecs, gr = e0 / vecs, g = e / (HD / 4);
                    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
                    const int i1 = min(count, (gr + 1) * chunk);
#pragma unroll 8
                    for (int i = gr * chunk; i < i1; ++i) {
                        const float f = wgt[i * G + g];
                        const float4 y = __ldcg(reinterpret_cast<const float4*>(
                                                    a.part_o + (int64_t)slot_of(i0 + i * step) * G * HD) + e);
                        o.x = fmaf(f, y.x, o.x); o.y = fmaf(f, y.y, o.y);
                        o.z = fmaf(f, y.z, o.z); o.w = fmaf(f, y.w, o.w);
                    }
                    sums[e0] = o;
                }
                __syncthreads();
                for (int e = tid; e < vecs; e += kThreads) {
                    float4 o = sums[e];
                    for (int gr = 1; gr < groups; ++gr) {
                        const float4 y = sums[gr * vecs + e];
                        o.x += y.x; o.y += y.y; o.z += y.z; o.w += y.w;
                    }
                    const int g = e / (HD / 4);
                    if (last) {
                        finish(e, o, ml[g].x, ml[g].y);
                    } else {
                        reinterpret_cast<float4*>(a.part_o + (int64_t)slot_of(i0) * G * HD)[e] = o;
                        if (e % (HD / 4) == 0) a.part_ml[slot_of(i0) * G + g] = ml[g];
                    }
                }
            };
            if (parts <= 2 * kJoin) {
                if (arrive(a.counters + slot0, parts)) join(0, 1, parts, true);
            } else {
                const int i0 = (int)(blockIdx.x - c0) / kJoin * kJoin, groups = (parts + kJoin - 1) / kJoin;
                const int count = min(kJoin, parts - i0);
                if (arrive(a.counters + slot_of(i0), count)) {
                    join(i0, 1, count, false);
                    if (arrive(a.counters + 2 * kMaxCtas + c0, groups)) join(0, kJoin, groups, true);
                }
            }
        }
        __syncthreads();  // the last tile's stage and ml are free
        first = false;
        w0 += cur.n;
        cur = nxt;
        ent = nxt_ent;
        ent_more = nxt_more;
        buf ^= 1;
        st0 = st;
    }
    // ---- rows that see nothing, and what is wrong with rows -------------------------------
    for (int r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const Range rg = row_range(a, tb, shift, r);
        if (rg.status && tid == 0) report(a.err, rg.status);
        if (rg.hi > rg.lo) continue;
        for (int i = tid; i < a.n_head * (HD / 4); i += kThreads)
            reinterpret_cast<float4*>(a.out + (int64_t)r * a.n_head * HD)[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (a.lse)
            for (int i = tid; i < a.n_head; i += kThreads) a.lse[(int64_t)r * a.n_head + i] = -INFINITY;
    }
}

template <typename T, int HD, int GP>
cudaError_t launch_one(const AttnArgs& a, const llama_q8_pages* p, int layer, const TableView& tb, cudaStream_t s) {
    // no more CTAs than units the table can hold, or than rows where those are more
    const int64_t units = (((int64_t)tb.stride * p->page + Shape<T, HD>::kUnit - 1) / Shape<T, HD>::kUnit + 1) *
                          a.rows * p->n_head_kv;
    const int64_t grid = std::min<int64_t>(kMaxCtas, std::max<int64_t>(1, (units + kMinShare - 1) / kMinShare));
    return launch_ex(attention_paged_kernel<T, HD, GP>, dim3((unsigned)grid), dim3(kThreads), kSmemBytes, s, false, a,
                     page_view<T>(p, layer), tb);
}

template <typename T>
cudaError_t launch_attention(const AttnArgs& a, const llama_q8_pages* p, int layer, const TableView& tb, cudaStream_t s) {
    if constexpr (!std::is_same<T, __half>::value) {
        if (a.n_head / p->n_head_kv > 4)
            return p->head_dim == 64 ? launch_one<T, 64, 8>(a, p, layer, tb, s) : launch_one<T, 128, 8>(a, p, layer, tb, s);
    }
    return p->head_dim == 64 ? launch_one<T, 64, 4>(a, p, layer, tb, s) : launch_one<T, 128, 4>(a, p, layer, tb, s);
}

template <typename T, int HD, int GP>
cudaError_t set_attr() {
    return cudaFuncSetAttribute(attention_paged_kernel<T, HD, GP>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
}

}  // namespace

cudaError_t init_attention_paged_attributes() {
    cudaError_t e = set_attr<float, 64, 4>();
    if (e == cudaSuccess) e = set_attr<float, 64, 8>();
    if (e == cudaSuccess) e = set_attr<float, 128, 4>();
    if (e == cudaSuccess) e = set_attr<float, 128, 8>();
    if (e == cudaSuccess) e = set_attr<__half, 64, 4>();
    if (e == cudaSuccess) e = set_attr<__half, 128, 4>();
    if (e == cudaSuccess) e = set_attr<__nv_bfloat16, 64, 4>();
    if (e == cudaSuccess) e = set_attr<__nv_bfloat16, 128, 4>();
    if (e == cudaSuccess) e = set_attr<__nv_bfloat16, 64, 8>();
    if (e == cudaSuccess) e = set_attr<__nv_bfloat16, 128, 8>();
    return e;
}
}  // namespace lq8

using namespace lq8;

extern "C" {

size_t llama_q8_attention_paged_workspace_bytes(int32_t rows, int32_t n_head, int32_t n_head_kv, int32_t head_dim) {
    if (rows < 0 || n_head <= 0 || n_head_kv <= 0 || n_head % n_head_kv || head_dim <= 0) return 0;
    return attn_paged_workspace(n_head, n_head_kv, head_dim, nullptr, nullptr);
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
    // units of 32 positions or more over all rows and KV heads are counted in 31 bits, a CTA's share past them included
    const int64_t reach = std::min<int64_t>((int64_t)table_stride * pages->page, INT32_MAX);
    if ((double)(reach / 32 + 2) * rows * pages->n_head_kv > INT32_MAX - 4096.0) return LQ8_ERR_UNSUPPORTED;
    if (((uintptr_t)q | (uintptr_t)out | (uintptr_t)workspace) & 15) return LQ8_ERR_ARG;
    if (((uintptr_t)pos | (uintptr_t)seq | (uintptr_t)table | (uintptr_t)lse | (uintptr_t)err) & 3) return LQ8_ERR_ARG;
    AttnArgs a{};
    if (workspace_bytes < attn_paged_workspace(n_head, pages->n_head_kv, pages->head_dim, &a, workspace))
        return LQ8_ERR_ARG;
    if (rows == 0) return LQ8_OK;
    if (ensure_kernel_attributes() != cudaSuccess) return LQ8_ERR_CUDA;
    a.q = q, a.pos = pos, a.seq = seq, a.rows = rows, a.n_head = n_head, a.window = window;
    a.scale_log2 = (scale > 0.0f ? scale : 1.0f / sqrtf((float)pages->head_dim)) * 1.4426950408889634f;
    a.out = out, a.lse = lse, a.err = err;
    const TableView tb{table, n_seq, table_stride};
    cudaStream_t s = (cudaStream_t)stream;
    cudaError_t e = pages->type == LLAMA_Q8_GGUF_F32   ? launch_attention<float>(a, pages, layer, tb, s)
                    : pages->type == LLAMA_Q8_GGUF_F16 ? launch_attention<__half>(a, pages, layer, tb, s)
                                                       : launch_attention<__nv_bfloat16>(a, pages, layer, tb, s);
    return e == cudaSuccess ? LQ8_OK : LQ8_ERR_CUDA;
}

}  // extern "C"
