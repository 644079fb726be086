// Quantisers that feed the 8-bit integer product: rows of numbers v[k] become
// int8 codes and one f32 scale.
//
//   M = max |v_i|,  scale = M f / 127 (rounded to f32),  code_i = v_i 127 / M rounded, ties away from zero
//
//   rows:  v = x,                       f = 1
//   norm:  h = x + delta (stored),  v = h g,  f = 1 / sqrt(mean(h^2) + eps)
//   silu:  v = gate / (1 + exp(-gate)) up,  f = 1
//
// f is a positive factor of the whole row, so the codes do not depend on it and
// a norm's codes need no second look at the row once M is known. The codes are
// those of exact arithmetic: the f32 quotient t = v (127 / M) is off by a few
// 2^-24 of itself, so a code is settled in f32 unless t lies within kWindow of a
// half (a few elements in ten thousand). Those are settled at the end by the sign
// of 254 |v| - (2 q + 1) M, from v and M in two-part f32 (exact for rows and norm,
// to 2^-40 for silu), and where that is no more than the parts leave out, in
// double (a double instruction takes 64 times an f32 one's turn, and exact halves
// are common in 16-bit rows). The exact M comes from the elements next to the f32
// maximum. Rows whose f32 numbers leave the normal range are done in double as a
// whole.
//
// Bound: memory (norm of 8195 x 4096 f32 65 us, 6.7 TB/s), and with 16-bit types the
// instructions (an element of rows takes 16, of norm 28, of silu 26 with its share of
// the row's reductions; they fill half to two thirds of the issue slots) and the chain from
// a row's maximum to its last code. A warp,
// or a CTA with as many threads as the row has values for, keeps a row's v in registers
// (16 values a thread, or 32, up to 14336), so every input is read once and
// every output written once; at least two CTAs share an SM, so that one row's loads run
// under another's barriers; rows of more than 14336 values are read twice.
#include "kernels.cuh"
#include "llama_q8.h"
#include "ptx.cuh"

#include <cuda_bf16.h>
#include <type_traits>

namespace lq8 {

enum QuantOp : int { QUANT_ROWS = 0, QUANT_NORM = 1, QUANT_SILU = 2 };

struct QuantArgs {
    const void* x;  // rows: x, norm: x, silu: gate
    const void* b;  // norm: delta or null, silu: up
    void* out;      // norm: h or null
    int64_t xs, bs, os;  // row strides in elements
    const float* g;
    float eps;
    int rows, k;
    int8_t* codes;
    int64_t row_bytes;  // k rounded up to 16
    float* scale;
};

struct BlockQ8 {};  // Q8_0 blocks as an element type

// threads of a CTA, at most: two such CTAs share an SM's registers (64 a thread; 72 with 32 values each)
constexpr int kQuantThreads = 512, kQuantThreads32 = 448;
constexpr float kMagic = 12582912.0f;       // 1.5 2^23: adding it rounds to an integer
// Half width of the band around a half in which f32 does not settle a code. t = v (127 / M) is at most 127 and off by
// the relative errors, in units of 2^-24, of 127 / M (1), of M (rows 0, norm 1, silu as v) and of v (rows 0, norm 1, silu
// 9: see silu_up): 127 * 19 * 2^-24 = 1.44e-4 for silu, 127 * 3 * 2^-24 = 2.3e-5 for the others; t itself is rounded at a
// few 2^-27 next to a half.
template <int OP> constexpr float kWindow = OP == QUANT_SILU ? 1.5e-4f : 3e-5f;
// v within this factor of the f32 maximum may be the exact maximum: f32 products round in order (norm), silu's are off
// by 9 * 2^-24 (2 * 9 * 2^-24 < 2^-19)
template <int OP> constexpr float kNearMax = OP == QUANT_SILU ? 1.0f - 1.0f / 262144.0f : 1.0f;
// M outside: the row is done in double. Above kTiny the products next to a half are 2^-100 and more, and the part of a norm's
// h g below f32 is a multiple of the smallest f32, 2^-149.
constexpr float kTiny = 0x1p-92f, kHuge = 1e36f;

template <typename T> struct Piece { static constexpr int n = 16 / sizeof(T); };
template <> struct Piece<BlockQ8> { static constexpr int n = 16; };

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// two numbers rounded to the type, as they lie in a word of memory (f32: not used), and back
template <typename T> __device__ __forceinline__ uint32_t pair_raw(uint64_t v) {
    if constexpr (std::is_same<T, __half>::value) {
        const __half2 h = __floats2half2_rn(f2_lo(v), f2_hi(v));
        return *reinterpret_cast<const uint32_t*>(&h);
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(f2_lo(v), f2_hi(v));
        return *reinterpret_cast<const uint32_t*>(&h);
    }
}
template <typename T> __device__ __forceinline__ void pair_open(uint32_t u, float& lo, float& hi) {
    if constexpr (std::is_same<T, __half>::value) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u));
        lo = f.x, hi = f.y;
    } else {
        lo = __uint_as_float(u << 16), hi = __uint_as_float(u & 0xffff0000u);
    }
}

// Element i of a row (any i < k).
template <typename T> __device__ __forceinline__ float load_one(const void* x, int64_t row_at, int i) {
    return to_f32(reinterpret_cast<const T*>(x)[row_at + i]);
}
template <> __device__ __forceinline__ float load_one<BlockQ8>(const void* x, int64_t row_at, int i) {
    const uint8_t* blk = reinterpret_cast<const uint8_t*>(x) + (row_at / 32 + i / 32) * 34;
    const float d = __half2float(__ushort_as_half(*reinterpret_cast<const unsigned short*>(blk)));
    return d * (float)reinterpret_cast<const int8_t*>(blk)[2 + i % 32];
}

// Elements i .. i + n - 1 of a row as they lie in memory (i a multiple of n, 16-byte aligned), zeros past k.
template <typename T> __device__ __forceinline__ uint4 load_raw(const void* x, int64_t row_at, int i, int k) {
    uint4 u = make_uint4(0u, 0u, 0u, 0u);
    if (i < k)
        asm volatile("ld.global.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
                     : "l"(reinterpret_cast<const T*>(x) + row_at + i));
    return u;
}
template <typename T> __device__ __forceinline__ void from_raw(const uint4& u, float (&v)[Piece<T>::n]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if constexpr (sizeof(T) == 4) v[j] = __uint_as_float(w[j]);
        else pair_open<T>(w[j], v[2 * j], v[2 * j + 1]);
    }
}

// Elements i .. i + n - 1 of a row (i a multiple of n), zeros past k. ALIGNED: 16-byte loads, k a multiple of n.
template <typename T, bool ALIGNED>
__device__ __forceinline__ void load_piece(const void* x, int64_t row_at, int i, int k, float (&v)[Piece<T>::n]) {
    if constexpr (ALIGNED) {
        from_raw<T>(load_raw<T>(x, row_at, i, k), v);
    } else {
#pragma unroll
        for (int j = 0; j < Piece<T>::n; ++j) v[j] = i + j < k ? load_one<T>(x, row_at, i + j) : 0.0f;
    }
}
// Half a Q8_0 block. Blocks lie on 2-byte boundaries, every other one off the words': its 16 codes are the words from two
// bytes before them on, shifted, the last half word read by itself (nothing past the codes is touched).
struct RawQ8 {
    uint32_t w[5];
    uint32_t d;  // the fp16 scale, and above it the shift
};
__device__ __forceinline__ RawQ8 load_raw_q8(const void* x, int64_t row_at, int i, int k) {
    RawQ8 r = {};
    if (i < k) {
        const uint8_t* blk = reinterpret_cast<const uint8_t*>(x) + (row_at / 32 + i / 32) * 34;
        const uint8_t* q = blk + 2 + i % 32;
        const uint32_t shift = ((uint32_t)(uintptr_t)q & 2u) * 8u;
        const uint32_t* word = reinterpret_cast<const uint32_t*>((uintptr_t)q & ~(uintptr_t)3);
        r.d = *reinterpret_cast<const unsigned short*>(blk) | shift << 16;
#pragma unroll
        for (int j = 0; j < 4; ++j) r.w[j] = word[j];
        if (shift) r.w[4] = *reinterpret_cast<const unsigned short*>(q + 14);
    }
    return r;
}
__device__ __forceinline__ void from_raw_q8(const RawQ8& r, float (&v)[16]) {
    const float d = __half2float(__ushort_as_half((unsigned short)(r.d & 0xffffu)));
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t u = __funnelshift_r(r.w[j], r.w[j + 1], r.d >> 16) ^ 0x80808080u;
        const uint64_t a = codes2_f2<0>(u), b = codes2_f2<2>(u);
        v[4 * j] = d * f2_lo(a), v[4 * j + 1] = d * f2_hi(a), v[4 * j + 2] = d * f2_lo(b), v[4 * j + 3] = d * f2_hi(b);
    }
}

template <typename T, bool ALIGNED>
__device__ __forceinline__ void store_piece(void* x, int64_t row_at, int i, int k, const float (&v)[Piece<T>::n]) {
    constexpr int n = Piece<T>::n;
    T* at = reinterpret_cast<T*>(x) + row_at + i;
    if constexpr (ALIGNED) {
        if (i >= k) return;
        uint4 u;
        T* e = reinterpret_cast<T*>(&u);
#pragma unroll
        for (int j = 0; j < n; ++j) e[j] = from_f32<T>(v[j]);
        *reinterpret_cast<uint4*>(at) = u;
    } else {
#pragma unroll
        for (int j = 0; j < n; ++j)
            if (i + j < k) at[j] = from_f32<T>(v[j]);
    }
}

// The largest magnitude of three; NaN if any is (its sign is left open).
__device__ __forceinline__ float max_magnitude(float a, float v, float w) {
    asm("max.NaN.abs.f32 %0, %0, %1, %2;" : "+f"(a) : "f"(v), "f"(w));
    return a;
}
__device__ __forceinline__ float min3(float a, float v, float w) {
    asm("min.f32 %0, %0, %1, %2;" : "+f"(a) : "f"(v), "f"(w));
    return a;
}

// silu(gate) up in double
__device__ __noinline__ double silu_up_f64(float gate, float up) {
    return (double)gate / (1.0 + exp(-(double)gate)) * (double)up;
}
// The same in f32 for gate >= -80: exp(x) = 2^h (1 + r) with h = x / ln 2 rounded and r what the rounding left, in six
// operations and two approximations (expf and a division take 12 more instructions per element). Off by 6.6 * 2^-24 of itself
// at most for any gate of -80 .. 80 (up = 1; measured over all f32 numbers of 1e-9 and more, against double), and by one
// product's rounding. gate and the quotient alone do not make the first product: it would lose bits where gate lies next to the
// subnormal range, which an up of 1e20 brings back among the row's numbers. Gate times up does so only where all of v is
// far below a row's smallest code (or leaves the range above, and the row goes through double), and so does the quotient
// times up, unless the quotient is 1. 16-bit types have the better time with the first order (2048 x 14336 bf16 42.6 us,
// 45.8 with the second), f32 with the second (61.4 us, 64.5).
template <typename T> __device__ __forceinline__ float silu_up(float gate, float up) {
    const float h = gate * -1.442695041f, r = fmaf(-h, 0.6931471806f, -gate);
    float e, q;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(h));
    e = fmaf(e, r, e);
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(q) : "f"(1.0f + e));
    if constexpr (sizeof(T) == 2) return gate * up * q;
    return gate * (q * up);
}

// ---- two-part f32 numbers: hi is the sum rounded to f32
struct Two {
    float hi, lo;
};
__device__ __forceinline__ Two two_sum(float a, float b) {
    const float s = a + b, t = s - a;
    return {s, (a - (s - t)) + (b - t)};
}
__device__ __forceinline__ Two two_renorm(float hi, float lo) {  // |hi| >= |lo|
    const float s = hi + lo;
    return {s, lo - (s - hi)};
}
__device__ __forceinline__ Two two_prod(float a, float b) {
    const float p = a * b;
    return {p, fmaf(a, b, -p)};
}

// silu(gate) up to about 2^-40 of itself, for the elements that a row's maximum and codes are settled by (of 2^-101 and more):
// exp(x) = 2^n exp(r) with x = n ln 2 + r, ln 2 in three parts of which n times the first is exact (the range reduction of
// Cody and Waite); exp(r), |r| <= ln 2 / 2, by its Taylor series to r^11 (what is left out is below 2^-47), the terms up to
// r^5 in two parts. Powers of two go from one factor to the other where a quotient's remainder would fall under the smallest f32:
// 2^n of a far gate (1 beside it is nothing) and 2^64 of a tiny one. An up that brings such a gate back is large.
__device__ __noinline__ Two silu_up_two(float gate, float up) {
    const float x = -gate;
    Two y = {1.0f, 0.0f};  // 1 + exp(x)
    if (x > -60.0f) {
        const float n = rintf(x * 1.442695041f);
        const float r1 = fmaf(-n, 0x1.62e4p-1f, x);
        const Two p = two_prod(n, 0x1.7f7d1cp-20f);
        Two r = two_sum(r1, -p.hi);
        r = two_renorm(r.hi, r.lo - p.lo - n * 0x1.ef357ap-45f);
        float q = 1.0f / 39916800.0f;
        q = fmaf(q, r.hi, 1.0f / 3628800.0f);
        q = fmaf(q, r.hi, 1.0f / 362880.0f);
        q = fmaf(q, r.hi, 1.0f / 40320.0f);
        q = fmaf(q, r.hi, 1.0f / 5040.0f);
        q = fmaf(q, r.hi, 1.0f / 720.0f);
        Two s = {q, 0.0f};
        const Two c[6] = {{1.0f, 0.0f}, {1.0f, 0.0f}, {0.5f, 0.0f}, {0x1.555556p-3f, -0x1.555556p-28f},
                          {0x1.555556p-5f, -0x1.555556p-30f}, {0x1.111112p-7f, -0x1.ddddep-32f}};  // 1 / i!
#pragma unroll
        for (int i = 5; i >= 0; --i) {
            Two m = two_prod(s.hi, r.hi);
            m.lo = fmaf(s.lo, r.hi, fmaf(s.hi, r.lo, m.lo));
            const Two t = two_sum(c[i].hi, m.hi);
            s = two_renorm(t.hi, t.lo + (c[i].lo + m.lo));
        }
        if (n < 60.0f) {
            const float scale = pow2f((int)n);
            y = two_sum(1.0f, s.hi * scale);
            y = two_renorm(y.hi, y.lo + s.lo * scale);
        } else {
            const int half = (int)n >> 1;
            y = s, up = up * pow2f(-half) * pow2f(half - (int)n);
        }
    }
    if (fabsf(gate) < 0x1p-100f) gate *= 0x1p64f, up *= 0x1p-64f;
    const float q0 = __fdiv_rn(gate, y.hi);
    const float q1 = __fdiv_rn(fmaf(-q0, y.lo, fmaf(-q0, y.hi, gate)), y.hi);
    const Two v = two_prod(q0, up);
    return two_renorm(v.hi, fmaf(q1, up, v.lo));
}

template <int OP, typename T, bool ALIGNED> struct Row {
    static constexpr int n = Piece<T>::n;
    const QuantArgs& a;
    int64_t xa, ba, oa;
    __device__ Row(const QuantArgs& args, int64_t r) : a(args), xa(r * args.xs), ba(r * args.bs), oa(r * args.os) {}

    // x (gate) and delta (up) of elements i .. i + n - 1
    __device__ __forceinline__ void load(int i, float (&x)[n], float (&b)[n]) const {
        load_piece<T, ALIGNED>(a.x, xa, i, a.k, x);
        if (OP == QUANT_SILU || (OP == QUANT_NORM && a.b)) load_piece<T, ALIGNED>(a.b, ba, i, a.k, b);
    }
    // the same as they lie in memory (ALIGNED), and from there
    struct Raw {
        uint4 x, b;
    };
    __device__ __forceinline__ void load(int i, Raw& r) const {
        r.x = load_raw<T>(a.x, xa, i, a.k);
        if (OP == QUANT_SILU || (OP == QUANT_NORM && a.b)) r.b = load_raw<T>(a.b, ba, i, a.k);
    }
    __device__ __forceinline__ void open(const Raw& r, float (&x)[n], float (&b)[n]) const {
        from_raw<T>(r.x, x);
        from_raw<T>(r.b, b);  // not used where it was not read
    }
    // v from them, into x; a norm's h is written out and the sum of its squares added to ss
    __device__ __forceinline__ void values(int i, float (&x)[n], const float (&b)[n], float& ss) const {
        if constexpr (OP == QUANT_SILU) {
            float low = 0.0f;
#pragma unroll
            for (int j = 0; j < n; j += 2) low = min3(low, x[j], x[j + 1]);
            if (low < -80.0f) {  // outside of silu_up's range
#pragma unroll
                for (int j = 0; j < n; ++j) x[j] = (float)silu_up_f64(x[j], b[j]);
            } else {
#pragma unroll
                for (int j = 0; j < n; ++j) x[j] = silu_up<T>(x[j], b[j]);
            }
        } else if constexpr (OP == QUANT_NORM) {
            if constexpr (ALIGNED && sizeof(T) == 2) {
                uint32_t w[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint64_t h = pack_f2(x[2 * j], x[2 * j + 1]);
                    if (a.b) h = add_f2(h, pack_f2(b[2 * j], b[2 * j + 1]));
                    w[j] = pair_raw<T>(h);
                    pair_open<T>(w[j], x[2 * j], x[2 * j + 1]);
                }
                if (a.out && i < a.k)
                    *reinterpret_cast<uint4*>(reinterpret_cast<T*>(a.out) + oa + i) = make_uint4(w[0], w[1], w[2], w[3]);
            } else {
                if (a.b) {
#pragma unroll
                    for (int j = 0; j < n; ++j) x[j] = to_f32(from_f32<T>(x[j] + b[j]));
                }
                if (a.out) store_piece<T, ALIGNED>(a.out, oa, i, a.k, x);
            }
#pragma unroll
            for (int j = 0; j < n; ++j) ss = fmaf(x[j], x[j], ss);
            gained(i, x);
        }
    }
    // h times g
    __device__ __forceinline__ void gained(int i, float (&x)[n]) const {
        if constexpr (ALIGNED) {
#pragma unroll
            for (int j = 0; j < n; j += 4) {
                float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
                if (i < a.k) f = __ldca(reinterpret_cast<const float4*>(a.g + i + j));
                x[j] *= f.x, x[j + 1] *= f.y, x[j + 2] *= f.z, x[j + 3] *= f.w;
            }
        } else {
#pragma unroll
            for (int j = 0; j < n; ++j) x[j] *= i + j < a.k ? a.g[i + j] : 0.0f;
        }
    }
    // v of elements i .. i + n - 1 after the first pass (which may have written h over x or delta)
    __device__ __forceinline__ void again(int i, float (&v)[n]) const {
        if constexpr (OP == QUANT_NORM) {
            if (a.out) {
                load_piece<T, ALIGNED>(a.out, oa, i, a.k, v);
            } else {
                float b[n];
                load(i, v, b);
                if (a.b) {
#pragma unroll
                    for (int j = 0; j < n; ++j) v[j] = to_f32(from_f32<T>(v[j] + b[j]));
                }
            }
            gained(i, v);
        } else {
            float b[n], unused = 0.0f;
            load(i, v, b);
            values(i, v, b, unused);
        }
    }
    // h of element i after the first pass
    __device__ __forceinline__ float h_again(int i) const {
        if (OP == QUANT_NORM && a.out) return load_one<T>(a.out, oa, i);
        float h = load_one<T>(a.x, xa, i);
        if constexpr (OP == QUANT_NORM)
            if (a.b) h = to_f32(from_f32<T>(h + load_one<T>(a.b, ba, i)));
        return h;
    }
    // whether v of element i is zero in fact
    __device__ __forceinline__ bool zero(int i) const {
        if (OP == QUANT_SILU) return load_one<T>(a.x, xa, i) == 0.0f || load_one<T>(a.b, ba, i) == 0.0f;
        return h_again(i) == 0.0f || (OP == QUANT_NORM && a.g[i] == 0.0f);
    }
    // v of element i in two parts
    __device__ __forceinline__ Two v_two(int i) const {
        if constexpr (OP == QUANT_SILU) {
            return silu_up_two(load_one<T>(a.x, xa, i), load_one<T>(a.b, ba, i));
        }
        if constexpr (OP == QUANT_NORM) return two_prod(h_again(i), a.g[i]);
        return {load_one<T>(a.x, xa, i), 0.0f};
    }
    // v of element i in double: exact for rows (one number) and norm (a product of two f32)
    __device__ double v_f64(int i) const {
        if constexpr (OP == QUANT_SILU) return silu_up_f64(load_one<T>(a.x, xa, i), load_one<T>(a.b, ba, i));
        if constexpr (OP == QUANT_NORM) return (double)h_again(i) * (double)a.g[i];
        return (double)load_one<T>(a.x, xa, i);
    }
};
// Q8_0 blocks stand under rows_quant alone
template <bool ALIGNED> struct Row<QUANT_ROWS, BlockQ8, ALIGNED> {
    static constexpr int n = Piece<BlockQ8>::n;
    const QuantArgs& a;
    int64_t xa;
    __device__ Row(const QuantArgs& args, int64_t r) : a(args), xa(r * args.xs) {}
    using Raw = RawQ8;
    __device__ __forceinline__ void load(int i, float (&x)[n], float (&)[n]) const { again(i, x); }
    __device__ __forceinline__ void values(int, float (&)[n], const float (&)[n], float&) const {}
    __device__ __forceinline__ void again(int i, float (&v)[n]) const { from_raw_q8(load_raw_q8(a.x, xa, i, a.k), v); }
    __device__ __forceinline__ float h_again(int i) const { return load_one<BlockQ8>(a.x, xa, i); }
    __device__ __forceinline__ bool zero(int i) const { return h_again(i) == 0.0f; }
    __device__ __forceinline__ Two v_two(int i) const { return {load_one<BlockQ8>(a.x, xa, i), 0.0f}; }
    __device__ double v_f64(int i) const { return (double)load_one<BlockQ8>(a.x, xa, i); }
};

// Whether 127 |v| / M is at least q + 1/2, in double. rows and norm have exact v and M: the sign of 254 |v| - (2 q + 1) M
// (where the two products are close their difference is exact, and so is the rounding error that is taken off). silu's are
// rounded, and halves that are exact in fact (one gate, two ups) are taken as the quotient in double has them.
template <int OP> __device__ __forceinline__ bool above_half(double v, double M, float q) {
    if constexpr (OP == QUANT_SILU) return 127.0 * fabs(v) / M - (double)q >= 0.5;
    const double odd = 2.0 * (double)q + 1.0, p = odd * M, e = fma(odd, M, -p);
    return fma(254.0, fabs(v), -p) - e >= 0.0;
}
// The same from two-part numbers: 1 or 0, or -1 where the difference is within what they leave out (2^-36 of either
// product; nothing for one-part numbers).
__device__ __forceinline__ int above_half(Two v, Two M, float q) {
    const float odd = 2.0f * q + 1.0f, p = odd * M.hi, e = fmaf(odd, M.hi, -p);
    const float lo = v.hi < 0.0f ? -v.lo : v.lo;
    const float off = (fmaf(254.0f, fabsf(v.hi), -p) - e) + fmaf(254.0f, lo, -(odd * M.lo));
    if (v.lo == 0.0f && M.lo == 0.0f) return off >= 0.0f;
    return fabsf(off) <= p * 0x1p-36f ? -1 : off > 0.0f;
}


// A row's reduction area; a warp's or a CTA's.
struct QuantShared {
    uint32_t max[32];
    float ss[32];
    unsigned long long exact;  // the exact maximum (key below)
};
struct QuantSharedF64 {
    unsigned long long max;
    double ss;
    int poison;
};

template <bool WARP> __device__ __forceinline__ void row_sync() {
    if constexpr (WARP) __syncwarp();
    else __syncthreads();
}

// A row whose numbers leave the range in which f32 settles codes, or are not finite, in double.
template <int OP, bool WARP, typename R>
__device__ __forceinline__ void quant_row_f64(const QuantArgs& a, int64_t r, int t, int G, QuantSharedF64& sh) {
    const R row(a, r);
    const int k = a.k, k16 = (int)a.row_bytes;
    int8_t* codes = a.codes + r * a.row_bytes;
    row_sync<WARP>();
    if (t == 0) sh.max = 0ull, sh.ss = 0.0, sh.poison = 0;
    row_sync<WARP>();
    double top = 0.0, sum = 0.0;
    bool bad = false;
    for (int i = t; i < k; i += G) {
        const double w = row.v_f64(i);
        if (OP == QUANT_NORM) {
            const double h = row.h_again(i);
            sum += h * h;
            bad |= !isfinite(h);
        }
        bad |= !isfinite(w);
        top = fmax(top, fabs(w));
    }
    if (bad) atomicOr(&sh.poison, 1);
    // the largest by its bits; the warps' sums in a fixed order, so that equal calls give equal bits
    atomicMax(&sh.max, (unsigned long long)__double_as_longlong(top));
    if constexpr (OP == QUANT_NORM) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        for (int w = 0; w < G >> 5; ++w) {
            if ((t & 31) == 0 && t >> 5 == w) sh.ss += sum;
            row_sync<WARP>();
        }
    }
    row_sync<WARP>();
    const double M = __longlong_as_double((long long)sh.max);
    const bool poison = sh.poison != 0;
    for (int i = t; i < k16; i += G) {
        int c = 0;
        if (i < k && !poison && M > 0.0) {
            const double w = row.v_f64(i);
            c = (int)fmax(floor(127.0 * fabs(w) / M - 0.25), 0.0);  // the code or the one below
            while (c < 127 && above_half<OP>(w, M, (float)c)) ++c;
            if (w < 0.0) c = -c;
        }
        codes[i] = (int8_t)c;
    }
    if (t == 0) {
        const double f = OP == QUANT_NORM ? 1.0 / sqrt(sh.ss / k + (double)a.eps) : 1.0;
        a.scale[r] = poison ? __int_as_float(0x7fffffff) : (float)(M == 0.0 ? 0.0 : M * f / 127.0);
    }
    row_sync<WARP>();
}

// The candidates for the exact maximum, ordered by one integer: the steps of f32 above `near` (they are few), the lower
// part's sign and magnitude, the element's number (any of equal ones).
__device__ __forceinline__ unsigned long long max_key(Two v, float near, int i) {
    const float lo = v.hi < 0.0f ? -v.lo : v.lo;
    return (unsigned long long)(__float_as_uint(fabsf(v.hi)) - __float_as_uint(near)) << 49 |
           (unsigned long long)f32_order_key(lo) << 17 | (unsigned)i;
}
__device__ __forceinline__ Two max_of_key(unsigned long long key, float near) {
    const uint32_t u = (uint32_t)(key >> 17);
    return {__uint_as_float(__float_as_uint(near) + (uint32_t)(key >> 49)),
            __uint_as_float(u & 0x80000000u ? u & 0x7fffffffu : ~u)};
}
static_assert(LLAMA_Q8_I8_MAX_K <= 1 << 17, "an element's number in a key");

// A row per warp (threads == 32, four per CTA) or per CTA of up to `threads`; E values of it a thread. E == 0: rows too
// long for the registers, read again. AHEAD: a CTA takes several rows, and asks for the next one's values when it has
// turned this one's into v.
template <int OP, typename T, bool ALIGNED, int E, int threads, bool AHEAD>
__global__ void __launch_bounds__(threads == 32 ? 128 : threads, threads == 32 ? 6 : threads > 512 ? 1 : 2)
    quant_kernel(const QuantArgs a) {
    using R = Row<OP, T, ALIGNED>;
    constexpr bool WARP = threads == 32, LOOP = E == 0;
    constexpr int n = R::n, pieces = E / n;
    constexpr int kRowsPerCta = WARP ? 4 : 1;
    __shared__ QuantShared shared[WARP ? 4 : 2];
    __shared__ QuantSharedF64 shared64[kRowsPerCta];
    const int G = WARP ? 32 : blockDim.x;
    const int t = WARP ? threadIdx.x & 31 : threadIdx.x, lane = threadIdx.x & 31, warp = t >> 5;
    const int k = a.k, k16 = (int)a.row_bytes;
    int64_t r = (int64_t)blockIdx.x * kRowsPerCta + (WARP ? threadIdx.x >> 5 : 0);
    if (r >= a.rows) return;  // a whole warp (WARP) or none
    pdl_wait();  // the launch may overlap the end of the kernel before (1 x 576 f32 2.5 -> 2.2 us)
    // two areas in turn: a row's first barrier is behind the last look at the area of the row before the last
    int area = WARP ? threadIdx.x >> 5 : 0;
    if (t == 0) {
        shared[area].exact = 0ull;
        if (!WARP) shared[1].exact = 0ull;
    }
    typename R::Raw raw[AHEAD ? pieces : 1];
    if constexpr (AHEAD) {
        const R row(a, r);
#pragma unroll
        for (int p = 0; p < pieces; ++p) row.load((p * G + t) * n, raw[p]);
    }
    for (;;) {
        const R row(a, r);
        QuantShared& sh = shared[area];
        int8_t* codes = a.codes + r * a.row_bytes;

        // the row once: v in registers, the largest magnitude, the sum of squares
        float v[LOOP ? n : E];
        float ss = 0.0f, own = 0.0f;
        if constexpr (LOOP) {
            float part[4] = {0.f, 0.f, 0.f, 0.f};  // short chains: a thread has many squares to add
            for (int i = t * n, p = 0; i < k; i += G * n, ++p) {
                float w[n], b[n], s = 0.0f;
                row.load(i, w, b);
                row.values(i, w, b, s);
                part[p & 3] += s;
#pragma unroll
                for (int j = 0; j < n; j += 2) own = max_magnitude(own, w[j], w[j + 1]);
            }
            ss = (part[0] + part[1]) + (part[2] + part[3]);
        } else {
            constexpr int batch = E == 32 ? (n == 16 ? 1 : 2) : pieces;  // pieces whose loads are in flight together
#pragma unroll
            for (int p0 = 0; p0 < pieces; p0 += batch) {
                float x[batch][n], b[batch][n];
#pragma unroll
                for (int p = 0; p < batch; ++p) {
                    if constexpr (AHEAD) row.open(raw[p0 + p], x[p], b[p]);
                    else row.load(((p0 + p) * G + t) * n, x[p], b[p]);
                }
                // 16 squares at most in a chain (a sum beside ss where one batch is all: 8195 x 14336 bf16 133 -> 143 us)
                float batch_ss = 0.0f, &part = batch == pieces ? ss : batch_ss;
#pragma unroll
                for (int p = 0; p < batch; ++p) {
                    row.values(((p0 + p) * G + t) * n, x[p], b[p], part);
#pragma unroll
                    for (int j = 0; j < n; j += 2) own = max_magnitude(own, x[p][j], x[p][j + 1]);
#pragma unroll
                    for (int j = 0; j < n; ++j) v[(p0 + p) * n + j] = x[p][j];
                }
                if constexpr (batch != pieces) ss += part;
            }
            if constexpr (AHEAD) {
                if (r + gridDim.x < a.rows) {
                    const R next(a, r + gridDim.x);
#pragma unroll
                    for (int p = 0; p < pieces; ++p) next.load((p * G + t) * n, raw[p]);
                }
            }
        }
        // the bits of magnitudes order like the magnitudes, NaN above infinity
        own = fabsf(own);
        uint32_t mx = __reduce_max_sync(0xffffffffu, __float_as_uint(own));
        if constexpr (OP == QUANT_NORM) ss = warp_sum(ss);
        if constexpr (!WARP) {
            if (lane == 0) sh.max[warp] = mx, sh.ss[warp] = ss;
            __syncthreads();
            mx = __reduce_max_sync(0xffffffffu, lane < G >> 5 ? sh.max[lane] : 0u);
            if constexpr (OP == QUANT_NORM) ss = warp_sum(lane < G >> 5 ? sh.ss[lane] : 0.0f);
            area ^= 1;
            if (t == 0) shared[area].exact = 0ull;
        } else {
            __syncwarp();
        }
        const float M = __uint_as_float(mx);
        if (!(M >= kTiny && M <= kHuge) || (OP == QUANT_NORM && !(ss >= 1e-28f && ss <= kHuge))) {
            bool zero = mx == 0u && !(OP == QUANT_NORM && !(ss <= kHuge));
            if (zero) {  // all zeros, or v below the smallest f32?
                for (int i = t; i < k; i += G) zero &= row.zero(i);
                if constexpr (WARP) zero = __all_sync(0xffffffffu, zero);
                else zero = __syncthreads_and(zero);
            }
            if (zero) {
                for (int i = t * 4; i < k16; i += G * 4) *reinterpret_cast<uint32_t*>(codes + i) = 0u;
                if (t == 0) a.scale[r] = 0.0f;
            } else {
                quant_row_f64<OP, WARP, R>(a, r, t, G, shared64[WARP ? threadIdx.x >> 5 : 0]);
            }
            if (!AHEAD || (r += gridDim.x) >= a.rows) return;
            continue;
        }

        // the exact maximum, of the elements that may be it
        const float near = M * kNearMax<OP>;
        if (OP != QUANT_ROWS && own >= near) {
            auto offer = [&](int i, float w) {
                if (fabsf(w) >= near) {
                    const Two e = row.v_two(i);
                    if (fabsf(e.hi) >= near) atomicMax(&sh.exact, max_key(e, near, i));
                }
            };
            if constexpr (!LOOP) {
#pragma unroll
                for (int p = 0; p < pieces; ++p)
#pragma unroll
                    for (int j = 0; j < n; ++j) offer((p * G + t) * n + j, v[p * n + j]);
            } else {
                for (int i = t * n; i < k; i += G * n) {
                    float w[n];
                    row.again(i, w);
#pragma unroll
                    for (int j = 0; j < n; ++j) offer(i + j, w[j]);
                }
            }
        }

        // codes, rounded in f32; the elements next to a border are noted, as bits of a piece
        const float inv = __fdiv_rn(127.0f, M);
        // two elements an instruction where the registers' pairs come for nothing (norm of 8195 x 4096 bf16 49 -> 42 us, but
        // Q8_0 rows 74 -> 80, silu of 2048 x 14336 bf16 43 -> 46)
        constexpr bool packed = OP == QUANT_NORM && sizeof(T) == 2;
        auto store = [&](int i, const float* w) -> uint32_t {
            uint32_t word[n / 4], border = 0u;
            float off = 0.0f;
            const uint64_t inv2 = pack_f2(inv, inv), magic = pack_f2(kMagic, kMagic);
#pragma unroll
            for (int q = 0; q < n / 4; ++q) {
                uint32_t c[4];
#pragma unroll
                for (int j = 0; j < 4; j += 2) {
                    const float x0 = w[4 * q + j], x1 = w[4 * q + j + 1];
                    if constexpr (packed) {
                        const uint64_t x = pack_f2(x0, x1), m = fma_f2(x, inv2, magic);
                        const uint64_t r = fma_f2(x, inv2, sub_f2(magic, m));
                        off = max_magnitude(off, f2_lo(r), f2_hi(r));
                        c[j] = (uint32_t)m, c[j + 1] = (uint32_t)(m >> 32);
                    } else {
                        const float m0 = fmaf(x0, inv, kMagic), m1 = fmaf(x1, inv, kMagic);  // rounded; the low byte is the code
                        off = max_magnitude(off, fmaf(x0, inv, kMagic - m0), fmaf(x1, inv, kMagic - m1));
                        c[j] = __float_as_uint(m0), c[j + 1] = __float_as_uint(m1);
                    }
                }
                word[q] = __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
            }
            if (i < k16) {
                if constexpr (n == 16)
                    *reinterpret_cast<uint4*>(codes + i) = make_uint4(word[0], word[1], word[2], word[3]);
                else if constexpr (n == 8) *reinterpret_cast<uint2*>(codes + i) = make_uint2(word[0], word[1]);
                else *reinterpret_cast<uint32_t*>(codes + i) = word[0];
            }
            if (fabsf(off) > 0.5f - kWindow<OP>) {
#pragma unroll
                for (int j = 0; j < n; ++j) {
                    const float m = fmaf(w[j], inv, kMagic);
                    if (fabsf(fmaf(w[j], inv, kMagic - m)) > 0.5f - kWindow<OP>) border |= 1u << j;
                }
            }
            return border;
        };
        // a noted element, with the exact maximum
        auto settle = [&](int at, Two w) {
            const unsigned long long key = sh.exact;
            const Two M2 = OP == QUANT_ROWS ? Two{M, 0.0f} : max_of_key(key, near);
            const float q = floorf(fabsf(w.hi) * inv);
            int up = above_half(w, M2, q);
            if (up < 0) up = above_half<OP>(row.v_f64(at), fabs(row.v_f64((int)(key & 0x1ffffu))), q);
            const int c = (int)q + up;
            codes[at] = (int8_t)(w.hi < 0.0f ? -c : c);
        };
        if constexpr (!LOOP) {
            uint32_t border = 0u;  // E <= 32
#pragma unroll
            for (int p = 0; p < pieces; ++p) border |= store((p * G + t) * n, v + p * n) << (p * n);
            auto place = [&] {
                const int bit = __ffs(border) - 1;
                border &= border - 1u;
                return (bit / n * G + t) * n + bit % n;
            };
            if constexpr (OP == QUANT_SILU) {
                // a thread's first noted element is looked up while the exact maximum is still on its way
                int first = -1;
                Two w = {0.0f, 0.0f};
                if (border) first = place(), w = row.v_two(first);
                row_sync<WARP>();
                if (first >= 0) settle(first, w);
            } else if constexpr (OP == QUANT_NORM) {
                row_sync<WARP>();
            }
            if constexpr (OP == QUANT_NORM) {  // piece by piece (8195 x 14336 bf16: 134 us, as below 180)
#pragma unroll 1
                for (int p = 0; border; ++p, border >>= n)
#pragma unroll 1
                    for (uint32_t bits = border & ((1u << n) - 1u); bits; bits &= bits - 1u) {
                        const int at = (p * G + t) * n + __ffs(bits) - 1;
                        settle(at, row.v_two(at));
                    }
            } else {
#pragma unroll 1
                while (border) {
                    const int at = place();
                    settle(at, row.v_two(at));
                }
            }
        } else {
            row_sync<WARP>();
            for (int i = t * n; i < k16; i += G * n) {
                float w[n];
                row.again(i, w);
                uint32_t bits = store(i, w);
#pragma unroll 1
                for (; bits; bits &= bits - 1u) {
                    const int at = i + __ffs(bits) - 1;
                    settle(at, row.v_two(at));
                }
            }
        }
        if (t == 0) {  // a norm's M is the exact maximum rounded
            if constexpr (OP == QUANT_SILU) {  // both parts, rounded once
                const Two top = max_of_key(sh.exact, near);
                const float q = __fdiv_rn(top.hi, 127.0f);
                a.scale[r] = fmaf(fmaf(-q, 127.0f, top.hi) + top.lo, 1.0f / 127.0f, q);
            } else {
                a.scale[r] = __fdiv_rn(M, OP == QUANT_NORM ? 127.0f * __fsqrt_rn(ss / (float)k + a.eps) : 127.0f);
            }
        }
        if (!AHEAD || (r += gridDim.x) >= a.rows) return;
    }
}

template <int OP, typename T, bool ALIGNED>
static cudaError_t launch_quant(const QuantArgs& a, cudaStream_t s) {
    auto go = [&](auto kernel, int64_t rows_per_cta, int64_t threads) {
        const int64_t grid = (a.rows + rows_per_cta - 1) / rows_per_cta;
        return launch_ex(kernel, dim3((unsigned)grid), dim3((unsigned)((threads + 31) / 32 * 32)), 0, s, true, a);
    };
    const int64_t k = a.row_bytes;
    if (k <= 16 * 32) return go(quant_kernel<OP, T, ALIGNED, 16, 32, false>, 4, 128);
    // 16 values a thread, or 32 with rows by themselves where 16 would take more than one wave of CTAs: half the warps share
    // the row's reductions (28672 x 4096 bf16 84 -> 63 us, f32 91 -> 82, Q8_0 74 -> 71; 512 x 4096 f32 4.1 -> 4.2 us; silu
    // of f32 loses more registers than it gains: 8195 x 1536 22.5 -> 33 us).
    const bool half = OP == QUANT_ROWS && ALIGNED && k > 2048 && a.rows * (k / 16) > 152 * 1024;
    // Several rows per CTA, as many CTAs as the SMs hold, for norms of 16-bit types, whose next row fits the registers beside
    // v (8195 x 4096 bf16 67 -> 42 us). Two arrays of f32 do not, and keep memory busy without; silu is bound by the chain
    // between its barriers, which more CTAs hide better (8195 x 4096 bf16 51.6 us in this form, 47.1 without).
    constexpr bool ahead = ALIGNED && OP == QUANT_NORM && sizeof(T) == 2;
    if constexpr (ahead) {
        const int64_t threads = (k / 16 + 31) / 32 * 32, ctas = 152 * (threads > 512 ? 1 : 1024 / threads);
        const int64_t per = a.rows > ctas ? (a.rows + ctas - 1) / ctas : 1;
        if (k <= 16 * kQuantThreads) return go(quant_kernel<OP, T, ALIGNED, 16, kQuantThreads, true>, per, threads);
        if (k <= 32 * kQuantThreads32) return go(quant_kernel<OP, T, ALIGNED, 16, 2 * kQuantThreads32, true>, per, threads);
    } else {
        if (k <= 16 * kQuantThreads && !half) return go(quant_kernel<OP, T, ALIGNED, 16, kQuantThreads, false>, 1, k / 16);
        if (k <= 32 * kQuantThreads32) return go(quant_kernel<OP, T, ALIGNED, 32, kQuantThreads32, false>, 1, (k + 31) / 32);
    }
    return go(quant_kernel<OP, T, ALIGNED, 0, kQuantThreads, false>, 1, kQuantThreads);
}

// 16-byte loads and stores: k a multiple of a piece, rows and bases on 16-byte boundaries.
template <int OP, typename T> static cudaError_t launch_quant_type(const QuantArgs& a, cudaStream_t s) {
    constexpr int n = Piece<T>::n;
    uintptr_t bases = (uintptr_t)a.x;
    int64_t counts = (int64_t)a.k | a.xs;
    if (OP != QUANT_ROWS && a.b) bases |= (uintptr_t)a.b, counts |= a.bs;
    if (OP == QUANT_NORM) {
        bases |= (uintptr_t)a.g;
        if (a.out) bases |= (uintptr_t)a.out, counts |= a.os;
    }
    if ((bases & 15) == 0 && counts % n == 0) return launch_quant<OP, T, true>(a, s);
    return launch_quant<OP, T, false>(a, s);
}

template <int OP> static llama_q8_status quant_types(int32_t type, const QuantArgs& a, cudaStream_t s) {
    cudaError_t e;
    switch (type) {
        case LLAMA_Q8_GGUF_F32: e = launch_quant_type<OP, float>(a, s); break;
        case LLAMA_Q8_GGUF_F16: e = launch_quant_type<OP, __half>(a, s); break;
        case LLAMA_Q8_GGUF_BF16: e = launch_quant_type<OP, __nv_bfloat16>(a, s); break;
        default: return LQ8_ERR_UNSUPPORTED;
    }
    return e == cudaSuccess ? LQ8_OK : LQ8_ERR_CUDA;
}

// What every quantiser asks of its outputs and sizes.
static llama_q8_status check_quant(int32_t type, int32_t rows, int32_t k, const int8_t* codes, const float* scale) {
    if (rows < 0 || k <= 0 || !codes || !scale || ((uintptr_t)codes & 15) || ((uintptr_t)scale & 3))
        return LQ8_ERR_ARG;
    if (type != LLAMA_Q8_GGUF_F32 && type != LLAMA_Q8_GGUF_F16 && type != LLAMA_Q8_GGUF_BF16 &&
        type != LLAMA_Q8_GGUF_Q8_0)
        return LQ8_ERR_UNSUPPORTED;
    if (k > LLAMA_Q8_I8_MAX_K) return LQ8_ERR_UNSUPPORTED;
    return LQ8_OK;
}

static uintptr_t type_mask(int32_t type) { return type == LLAMA_Q8_GGUF_F32 ? 3 : 1; }

}  // namespace lq8

using namespace lq8;

extern "C" {

int64_t llama_q8_i8_row_bytes(int64_t k) { return k <= 0 ? 0 : (k + 15) / 16 * 16; }

llama_q8_status llama_q8_rows_quant(int32_t type, const void* x, int64_t x_stride, int32_t rows, int32_t k,
                                    int8_t* codes, float* scale, void* stream) {
    if (!x) return LQ8_ERR_ARG;
    const llama_q8_status st = check_quant(type, rows, k, codes, scale);
    if (st != LQ8_OK) return st;
    if (x_stride < k || ((uintptr_t)x & type_mask(type))) return LQ8_ERR_ARG;
    QuantArgs a{};
    a.x = x, a.xs = x_stride, a.rows = rows, a.k = k, a.codes = codes, a.scale = scale;
    a.row_bytes = llama_q8_i8_row_bytes(k);
    if (type == LLAMA_Q8_GGUF_Q8_0) {
        if (k % 32 || x_stride % 32) return LQ8_ERR_ARG;
        if (rows == 0) return LQ8_OK;
        return launch_quant<QUANT_ROWS, BlockQ8, true>(a, (cudaStream_t)stream) == cudaSuccess ? LQ8_OK : LQ8_ERR_CUDA;
    }
    if (rows == 0) return LQ8_OK;
    return quant_types<QUANT_ROWS>(type, a, (cudaStream_t)stream);
}

llama_q8_status llama_q8_norm_quant(int32_t type, const void* x, int64_t x_stride, const void* delta,
                                    int64_t delta_stride, void* x_out, int64_t out_stride, const float* g, float eps,
                                    int32_t rows, int32_t k, int8_t* codes, float* scale, void* stream) {
    if (!x || !g) return LQ8_ERR_ARG;
    const llama_q8_status st = check_quant(type, rows, k, codes, scale);
    if (st != LQ8_OK) return st;
    if (type == LLAMA_Q8_GGUF_Q8_0) return LQ8_ERR_UNSUPPORTED;
    const uintptr_t mask = type_mask(type);
    if (x_stride < k || ((uintptr_t)x & mask) || ((uintptr_t)g & 3) || !(eps >= 0.0f) || eps > 3.4e38f)
        return LQ8_ERR_ARG;
    if (delta && (delta_stride < k || ((uintptr_t)delta & mask))) return LQ8_ERR_ARG;
    if (x_out && (out_stride < k || ((uintptr_t)x_out & mask))) return LQ8_ERR_ARG;
    // the sum in the place of one of its parts: row on row
    if ((x_out == x && out_stride != x_stride) || (x_out && x_out == delta && out_stride != delta_stride))
        return LQ8_ERR_ARG;
    if (rows == 0) return LQ8_OK;
    QuantArgs a{};
    a.x = x, a.xs = x_stride, a.b = delta, a.bs = delta_stride, a.out = x_out, a.os = out_stride, a.g = g, a.eps = eps;
    a.rows = rows, a.k = k, a.codes = codes, a.scale = scale, a.row_bytes = llama_q8_i8_row_bytes(k);
    return quant_types<QUANT_NORM>(type, a, (cudaStream_t)stream);
}

llama_q8_status llama_q8_silu_quant(int32_t type, const void* gate, const void* up, int64_t stride, int32_t rows,
                                    int32_t k, int8_t* codes, float* scale, void* stream) {
    if (!gate || !up) return LQ8_ERR_ARG;
    const llama_q8_status st = check_quant(type, rows, k, codes, scale);
    if (st != LQ8_OK) return st;
    if (type == LLAMA_Q8_GGUF_Q8_0) return LQ8_ERR_UNSUPPORTED;
    if (stride < k || (((uintptr_t)gate | (uintptr_t)up) & type_mask(type))) return LQ8_ERR_ARG;
    if (rows == 0) return LQ8_OK;
    QuantArgs a{};
    a.x = gate, a.xs = stride, a.b = up, a.bs = stride, a.rows = rows, a.k = k, a.codes = codes, a.scale = scale;
    a.row_bytes = llama_q8_i8_row_bytes(k);
    return quant_types<QUANT_SILU>(type, a, (cudaStream_t)stream);
}

}  // extern "C"
