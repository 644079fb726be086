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
// half (a few elements in ten thousand), and those are decided in double from
// the stored numbers, as is M (from the few elements within 2^-18 of the f32
// maximum). Rows whose f32 numbers leave the normal range are done in double as
// a whole.
//
// Bound: memory. One CTA of G threads (or one warp) per row keeps the row's v in
// registers (16 values a thread), so every input is read once and every output
// written once; rows of more than 16384 values are read twice.
#include "kernels.cuh"
#include "llama_q8.h"
#include "ptx.cuh"

#include <cuda_bf16.h>

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

constexpr int kPerThread = 16;             // values of a row that a thread keeps
constexpr int kQuantMaxThreads = 1024;
constexpr float kMagic = 12582912.0f;       // 1.5 2^23: adding it rounds to an integer
// Half width of the band around a half in which f32 does not settle a code. t = v (127 / M)
// is at most 127 and off by the relative errors, in units of 2^-24, of: 127 / M 1, M 1, the
// product by it 1, and v (rows 0, norm 1, silu: exp 4, 1 + e 1, the quotient 4, the product 1):
// 127 * 13 * 2^-24 = 9.9e-5 for silu, 3.1e-5 for the others.
template <int OP> constexpr float kWindow = OP == QUANT_SILU ? 1.6e-4f : 5e-5f;
// v within this factor of the f32 maximum may be the exact maximum (2 * 11 * 2^-24 < 2^-19)
constexpr float kNearMax = 1.0f - 1.0f / 262144.0f;
constexpr float kTiny = 7.9e-31f, kHuge = 1e36f;  // M outside: the row is done in double

template <typename T> struct Piece { static constexpr int n = 16 / sizeof(T); };
template <> struct Piece<BlockQ8> { static constexpr int n = 8; };

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// Element i of a row (any i < k).
template <typename T> __device__ __forceinline__ float load_one(const void* x, int64_t row_at, int i) {
    return to_f32(reinterpret_cast<const T*>(x)[row_at + i]);
}
template <> __device__ __forceinline__ float load_one<BlockQ8>(const void* x, int64_t row_at, int i) {
    const uint8_t* blk = reinterpret_cast<const uint8_t*>(x) + (row_at / 32 + i / 32) * 34;
    const float d = __half2float(__ushort_as_half(*reinterpret_cast<const unsigned short*>(blk)));
    return d * (float)reinterpret_cast<const int8_t*>(blk)[2 + i % 32];
}

// Elements i .. i + n - 1 of a row (i a multiple of n), zeros past k. ALIGNED: 16-byte loads, k a multiple of n.
template <typename T, bool ALIGNED>
__device__ __forceinline__ void load_piece(const void* x, int64_t row_at, int i, int k, float (&v)[Piece<T>::n]) {
    constexpr int n = Piece<T>::n;
    if constexpr (ALIGNED) {
        uint4 u = make_uint4(0u, 0u, 0u, 0u);
        if (i < k)
            asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                         : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
                         : "l"(reinterpret_cast<const T*>(x) + row_at + i));
        const T* e = reinterpret_cast<const T*>(&u);
#pragma unroll
        for (int j = 0; j < n; ++j) v[j] = to_f32(e[j]);
    } else {
#pragma unroll
        for (int j = 0; j < n; ++j) v[j] = i + j < k ? load_one<T>(x, row_at, i + j) : 0.0f;
    }
}
template <>
__device__ __forceinline__ void load_piece<BlockQ8, true>(const void* x, int64_t row_at, int i, int k, float (&v)[8]) {
    // 8 codes of one block (blocks lie on 2-byte boundaries)
    if (i >= k) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = 0.0f;
        return;
    }
    const unsigned short* blk = reinterpret_cast<const unsigned short*>(
        reinterpret_cast<const uint8_t*>(x) + (row_at / 32 + i / 32) * 34);
    const float d = __half2float(__ushort_as_half(blk[0]));
    const unsigned short* q = blk + 1 + (i % 32) / 2;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const unsigned short w = q[j];
        v[2 * j] = d * (float)(int8_t)(w & 0xff);
        v[2 * j + 1] = d * (float)(int8_t)(w >> 8);
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

// silu(gate) up in double
__device__ __noinline__ double silu_up_f64(float gate, float up) {
    return (double)gate / (1.0 + exp(-(double)gate)) * (double)up;
}
__device__ __forceinline__ float silu_up(float gate, float up) {
    // below -80 the quotient's divisor passes the range of the quick division
    if (gate < -80.0f) return (float)silu_up_f64(gate, up);
    return __fdividef(gate, 1.0f + expf(-gate)) * up;
}

template <int OP, typename T, bool ALIGNED> struct Row {
    static constexpr int n = Piece<T>::n;
    const QuantArgs& a;
    int64_t xa, ba, oa;
    __device__ Row(const QuantArgs& args, int64_t r) : a(args), xa(r * args.xs), ba(r * args.bs), oa(r * args.os) {}

    // h of elements i .. i + n - 1 as the first pass makes it; STORE writes it out
    template <bool STORE> __device__ __forceinline__ void sums(int i, float (&h)[n]) const {
        load_piece<T, ALIGNED>(a.x, xa, i, a.k, h);
        if constexpr (OP == QUANT_NORM) {
            if (a.b) {
                float d[n];
                load_piece<T, ALIGNED>(a.b, ba, i, a.k, d);
#pragma unroll
                for (int j = 0; j < n; ++j) h[j] = to_f32(from_f32<T>(h[j] + d[j]));
            }
            if (STORE && a.out) store_piece<T, ALIGNED>(a.out, oa, i, a.k, h);
        }
    }
    // v of the same elements, the sum of the squares of h added to ss
    template <bool STORE> __device__ __forceinline__ void values(int i, float (&v)[n], float& ss) const {
        if constexpr (OP == QUANT_SILU) {
            float up[n];
            load_piece<T, ALIGNED>(a.x, xa, i, a.k, v);
            load_piece<T, ALIGNED>(a.b, ba, i, a.k, up);
#pragma unroll
            for (int j = 0; j < n; ++j) v[j] = silu_up(v[j], up[j]);
        } else {
            sums<STORE>(i, v);
            if constexpr (OP == QUANT_NORM) {
                float g[n];
#pragma unroll
                for (int j = 0; j < n; ++j) ss = fmaf(v[j], v[j], ss);
                if constexpr (ALIGNED) {
#pragma unroll
                    for (int j = 0; j < n; j += 4) {
                        float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
                        if (i < a.k) f = *reinterpret_cast<const float4*>(a.g + i + j);
                        g[j] = f.x, g[j + 1] = f.y, g[j + 2] = f.z, g[j + 3] = f.w;
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < n; ++j) g[j] = i + j < a.k ? a.g[i + j] : 0.0f;
                }
#pragma unroll
                for (int j = 0; j < n; ++j) v[j] *= g[j];
            }
        }
    }
    // h of element i after the first pass (which may have written it over x or delta)
    __device__ __forceinline__ float h_again(int i) const {
        if (OP == QUANT_NORM && a.out) return load_one<T>(a.out, oa, i);
        float h = load_one<T>(a.x, xa, i);
        if constexpr (OP == QUANT_NORM)
            if (a.b) h = to_f32(from_f32<T>(h + load_one<T>(a.b, ba, i)));
        return h;
    }
    // v of element i in double: exact for rows (one number) and norm (a product of two f32)
    __device__ double v_f64(int i) const {
        if constexpr (OP == QUANT_SILU) return silu_up_f64(load_one<T>(a.x, xa, i), load_one<T>(a.b, ba, i));
        if constexpr (OP == QUANT_NORM) return (double)h_again(i) * (double)a.g[i];
        return (double)load_one<T>(a.x, xa, i);
    }
};
// no element type but BlockQ8 stands only under rows_quant
template <bool ALIGNED> struct Row<QUANT_ROWS, BlockQ8, ALIGNED> {
    static constexpr int n = 8;
    const QuantArgs& a;
    int64_t xa;
    __device__ Row(const QuantArgs& args, int64_t r) : a(args), xa(r * args.xs) {}
    template <bool STORE> __device__ __forceinline__ void values(int i, float (&v)[n], float&) const {
        load_piece<BlockQ8, true>(a.x, xa, i, a.k, v);
    }
    __device__ __forceinline__ float h_again(int i) const { return load_one<BlockQ8>(a.x, xa, i); }
    __device__ double v_f64(int i) const { return (double)load_one<BlockQ8>(a.x, xa, i); }
};

// Whether 127 |v| / M is at least q + 1/2, from exact v and M: the sign of 254 |v| - (2 q + 1) M. Where the two
// products are close their difference is exact, and so is the rounding error that is taken off.
__device__ __forceinline__ bool above_half(double v, double M, float q) {
    const double odd = 2.0 * (double)q + 1.0, p = odd * M, e = fma(odd, M, -p);
    return fma(254.0, fabs(v), -p) - e >= 0.0;
}

// The bits of a magnitude order like the magnitude, NaN above infinity.
__device__ __forceinline__ uint32_t magnitude_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// One row's reduction area; a warp's or a CTA's.
struct QuantShared {
    uint32_t max[32];
    float ss[32];
    unsigned long long exact;  // the exact maximum as the bits of a double
    double ss64;
    int poison;
};

template <int G> __device__ __forceinline__ void row_sync() {
    if constexpr (G == 32) __syncwarp();
    else __syncthreads();
}

// G threads per row (32: a warp; 128 / G rows per CTA below 128). LOOP: rows too long for the registers, read again.
template <int OP, typename T, bool ALIGNED, int G, bool LOOP>
__global__ void __launch_bounds__(G < 128 ? 128 : G) quant_kernel(const QuantArgs a) {
    using R = Row<OP, T, ALIGNED>;
    constexpr int n = R::n, pieces = kPerThread / n;
    constexpr int kRowsPerCta = G == 32 ? 4 : 1;
    __shared__ QuantShared shared[kRowsPerCta];
    const int t = G == 32 ? threadIdx.x & 31 : threadIdx.x, lane = threadIdx.x & 31, warp = t >> 5;
    QuantShared& sh = shared[G == 32 ? threadIdx.x >> 5 : 0];
    const int64_t r = (int64_t)blockIdx.x * kRowsPerCta + (G == 32 ? threadIdx.x >> 5 : 0);
    if (r >= a.rows) return;  // a whole warp (G == 32) or none
    const R row(a, r);
    const int k = a.k, k16 = (int)a.row_bytes;
    int8_t* codes = a.codes + r * a.row_bytes;
    if (t == 0) sh.exact = 0ull, sh.ss64 = 0.0, sh.poison = 0;

    // the row once: v in registers, the largest magnitude, the sum of squares
    float v[LOOP ? n : kPerThread];
    float ss = 0.0f;
    uint32_t mx = 0u;
    if constexpr (!LOOP) {
#pragma unroll
        for (int p = 0; p < pieces; ++p) {
            float w[n];
            row.template values<true>((p * G + t) * n, w, ss);
#pragma unroll
            for (int j = 0; j < n; ++j) v[p * n + j] = w[j], mx = max(mx, magnitude_bits(w[j]));
        }
    } else {
        float part[4] = {0.f, 0.f, 0.f, 0.f};  // short chains: a thread has many squares to add
        for (int i = t * n, p = 0; i < k; i += G * n, ++p) {
            float w[n], s = 0.0f;
            row.template values<true>(i, w, s);
            part[p & 3] += s;
#pragma unroll
            for (int j = 0; j < n; ++j) mx = max(mx, magnitude_bits(w[j]));
        }
        ss = (part[0] + part[1]) + (part[2] + part[3]);
    }
    mx = __reduce_max_sync(0xffffffffu, mx);
    if constexpr (OP == QUANT_NORM) ss = warp_sum(ss);
    if constexpr (G > 32) {
        if (lane == 0) sh.max[warp] = mx, sh.ss[warp] = ss;
        __syncthreads();
        mx = __reduce_max_sync(0xffffffffu, lane < G / 32 ? sh.max[lane] : 0u);
        if constexpr (OP == QUANT_NORM) ss = warp_sum(lane < G / 32 ? sh.ss[lane] : 0.0f);
    } else {
        __syncwarp();
    }
    const float M = __uint_as_float(mx);
    if (mx == 0u && (OP != QUANT_NORM || ss < kHuge)) {
        // zeros (a norm whose sum of squares is NaN or beyond f32 is looked at below), or v below the smallest f32
        bool zero = true;
        if constexpr (OP != QUANT_ROWS) {
            for (int i = t; i < k; i += G) zero &= row.v_f64(i) == 0.0;
            if constexpr (G == 32) zero = __all_sync(0xffffffffu, zero);
            else zero = __syncthreads_and(zero);
        }
        if (zero) {
            for (int i = t * 4; i < k16; i += G * 4) *reinterpret_cast<uint32_t*>(codes + i) = 0u;
            if (t == 0) a.scale[r] = 0.0f;
            return;
        }
    }

    if (!(M >= kTiny && M <= kHuge) || (OP == QUANT_NORM && !(ss >= 1e-28f && ss <= kHuge))) {
        // outside the range in which f32 settles codes (or not finite): the row in double
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
        atomicMax(&sh.exact, (unsigned long long)__double_as_longlong(top));
        if constexpr (OP == QUANT_NORM) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            for (int w = 0; w < (G + 31) / 32; ++w) {
                if (lane == 0 && warp == w) sh.ss64 += sum;
                row_sync<G>();
            }
        }
        row_sync<G>();
        const double M64 = __longlong_as_double((long long)sh.exact);
        const bool poison = sh.poison != 0;
        for (int i = t; i < k16; i += G) {
            int c = 0;
            if (i < k && !poison && M64 > 0.0) {
                const double w = row.v_f64(i);
                const float q = (float)floor(127.0 * fabs(w) / M64 - 0.25);  // the code or the one below
                c = (int)fmaxf(q, 0.0f);
                while (c < 127 && above_half(w, M64, (float)c)) ++c;
                if (w < 0.0) c = -c;
            }
            codes[i] = (int8_t)c;
        }
        if (t == 0) {
            double f = 1.0;
            if constexpr (OP == QUANT_NORM) f = 1.0 / sqrt(sh.ss64 / k + (double)a.eps);
            a.scale[r] = poison ? __int_as_float(0x7fffffff) : (float)(M64 == 0.0 ? 0.0 : M64 * f / 127.0);
        }
        return;
    }

    // v of elements i .. i + n - 1 once more (h from where the first pass left it)
    auto again = [&](int i, float(&w)[n]) {
        if constexpr (OP == QUANT_NORM) {
#pragma unroll
            for (int j = 0; j < n; ++j) w[j] = i + j < k ? row.h_again(i + j) * a.g[i + j] : 0.0f;
        } else {
            float unused = 0.0f;
            row.template values<false>(i, w, unused);
        }
    };
    // the exact maximum, of the elements that may be it
    double M64 = M;
    if constexpr (OP != QUANT_ROWS) {
        const float near = M * kNearMax;
        auto offer = [&](int i, float w) {
            if (fabsf(w) >= near)
                atomicMax(&sh.exact, (unsigned long long)__double_as_longlong(fabs(row.v_f64(i))));
        };
        if constexpr (!LOOP) {
#pragma unroll
            for (int p = 0; p < pieces; ++p)
#pragma unroll
                for (int j = 0; j < n; ++j) offer((p * G + t) * n + j, v[p * n + j]);
        } else {
            for (int i = t * n; i < k; i += G * n) {
                float w[n];
                again(i, w);
#pragma unroll
                for (int j = 0; j < n; ++j) offer(i + j, w[j]);
            }
        }
        row_sync<G>();
        M64 = __longlong_as_double((long long)sh.exact);
    }

    // codes
    const float inv = __fdiv_rn(127.0f, M);
    auto code = [&](int i, float w) -> uint32_t {
        const float m = fmaf(w, inv, kMagic);  // rounded; its low byte is the code
        const float off = fabsf(fmaf(w, inv, kMagic - m));
        int c = __float_as_int(m);
        if (off > 0.5f - kWindow<OP>) {
            const float q = floorf(fabsf(w) * inv);
            const int u = (int)q + (above_half(row.v_f64(i), M64, q) ? 1 : 0);
            c = w < 0.0f ? -u : u;
        }
        return (uint32_t)c & 0xffu;
    };
    auto store = [&](int i, const float* w) {
        uint32_t word[n / 4];
#pragma unroll
        for (int j = 0; j < n / 4; ++j)
            word[j] = code(i + 4 * j, w[4 * j]) | code(i + 4 * j + 1, w[4 * j + 1]) << 8 |
                      code(i + 4 * j + 2, w[4 * j + 2]) << 16 | code(i + 4 * j + 3, w[4 * j + 3]) << 24;
        if (i < k16) {
            if constexpr (n == 8) *reinterpret_cast<uint2*>(codes + i) = make_uint2(word[0], word[1]);
            else *reinterpret_cast<uint32_t*>(codes + i) = word[0];
        }
    };
    if constexpr (!LOOP) {
#pragma unroll
        for (int p = 0; p < pieces; ++p) store((p * G + t) * n, v + p * n);
    } else {
        for (int i = t * n; i < k16; i += G * n) {
            float w[n];
            again(i, w);
            store(i, w);
        }
    }
    if (t == 0) {
        float d;
        if constexpr (OP == QUANT_NORM) d = __fdiv_rn((float)M64, 127.0f * __fsqrt_rn(ss / (float)k + a.eps));
        else d = __fdiv_rn((float)M64, 127.0f);
        a.scale[r] = d;
    }
}

template <int OP, typename T, bool ALIGNED>
static cudaError_t launch_quant(const QuantArgs& a, cudaStream_t s) {
    const int threads = (int)((a.row_bytes + kPerThread - 1) / kPerThread);
    auto go = [&](auto kernel, int rows_per_cta, int block) {
        const unsigned grid = (unsigned)(((int64_t)a.rows + rows_per_cta - 1) / rows_per_cta);
        return launch_ex(kernel, dim3(grid), dim3((unsigned)block), 0, s, false, a);
    };
    if (threads <= 32) return go(quant_kernel<OP, T, ALIGNED, 32, false>, 4, 128);
    if (threads <= 128) return go(quant_kernel<OP, T, ALIGNED, 128, false>, 1, 128);
    if (threads <= 256) return go(quant_kernel<OP, T, ALIGNED, 256, false>, 1, 256);
    if (threads <= 512) return go(quant_kernel<OP, T, ALIGNED, 512, false>, 1, 512);
    if (threads <= 1024) return go(quant_kernel<OP, T, ALIGNED, 1024, false>, 1, 1024);
    return go(quant_kernel<OP, T, ALIGNED, 1024, true>, 1, 1024);
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
