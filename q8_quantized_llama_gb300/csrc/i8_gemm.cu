// Many tokens: the int8 product on the 5th-generation tensor cores.
//
// The GPU has no fast integer tensor rate, but int8 codes are exact in f16, a
// product of two is exact in f32 (14 bits), and a tensor-core sum in f32 is the
// exact integer as long as no partial sum passes 2^24. By the Cauchy-Schwarz
// inequality no partial sum of a row and a token passes |a| |w|, so a tile whose
// largest norms multiply to no more than 2^24 is summed in one go (activations
// and weights of models lie a factor of four and more below, at k = 14336);
// the others are read out as integers after every 1024 products (1024 * 128^2 =
// 2^24).
//
// i8_widen_kernel turns the token rows into f16 once per call and notes their
// norms. i8_gemm_kernel: CTA tile 128 channels (M) x bn tokens (N, a multiple of
// 16 up to 256), 64 codes of k per stage, one CTA per SM, persistent. Warp roles:
//  - producer: per stage two tensor copies, the f16 token tile (128-byte rows of 64
//    values, 128-byte swizzle: the K-major B operand, used in place) and the codes
//    of the four 32-row tiles;
//  - 4 converter warps: row r's 64 codes as f16 into lane r of tensor memory (the A
//    operand), one stage's columns next to the other's;
//  - MMA warp: one thread issues four 128 x bn x 16 products per stage;
//  - 8 accumulator warps read the finished sums (every second group of 16 columns
//    each), apply the scales and store: a warp's 32 lanes hold 32 neighbouring
//    channels of a token, 128 bytes of y.
//
// Work is dealt in whole tiles (tokens fastest, so that the CTAs that share a weight
// tile run together), or, where whole tiles would leave SMs idle, in equal runs of
// k-blocks: tiles that are cut meet as integers in the workspace, where the last CTA
// to finish its part adds them (integers: in any order the same).
#include "i8.cuh"
#include "kernels.cuh"
#include "llama_q8.h"
#include "paged.cuh"
#include "tc.cuh"

namespace lq8 {

constexpr int kI8BM = 128;
constexpr int kI8Ctas = 152;       // SMs of a GB300; the plan does not depend on the device at hand
constexpr int kI8ConvWarps = 4, kI8AccWarps = 8;
constexpr int kI8AccWarp0 = kI8ConvWarps, kI8ProducerWarp = kI8ConvWarps + kI8AccWarps, kI8MmaWarp = kI8ProducerWarp + 1;
constexpr int kI8Threads = (kI8MmaWarp + 1) * 32;
constexpr int kI8StagesMax = 8;
constexpr int kI8CodeBytes = kI8BM * 64;  // a stage's codes
constexpr int kI8Smem = 220 * 1024;       // stages, in units of what a tile's width needs
constexpr int kI8Exact = 16;              // k-blocks whose products cannot pass 2^24
constexpr int kI8ACols = 32;              // tensor-memory columns of a stage's A
constexpr int kI8Slots = 3;               // parts a CTA can hold: the tile it begins in, the one it ends in, one between

struct I8Gemm {
    I8Weights W;
    const float* anorm;  // per token
    const float* sa;
    int m, bn, token_tiles, kb;
    int stages, buffers;
    int64_t tiles;
    int64_t y_stride;
    int32_t* slots;      // [CTA][kI8Slots][bn][128]
    unsigned* counters;  // per CTA: parts of the tile it ends in
    bool cut;            // equal runs of k-blocks instead of whole tiles
    int32_t* err;
};

__device__ __forceinline__ bool i8_try(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
// One thread of the warp, the same at every call (the single-thread instructions of the tensor cores take uniform
// operands: behind a comparison with the lane's number each of them took 65 cycles to issue).
__device__ __forceinline__ bool i8_elect() {
    uint32_t one;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(one));
    return one != 0;
}
__device__ __forceinline__ void i8_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void i8_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
// a tensor copy of a box at (x, y), completing on the barrier
__device__ __forceinline__ void i8_box(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
        "[%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

// The segments of tiles that a CTA works on, the same for all its warps.
struct I8Segments {
    const I8Gemm& g;
    int64_t at, end, tile;
    int k0, k1;
    __device__ I8Segments(const I8Gemm& args) : g(args) {
        const int64_t units = g.tiles * g.kb, c = blockIdx.x, n = gridDim.x;
        at = g.cut ? units * c / n : c, end = g.cut ? units * (c + 1) / n : g.tiles;
    }
    __device__ bool next() {
        if (at >= end) return false;
        if (g.cut) {
            tile = at / g.kb, k0 = (int)(at % g.kb);
            k1 = (int)(end - at < g.kb - k0 ? k0 + (end - at) : g.kb);
            at += k1 - k0;
        } else {
            tile = at, k0 = 0, k1 = g.kb;
            at += gridDim.x;
        }
        return true;
    }
    __device__ int channel0() const { return (int)(tile / g.token_tiles) * kI8BM; }
    __device__ int token0() const { return (int)(tile % g.token_tiles) * g.bn; }
};

// A position in a ring of buffers and the parity of its pass. What a role does for each stage is a chain of
// dependent instructions that one thread or warp issues alone, so it is kept short: positions are counted up (a
// quotient by a number that is not known when compiling takes longer than a stage's products) and barriers are
// addressed in shared memory.
struct I8Ring {
    int n, at = 0;
    uint32_t parity = 0;
    __device__ explicit I8Ring(int count) : n(count) {}
    __device__ __forceinline__ void next() {
        if (++at == n) at = 0, parity ^= 1u;
    }
};

// The bounded wait of mbar_wait_bounded with its timer out of the way.
__device__ __noinline__ bool i8_wait_long(uint32_t bar, uint32_t parity, int32_t* err) {
    const uint64_t t0 = global_timer_ns();
    while (!i8_try(bar, parity))
        if (global_timer_ns() - t0 > 1000000000ull) {
            report(err, LQ8_ERR_CUDA);
            return false;
        }
    return true;
}
__device__ __forceinline__ bool i8_wait(uint32_t bar, uint32_t parity, int32_t* err) {
    return i8_try(bar, parity) || i8_try(bar, parity) || i8_try(bar, parity) || i8_wait_long(bar, parity, err);
}

// Whether no sum of the tile can pass 2^24 (one warp; the same answer in every warp).
__device__ __forceinline__ bool i8_one_sum(const I8Gemm& g, int channel0, int token0, int lane) {
    float w = 0.0f, a = 0.0f;
    const int t = channel0 / 32 + lane;
    if (lane < 4 && t < g.W.rows_pad / 32) w = g.W.norm[t];
    for (int i = lane; i < g.bn; i += 32)
        if (token0 + i < g.m) a = fmaxf(a, __ldcg(g.anorm + token0 + i));
    return warp_max(w) * warp_max(a) <= 16777216.0f;
}

template <typename T>
__global__ void __launch_bounds__(kI8Threads, 1)
    i8_gemm_kernel(const I8Gemm g, const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap wmap,
                   T* __restrict__ y) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ __align__(8) uint64_t full_bar[kI8StagesMax];  // copies landed
    __shared__ __align__(8) uint64_t conv_bar[kI8StagesMax];  // A in tensor memory
    __shared__ __align__(8) uint64_t done_bar[kI8StagesMax];  // products of the stage complete
    __shared__ __align__(8) uint64_t sum_full[2];             // a chunk's sums complete
    __shared__ __align__(8) uint64_t sum_empty[2];            // and read
    __shared__ uint32_t tmem_holder;
    __shared__ unsigned ticket;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int stages = g.stages, token_bytes = g.bn * 128, stage_bytes = token_bytes + kI8CodeBytes;
    if (tid == 0) {
        for (int s = 0; s < kI8StagesMax; ++s) {
            mbar_init(&full_bar[s], 1);
            mbar_init(&conv_bar[s], kI8ConvWarps);
            mbar_init(&done_bar[s], 1);
        }
        for (int p = 0; p < 2; ++p) {
            mbar_init(&sum_full[p], 1);
            mbar_init(&sum_empty[p], kI8AccWarps);
        }
        fence_mbar_init();
    }
    if (warp == kI8MmaWarp) tmem_alloc(&tmem_holder, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_holder, tmem_a = tmem + (uint32_t)(g.buffers * g.bn);
    const uint32_t data = smem_u32(smem), full = smem_u32(full_bar), conv = smem_u32(conv_bar), done = smem_u32(done_bar),
                   sfull = smem_u32(sum_full), sempty = smem_u32(sum_empty);
    bool alive = true;  // cleared by a wait that ran out; the role then ends

    if (warp == kI8ProducerWarp) {
        if (lane == 0) {
            // boxes are whole: codes past the last chunk or tile and tokens past the last arrive as zeros
            auto issue_codes = [&](int channel0, int kb, int s) {
                const uint32_t bar = full + s * 8;
                asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(stage_bytes)
                             : "memory");
                i8_box(data + s * stage_bytes + token_bytes, &wmap, kb * 256, channel0 / 32, bar);
            };
            auto issue_tokens = [&](int token0, int kb, int s) {
                i8_box(data + s * stage_bytes, &amap, kb * 64, token0, full + s * 8);
            };
            // the first stages' codes do not depend on the kernel before
            int ahead = 0;
            {
                I8Segments seg(g);
                while (ahead < stages && seg.next()) {
                    const int channel0 = seg.channel0();
                    for (int kb = seg.k0; kb < seg.k1 && ahead < stages; ++kb) issue_codes(channel0, kb, ahead++);
                }
            }
            pdl_wait();
            I8Segments seg(g);
            I8Ring ring(stages);
            bool again = false;  // past the first pass over the stages
            while (alive && seg.next()) {
                const int channel0 = seg.channel0(), token0 = seg.token0();
                for (int kb = seg.k0; kb < seg.k1; ++kb) {
                    const int s = ring.at;
                    if (again) {
                        alive = i8_wait(done + s * 8, ring.parity ^ 1u, g.err);
                        if (!alive) break;
                        issue_codes(channel0, kb, s);
                    }
                    issue_tokens(token0, kb, s);
                    ring.next();
                    again |= ring.at == 0;
                }
            }
            // every copy has landed before the CTA may exit: the last of each stage
            for (int i = 0; i < stages; ++i) {
                if (i >= ring.at && !again) break;
                i8_wait(full + i * 8, i < ring.at ? ring.parity : ring.parity ^ 1u, g.err);
            }
        }
        __syncwarp();
    } else if (warp == kI8MmaWarp) {
        pdl_wait();
        const uint32_t idesc = idesc_f16(kI8BM, (uint32_t)g.bn);
        const uint64_t desc0 = sw128_desc(data);
        I8Segments seg(g);
        I8Ring ring(stages), sums(g.buffers);
        bool again = false;  // past the first pass over the sum buffers
        uint32_t last = 0, last_parity = 0;
        while (alive && seg.next()) {
            const int n = seg.k1 - seg.k0;
            const bool one = n <= kI8Exact || i8_one_sum(g, seg.channel0(), seg.token0(), lane);
            for (int left = n; left > 0 && alive;) {
                int blocks = one ? left : min(left, kI8Exact);
                left -= blocks;
                if (again) alive = __all_sync(0xffffffffu, i8_wait(sempty + sums.at * 8, sums.parity ^ 1u, g.err));
                const uint32_t d = tmem + (uint32_t)(sums.at * g.bn);
                uint32_t accumulate = 0;
                for (; blocks > 0 && alive; --blocks) {
                    const int s = ring.at;
                    // the converters arrive after the stage's copies: the token tile has landed too
                    alive = __all_sync(0xffffffffu, i8_wait(conv + s * 8, ring.parity, g.err));
                    if (!alive) break;
                    tc_fence_after();
                    const uint64_t b = desc0 + (uint32_t)(s * stage_bytes >> 4);
                    const uint32_t a = tmem_a + (uint32_t)(s * kI8ACols);
                    if (i8_elect()) {
                        mma_f16_ts(d, a, b, idesc, accumulate);  // 16 k: 8 columns of A, 32 bytes of B's rows
                        mma_f16_ts(d, a + 8, b + 2, idesc, 1u);
                        mma_f16_ts(d, a + 16, b + 4, idesc, 1u);
                        mma_f16_ts(d, a + 24, b + 6, idesc, 1u);
                        i8_commit(done + s * 8);
                        if (blocks == 1) i8_commit(sfull + sums.at * 8);
                    }
                    accumulate = 1u;
                    last = done + s * 8, last_parity = ring.parity;
                    ring.next();
                }
                sums.next();
                again |= sums.at == 0;
            }
        }
        // products in flight read shared memory and write tensor memory: the last is complete before the CTA exits
        if (last) i8_wait(last, last_parity, g.err);
        __syncwarp();
    } else if (warp < kI8ConvWarps) {
        const uint32_t base = tmem_a + ((uint32_t)(warp * 32) << 16);
        I8Segments seg(g);
        I8Ring ring(stages);
        while (alive && seg.next())
            for (int kb = seg.k0; kb < seg.k1; ++kb, ring.next()) {
                const int s = ring.at;
                alive = i8_wait(full + s * 8, ring.parity, g.err);
                if (!__all_sync(0xffffffffu, alive)) {
                    alive = false;
                    break;
                }
                tc_fence_after();
                const uint4* q = reinterpret_cast<const uint4*>(smem + s * stage_bytes + token_bytes + warp * 2048) + lane;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t u[16];
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const uint4 v = q[(2 * h + c) * 32];
                        codes_to_f16x2(v.x, u[8 * c + 0], u[8 * c + 1]);
                        codes_to_f16x2(v.y, u[8 * c + 2], u[8 * c + 3]);
                        codes_to_f16x2(v.z, u[8 * c + 4], u[8 * c + 5]);
                        codes_to_f16x2(v.w, u[8 * c + 6], u[8 * c + 7]);
                    }
                    tmem_st16(base + (uint32_t)(s * kI8ACols + h * 16), u);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) i8_arrive(conv + s * 8);
            }
    } else {
        pdl_wait();
        const int aw = warp - kI8AccWarp0, quarter = warp & 3, half = aw >> 2;
        const int groups = g.bn / 16;
        const uint32_t base = tmem + ((uint32_t)(quarter * 32) << 16);
        // a warp whose wait ran out still meets the others at their barriers
        I8Segments seg(g);
        I8Ring sums(g.buffers);
        while (seg.next()) {
            const int n = seg.k1 - seg.k0, channel0 = seg.channel0(), token0 = seg.token0();
            const bool one = n <= kI8Exact || i8_one_sum(g, channel0, token0, lane);
            const bool whole = n == g.kb;
            const int channel = channel0 + quarter * 32 + lane;
            const bool mine = channel < g.W.rows;
            const float sw = mine ? g.W.scale[channel] : 0.0f;
            // parts: 0 the tile the CTA begins in, 1 the one it ends in, 2 a whole tile in more than one chunk
            int32_t* slot = g.slots + ((int64_t)blockIdx.x * kI8Slots + (whole ? 2 : seg.k0 > 0 ? 0 : 1)) * g.bn * kI8BM +
                            quarter * 32 + lane;
            auto store = [&](int c, auto v) {  // an exact sum, as an integer or as f32
                const int t = token0 + c;
                if (mine && t < g.m) y[(int64_t)t * g.y_stride + channel] = i8_scaled<T>(v, g.sa[t], sw);
            };
            const int chunks = one ? 1 : (n + kI8Exact - 1) / kI8Exact;
            for (int ch = 0; ch < chunks; ++ch, sums.next()) {
                const int p = sums.at;
                if (alive) alive = i8_wait(sfull + p * 8, sums.parity, g.err);
                alive = __all_sync(0xffffffffu, alive);
                if (!alive) break;
                tc_fence_after();
                for (int gr = half; gr < groups; gr += 2) {
                    float v[16];
                    tmem_ld16(base + (uint32_t)(p * g.bn + gr * 16), v);
                    int32_t* at = slot + (int64_t)gr * 16 * kI8BM;
                    if (whole && chunks == 1) {
#pragma unroll
                        for (int j = 0; j < 16; ++j) store(gr * 16 + j, v[j]);
                    } else {
                        int i[16];
#pragma unroll
                        for (int j = 0; j < 16; ++j) i[j] = __float2int_rn(v[j]) + (ch > 0 ? at[j * kI8BM] : 0);
                        if (whole && ch == chunks - 1) {
#pragma unroll
                            for (int j = 0; j < 16; ++j) store(gr * 16 + j, i[j]);
                        } else {
#pragma unroll
                            for (int j = 0; j < 16; ++j) at[j * kI8BM] = i[j];
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) i8_arrive(sempty + p * 8);
            }
            if (!whole) {
                // the part is in the workspace; the CTA that brings the tile's last one adds them all
                const int64_t units = g.tiles * g.kb, u0 = seg.tile * g.kb, u1 = u0 + g.kb;
                const int G = gridDim.x;
                // the CTAs whose runs hold the tile's first and last unit: unit u is in run c with
                // units * c / G <= u < units * (c + 1) / G, rounded down
                auto owner = [&](int64_t u) { return (int)(((u + 1) * G - 1) / units); };
                const int c0 = owner(u0), c1 = owner(u1 - 1);
                named_bar_sync(1, kI8AccWarps * 32);
                if (tid == kI8AccWarp0 * 32) ticket = take_ticket(&g.counters[c0]);
                named_bar_sync(1, kI8AccWarps * 32);
                if (alive && ticket == (unsigned)(c1 - c0)) {
                    if (tid == kI8AccWarp0 * 32) g.counters[c0] = 0u;
                    const int64_t part = (int64_t)g.bn * kI8BM;
                    const int32_t* first = g.slots + ((int64_t)c0 * kI8Slots + 1) * part + quarter * 32 + lane;
                    for (int gr = half; gr < groups; gr += 2) {
                        int i[16];
                        const int64_t off = (int64_t)gr * 16 * kI8BM;
#pragma unroll
                        for (int j = 0; j < 16; ++j) i[j] = __ldcg(first + off + j * kI8BM);
                        for (int c = c0 + 1; c <= c1; ++c) {
                            const int32_t* other =
                                g.slots + (int64_t)c * kI8Slots * part + off + quarter * 32 + lane;
#pragma unroll
                            for (int j = 0; j < 16; ++j) i[j] += __ldcg(other + j * kI8BM);
                        }
#pragma unroll
                        for (int j = 0; j < 16; ++j) store(gr * 16 + j, i[j]);
                    }
                }
                named_bar_sync(1, kI8AccWarps * 32);  // `ticket` has been read
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kI8MmaWarp) tmem_dealloc(tmem, 512);
}

// The token rows as f16 and their norms, rounded up: one CTA per row.
__global__ void __launch_bounds__(256) i8_widen_kernel(const uint4* __restrict__ codes, int64_t chunks,
                                                       uint4* __restrict__ wide, float* __restrict__ norm) {
    __shared__ uint32_t part[8];
    pdl_launch_dependents();
    const int64_t row = blockIdx.x;
    int sum = 0;
    for (int64_t c = threadIdx.x; c < chunks; c += 256) {
        const uint4 q = codes[row * chunks + c];
        uint4 lo, hi;
        codes_to_f16x2(q.x, lo.x, lo.y);
        codes_to_f16x2(q.y, lo.z, lo.w);
        codes_to_f16x2(q.z, hi.x, hi.y);
        codes_to_f16x2(q.w, hi.z, hi.w);
        wide[(row * chunks + c) * 2] = lo;
        wide[(row * chunks + c) * 2 + 1] = hi;
        sum = __dp4a((int)q.x, (int)q.x, sum);
        sum = __dp4a((int)q.y, (int)q.y, sum);
        sum = __dp4a((int)q.z, (int)q.z, sum);
        sum = __dp4a((int)q.w, (int)q.w, sum);
    }
    const uint32_t s = __reduce_add_sync(0xffffffffu, (uint32_t)sum);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        uint32_t all = 0;
        for (int w = 0; w < 8; ++w) all += part[w];  // at most 131056 * 2^14 < 2^31
        norm[row] = __fsqrt_ru(__uint2float_ru(all));
    }
}

// ---- the plan of a call, from its sizes alone ------------------------------------------
struct I8Plan {
    int64_t tokens;  // of one launch
    int bn, token_tiles, kb, stages, buffers;
    int64_t tiles;
    bool cut;
    size_t wide, norms, slots, total;  // byte offsets in the workspace
};

static I8Plan i8_plan(int64_t rows, int64_t k, int64_t m) {
    I8Plan p{};
    const int64_t k16 = (k + 15) / 16 * 16;
    // tokens widened at a time: 512 MB of f16, and enough of them to fill the GPU
    int64_t most = (512ll << 20) / (2 * k16) / 256 * 256;
    most = most < 2048 ? 2048 : most > 65536 ? 65536 : most;
    p.tokens = m < most ? m : most;
    p.token_tiles = (int)((p.tokens + 255) / 256);
    p.bn = (int)(((p.tokens + p.token_tiles - 1) / p.token_tiles + 15) / 16 * 16);
    if (p.bn < 32) p.bn = 32;
    const int64_t tiles = (rows + kI8BM - 1) / kI8BM * p.token_tiles;
    p.tiles = tiles;
    p.kb = (int)((k16 + 63) / 64);
    p.stages = kI8Smem / (p.bn * 128 + kI8CodeBytes);
    if (p.stages > kI8StagesMax) p.stages = kI8StagesMax;
    // two buffers of sums where four stages still fit beside them
    p.buffers = (512 - 2 * p.bn) / kI8ACols >= 4 ? 2 : 1;
    const int room = (512 - p.buffers * p.bn) / kI8ACols;
    if (p.stages > room) p.stages = room;
    // whole tiles take waves * kb blocks of time, equal runs their share and the exchange of parts (about 8 blocks)
    const int64_t waves = (tiles + kI8Ctas - 1) / kI8Ctas;
    p.cut = waves * p.kb > (tiles * p.kb + kI8Ctas - 1) / kI8Ctas + 8;
    auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    p.wide = kCounterBytes;
    p.norms = up(p.wide + (size_t)p.tokens * k16 * 2);
    p.slots = up(p.norms + (size_t)p.tokens * 4);
    p.total = up(p.slots + (size_t)kI8Ctas * kI8Slots * p.bn * kI8BM * 4);
    return p;
}

size_t i8_gemm_workspace(int64_t rows, int64_t k, int64_t m) { return i8_plan(rows, k, m).total; }

cudaError_t init_i8_gemm_attributes() {
    cudaError_t e = cudaFuncSetAttribute(i8_gemm_kernel<float>, cudaFuncAttributeMaxDynamicSharedMemorySize, kI8Smem + 1024);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(i8_gemm_kernel<__half>, cudaFuncAttributeMaxDynamicSharedMemorySize, kI8Smem + 1024);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(i8_gemm_kernel<__nv_bfloat16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kI8Smem + 1024);
    return e;
}

template <typename T>
cudaError_t launch_i8_gemm(const I8Weights& W, int64_t k, const int8_t* a, const float* sa, int64_t m,
                           T* y, int64_t y_stride, void* workspace, int32_t* err, cudaStream_t s) {
    const I8Plan full = i8_plan(W.rows, k, m);
    cudaError_t e = get_encode_tiled();
    if (e != cudaSuccess) return e;
    uint8_t* ws = reinterpret_cast<uint8_t*>(workspace);
    // the packed codes as rows of 8-byte words, a row per 32-row tile: boxes of 4 tiles x 64 k (2 KB of a row)
    CUtensorMap wmap;
    {
        const cuuint64_t dims[2] = {(cuuint64_t)W.chunks * 64, (cuuint64_t)W.rows_pad / 32};
        const cuuint64_t strides[1] = {(cuuint64_t)W.chunks * 512};
        const cuuint32_t box[2] = {256, 4}, elem[2] = {1, 1};
        if (g_encode_tiled(&wmap, CU_TENSOR_MAP_DATA_TYPE_FLOAT64, 2, const_cast<int8_t*>(W.codes), dims, strides, box, elem,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return cudaErrorInvalidValue;
    }
    const int64_t k16 = W.chunks * 16;
    for (int64_t t = 0; t < m; t += full.tokens) {
        const int64_t part = m - t < full.tokens ? m - t : full.tokens;
        I8Plan p = i8_plan(W.rows, k, part);
        __half* wide = reinterpret_cast<__half*>(ws + full.wide);
        float* norms = reinterpret_cast<float*>(ws + full.norms);
        e = launch_ex(i8_widen_kernel, dim3((unsigned)part), dim3(256), 0, s, false,
                      reinterpret_cast<const uint4*>(a + t * k16), W.chunks, reinterpret_cast<uint4*>(wide), norms);
        if (e != cudaSuccess) return e;
        CUtensorMap map;
        const cuuint64_t dims[2] = {(cuuint64_t)k16, (cuuint64_t)part};
        const cuuint64_t strides[1] = {(cuuint64_t)k16 * sizeof(__half)};
        const cuuint32_t box[2] = {64, (cuuint32_t)p.bn};
        const cuuint32_t elem[2] = {1, 1};
        if (g_encode_tiled(&map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, wide, dims, strides, box, elem,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return cudaErrorInvalidValue;
        I8Gemm g{};
        g.W = W, g.anorm = norms, g.sa = sa + t, g.m = (int)part, g.bn = p.bn;
        g.token_tiles = p.token_tiles, g.tiles = p.tiles, g.kb = p.kb, g.stages = p.stages, g.buffers = p.buffers;
        g.y_stride = y_stride, g.slots = reinterpret_cast<int32_t*>(ws + full.slots);
        g.counters = reinterpret_cast<unsigned*>(ws), g.cut = p.cut, g.err = err;
        const int64_t units = p.tiles * p.kb;
        const int64_t ctas = p.cut ? (units < kI8Ctas ? units : kI8Ctas) : (p.tiles < kI8Ctas ? p.tiles : kI8Ctas);
        e = launch_ex(i8_gemm_kernel<T>, dim3((unsigned)ctas), dim3(kI8Threads), (size_t)kI8Smem + 1024, s, true, g, map, wmap,
                      y + t * y_stride);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

template cudaError_t launch_i8_gemm<float>(const I8Weights&, int64_t, const int8_t*, const float*, int64_t,
                                           float*, int64_t, void*, int32_t*, cudaStream_t);
template cudaError_t launch_i8_gemm<__half>(const I8Weights&, int64_t, const int8_t*, const float*, int64_t,
                                            __half*, int64_t, void*, int32_t*, cudaStream_t);
template cudaError_t launch_i8_gemm<__nv_bfloat16>(const I8Weights&, int64_t, const int8_t*, const float*,
                                                   int64_t, __nv_bfloat16*, int64_t, void*, int32_t*, cudaStream_t);

}  // namespace lq8
