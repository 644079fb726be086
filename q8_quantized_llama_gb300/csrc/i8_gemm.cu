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
// i8_gemm_kernel: CTA tile 128 channels (M) x bn tokens (N, a multiple of 16 up to
// 256), one CTA per SM, persistent; a stage holds KS blocks of 64 codes of k (two up
// to 128 tokens, where the products are shorter than what surrounds them). More than
// 64 tokens are turned into f16 once per call by i8_widen_kernel, which also notes
// their norms; fewer (NARROW) are turned into f16 by every CTA for itself, which saves
// the launch before and the wait for it (48 tokens over 4096 x 14336: 5 of 24 us).
// Warp roles:
//  - two producers: the token tile (f16: 128-byte rows of 64 values, 128-byte swizzle,
//    the K-major B operand, used in place; NARROW: codes) and the codes of the four
//    32-row tiles, by tensor copies, each into a ring of its own: codes make room as soon
//    as they are converted, tokens when they are multiplied;
//  - two groups of 4 converter warps, taking stages in turn: row r's codes as f16 into
//    lane r of tensor memory (the A operand), one stage's columns next to the other's;
//    NARROW: 4 warps more for the tokens' codes;
//  - MMA warp: one thread issues four 128 x bn x 16 products per block;
//  - 8 accumulator warps read the finished sums (every second group of 16 columns
//    each), apply the scales and store: a warp's 32 lanes hold 32 neighbouring
//    channels of a token, 128 bytes of y.
//
// Work is dealt in whole tiles (tokens fastest, so that the CTAs that share a weight
// tile run together). The tiles that do not fill a wave are cut along k into parts,
// one per CTA, where that is shorter. Where all tiles are cut, the CTAs of a tile are a
// cluster: each leaves its sums (integers) in its shared memory and stores a share of the
// tile's tokens (512 tokens over 4096 x 14336 56 -> 49 us, 65 26 -> 20, against the other
// way). Behind whole tiles each leaves them in the workspace, and the one that brings a
// tile's last part adds the others to its own and stores.
#include "i8.cuh"
#include "kernels.cuh"
#include "llama_q8.h"
#include "paged.cuh"
#include "ptx.cuh"
#include "tc.cuh"

namespace lq8 {

constexpr int kI8BM = 128;
constexpr int kI8Ctas = 152;       // SMs of a GB300; the plan does not depend on the device at hand
constexpr int kI8AccWarps = 8;
// warps: accumulators, code converters, producers of tokens and of codes, MMA issuer, NARROW: token converters
constexpr int kI8ConvWarp0 = kI8AccWarps, kI8TokenWarp = kI8ConvWarp0 + 8, kI8CodeWarp = kI8TokenWarp + 1,
              kI8MmaWarp = kI8CodeWarp + 1, kI8WidenWarp0 = kI8MmaWarp + 1;
constexpr int i8_threads(bool narrow) { return (kI8WidenWarp0 + (narrow ? 4 : 0)) * 32; }
constexpr int kI8StagesMax = 8;
constexpr int kI8CodeBytes = kI8BM * 64;  // a block's codes
constexpr int kI8Smem = 224 * 1024;       // both rings
constexpr int kI8Exact = 16;              // blocks whose products cannot pass 2^24
constexpr int kI8Narrow = 64;             // tokens up to which every CTA makes its own f16 of them
constexpr int kI8ACols = 32;              // tensor-memory columns of a block's A
static_assert(256 * kI8BM * 4 <= kI8Smem, "a tile's sums fit in the rings' place");

struct I8Gemm {
    I8Weights W;
    const float* anorm;  // per token
    const float* sa;
    int m, bn, token_tiles, kb;
    int stages, code_stages, buffers;
    int64_t tiles, cut0;  // tiles from cut0 on are cut into `parts`, one for each of the first (tiles - cut0) parts CTAs
    int parts;
    bool cluster;  // every tile is cut, and a tile's CTAs are a cluster
    int64_t y_stride;
    int32_t* part;       // [CTA][bn][128]: the sums of its part
    int32_t* spare;      // [CTA][bn][128]: sums so far of a whole tile that is read out more than once
    unsigned* counters;  // per cut tile: parts that have arrived
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
// whether the phase is complete now
__device__ __forceinline__ bool i8_test(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ void i8_expect(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
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

// The segments of tiles that a CTA works on, the same for all its warps: its part of a cut tile, then whole tiles.
struct I8Segments {
    const I8Gemm& g;
    int64_t whole, tile;
    int k0, k1;
    bool cut;  // the segment to come or at hand is a part
    __device__ I8Segments(const I8Gemm& args) : g(args), whole(-1) {}
    __device__ bool next() {
        if (whole < 0) {
            whole = blockIdx.x;
            const int64_t at = g.cut0 + blockIdx.x / g.parts;
            cut = g.parts > 1 && at < g.tiles;
            if (cut) {
                const int64_t p = blockIdx.x % g.parts;
                tile = at, k0 = (int)(g.kb * p / g.parts), k1 = (int)(g.kb * (p + 1) / g.parts);
                return true;
            }
        }
        if (whole >= g.cut0) return false;
        cut = false, tile = whole, k0 = 0, k1 = g.kb;
        whole += gridDim.x;
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

// The products of stage s: 16 k each, 8 columns of A and 32 bytes of B's rows on.
template <int KS>
__device__ __forceinline__ void i8_stage(uint32_t d, uint32_t tmem_a, uint64_t desc0, int s, int tok_bytes, int token_bytes,
                                         uint32_t idesc, uint32_t accumulate, bool two) {
    const uint64_t b = desc0 + (uint32_t)(s * tok_bytes >> 4);
    const uint32_t a = tmem_a + (uint32_t)(s * KS * kI8ACols);
    mma_f16_ts(d, a, b, idesc, accumulate);
    mma_f16_ts(d, a + 8, b + 2, idesc, 1u);
    mma_f16_ts(d, a + 16, b + 4, idesc, 1u);
    mma_f16_ts(d, a + 24, b + 6, idesc, 1u);
    if (KS == 2 && two) {
        const uint64_t b1 = b + (uint32_t)(token_bytes >> 4);
        mma_f16_ts(d, a + 32, b1, idesc, 1u);
        mma_f16_ts(d, a + 40, b1 + 2, idesc, 1u);
        mma_f16_ts(d, a + 48, b1 + 4, idesc, 1u);
        mma_f16_ts(d, a + 56, b1 + 6, idesc, 1u);
    }
}

template <typename T, int KS, bool NARROW>
__global__ void __launch_bounds__(i8_threads(NARROW), 1)
    i8_gemm_kernel(const I8Gemm g, const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap wmap,
                   T* __restrict__ y) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ __align__(8) uint64_t tok_full[kI8StagesMax];    // token copies landed
    __shared__ __align__(8) uint64_t code_full[kI8StagesMax];   // code copies landed
    __shared__ __align__(8) uint64_t code_empty[kI8StagesMax];  // and read
    __shared__ __align__(8) uint64_t conv_bar[kI8StagesMax];    // A in tensor memory (NARROW: B in shared memory)
    __shared__ __align__(8) uint64_t done_bar[kI8StagesMax];    // products of the stage complete
    __shared__ __align__(8) uint64_t sum_full[2];               // a chunk's sums complete
    __shared__ __align__(8) uint64_t sum_empty[2];              // and read
    __shared__ uint32_t tmem_holder;
    __shared__ unsigned arrived;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // a stage's tokens: KS tiles, NARROW: then their codes; the code ring follows the token ring
    const int stages = g.stages, token_bytes = g.bn * 128, tok_bytes = (KS + (NARROW ? 1 : 0)) * token_bytes;
    constexpr int code_bytes = KS * kI8CodeBytes;
    if (tid == 0) {
        for (int s = 0; s < kI8StagesMax; ++s) {
            mbar_init(&tok_full[s], 1);
            mbar_init(&code_full[s], 1);
            mbar_init(&code_empty[s], 4);
            mbar_init(&conv_bar[s], NARROW ? 8 : 4);
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
    if (NARROW) {
        pdl_wait();
        pdl_launch_dependents();  // behind the allocation, too: a kernel that waits for this one cannot hold its columns
    }
    const uint32_t tmem = tmem_holder, tmem_a = tmem + (uint32_t)(g.buffers * g.bn);
    const uint32_t data = smem_u32(smem), code_data = data + stages * tok_bytes, tfull = smem_u32(tok_full),
                   cfull = smem_u32(code_full), cempty = smem_u32(code_empty), conv = smem_u32(conv_bar),
                   done = smem_u32(done_bar), sfull = smem_u32(sum_full), sempty = smem_u32(sum_empty);
    bool alive = true;  // cleared by a wait that ran out; the role then ends

    if (warp == kI8TokenWarp || warp == kI8CodeWarp) {
        // boxes are whole: codes past the last chunk or tile and tokens past the last arrive as zeros
        const bool codes = warp == kI8CodeWarp;
        const CUtensorMap* map = codes ? &wmap : &amap;
        const uint32_t to = codes ? code_data : data + (NARROW ? KS * token_bytes : 0), slot = codes ? code_bytes : tok_bytes;
        const uint32_t size = codes ? kI8CodeBytes : token_bytes, full = codes ? cfull : tfull, empty = codes ? cempty : done;
        const int step = codes ? 256 : 64;  // a block in the map's elements
        if (!NARROW && !codes) pdl_wait();  // the codes do not depend on the kernel before
        I8Segments seg(g);
        I8Ring ring(codes ? g.code_stages : stages);
        bool again = false;  // past the first pass over the ring
        while (alive && seg.next()) {
            const int row = codes ? seg.channel0() / 32 : seg.token0();
            for (int kb = seg.k0; kb < seg.k1; kb += KS) {
                const int s = ring.at;
                if (again) {
                    alive = __all_sync(0xffffffffu, i8_wait(empty + s * 8, ring.parity ^ 1u, g.err));
                    if (!alive) break;
                }
                if (i8_elect()) {
                    const uint32_t bar = full + s * 8, at = to + s * slot;
                    const bool two = KS == 2 && kb + 1 < seg.k1 && (codes || !NARROW);  // a box of token codes is a stage
                    i8_expect(bar, two ? 2 * size : size);
                    i8_box(at, map, kb * step, row, bar);
                    if (two) i8_box(at + size, map, (kb + 1) * step, row, bar);
                }
                ring.next();
                again |= ring.at == 0;
            }
        }
        // every copy has landed before the CTA may exit: the last of each slot
        if (!NARROW && codes) pdl_wait();
        for (int i = 0; i < ring.n; ++i) {
            if (i >= ring.at && !again) break;
            i8_wait(full + i * 8, i < ring.at ? ring.parity : ring.parity ^ 1u, g.err);
        }
        __syncwarp();
    } else if (warp == kI8MmaWarp) {
        if (!NARROW) pdl_wait();
        const uint32_t idesc = idesc_f16(kI8BM, (uint32_t)g.bn);
        const uint64_t desc0 = sw128_desc(data);
        I8Segments seg(g);
        I8Ring ring(stages), sums(g.buffers);
        bool again = false;  // past the first pass over the sum buffers
        bool ready = false;  // the next stages are known to be
        constexpr int U = KS == 1 ? 2 : 1;  // stages issued together: what is around the products takes half as long as they
        uint32_t last = 0, last_parity = 0;
        while (alive && seg.next()) {
            const int n = seg.k1 - seg.k0;
            const bool one = n <= kI8Exact || (!NARROW && i8_one_sum(g, seg.channel0(), seg.token0(), lane));
            for (int left = n; left > 0 && alive;) {
                int blocks = one ? left : min(left, kI8Exact);
                left -= blocks;
                if (again) alive = __all_sync(0xffffffffu, i8_wait(sempty + sums.at * 8, sums.parity ^ 1u, g.err));
                const uint32_t d = tmem + (uint32_t)(sums.at * g.bn);
                uint32_t accumulate = 0;
                for (; blocks > 0 && alive; blocks -= U * KS) {
                    const bool more = U == 2 && blocks > KS;  // a second stage
                    const int s0 = ring.at;
                    const uint32_t parity0 = ring.parity;
                    ring.next();
                    const int s1 = ring.at;
                    if (!ready) {
                        bool ok = i8_wait(conv + s0 * 8, parity0, g.err);
                        if (!NARROW) ok = i8_wait(tfull + s0 * 8, parity0, g.err) && ok;
                        if (more) {
                            ok = i8_wait(conv + s1 * 8, ring.parity, g.err) && ok;
                            if (!NARROW) ok = i8_wait(tfull + s1 * 8, ring.parity, g.err) && ok;
                        }
                        alive = __all_sync(0xffffffffu, ok);
                    }
                    if (!alive) break;
                    tc_fence_after();
                    if (i8_elect()) {
                        i8_stage<KS>(d, tmem_a, desc0, s0, tok_bytes, token_bytes, idesc, accumulate, blocks > 1);
                        i8_commit(done + s0 * 8);
                        if (more) {
                            i8_stage<KS>(d, tmem_a, desc0, s1, tok_bytes, token_bytes, idesc, 1u, true);
                            i8_commit(done + s1 * 8);
                        }
                        if (blocks <= U * KS) i8_commit(sfull + sums.at * 8);
                    }
                    accumulate = 1u;
                    last = done + (more ? s1 : s0) * 8, last_parity = more ? ring.parity : parity0;
                    if (more) ring.next();
                    // asked for while the products are on their way to the tensor cores
                    I8Ring then = ring;
                    ready = i8_test(conv + then.at * 8, then.parity);
                    if (!NARROW) ready &= i8_test(tfull + then.at * 8, then.parity);
                    if (U == 2) {
                        then.next();
                        ready &= i8_test(conv + then.at * 8, then.parity);
                        if (!NARROW) ready &= i8_test(tfull + then.at * 8, then.parity);
                    }
                    ready = __all_sync(0xffffffffu, ready);
                }
                sums.next();
                again |= sums.at == 0;
            }
        }
        // products in flight read shared memory and write tensor memory: the last is complete before the CTA exits
        if (last) i8_wait(last, last_parity, g.err);
        __syncwarp();
    } else if (NARROW && warp >= kI8WidenWarp0) {
        // the tokens' codes as f16: 16 codes are two 16-byte pieces of a token's row, each swizzled by the row
        I8Segments seg(g);
        I8Ring ring(stages);
        while (alive && seg.next())
            for (int n = seg.k1 - seg.k0; n > 0; n -= KS, ring.next()) {
                const int s = ring.at;
                alive = __all_sync(0xffffffffu, i8_wait(tfull + s * 8, ring.parity, g.err));
                if (!alive) break;
                const uint32_t to = data + s * tok_bytes, codes = to + KS * token_bytes;
                uint4 q[kI8Narrow / 16];  // all loads first
#pragma unroll
                for (int p = 0; p < kI8Narrow / 16; ++p) {
                    const int i = tid - kI8WidenWarp0 * 32 + p * 128;
                    if (i < g.bn * 8)
                        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                                     : "=r"(q[p].x), "=r"(q[p].y), "=r"(q[p].z), "=r"(q[p].w)
                                     : "r"(codes + i * 16));
                }
#pragma unroll
                for (int p = 0; p < kI8Narrow / 16; ++p) {
                    const int i = tid - kI8WidenWarp0 * 32 + p * 128, row = i >> 3, c = i & 7;
                    if (i >= g.bn * 8) break;
                    uint4 lo, hi;
                    codes_to_f16x2(q[p].x, lo.x, lo.y);
                    codes_to_f16x2(q[p].y, lo.z, lo.w);
                    codes_to_f16x2(q[p].z, hi.x, hi.y);
                    codes_to_f16x2(q[p].w, hi.z, hi.w);
                    const uint32_t at = to + (c >> 2) * token_bytes + row * 128, j = (uint32_t)((c & 3) * 2);
                    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at + ((j ^ (row & 7)) << 4)), "r"(lo.x),
                                 "r"(lo.y), "r"(lo.z), "r"(lo.w)
                                 : "memory");
                    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at + (((j + 1) ^ (row & 7)) << 4)),
                                 "r"(hi.x), "r"(hi.y), "r"(hi.z), "r"(hi.w)
                                 : "memory");
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the tensor cores read what was stored
                __syncwarp();
                if (lane == 0) i8_arrive(conv + s * 8);
            }
    } else if (warp >= kI8ConvWarp0) {
        // The groups take stages in turn. The code ring's slots are an even number, so that each is always read by the same
        // group and a wait never meets a barrier two phases behind (products complete in order, so those of the slot's
        // stage before the last are complete when a group waits for the last's).
        const int quarter = warp & 3, group = (warp - kI8ConvWarp0) >> 2;
        const uint32_t base = tmem_a + ((uint32_t)(quarter * 32) << 16);
        const uint32_t from = code_data + quarter * 2048 + lane * 16;
        I8Segments seg(g);
        I8Ring ring(stages), slots(g.code_stages);
        bool again = false, mine = group == 0;
        while (alive && seg.next())
            for (int n = seg.k1 - seg.k0; n > 0; n -= KS) {
                if (mine) {
                    const int s = ring.at, c = slots.at;
                    alive = __all_sync(0xffffffffu, i8_wait(cfull + c * 8, slots.parity, g.err));
                    if (!alive) break;
                    uint4 q[4 * KS];
#pragma unroll
                    for (int i = 0; i < 4 * KS; ++i)  // the second block may be missing: not used
                        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                                     : "=r"(q[i].x), "=r"(q[i].y), "=r"(q[i].z), "=r"(q[i].w)
                                     : "r"(from + c * code_bytes + (i >> 2) * kI8CodeBytes + (i & 3) * 512));
                    // the products that read the columns before
                    if (again) alive = __all_sync(0xffffffffu, i8_wait(done + s * 8, ring.parity ^ 1u, g.err));
                    if (!alive) break;
                    tc_fence_after();
#pragma unroll
                    for (int h = 0; h < 2 * KS; ++h) {
                        uint32_t u[16];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            codes_to_f16x2(q[2 * h + i].x, u[8 * i + 0], u[8 * i + 1]);
                            codes_to_f16x2(q[2 * h + i].y, u[8 * i + 2], u[8 * i + 3]);
                            codes_to_f16x2(q[2 * h + i].z, u[8 * i + 4], u[8 * i + 5]);
                            codes_to_f16x2(q[2 * h + i].w, u[8 * i + 6], u[8 * i + 7]);
                        }
                        tmem_st16(base + (uint32_t)(s * KS * kI8ACols + h * 16), u);
                    }
                    __syncwarp();
                    if (lane == 0) i8_arrive(cempty + c * 8);  // the codes are in registers, and converted
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) i8_arrive(conv + s * 8);
                }
                mine = !mine;
                ring.next();
                slots.next();
                again |= ring.at == 0;
            }
    } else {
        if (!NARROW) pdl_wait();
        const int quarter = warp & 3, half = warp >> 2, groups = g.bn / 16;
        const uint32_t base = tmem + ((uint32_t)(quarter * 32) << 16);
        const int64_t part = (int64_t)g.bn * kI8BM, off = quarter * 32 + lane;
        // a warp whose wait ran out still meets the others at their barriers
        I8Segments seg(g);
        I8Ring sums(g.buffers);
        while (seg.next()) {
            const int n = seg.k1 - seg.k0, channel0 = seg.channel0(), token0 = seg.token0();
            const bool one = n <= kI8Exact || (!NARROW && i8_one_sum(g, channel0, token0, lane));
            const int channel = channel0 + quarter * 32 + lane;
            const bool mine = channel < g.W.rows;
            const float sw = mine ? g.W.scale[channel] : 0.0f;
            // 16 tokens' exact sums, as integers or as f32
            auto store = [&](int gr, const auto* v) {
                const int t0 = token0 + gr * 16;
                T* at = y + (int64_t)t0 * g.y_stride + channel;
                float sa[16];  // before the stores, which the compiler takes for possible writes to them
#pragma unroll
                for (int j = 0; j < 16; ++j) sa[j] = t0 + j < g.m ? __ldca(g.sa + t0 + j) : 0.0f;
                if (t0 + 16 <= g.m) {
                    if (mine) {
#pragma unroll
                        for (int j = 0; j < 16; ++j, at += g.y_stride) *at = i8_scaled<T>(v[j], sa[j], sw);
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 16; ++j, at += g.y_stride)
                        if (mine && t0 + j < g.m) *at = i8_scaled<T>(v[j], sa[j], sw);
                }
            };
            const int chunks = one ? 1 : (n + kI8Exact - 1) / kI8Exact;
            // whether this CTA brings its cut tile's last part: the others' are in memory for it then
            int32_t* const parts = g.part + off;
            int32_t* const staged = reinterpret_cast<int32_t*>(smem) + off;  // the rings are done with when it is written
            const int first = (int)(blockIdx.x - blockIdx.x % g.parts);
            auto last_of_tile = [&] {
                unsigned* counter = &g.counters[blockIdx.x / g.parts];
                named_bar_sync(1, kI8AccWarps * 32);
                if (tid == 0) {
                    arrived = take_ticket(counter) + 1;
                    if (arrived == (unsigned)g.parts) *counter = 0u;
                }
                named_bar_sync(1, kI8AccWarps * 32);
                return arrived == (unsigned)g.parts && alive;
            };
            if constexpr (NARROW) {
                // up to 64 tokens: a warp's two groups of sums stay in registers
                int sum[2][16];
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int j = 0; j < 16; ++j) sum[h][j] = 0;
                for (int ch = 0; ch < chunks; ++ch, sums.next()) {
                    const int p = sums.at;
                    if (alive) alive = i8_wait(sfull + p * 8, sums.parity, g.err);
                    alive = __all_sync(0xffffffffu, alive);
                    if (!alive) break;
                    tc_fence_after();
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if (half + 2 * h >= groups) break;
                        float v[16];
                        tmem_ld16(base + (uint32_t)(p * g.bn + (half + 2 * h) * 16), v);
#pragma unroll
                        for (int j = 0; j < 16; ++j) sum[h][j] += __float2int_rn(v[j]);
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) i8_arrive(sempty + p * 8);
                }
                if (g.cluster) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if (half + 2 * h >= groups) break;
#pragma unroll
                        for (int j = 0; j < 16; ++j) staged[((half + 2 * h) * 16 + j) * kI8BM] = sum[h][j];
                    }
                    continue;
                }
                if (seg.cut) {
                    int32_t* mypart = parts + blockIdx.x * part;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if (half + 2 * h >= groups) break;
#pragma unroll
                        for (int j = 0; j < 16; ++j) mypart[((half + 2 * h) * 16 + j) * kI8BM] = sum[h][j];
                    }
                    if (!last_of_tile()) continue;
                    for (int c = first; c < first + g.parts; ++c) {
                        if (c == (int)blockIdx.x) continue;
                        const int32_t* other = parts + c * part;
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            if (half + 2 * h >= groups) break;
#pragma unroll
                            for (int j = 0; j < 16; ++j) sum[h][j] += __ldcg(other + ((half + 2 * h) * 16 + j) * kI8BM);
                        }
                    }
                }
                if (!alive) continue;
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    if (half + 2 * h < groups) store(half + 2 * h, sum[h]);
            } else {
                int32_t* sum = seg.cut && !g.cluster ? parts + blockIdx.x * part : g.spare + blockIdx.x * part + off;
                for (int ch = 0; ch < chunks; ++ch, sums.next()) {
                    const int p = sums.at;
                    if (alive) alive = i8_wait(sfull + p * 8, sums.parity, g.err);
                    alive = __all_sync(0xffffffffu, alive);
                    if (!alive) break;
                    tc_fence_after();
                    for (int gr = half; gr < groups; gr += 2) {
                        float v[16];
                        tmem_ld16(base + (uint32_t)(p * g.bn + gr * 16), v);
                        int32_t* at = sum + gr * 16 * kI8BM;
                        if (chunks == 1 && !seg.cut) {
                            store(gr, v);
                            continue;
                        }
                        int i[16];
#pragma unroll
                        for (int j = 0; j < 16; ++j) i[j] = __float2int_rn(v[j]) + (ch > 0 ? at[j * kI8BM] : 0);
                        if (ch == chunks - 1 && !seg.cut) {
                            store(gr, i);
                        } else {
                            if (ch == chunks - 1 && g.cluster) at = staged + gr * 16 * kI8BM;
#pragma unroll
                            for (int j = 0; j < 16; ++j) at[j * kI8BM] = i[j];
                        }
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) i8_arrive(sempty + p * 8);
                }
                if (!seg.cut || g.cluster || !last_of_tile()) continue;
                // two groups' sums are asked for together
                for (int gr = half; gr < groups; gr += 4) {
                    int i[2][16];
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int j = 0; j < 16; ++j) i[h][j] = 0;
                    for (int c = first; c < first + g.parts; ++c) {
                        const int32_t* from = parts + c * part;
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int at = gr + 2 * h < groups ? gr + 2 * h : gr;
#pragma unroll
                            for (int j = 0; j < 16; ++j) i[h][j] += __ldcg(from + (at * 16 + j) * kI8BM);
                        }
                    }
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        if (gr + 2 * h < groups) store(gr + 2 * h, i[h]);
                }
            }
        }
    }
    if (g.cluster) {
        // the tile's tokens are dealt over its CTAs and their warps
        __syncwarp();
        cluster_sync();
        const int64_t tile = blockIdx.x / g.parts;
        const int rank = blockIdx.x % g.parts, channel = (int)(tile / g.token_tiles) * kI8BM + lane;
        const int token0 = (int)(tile % g.token_tiles) * g.bn;
        float sw[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) sw[q] = channel + q * 32 < g.W.rows ? g.W.scale[channel + q * 32] : 0.0f;
        for (int t = rank + g.parts * warp; t < g.bn && token0 + t < g.m; t += g.parts * (int)(blockDim.x >> 5)) {
            int s[4] = {0, 0, 0, 0};
#pragma unroll 4
            for (int c = 0; c < g.parts; ++c) {
                uint32_t from;
                asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(from) : "r"(data + (t * kI8BM + lane) * 4), "r"(c));
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    int v;
                    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(from + q * 128) : "memory");
                    s[q] += v;
                }
            }
            const float sa = __ldca(g.sa + token0 + t);
            T* at = y + (int64_t)(token0 + t) * g.y_stride + channel;
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if (channel + q * 32 < g.W.rows) at[q * 32] = i8_scaled<T>(s[q], sa, sw[q]);
        }
        cluster_sync();  // nobody leaves while its sums are read
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kI8MmaWarp) tmem_dealloc(tmem, 512);
}

// The token rows as f16 and their norms, rounded up: one CTA per row, a thread per 16 codes as far as there are threads.
constexpr int kWidenThreads = 1024;
__global__ void __launch_bounds__(kWidenThreads) i8_widen_kernel(const uint4* __restrict__ codes, int64_t chunks,
                                                       uint4* __restrict__ wide, float* __restrict__ norm) {
    __shared__ uint32_t part[kWidenThreads / 32];
    pdl_launch_dependents();
    const int64_t row = blockIdx.x;
    int sum = 0;
    for (int64_t c = threadIdx.x; c < chunks; c += blockDim.x) {
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
        for (int w = 0; w < (int)blockDim.x / 32; ++w) all += part[w];  // at most 131056 * 2^14 < 2^31
        norm[row] = __fsqrt_ru(__uint2float_ru(all));
    }
}

// ---- the plan of a call, from its sizes alone ------------------------------------------
struct I8Plan {
    int64_t tokens;  // of one launch
    int bn, ks, token_tiles, kb, stages, code_stages, buffers, parts;
    bool narrow, cluster;
    int64_t tiles, cut0;
    size_t at_wide, at_norms, at_part, at_spare;  // byte offsets in the workspace
};

// tokens of one launch: 512 MB of f16, and enough of them to fill the GPU
constexpr int64_t kI8Wide = 512ll << 20, kI8MinTokens = 2048, kI8MaxTokens = 65536;
static int64_t i8_launch_tokens(int64_t k16, int64_t m) {
    const int64_t fit = kI8Wide / (2 * k16) / 256 * 256;
    const int64_t most = fit < kI8MinTokens ? kI8MinTokens : fit > kI8MaxTokens ? kI8MaxTokens : fit;
    return m < most ? m : most;
}
static size_t i8_up256(size_t x) { return (x + 255) / 256 * 256; }
// The workspace of any plan for up to m tokens: counters, a launch's tokens as f16 and their norms, a tile of sums per CTA
// for the parts and one for sums so far. It never falls as m or k grows (a launch's tokens may, as k grows: hence bounds
// in their place), so that one workspace serves many sizes.
size_t i8_gemm_workspace(int64_t k, int64_t m) {
    const int64_t k16 = (k + 15) / 16 * 16, tokens = m < kI8MaxTokens ? m : kI8MaxTokens;
    const int64_t bn = tokens < 32 ? 32 : tokens > 256 ? 256 : (tokens + 15) / 16 * 16;
    const size_t slots = (size_t)kI8Ctas * bn * kI8BM * 4;
    if (m <= kI8Narrow) return kCounterBytes + slots;
    const int64_t all = tokens * k16 * 2, most = kI8MinTokens * k16 * 2 > kI8Wide ? kI8MinTokens * k16 * 2 : kI8Wide;
    return i8_up256(kCounterBytes + (size_t)(all < most ? all : most)) + i8_up256((size_t)tokens * 4) + 2 * slots;
}

// Clusters of so many CTAs that a GB300 holds at once, a CTA taking an SM (what cudaOccupancyMaxActiveClusters reports).
constexpr int kI8Clusters[9] = {0, 152, 76, 46, 36, 28, 23, 15, 15};
static bool i8_clusters(int64_t tiles, int parts) { return parts > 1 && tiles <= kI8Clusters[parts]; }

// Microseconds of a launch with token tiles of bn and `parts` parts of each tile past the last full wave, from what was
// measured: a block takes 0.20 us with 32 tokens, 0.23 with 128 and 0.32 with 256, storing a tile 0.5 us and 1 / 100 us per
// token. Parts that meet in a cluster share the stores, all in all 2.25 us, 1 / 64 us per token and 0.45 us for each part
// after the second; through the workspace they take 2 us and another 1 us for every 64 tokens of each part after the first.
static double i8_cost(int64_t tiles, int kb, int bn, int parts) {
    const double block = bn <= 128 ? 0.19 + 0.0003 * bn : 0.24 + 0.00033 * bn, out = 0.5 + 0.01 * bn;
    const int64_t rest = tiles % kI8Ctas;
    double t = (double)(tiles / kI8Ctas) * (kb * block + out);
    if (rest) {
        t += (double)((kb + parts - 1) / parts) * block;
        t += i8_clusters(tiles, parts) ? 2.25 + bn / 64.0 + (parts - 2) * 0.45
                                       : out + (parts > 1 ? 2.0 + (parts - 1) * bn / 64.0 : 0.0);
    }
    return t;
}

static I8Plan i8_plan(int64_t rows, int64_t k, int64_t m) {
    I8Plan p{};
    const int64_t k16 = (k + 15) / 16 * 16;
    p.tokens = i8_launch_tokens(k16, m);
    p.kb = (int)((k16 + 63) / 64);
    p.narrow = p.tokens <= kI8Narrow;
    // token tiles from the fewest on, and parts
    const int64_t row_tiles = (rows + kI8BM - 1) / kI8BM;
    double best = 0.0;
    for (int64_t tt = (p.tokens + 255) / 256, tries = 0; tries < 8; ++tt, ++tries) {
        int bn = (int)(((p.tokens + tt - 1) / tt + 15) / 16 * 16);
        if (bn < 32) bn = 32;
        const int64_t tiles = row_tiles * tt, rest = tiles % kI8Ctas;
        for (int parts = 1; parts == 1 || (rest && parts * rest <= kI8Ctas && parts <= 8 && p.kb >= 4 * parts); ++parts) {
            const double t = i8_cost(tiles, p.kb, bn, parts);
            if (p.bn == 0 || t < best)
                best = t, p.bn = bn, p.token_tiles = (int)tt, p.tiles = tiles, p.parts = parts,
                p.cut0 = parts > 1 ? tiles - rest : tiles;
        }
        if (bn == 32) break;
    }
    p.cluster = i8_clusters(p.tiles, p.parts);
    p.ks = p.bn <= 128 ? 2 : 1;
    // the token ring: as many stages as tensor memory has columns for their A beside the sums (two buffers of them where
    // four stages still fit); the code ring: the rest, an even number of stages, four at least
    const int cols = p.ks * kI8ACols, token = (p.ks + (p.narrow ? 1 : 0)) * p.bn * 128, code = p.ks * kI8CodeBytes;
    p.buffers = (512 - 2 * p.bn) / cols >= 4 ? 2 : 1;
    p.stages = (512 - p.buffers * p.bn) / cols;
    p.stages = p.stages < kI8StagesMax ? p.stages : kI8StagesMax;
    while (p.stages * token + 4 * code > kI8Smem) --p.stages;
    p.code_stages = (kI8Smem - p.stages * token) / code / 2 * 2;
    p.code_stages = p.code_stages < kI8StagesMax ? p.code_stages : kI8StagesMax;
    p.at_wide = kCounterBytes;
    p.at_norms = i8_up256(p.at_wide + (p.narrow ? 0 : (size_t)p.tokens * k16 * 2));
    p.at_part = i8_up256(p.at_norms + (p.narrow ? 0 : (size_t)p.tokens * 4));
    p.at_spare = p.at_part + (p.parts > 1 ? (size_t)(p.tiles - p.cut0) * p.parts * p.bn * kI8BM * 4 : 0);
    return p;
}

template <typename T> static cudaError_t i8_gemm_attributes() {
    cudaError_t e = cudaSuccess;
    for (auto kernel : {i8_gemm_kernel<T, 1, false>, i8_gemm_kernel<T, 2, false>, i8_gemm_kernel<T, 2, true>})
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kI8Smem + 1024);
    return e;
}
cudaError_t init_i8_gemm_attributes() {
    cudaError_t e = i8_gemm_attributes<float>();
    if (e == cudaSuccess) e = i8_gemm_attributes<__half>();
    if (e == cudaSuccess) e = i8_gemm_attributes<__nv_bfloat16>();
    return e;
}

// A tensor map of rows of 8-byte words, f16 numbers or bytes: boxes of box_x x box_y.
static bool i8_map(CUtensorMap* map, CUtensorMapDataType type, const void* base, int64_t width, int64_t rows,
                   int64_t row_bytes, int box_x, int box_y, CUtensorMapSwizzle swizzle) {
    const cuuint64_t dims[2] = {(cuuint64_t)width, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)row_bytes};
    const cuuint32_t box[2] = {(cuuint32_t)box_x, (cuuint32_t)box_y}, elem[2] = {1, 1};
    return g_encode_tiled(map, type, 2, const_cast<void*>(base), dims, strides, box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// One launch: tokens a[m] by the plan.
template <typename T>
static cudaError_t i8_gemm_part(const I8Plan& p, const I8Weights& W, const int8_t* a, const float* sa, int m, T* y,
                                int64_t y_stride, uint8_t* ws, int32_t* err, cudaStream_t s) {
    __half* wide = reinterpret_cast<__half*>(ws + p.at_wide);
    float* norms = reinterpret_cast<float*>(ws + p.at_norms);
    const int64_t k16 = W.chunks * 16;
    // the packed codes: a row per 32-row tile, boxes of 4 tiles x 64 k (2 KB of a row)
    CUtensorMap wmap, amap;
    const bool mapped =
        i8_map(&wmap, CU_TENSOR_MAP_DATA_TYPE_FLOAT64, W.codes, W.chunks * 64, W.rows_pad / 32, W.chunks * 512, 256, 4,
               CU_TENSOR_MAP_SWIZZLE_NONE) &&
        (p.narrow ? i8_map(&amap, CU_TENSOR_MAP_DATA_TYPE_UINT8, a, k16, m, k16, 128, p.bn, CU_TENSOR_MAP_SWIZZLE_NONE)
                  : i8_map(&amap, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, wide, k16, m, k16 * 2, 64, p.bn, CU_TENSOR_MAP_SWIZZLE_128B));
    if (!mapped) return cudaErrorInvalidValue;
    if (!p.narrow) {
        const int64_t threads = W.chunks < kWidenThreads ? (W.chunks + 31) / 32 * 32 : kWidenThreads;
        const cudaError_t e = launch_ex(i8_widen_kernel, dim3((unsigned)m), dim3((unsigned)threads), 0, s, false,
                                        reinterpret_cast<const uint4*>(a), W.chunks, reinterpret_cast<uint4*>(wide), norms);
        if (e != cudaSuccess) return e;
    }
    I8Gemm g{};
    g.W = W, g.anorm = norms, g.sa = sa, g.m = m, g.bn = p.bn, g.token_tiles = p.token_tiles, g.kb = p.kb;
    g.stages = p.stages, g.code_stages = p.code_stages, g.buffers = p.buffers, g.tiles = p.tiles, g.cut0 = p.cut0;
    g.parts = p.parts, g.cluster = p.cluster, g.y_stride = y_stride, g.part = reinterpret_cast<int32_t*>(ws + p.at_part);
    g.spare = reinterpret_cast<int32_t*>(ws + p.at_spare), g.counters = reinterpret_cast<unsigned*>(ws), g.err = err;
    const int64_t cutters = p.parts > 1 ? (p.tiles - p.cut0) * p.parts : 0;
    const int64_t ctas = p.cut0 >= kI8Ctas ? kI8Ctas : p.cut0 > cutters ? p.cut0 : cutters;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(i8_threads(p.narrow));
    cfg.dynamicSmemBytes = (size_t)kI8Smem + 1024;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    cfg.attrs = attr;
    attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[cfg.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
    if (p.cluster) {
        attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
        attr[cfg.numAttrs].val.clusterDim.x = (unsigned)p.parts;
        attr[cfg.numAttrs].val.clusterDim.y = attr[cfg.numAttrs].val.clusterDim.z = 1;
        ++cfg.numAttrs;
    }
    return cudaLaunchKernelEx(&cfg, p.narrow ? i8_gemm_kernel<T, 2, true> : p.ks == 2 ? i8_gemm_kernel<T, 2, false> : i8_gemm_kernel<T, 1, false>,
                              g, amap, wmap, y);
}

template <typename T>
llama_q8_status launch_i8_gemm(const I8Weights& W, int64_t k, const int8_t* a, const float* sa, int64_t m, T* y,
                               int64_t y_stride, void* workspace, size_t workspace_bytes, int32_t* err, cudaStream_t s) {
    const I8Plan first = i8_plan(W.rows, k, m);
    if (!workspace || workspace_bytes < i8_gemm_workspace(k, m)) return LQ8_ERR_ARG;
    if (ensure_kernel_attributes() != cudaSuccess || get_encode_tiled() != cudaSuccess) return LQ8_ERR_CUDA;
    for (int64_t t = 0; t < m; t += first.tokens) {
        const int64_t part = m - t < first.tokens ? m - t : first.tokens;
        const cudaError_t e = i8_gemm_part(part == first.tokens ? first : i8_plan(W.rows, k, part), W, a + t * W.chunks * 16,
                                           sa + t, (int)part, y + t * y_stride, y_stride,
                                           reinterpret_cast<uint8_t*>(workspace), err, s);
        if (e != cudaSuccess) return LQ8_ERR_CUDA;
    }
    return LQ8_OK;
}

template llama_q8_status launch_i8_gemm<float>(const I8Weights&, int64_t, const int8_t*, const float*, int64_t,
                                           float*, int64_t, void*, size_t, int32_t*, cudaStream_t);
template llama_q8_status launch_i8_gemm<__half>(const I8Weights&, int64_t, const int8_t*, const float*, int64_t,
                                            __half*, int64_t, void*, size_t, int32_t*, cudaStream_t);
template llama_q8_status launch_i8_gemm<__nv_bfloat16>(const I8Weights&, int64_t, const int8_t*, const float*,
                                                   int64_t, __nv_bfloat16*, int64_t, void*, size_t, int32_t*, cudaStream_t);

}  // namespace lq8
