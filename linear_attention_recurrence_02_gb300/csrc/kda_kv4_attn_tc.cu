// kda_kv4_attn_tc.cu -- softmax attention of many rows over the 4-bit cache (kda_kv4_attention, bf16):
// prompts, chunks of prompts, many query heads over one key/value head.
//
// Rows (new tokens times the query heads of a key/value head) come in blocks of two tiles of 128, over tiles
// of 128 cached tokens. Bound by the tensor cores together with what feeds them: per pair of tiles 4 products
// of 128 x 128 x D, 2 x 128 x 128 exponentials, and the expansion of 2 x 128 x D codes, which the two row
// tiles share. One CTA an SM, roles by warp group:
//
//   groups 0, 1  softmax of row tile 0, 1: a thread owns a row, reads its 128 scores from TMEM, writes the
//                factors back over them in two bf16 terms (the second product's A operand), rescales its row of
//                the output in TMEM in the rare case that the running maximum moves
//   group 2      codes from global memory through registers, expanded to bf16 (exact), into the 128-byte
//                swizzled tiles that the tensor cores read: keys K-major, values as they come (MN-major)
//   group 3      a warp issues S_i = Q_i K^T and O_i += P_i V for the two row tiles in turn: while one
//                tile's softmax runs, the tensor cores have the other's products. Where a block has one row
//                tile only, the two groups take its even and odd tiles of cached tokens and join their outputs
//
// TMEM: S_0, S_1 (128 columns each, P_i over S_i), O_0, O_1 (D columns each).
//
// A factor is two bf16 terms, off by 2^-16 at most: with one, its rounding (2^-8) costs an output as much as the output's
// own (0.0023 of its root mean square against 0.0017), and the same query over the same cache would be less exact here than
// in the kernel for few rows. The second term is half as many products again.
//
// 4096 queries of 32 heads over 8192 cached tokens of 8 heads of 128: 428 us (0.96 PFLOP/s; with one term 364). A pair of
// tiles takes about 4600 cycles, of which the tensor cores need 3200, and the products of Q and K read shared memory at
// its full rate. Measured with one term and not taken: half the codes to expand (as two CTAs would share them) 347 us;
// scores read from TMEM once, the maximum kept per 64 tokens, 369; 64 tokens' scores computed under the other 64's
// softmax 420, because a product that narrow reads more of shared memory than the tensor cores can wait for. fp16 factors and
// values in tiles whose scales fit fp16, two bf16 terms in the others: 426 us, and a row's last bits would then depend on
// tokens that it does not see.
#include <string>

#include "kda_kv4_attn.cuh"
#include "kda_prefill.cuh"
#include "kda_tc.cuh"

namespace kda {
namespace kv4 {
namespace many {

constexpr int R = 256, TILE = 128, NT = 512;
constexpr long long WAIT_LIMIT = 2000000000LL;  // clock cycles of a wait before it gives up (about 1 s)
constexpr long long TILE_LIMIT = 100000;        // and for every tile that it is behind (one takes some 2500)
constexpr float SLACK = 8.f;                    // log2 of how far scores may pass the reference maximum
// What starting and finishing an item costs, in tiles: a run of many short items has as much less to compute (8192 queries
// of a prompt, 32 over 8 heads: 489 us; counted as two tiles 546, as one 664).
constexpr int ITEM_COST = 3;
constexpr int SUMS = 4096;                      // sums of work kept while a CTA looks for its run

// A place in the line of tiles; items are (sequence, block of rows, key/value head).
struct Place {
    int64_t left;
    int64_t t0;
    int b, n, len, blocks;
    int block, h, t;      // of the item, and its next tile
    int first, tiles;     // the block's tiles: [first, first + tiles), at least one; ITEM_COST more in the line
};
// What a run has of an item.
struct Part {
    int64_t t0;
    int b, n, len, block, h, first, last, piece, rest;
    bool there;
};

constexpr int PITCH = 80;  // of a row's 64 bytes on their way out: an odd number of 16 bytes

template <int D> struct Smem {
    static constexpr int HALF = 128 * 128;             // 128 rows x 64 channels
    static constexpr int TILE_BYTES = 128 * D * 2;
    static constexpr int Q = 0, K = 2 * TILE_BYTES, V = K + 2 * TILE_BYTES, BAR = V + 2 * TILE_BYTES;
    static constexpr int OTHER = BAR + 256, PLACES = OTHER + 1024, PARTS = PLACES + 16 * 64, STAGE = PARTS + 16 * 128;
    static constexpr int BYTES = STAGE + 8 * 32 * PITCH + 1024;
};
static_assert(sizeof(Place) <= 64 && sizeof(Part) <= 64, "room for a place");

struct Bars {
    uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2], q_full[2], q_empty[2], s_full[2], p_half[2], p_full[2], pv_done[2], other_done,
        other_read;
    uint32_t taddr;
};

__device__ __forceinline__ void enter_block(const AttnArgs &a, Place &w) {
    block_tiles<R, TILE>(a, w.n, w.len, w.block, w.first, w.tiles);
    w.h = w.t = 0;
}
__device__ __forceinline__ void enter_sequence(const AttnArgs &a, Place &w) {
    const Seq s = seq_at<R, TILE>(a, w.b, false);
    w.t0 = s.t0;
    w.n = s.n;
    w.len = s.len;
    w.blocks = s.blocks;
    w.block = 0;
}

__device__ __forceinline__ void next_part(const AttnArgs &a, Place &w, Part &g) {
    g.there = false;
    for (;;) {
        if (w.left <= 0) return;
        if (w.h >= a.c.Hk) {
            ++w.block;
            while (w.block >= w.blocks) {
                if (++w.b >= a.c.B) return;
                enter_sequence(a, w);
            }
            enter_block(a, w);
        }
        const int from = w.t, take = (int)min((int64_t)(w.tiles + ITEM_COST - w.t), w.left), to = min(from + take, w.tiles);
        const int h = w.h;
        w.left -= take;
        w.t += take;
        if (w.t == w.tiles + ITEM_COST) {
            w.t = 0;
            ++w.h;
        }
        if (from >= w.tiles) continue;  // the item ended in the run before
        g.t0 = w.t0;
        g.b = w.b;
        g.n = w.n;
        g.len = w.len;
        g.block = w.block;
        g.h = h;
        g.piece = from > 0 ? 0 : to < w.tiles ? 1 : -1;
        g.rest = w.tiles - to;
        g.first = w.first + from;
        // a block that sees nothing has one tile in the line and none to compute
        const bool nothing = g.first * TILE >= w.len ||
                             (a.causal && w.len - w.n + a.by_group(min(w.n * a.group - 1, w.block * R + R - 1)) < 0);
        g.last = nothing ? g.first : w.first + to;
        g.there = true;
        return;
    }
}

// ---------------------------------------------------------------- issuing
// Four products along K by the warp's elected lane, all lanes calling: a branch around the issue instead makes
// every descriptor a per-lane value that has to be moved back to uniform registers (137 cycles a product, which
// then bounded the kernel). D (+)= A B^T with A and B K-major in shared memory (steps of 32 bytes).
__device__ __forceinline__ void mma4_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q, t;\n\t.reg .b64 a1, a2, a3, b1, b2, b3;\n\t"
        "setp.ne.u32 q, %4, 0;\n\tsetp.eq.u32 t, 0, 0;\n\t"
        "add.s64 a1, %1, 2;\n\tadd.s64 a2, %1, 4;\n\tadd.s64 a3, %1, 6;\n\t"
        "add.s64 b1, %2, 2;\n\tadd.s64 b2, %2, 4;\n\tadd.s64 b3, %2, 6;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "@p tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, q;\n\t"
        "@p tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, t;\n\t"
        "@p tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %3, t;\n\t"
        "@p tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %3, t;\n\t}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
// A in TMEM, for 64 tokens: the first terms of 32 in 16 columns, their second terms in the next 16; then the other 32
// tokens'. B MN-major in shared memory (2048 bytes a step of 16 tokens).
__device__ __forceinline__ void mma8_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q, t;\n\t.reg .b32 a1, a2, a3, a4, a5, a6, a7;\n\t.reg .b64 b1, b2, b3;\n\t"
        "setp.ne.u32 q, %4, 0;\n\tsetp.eq.u32 t, 0, 0;\n\t"
        "add.u32 a1, %1, 8;\n\tadd.u32 a2, %1, 16;\n\tadd.u32 a3, %1, 24;\n\t"
        "add.u32 a4, %1, 32;\n\tadd.u32 a5, %1, 40;\n\tadd.u32 a6, %1, 48;\n\tadd.u32 a7, %1, 56;\n\t"
        "add.s64 b1, %2, 128;\n\tadd.s64 b2, %2, 256;\n\tadd.s64 b3, %2, 384;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "@p tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, q;\n\t"
        "@p tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %3, t;\n\t"
        "@p tcgen05.mma.cta_group::1.kind::f16 [%0], [a2], %2, %3, t;\n\t"
        "@p tcgen05.mma.cta_group::1.kind::f16 [%0], [a3], b1, %3, t;\n\t"
        "@p tcgen05.mma.cta_group::1.kind::f16 [%0], [a4], b2, %3, t;\n\t"
        "@p tcgen05.mma.cta_group::1.kind::f16 [%0], [a5], b3, %3, t;\n\t"
        "@p tcgen05.mma.cta_group::1.kind::f16 [%0], [a6], b2, %3, t;\n\t"
        "@p tcgen05.mma.cta_group::1.kind::f16 [%0], [a7], b3, %3, t;\n\t}\n" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Arrives on `bar` when the elected lane's products so far are complete.
__device__ __forceinline__ void commit(uint64_t *bar) {
    asm volatile(
        "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\t"
        "@p tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}\n" ::"r"(tc::smem_u32(bar))
        : "memory");
}

// Waits for this thread's TMEM loads; what was loaded is not looked at before.
__device__ __forceinline__ void landed(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                   "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]),
                   "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]),
                   "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29])
                 :
                 : "memory");
    asm volatile("" : "+r"(r[30]), "+r"(r[31]));
}

// ---------------------------------------------------------------- expanding
// One block of 16 tokens in a warp's registers. Lane (q, b2, j) = (lane / 8, lane / 4 % 2, lane % 4) has rows
// q + 4 b2 and q + 4 b2 + 8 of the keys, words j of every group, and token pair (q & 1) + 4 (q >> 1) + 2 b2 of
// the values, words j: eight lanes then store rows that differ in bit 2, so that the swizzle spreads their 16
// bytes over all banks.
template <int D> struct Raw {
    static constexpr int G = D / 32;
    uint32_t k[2][G], ks[2][G / 2], v[2][G], vs[G];
};
template <int N> __device__ __forceinline__ void ldg(uint32_t (&w)[N], const uint8_t *p) {
    if constexpr (N == 4) {
        const uint4 v = *reinterpret_cast<const uint4 *>(p);
        w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
    } else if constexpr (N == 2) {
        const uint2 v = *reinterpret_cast<const uint2 *>(p);
        w[0] = v.x; w[1] = v.y;
    } else {
        w[0] = *reinterpret_cast<const uint32_t *>(p);
    }
}

template <int D>
__global__ void __launch_bounds__(NT, 1) kv4_attn_many_kernel(const __grid_constant__ AttnArgs a) {
    using namespace tc;
    using Sm = Smem<D>;
    using bf16 = __nv_bfloat16;
    constexpr int G = D / 32, FB = Format<D>::BYTES;
    constexpr uint32_t ID_S = idesc_bf16(128, 128, 0, 0), ID_O = idesc_bf16(128, D, 0, 1);
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    Bars *bar = reinterpret_cast<Bars *>(sm + Sm::BAR);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        mbar_init(&bar->other_done, 4);
        mbar_init(&bar->other_read, 4);
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar->k_full + i, 4);
            mbar_init(bar->v_full + i, 4);
            mbar_init(bar->q_full + i, 3);
            mbar_init(bar->q_empty + i, 1);
            mbar_init(bar->p_half + i, 4);
            mbar_init(bar->p_full + i, 4);
            mbar_init(bar->k_empty + i, 1);
            mbar_init(bar->v_empty + i, 1);
            mbar_init(bar->s_full + i, 1);
            mbar_init(bar->pv_done + i, 1);
        }
        fence_mbar_init();
    }
    if (warp == 12) {
        tmem_alloc(&bar->taddr, 512);
        tmem_relinquish();
    }
    dependent_launch();

    // ------------------------------------------------ this CTA's run
    int64_t *sums = reinterpret_cast<int64_t *>(sm + Sm::K);  // of `per` sequences each
    const int per = (a.c.B + SUMS - 1) / SUMS, entries = (a.c.B + per - 1) / per;
    for (int e = warp; e < entries; e += NT / 32) {
        int64_t s = 0;
        for (int b = e * per; b < min((e + 1) * per, a.c.B); ++b) s += sequence_tiles<R, TILE, ITEM_COST>(a, b, lane, blockIdx.x == 0);
        if (lane == 0) sums[e] = s;
    }
    if (threadIdx.x == 0) a.joint[blockIdx.x].pieces = 0;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = bar->taddr;
    int64_t total = 0;
    for (int e = lane; e < entries; e += 32) total += sums[e];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    const int64_t run = run_length(total, a.ctas, 1), start = blockIdx.x * run;
    const bool work = start < total;
    Place *place = reinterpret_cast<Place *>(sm + Sm::PLACES + 64 * warp);
    Part *part = reinterpret_cast<Part *>(sm + Sm::PARTS + 128 * warp);  // [2], 64 bytes apart
    if (work && warp == 0) {
        int64_t before = 0;
        int e = 0;
        for (;; e += 32) {  // the entry, 32 at a time
            const int64_t mine = e + lane < entries ? sums[e + lane] : 0;
            const int l = lane_past(mine, start, lane, before);
            if (l >= 0) {
                e += l;
                break;
            }
        }
        Place w;
        w.b = e * per;
        for (;; ++w.b) {  // the sequence
            const int64_t s = sequence_tiles<R, TILE, ITEM_COST>(a, w.b, lane, false);
            if (before + s > start) break;
            before += s;
        }
        enter_sequence(a, w);
        for (int k = 0;; k += 32) {  // the block of rows
            int first = 0, tiles = 0;
            if (k + lane < w.blocks) block_tiles<R, TILE>(a, w.n, w.len, k + lane, first, tiles);
            const int64_t mine = k + lane < w.blocks ? (int64_t)(tiles + ITEM_COST) * a.c.Hk : 0;
            const int l = lane_past(mine, start, lane, before);
            if (l >= 0) {
                w.block = k + l;
                break;
            }
        }
        enter_block(a, w);
        w.h = (int)div64(start - before, w.tiles + ITEM_COST);
        w.t = (int)(start - before - (int64_t)w.h * (w.tiles + ITEM_COST));
        w.left = min(run, total - start);
        if (lane == 0)
            for (int x = 0; x < NT / 32; ++x) *reinterpret_cast<Place *>(sm + Sm::PLACES + 64 * x) = w;
    }
    __syncthreads();

    bool ok = true;  // no wait of this warp has given up
    auto wait = [&](uint64_t *b, int parity) {  // all lanes
        if (ok && !__all_sync(0xffffffffu, mbar_wait_lean<0>(b, parity, WAIT_LIMIT))) ok = false;
    };
    auto wait_idly = [&](uint64_t *b, int parity, int tiles) {
        if (ok && !__all_sync(0xffffffffu, mbar_wait_lean<100>(b, parity, WAIT_LIMIT + TILE_LIMIT * tiles))) ok = false;
    };
    // All lanes: the run's next part, in the one of the warp's two places that the current part does not have. Parts
    // stay in shared memory: they are looked at once per item, and registers are short.
    int slot = 0;
    auto advance = [&]() {
        slot ^= 64;
        Part *g = reinterpret_cast<Part *>(reinterpret_cast<uint8_t *>(part) + slot);
        __syncwarp();
        if (lane == 0) next_part(a, *place, *g);
        __syncwarp();
        return const_cast<const Part *>(g);
    };

    if (warp < 8) {
        // ------------------------------------------------ softmax
        const int i = warp >> 2, row = (warp & 3) * 32 + lane;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t ts = tbase + lanes + 128 * i, to = tbase + lanes + 256 + D * i;
        int done = 0;    // tiles of this stream so far
        int joined = 0;  // items whose streams were joined so far
        const float slack = SLACK / a.scale_log2;
        const Part *at_hand = nullptr;
        if (work) at_hand = advance();
        while (at_hand && at_hand->there) {
            const Part &g = *at_hand;
            const Part *next = advance();
            const bool alone = g.n * a.group - g.block * R <= 128;  // one row tile: the streams share its cached tokens
            const int rr = g.block * R + (alone ? 0 : 128 * i) + row, ti = a.by_group(rr), pos = g.len - g.n + ti;
            const int hi = a.causal ? min(pos + 1, g.len) : g.len, lo = a.window > 0 ? pos - a.window + 1 : 0;
            const int i0 = a.by_group(g.block * R), i1 = a.by_group(min(g.n * a.group - 1, g.block * R + R - 1));
            const int whole_hi = a.causal ? min(g.len - g.n + i0 + 1, g.len) : g.len;
            const int whole_lo = a.window > 0 ? g.len - g.n + i1 - a.window + 1 : 0;
            const int first = g.first + (alone ? i : 0), step = alone ? 2 : 1;
            float neg = 0.f, top = -INFINITY, l = 0.f;
            for (int tile = first, last = g.last; tile < last; tile += step) {
                    wait(bar->s_full + i, done & 1);
                    tc_fence_after();
                    const int tok0 = tile * TILE;
                    if (tok0 + TILE > whole_hi || tok0 < whole_lo) {  // tokens that a row does not see
#pragma unroll 1
                        for (int c = 0; c < 4; ++c) {
                            uint32_t x[32];
                            tmem_ld32(ts + 32 * c, x);
                            landed(x);
                            const int t0 = tok0 + 32 * c;
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (t0 + e >= hi || t0 + e < lo) x[e] = 0xff800000u;  // -infinity
                            tmem_st32(ts + 32 * c, x);
                        }
                        tmem_st_wait();
                    }
                    float m = -INFINITY;
#pragma unroll 1
                    for (int c = 0; c < 2; ++c) {
                        uint32_t x[32], y[32];
                        tmem_ld32(ts + 64 * c, x);
                        tmem_ld32(ts + 64 * c + 32, y);
                        landed(x);
                        landed(y);
                        float m2 = -INFINITY;
#pragma unroll
                        for (int e = 0; e < 32; e += 2) {
                            m = fmaxf(m, fmaxf(__uint_as_float(x[e]), __uint_as_float(x[e + 1])));
                            m2 = fmaxf(m2, fmaxf(__uint_as_float(y[e]), __uint_as_float(y[e + 1])));
                        }
                        m = fmaxf(m, m2);
                    }
                    if (__any_sync(0xffffffffu, m > top)) {
                        float f = 1.f;
                        if (m > top - slack) {  // -infinity while there is no maximum
                            const float x = -m * a.scale_log2;
                            f = top == -INFINITY ? 0.f : exp2_fast(x - neg);
                            neg = x;
                            top = m + slack;
                        }
                        l *= f;
                        if (tile != first) {  // the output so far
                            wait(bar->pv_done + i, (done - 1) & 1);
                            tc_fence_after();
#pragma unroll 1
                            for (int c = 0; c < D / 32; ++c) {
                                uint32_t o[32];
                                tmem_ld32(to + 32 * c, o);
                                landed(o);
#pragma unroll
                                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                                tmem_st32(to + 32 * c, o);
                            }
                        }
                    }
                    // The factors, 32 at a time, in the columns of the scores that they come from: 16 columns of first terms, 16
                    // of second ones. The product starts on the first half of them. (64 at a time: 470 us instead of 442.)
                    float2 sum = make_float2(0.f, 0.f);
                    const float2 sc = make_float2(a.scale_log2, a.scale_log2), ng = make_float2(neg, neg);
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        uint32_t x[32], p[32];
                        tmem_ld32(ts + 32 * c, x);
                        landed(x);
                        float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            float2 u = __ffma2_rn(make_float2(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1])), sc, ng);
                            u.x = exp2_fast(u.x);
                            u.y = exp2_fast(u.y);
                            s2 = __fadd2_rn(s2, u);
                            uint32_t t[2];
                            split_bf16<2>(u, t);
                            p[e] = t[0];
                            p[16 + e] = t[1];
                        }
                        sum = __fadd2_rn(sum, s2);
                        tmem_st32(ts + 32 * c, p);
                        if (c % 2 == 0) continue;
                        tmem_st_wait();
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive((c == 1 ? bar->p_half : bar->p_full) + i);
                    }
                    l += sum.x + sum.y;
                    ++done;
                }
            if (l != l && top == -INFINITY) top = 0.f;  // scores that are all NaN leave no maximum
            float mx = top == -INFINITY ? -INFINITY : -neg;
            const bool any = first < g.last;
            if (any) {
                wait(bar->pv_done + i, (done - 1) & 1);
                tc_fence_after();
            }
            float2 *other = reinterpret_cast<float2 *>(sm + Sm::OTHER);
            if (alone && i == 1) {  // the first group joins both streams
                other[row] = make_float2(mx, l);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar->other_done);
                wait(&bar->other_read, joined++ & 1);
            } else {
                bool both = false;
                float f0 = 1.f, f1 = 0.f;
                if (alone) {
                    wait(&bar->other_done, joined++ & 1);
                    tc_fence_after();
                    both = g.first + 1 < g.last;
                    const float2 x = other[row];
                    const float m = fmaxf(mx, x.x);
                    f0 = mx == -INFINITY ? 0.f : exp2_fast(mx - m);
                    f1 = x.x == -INFINITY ? 0.f : exp2_fast(x.x - m);
                    l = l * f0 + x.y * f1;
                    mx = m;
                }
                const int64_t at = ((int64_t)blockIdx.x * 2 + g.piece) * R + (alone ? 0 : 128 * i) + row;
                const int head = g.h * a.group + rr - ti * a.group;
                const bool live = ti < g.n;
                const float inv = l == 0.f ? 0.f : 1.f / l;
                // Rows leave 64 bytes at a time through shared memory, four lanes a row: a store of a lane's own row
                // touches 32 lines (8192 queries of a prompt, 32 over 8 heads: 512 us so, 489 with this).
                const uint64_t mine = !live ? 0 : g.piece >= 0
                    ? (uint64_t)(a.part + at * D)
                    : (uint64_t)(static_cast<bf16 *>(a.out) + (g.t0 + ti) * a.out_stride + (int64_t)head * D);
                uint64_t dst[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) dst[k] = __shfl_sync(0xffffffffu, mine, 8 * k + (lane >> 2)) + 16 * (lane & 3);
                uint8_t *stage = sm + Sm::STAGE + warp * 32 * PITCH;
                auto put = [&](const uint32_t *w, int off) {  // a row's 64 bytes, `off` bytes from its start
                    __syncwarp();
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        *reinterpret_cast<uint4 *>(stage + lane * PITCH + 16 * k) = make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
                    __syncwarp();
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint4 v = *reinterpret_cast<const uint4 *>(stage + (8 * k + (lane >> 2)) * PITCH + 16 * (lane & 3));
                        if (dst[k] >= 64) *reinterpret_cast<uint4 *>(dst[k] + off) = v;
                    }
                };
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t o[32];
                    __syncwarp();
                    if (any) {
                        tmem_ld32(to + 32 * c, o);
                        landed(o);
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = 0;
                    }
                    if (both) {
                        uint32_t o1[32];
                        tmem_ld32(to + D + 32 * c, o1);
                        landed(o1);
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            o[e] = __float_as_uint(__uint_as_float(o[e]) * f0 + __uint_as_float(o1[e]) * f1);
                    }
                    if (g.piece >= 0) {
                        put(o, 128 * c);
                        put(o + 16, 128 * c + 64);
                    } else {
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            o[e] = pack_bf16(__uint_as_float(o[2 * e]) * inv, __uint_as_float(o[2 * e + 1]) * inv);
                        put(o, 64 * c);
                    }
                }
                __syncwarp();
                tc_fence_before();
                if (alone && lane == 0) mbar_arrive(&bar->other_read);
                if (live) {
                    if (g.piece >= 0) a.ml[at] = make_float2(mx, l);
                    else if (a.lse) a.lse[(g.t0 + ti) * a.Hq + head] = l == 0.f ? -INFINITY : (mx + log2f(l)) * 0.69314718f;
                }
                if (g.piece == 1 && i == 0 && row == 0)
                    a.joint[blockIdx.x] = Joint{g.t0, g.n, g.block, g.h, (int)div64(g.rest + run - 1, run) + 1};
            }
            at_hand = next;
        }
    } else if (warp < 12) {
        // ------------------------------------------------ expanding
        const Expand expand;
        const int w = warp - 8, q = lane >> 3, b2 = (lane >> 2) & 1, j = lane & 3;
        const int r0 = q + 4 * b2, pr = (q & 1) + 4 * (q >> 1) + 2 * b2;
        // the lane that has the values of the pair of rows r0 and r0 + 8 (pairs r0 / 2 and r0 / 2 + 4)
        const int pl = (((r0 >> 1) & 1) * 8) + ((r0 >> 2) & 1) * 4;
        int at = 0, last = 0, seq_len = 0, h = 0;  // the next tile, its item's last, its sequence and head
        const int32_t *row = a.c.table;
        bool there = work;
        auto settle = [&]() {
            while (there && at >= last) {
                const Part *g = advance();
                there = g->there;
                at = g->first;
                last = g->last;
                seq_len = g->len;
                h = g->h;
                row = a.c.table + g->b * a.c.table_stride;
            }
        };
        settle();
        // Blocks w and w + 4 of a tile. One behind the sequence's end, whose page need not exist, is read from the
        // tile's first page; a page outside the cache is read as page 0 and flagged. Three tiles are under way ahead of
        // the one that is expanded: one whose codes are on their way to registers, one on its way to L2, one whose
        // pages are looked up.
        bool bad = false;
        int page[2] = {0, 0};
        auto look = [&]() {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int t = at * TILE + 16 * (w + 4 * x);
                page[x] = row[(t < seq_len ? t : at * TILE) >> a.c.page_shift];
            }
        };
        struct Tile {
            const uint8_t *base[2];
            int tok, len;  // the first block's first token, the sequence's length
            bool there;
        };
        auto aim = [&]() {  // the tile whose pages were looked up; on to the one behind it
            Tile t;
            t.there = there;
            t.tok = at * TILE + 16 * w;
            t.len = seq_len;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const bool out = (uint32_t)page[x] >= (uint32_t)a.c.pages;
                bad |= out && there;
                const int block = ((t.tok + 64 * x) & ((1 << a.c.page_shift) - 1)) >> 4;
                t.base[x] = a.c.data + ((((int64_t)(out ? 0 : page[x]) * a.c.Hk + h) << (a.c.page_shift - 4)) + block) * FB;
            }
            if (there) {
                if (lane < 2) prefetch_l2_bulk(lane ? t.base[1] : t.base[0], FB);
                ++at;
                settle();
                if (there) look();
            }
            return t;
        };
        if (there) look();
        Tile load = aim(), next = aim();
        Raw<D> raw[2];
        auto load_keys = [&](int x) {
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                ldg<G>(raw[x].k[y], load.base[x] + (r0 + 8 * y) * (D / 2) + j * (D / 8));
                ldg<G / 2>(raw[x].ks[y], load.base[x] + Format<D>::KS + (r0 + 8 * y) * (D / 16));
            }
        };
        auto load_values = [&](int x) {
            const uint8_t *p = load.base[x] + Format<D>::V + pr * D + ((2 * j + 2 * pr) & 7) * (D / 8);
            ldg<G>(raw[x].v[0], p);
            ldg<G>(raw[x].v[1], p + D / 8);
            ldg<G>(raw[x].vs, load.base[x] + Format<D>::VS + pr * (D / 8));
        };
        if (load.there)
            for (int x = 0; x < 2; ++x) {
                load_keys(x);
                load_values(x);
            }
        for (int c = 0; load.there; ++c) {
            const int st = c & 1, ph = (c >> 1) & 1;
            const int tok_v = load.tok, len_v = load.len;
            wait(bar->k_empty + st, ph ^ 1);
            uint8_t *kt = sm + Sm::K + st * Sm::TILE_BYTES, *vt = sm + Sm::V + st * Sm::TILE_BYTES;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                // A value that is not finite would reach rows that do not see it (0 times NaN). Its scale is taken as
                // zero below, and the token's keys are NaN instead, for the rows that see it.
                uint32_t odd = 0, even = 0;
#pragma unroll
                for (int gr = 0; gr < G; ++gr) {
                    even |= not_finite16(raw[x].vs[gr]);
                    odd |= not_finite16(raw[x].vs[gr] >> 16);
                }
                const uint32_t be = __ballot_sync(0xffffffffu, even), bo = __ballot_sync(0xffffffffu, odd);
                const uint32_t of_row = (r0 & 1 ? bo : be) >> pl;
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const int t = 16 * (w + 4 * x) + r0 + 8 * y;
                    const bool nan = (of_row >> (16 * y)) & 1;
#pragma unroll
                    for (int gr = 0; gr < G; ++gr) {
                        uint32_t s2 = prmt(raw[x].ks[y][gr >> 1], 0, gr & 1 ? 0x3232 : 0x1010), f[4];
                        if (nan) s2 = 0x7fc07fc0u;
                        expand(raw[x].k[y][gr], swap_bytes(raw[x].k[y][gr]), s2, minus24(s2), f);
                        *reinterpret_cast<uint4 *>(kt + (gr >> 1) * Sm::HALF + t * 128 + ((((gr & 1) * 4 + j) ^ (t & 7)) << 4)) =
                            make_uint4(f[0], f[1], f[2], f[3]);
                    }
                }
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar->k_full + st);
            load = next;
            if (load.there) {
                load_keys(0);
                load_keys(1);
                next = aim();
            }
            wait(bar->v_empty + st, ph ^ 1);
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int t = 16 * (w + 4 * x) + 2 * pr + e;
                    const bool past = tok_v + 64 * x + 2 * pr + e >= len_v;
#pragma unroll
                    for (int gr = 0; gr < G; ++gr) {
                        uint32_t s2 = prmt(raw[x].vs[gr], 0, e ? 0x3232 : 0x1010), f[4];
                        if (past || not_finite16(s2)) s2 = 0;
                        const uint32_t lo = raw[x].v[0][e * (G / 2) + (gr >> 1)], hi = raw[x].v[1][e * (G / 2) + (gr >> 1)];
                        expand(prmt(lo, hi, gr & 1 ? 0x7632 : 0x5410), prmt(lo, hi, gr & 1 ? 0x6723 : 0x4501), s2, minus24(s2), f);
                        *reinterpret_cast<uint4 *>(vt + (gr >> 1) * Sm::HALF + t * 128 + ((((gr & 1) * 4 + j) ^ (t & 7)) << 4)) =
                            make_uint4(f[0], f[1], f[2], f[3]);
                    }
                }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar->v_full + st);
            if (load.there) {
                load_values(0);
                load_values(1);
            }
        }
        if (__any_sync(0xffffffffu, bad) && lane == 0) atomicOr(a.err, DEVERR_PAGES);
    } else {
        // ------------------------------------------------ issuing
        if (warp == 12 && work) {
            const uint32_t sbase = smem_u32(sm);
            int c = 0, nq[2] = {0, 0}, np[2] = {0, 0};  // tiles, row tiles loaded, factors taken
            const uint64_t q0 = sdesc_sw128(sbase + Sm::Q, 16, 1024), k0 = sdesc_sw128(sbase + Sm::K, 16, 1024),
                           v0 = sdesc_sw128(sbase + Sm::V, Sm::HALF, 1024);
            auto scores = [&](int i, int rows, int st) {  // of row tile `rows`
                if (!ok) return;
#pragma unroll
                for (int half = 0; half < D / 64; ++half)
                    mma4_ss(tbase + 128 * i, q0 + (rows * Sm::TILE_BYTES + half * Sm::HALF) / 16,
                            k0 + (st * Sm::TILE_BYTES + half * Sm::HALF) / 16, ID_S, half > 0);
                commit(bar->s_full + i);
            };
            auto outputs = [&](int i, int st, int half, bool more) {  // the first or second 64 tokens
                if (!ok) return;
                mma8_ts(tbase + 256 + D * i, tbase + 128 * i + 64 * half, v0 + st * (Sm::TILE_BYTES / 16) + 512 * half,
                        ID_O, more || half);
                if (half) commit(bar->pv_done + i);
            };
            auto release = [&](uint64_t *b) {
                if (ok) commit(b);
            };
            for (const Part *g = advance(), *after; g->there; g = after) {
                const int nt = g->last - g->first, rows = g->n * a.group - g->block * R;
                after = advance();
                if (nt <= 0) continue;
                if (rows <= 128) {
                    // One row tile: its even and odd tiles of cached tokens are two streams with an output each, so that
                    // here too one's products run while the other's factors are formed.
                    wait(bar->q_full, nq[0]++ & 1);
                    for (int n = 0; n < min(nt, 2); ++n) {
                        const int st = (c + n) & 1;
                        wait(bar->k_full + st, ((c + n) >> 1) & 1);
                        scores(n, 0, st);
                        release(bar->k_empty + st);
                    }
                    if (nt <= 2) release(bar->q_empty);
                    for (int n = 0; n < nt; ++n, ++c) {
                        const int st = c & 1, i = n & 1, turn = i ? np[1]++ : np[0]++;
                        wait(bar->v_full + st, (c >> 1) & 1);
                        wait(bar->p_half + i, turn & 1);
                        tc_fence_after();
                        outputs(i, st, 0, n > 1);
                        wait(bar->p_full + i, turn & 1);
                        tc_fence_after();
                        outputs(i, st, 1, true);
                        release(bar->v_empty + st);
                        if (n + 2 < nt) {
                            wait(bar->k_full + st, ((c + 2) >> 1) & 1);
                            scores(i, 0, st);
                            release(bar->k_empty + st);
                            if (n + 3 == nt) release(bar->q_empty);
                        }
                    }
                    continue;
                }
                wait(bar->k_full + (c & 1), (c >> 1) & 1);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    wait(bar->q_full + i, nq[i]++ & 1);
                    scores(i, i, c & 1);
                }
                release(bar->k_empty + (c & 1));
                if (nt == 1)
                    for (int i = 0; i < 2; ++i) release(bar->q_empty + i);
                for (int n = 0; n < nt; ++n, ++c) {
                    const int st = c & 1, s1 = (c + 1) & 1;
                    const bool next = n + 1 < nt;
                    wait(bar->v_full + st, (c >> 1) & 1);
                    if (next) wait(bar->k_full + s1, ((c + 1) >> 1) & 1);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        wait(bar->p_half + i, np[i] & 1);
                        tc_fence_after();
                        outputs(i, st, 0, n > 0);
                        wait(bar->p_full + i, np[i]++ & 1);
                        tc_fence_after();
                        outputs(i, st, 1, true);
                        if (next) scores(i, i, s1);
                        if (n + 2 == nt) release(bar->q_empty + i);
                    }
                    release(bar->v_empty + st);
                    if (next) release(bar->k_empty + s1);
                }
            }
            // the last releases arrive before shared memory goes away
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (nq[i] > 0) wait(bar->q_empty + i, (nq[i] - 1) & 1);
            for (int k = max(c - 2, 0); k < c; ++k) {
                wait(bar->k_empty + (k & 1), (k >> 1) & 1);
                wait(bar->v_empty + (k & 1), (k >> 1) & 1);
            }
        }
        if (warp > 12 && work) {
            // ------------------------------------------------ an item's rows of q, 16 bytes a lane
            const int c = lane & (D / 8 - 1);  // of a row's chunks
            int n[2] = {0, 0}, behind = 0;  // behind: tiles of the item whose rows are there
            for (const Part *g = advance(); g->there; g = advance()) {
                if (g->first >= g->last) continue;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int r0 = g->block * R + 128 * i, rows = g->n * a.group - r0;
                    if (rows <= 0) break;
                    wait_idly(bar->q_empty + i, (n[i]++ & 1) ^ 1, behind);
                    for (int row = (warp - 13) * (256 / D) + lane / (D / 8); row < 128; row += 3 * (256 / D)) {
                        const int ti = a.by_group(r0 + row);
                        const bool live = row < rows;
                        const bf16 *p = static_cast<const bf16 *>(a.q) +
                                        (live ? (g->t0 + ti) * a.q_stride + (int64_t)(g->h * a.group + r0 + row - ti * a.group) * D + 8 * c : 0);
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                                         smem_u32(sm + Sm::Q + i * Sm::TILE_BYTES) + (c >> 3) * Sm::HALF + row * 128 +
                                         (((c & 7) ^ (row & 7)) << 4)),
                                     "l"(p), "r"(live ? 16 : 0)
                                     : "memory");
                    }
                    asm volatile("cp.async.wait_all;" ::: "memory");
                    fence_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar->q_full + i);
                }
                behind = g->last - g->first;
            }
        }
    }
    if (!ok && lane == 0) atomicOr(a.err, DEVERR_TIMEOUT);  // said once, not at every wait: 439 -> 428 us
    tc_fence_before();
    __syncthreads();
    if (warp == 12) tmem_dealloc(tbase, 512);
}

}  // namespace many

template <int D> static kda_status run_many(AttnArgs a, cudaStream_t s) {
    using Sm = many::Smem<D>;
    constexpr auto kern = many::kv4_attn_many_kernel<D>;
    if (smem_attr_once<kern>(Sm::BYTES) != cudaSuccess) return check_launch("kv4_attn_many_kernel: shared memory");
    const int64_t blocks = a.c.T * a.group / many::R + a.c.B, tiles = ((int64_t)a.c.cols << a.c.page_shift) / many::TILE + 1;
    a.ctas = ctas_for(blocks, a.c.Hk, tiles, 1, a.sms);
    place_pieces(a, a.part, many::R, D);
    launch_dependent(kern, dim3(a.ctas), dim3(many::NT), Sm::BYTES, s, a);
    const kda_status st = check_launch("kv4_attn_many_kernel");
    if (st || a.ctas == 1) return st;
    return launch_join<D, __nv_bfloat16, many::R>(a, s);
}

kda_status attn_many(const AttnArgs &a, int D, cudaStream_t s) { return D == 128 ? run_many<128>(a, s) : run_many<64>(a, s); }

}  // namespace kv4
}  // namespace kda
