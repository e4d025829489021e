// kda_kv4_attn.cu -- softmax attention of a few rows over the 4-bit cache (kda_kv4_attention): decode
// steps, drafted tokens, and everything in fp32.
//
// Bound by memory: 9 D / 8 bytes of each cached token and key/value head, read once for all query heads
// that share it. The codes become bf16 pairs in registers, in the places where a matrix instruction wants
// them, so nothing expanded goes through shared memory. What has to be kept low is the instructions per
// code: two bf16 values take one mask-and-join, at most one shift and one fused product (kda_kv4.cuh).
//
//   S^T = K Q^T   16 cached tokens x 8 rows x 16 channels: the cache is the operand of 16 rows, so that
//                 one instruction takes 256 codes (the other way round it would take 128)
//   O^T = V^T P^T 16 channels x 8 rows x 16 tokens; P^T is S^T's accumulator turned by an 8 x 8 transpose
//
// tcgen05 takes its operands from shared memory or TMEM, where expanded codes would have to be written
// first: at the rate at which HBM delivers codes that alone is about all that shared memory can write.
//
// Each warp is on its own: it takes every fourth tile of 64 tokens of the CTA's run, brings its tiles in
// through a ring of two (by 16-byte asynchronous copies of all lanes: a bulk copy's issue by one lane, its
// barrier and the wait on it took as many issue slots as a third of the tile's arithmetic), and keeps a running
// maximum and sum (moved only when a score passes the maximum by 2^8: the factors stay in range and most
// tiles rescale nothing). At an item's end the four warps' results are joined through shared memory.
//
// 64 sequences of up to 8192 tokens, 96 over 8 heads of 128 in bf16: 152 us, 3.0 TB/s; one query head a
// cached one: 108 us. By then instructions bound it and their latencies, with eight warps an SM (255 registers each).
// While factors were one bf16 term, and it took 127 us, tiles of 32 tokens with three CTAs an SM took 136, with deeper rings
// 134 to 141, the tile's body as a loop over halves or quarters 136 or 139. One sequence of 4096 tokens takes 9 us, a single tile 6.
#include <algorithm>
#include <string>

#include "kda_fp8.cuh"
#include "kda_kv4_attn.cuh"
#include "kda_prefill.cuh"
#include "kda_tc.cuh"

namespace kda {
namespace kv4 {

constexpr int WARPS = 4, STAGES = 2, TILE = 64, BLOCKS = TILE / BLOCK;
constexpr int MOST_GROUP = 8;  // CTAs of a cluster
// Rows a key/value head up to which this kernel takes bf16 queries, in blocks of 16 that each go over the tokens once more;
// the kernel for many rows expands them once and works on 128 rows whatever it has. One token of 32 sequences of 8192, 8
// heads of 128, in us, this kernel and that one: 17 rows 184 and 203, 32 185 and 205, 48 270 and 206; heads of 64: 104 and
// 169, 105 and 170, 153 and 171; one key/value head: 37 and 41, 37 and 41, 47 and 41; 16 sequences of 1000: 28 and 32, 28
// and 32, 40 and 33. (Drafts of four tokens, which launch both: 20 rows 201 and 211, of heads of 64 116 and 176; one sequence 41
// and 36.)
constexpr int FEW_ROWS = 32;
constexpr float SLACK = 8.f;  // log2 of how far scores may pass the running maximum before it moves

// Where the run's computing (one for the CTA) and its copies (one a warp) stand. In shared memory, because
// they are needed once an item and would fill forty registers.
struct Places {
    Walk walk, ahead[WARPS];
    Segment seg[2], copied[WARPS];
};

template <int D, int NTL, int QS> struct FewSmem {
    static constexpr int R = 8 * NTL, STAGE = BLOCKS * Format<D>::BYTES;
    static constexpr int RING = WARPS * STAGES * STAGE;
    static constexpr int RAW = NTL * (D / 32) * 512 * (QS == 1 ? 1 : 2);  // an item's rows of q, [2] of them
    static constexpr int Q = RING, SPLIT = Q + 2 * RAW, ZERO = SPLIT + (QS == 1 ? 0 : NTL * (D / 32) * QS * 512);
    static constexpr int SUM = ZERO + NTL * (D / 32) * 64;
    static constexpr int ML = SUM + WARPS * 8 * 65 * 4;
    static constexpr int PLACES = ML + WARPS * R * 8, BYTES = PLACES + (int)sizeof(Places);
};

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// N words of shared memory.
template <int N> __device__ __forceinline__ void lds(uint32_t (&w)[N], const uint8_t *p) {
    if constexpr (N == 4) {
        const uint4 v = *reinterpret_cast<const uint4 *>(p);
        w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
    } else {
        const uint2 v = *reinterpret_cast<const uint2 *>(p);
        w[0] = v.x; w[1] = v.y;
    }
}

// A warp's copies: walks the CTA's run ahead of the computing, tile by tile. The pages of the next tile are
// looked up when the one before it is asked for, so that no copy waits for a lookup.
template <int D, int R> struct Loader {
    Walk *w;
    Segment *g;
    const int32_t *row;  // of the block table
    int tile, last, h, page;  // page: lane l's is that of block l of the tile
    bool more, bad;

    // All lanes: on to the run's next item that has a tile for this warp.
    __device__ __forceinline__ void next_item(const AttnArgs &a, int warp, int lane) {
        do {
            if (lane == 0) next_segment<R, TILE>(a, *w, *g);
            __syncwarp();
            more = g->there;
            row = a.c.table + g->b * a.c.table_stride;
            tile = g->first + warp;
            last = g->last;
            h = g->h;
            __syncwarp();
        } while (more && tile >= last);
        if (more) look(a, lane);
    }
    // Blocks behind the sequence's last token, whose page need not exist, are read from the tile's first page.
    __device__ __forceinline__ void look(const AttnArgs &a, int lane) {
        const int at = BLOCK * (lane & (BLOCKS - 1));
        page = row[(tile * TILE + (tile * TILE + at < g->len ? at : 0)) >> a.c.page_shift];
    }
    // Where a block of the page that stands for it begins; a page outside the cache is read as page 0 and flagged
    // at the end.
    __device__ __forceinline__ const uint8_t *block_at(const AttnArgs &a, int p, int block) {
        const bool out = (uint32_t)p >= (uint32_t)a.c.pages;
        bad |= out;
        return a.c.data + ((((int64_t)(out ? 0 : p) * a.c.Hk + h) << (a.c.page_shift - 4)) + block) * Format<D>::BYTES;
    }
    // The copies of the tile into `to` (a shared memory address), 16 bytes a lane at a time, and on to the next.
    __device__ __forceinline__ void issue(const AttnArgs &a, uint32_t to, int warp, int lane) {
        constexpr int BYTES = Format<D>::BYTES, CHUNKS = BYTES / 16;
        to += 16 * lane;
        const int in_page = (1 << (a.c.page_shift - 4)) - 1;
        if ((1 << a.c.page_shift) >= TILE) {  // one page
            const uint8_t *src = block_at(a, __shfl_sync(0xffffffffu, page, 0), BLOCKS * tile & in_page) + 16 * lane;
#pragma unroll
            for (int k = 0; k < (BLOCKS * CHUNKS + 31) / 32; ++k)
                if (BLOCKS * CHUNKS % 32 == 0 || 32 * k + lane < BLOCKS * CHUNKS)
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + 512 * k), "l"(src + 512 * k)
                                 : "memory");
        } else {
            for (int i = 0; i < BLOCKS; ++i) {
                const uint8_t *src = block_at(a, __shfl_sync(0xffffffffu, page, i), (BLOCKS * tile + i) & in_page) + 16 * lane;
#pragma unroll
                for (int k = 0; k < (CHUNKS + 31) / 32; ++k)
                    if (32 * k + lane < CHUNKS)
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + i * BYTES + 512 * k),
                                     "l"(src + 512 * k)
                                     : "memory");
            }
        }
        tile += WARPS;
        if (tile < last) look(a, lane);
        else next_item(a, warp, lane);
    }
};

// CTAs of an SM: as many as registers (without spills) and shared memory allow.
constexpr int few_per_sm(int D) { return D == 64 ? 3 : 2; }

__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The fp32 at shared memory address `at` of the cluster's CTA `rank`.
__device__ __forceinline__ float peer_float(uint32_t at, uint32_t rank) {
    float v;
    asm volatile("{\n\t.reg .u32 p;\n\tmapa.shared::cluster.u32 p, %1, %2;\n\tld.shared::cluster.f32 %0, [p];\n\t}"
                 : "=f"(v)
                 : "r"(at), "r"(rank)
                 : "memory");
    return v;
}

// GROUP: a cluster has one item, whose tiles its CTAs share and whose results they join through each other's shared
// memory. Else CTAs have runs of the line of tiles, and what they have of unfinished items goes to the workspace.
template <int D, typename T, int NTL, bool GROUP>
__global__ void __launch_bounds__(32 * WARPS, few_per_sm(D)) kv4_attn_few_kernel(const __grid_constant__ AttnArgs a) {
    constexpr int G = D / 32, QS = sizeof(T) == 4 ? 3 : 1, BYTES = Format<D>::BYTES;
    // Terms of bf16 that a factor is taken as. With bf16 queries one costs as much accuracy as the output's own rounding
    // (0.0023 against 0.0017 of the output's root mean square, up to half as much again where there are few heads); two
    // leave only the latter, whatever the form that a call's sizes choose. One sequence of 4096 tokens 9.2 -> 9.4 us; 64 x
    // 8192 tokens 128 -> 152 with 96 query heads over 8, 99 -> 108 with 8 over 8.
    constexpr int PT = QS > 1 ? 3 : 2;
    using Sm = FewSmem<D, NTL, QS>;
    constexpr int R = Sm::R;
    extern __shared__ __align__(128) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, j = lane & 3;
    const Expand expand;
    uint8_t *ring = smem + warp * STAGES * Sm::STAGE;
    float *sum = reinterpret_cast<float *>(smem + Sm::SUM);
    float2 *ml = reinterpret_cast<float2 *>(smem + Sm::ML);
    float4 *zero = reinterpret_cast<float4 *>(smem + Sm::ZERO);
    dependent_launch();

    Places *at = reinterpret_cast<Places *>(smem + Sm::PLACES);
    Walk w;
    int64_t run = 0;
    bool shared_out = false;  // GROUP: more than one CTA has tiles of the item
    if constexpr (GROUP) {
        const int size = cluster_size(), rank = cluster_rank();
        if (!item_at<R, TILE>(a, blockIdx.x / size, lane, blockIdx.x >= gridDim.x - size, w)) return;  // the whole cluster
        const int per = (w.s.tiles + size - 1) / size;
        w.t = min(rank * per, w.s.tiles);
        w.left = min(per, w.s.tiles - w.t);
        shared_out = per < w.s.tiles;
    } else {
        const int64_t total = line_tiles<R, TILE>(a, lane);
        run = run_length(total, a.ctas, WARPS);
        const int64_t start = blockIdx.x * run;
        if (threadIdx.x == 0) a.joint[blockIdx.x].pieces = 0;
        if (start >= total) return;  // the whole CTA
        w = walk_at<R, TILE>(a, start, lane);
        w.left = min(run, total - start);
    }
    if (lane == 0) {
        at->ahead[warp] = w;
        if (warp == 0) {
            at->walk = w;
            next_segment<R, TILE>(a, at->walk, at->seg[0]);
        }
    }
    __syncthreads();
    Loader<D, R> ld;
    ld.w = at->ahead + warp;
    ld.g = at->copied + warp;
    ld.bad = false;
    ld.next_item(a, warp, lane);
    const uint32_t ring_at = tc::smem_u32(ring);
    auto copy_next = [&](uint32_t dst) {  // one group a tile, an empty one behind the run's end
        if (ld.more) ld.issue(a, dst, warp, lane);
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    for (int i = 0; i < STAGES; ++i) copy_next(ring_at + i * Sm::STAGE);

    // An item's rows of q on their way: lane (r, j) has channels 32g + 8j + 0..7 of row r. Zeros for rows that the
    // last block does not have.
    auto copy_rows = [&](const Segment &g, uint8_t *dst) {
        for (int x = warp; x < NTL * G; x += WARPS) {
            const int nt = x / G, gr = x % G, rr = g.block * R + nt * 8 + r, i = a.by_group(rr);
            const bool live = i < g.n;
            const T *p = static_cast<const T *>(a.q) +
                         (live ? (g.t0 + i) * a.q_stride + (int64_t)(g.h * a.group + rr - i * a.group) * D + 8 * j + 32 * gr : 0);
#pragma unroll
            for (int k = 0; k < (QS == 1 ? 1 : 2); ++k)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                                 tc::smem_u32(dst + (x * (QS == 1 ? 1 : 2) + k) * 512 + lane * 16)),
                             "l"(p + 4 * k), "r"(live ? 16 : 0)
                             : "memory");
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };

    int stage = 0;
    bool idle = true;  // no tile of this warp's since its last copy of rows
    if (at->seg[0].there) copy_rows(at->seg[0], smem + Sm::Q);
    for (int turn = 0; at->seg[turn].there; turn ^= 1) {
        const Segment g = at->seg[turn];
        // The rows' copies have landed: behind them stands one tile's group at most where this warp had a tile
        // since, and none where it had not.
        if (idle) asm volatile("cp.async.wait_group 0;" ::: "memory");
        else asm volatile("cp.async.wait_group 1;" ::: "memory");
        idle = true;
        if (threadIdx.x == 0) {
            next_segment<R, TILE>(a, at->walk, at->seg[turn ^ 1]);
            if (!GROUP && g.piece == 1)
                a.joint[blockIdx.x] = Joint{g.t0, g.n, g.block, g.h, (int)div64(g.rest + run - 1, run) + 1};
        }
        if constexpr (QS > 1) {  // fp32: as three bf16 terms
            for (int x = warp; x < NTL * G; x += WARPS) {
                const float4 *p = reinterpret_cast<const float4 *>(smem + Sm::Q + turn * Sm::RAW) + x * 64 + lane;
                const float4 u = p[0], v = p[32];
                uint32_t f[4][QS];
                split_bf16<QS>(make_float2(u.x, u.y), f[0]);
                split_bf16<QS>(make_float2(u.z, u.w), f[1]);
                split_bf16<QS>(make_float2(v.x, v.y), f[2]);
                split_bf16<QS>(make_float2(v.z, v.w), f[3]);
#pragma unroll
                for (int k = 0; k < QS; ++k)
                    reinterpret_cast<uint4 *>(smem + Sm::SPLIT)[(x * QS + k) * 32 + lane] =
                        make_uint4(f[0][k], f[1][k], f[2][k], f[3][k]);
            }
        }
        const uint4 *qs = reinterpret_cast<const uint4 *>(smem + (QS == 1 ? Sm::Q + turn * Sm::RAW : Sm::SPLIT));
        int hi[NTL][2], lo[NTL][2];
#pragma unroll
        for (int nt = 0; nt < NTL; ++nt) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int pos = g.len - g.n + a.by_group(g.block * R + nt * 8 + 2 * j + e);
                hi[nt][e] = a.causal ? min(pos + 1, g.len) : g.len;
                lo[nt][e] = a.window > 0 ? pos - a.window + 1 : 0;
            }
        }
        // tiles between these two ends are seen whole by every row
        const int i0 = a.by_group(g.block * R), i1 = a.by_group(min(g.n * a.group - 1, g.block * R + R - 1));
        const int whole_hi = a.causal ? g.len - g.n + i0 + 1 : g.len;
        const int whole_lo = a.window > 0 ? g.len - g.n + i1 - a.window + 1 : 0;

        // of each column: its reference maximum (in log2 units, negated; 0 where there is none yet), the score that
        // moves it, and the sum of its factors
        float o[G][2][NTL][4], neg[NTL][2], bar[NTL][2], l[NTL][2];
        const float slack = SLACK / a.scale_log2;
#pragma unroll
        for (int nt = 0; nt < NTL; ++nt) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                neg[nt][e] = 0.f;
                bar[nt][e] = -INFINITY;
                l[nt][e] = 0.f;
            }
#pragma unroll
            for (int gr = 0; gr < G; ++gr)
#pragma unroll
                for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[gr][mt][nt][e] = 0.f;
        }

        __syncthreads();
        if constexpr (QS == 1) {
            // What a column's product with a group of codes starts from: -24 times the sum of its 32 channels, since
            // the codes come as 16 + c and stand for c - 8.
            for (int x = warp; x < NTL * G; x += WARPS) {
                const uint4 v = qs[x * 32 + lane];
                float z[4] = {0.f, 0.f, 0.f, 0.f};
                const uint32_t m24 = 0xC1C0C1C0u;
                mma16816(z, m24, m24, m24, m24, v.x, v.y);
                mma16816(z, m24, m24, m24, m24, v.z, v.w);
                if (r == 0) zero[x * 4 + j] = make_float4(z[0], z[1], z[0], z[1]);
            }
            __syncthreads();
        }
        if (at->seg[turn ^ 1].there) copy_rows(at->seg[turn ^ 1], smem + Sm::Q + (turn ^ 1) * Sm::RAW);
        for (int tile = g.first + warp; tile < g.last; tile += WARPS) {
            const uint8_t *buf = ring + stage * Sm::STAGE;
            asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 1) : "memory");
            __syncwarp();
            const int tok0 = tile * TILE;
            const bool edge = tok0 + TILE > min(whole_hi, g.len) || tok0 < whole_lo;
            float s[BLOCKS][NTL][4];
#pragma unroll
            for (int blk = 0; blk < BLOCKS; ++blk) {
                const uint8_t *kb = buf + blk * BYTES;
                uint32_t kw[2][G], ksc[2][(G + 1) / 2];
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    lds<G>(kw[x], kb + (r + 8 * x) * (D / 2) + j * (D / 8));
                    if constexpr (G == 4) {
                        lds<2>(ksc[x], kb + Format<D>::KS + (r + 8 * x) * 8);
                    } else {
                        ksc[x][0] = *reinterpret_cast<const uint32_t *>(kb + Format<D>::KS + (r + 8 * x) * 4);
                    }
                }
#pragma unroll
                for (int nt = 0; nt < NTL; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[blk][nt][e] = 0.f;
#pragma unroll
                for (int gr = 0; gr < G; ++gr) {
                    uint32_t f[2][4];
                    if constexpr (QS == 1) {
                        // bf16 queries: codes as they are, the group's scale on its scores. Sums of 32 products
                        // of eight and five bits lose nothing that matters against the factors' bf16.
                        float sc[2];
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            expand.codes16(kw[x][gr], swap_bytes(kw[x][gr]), f[x]);
                            sc[x] = __uint_as_float(gr & 1 ? ksc[x][gr >> 1] & 0xffff0000u : ksc[x][gr >> 1] << 16);
                        }
#pragma unroll
                        for (int nt = 0; nt < NTL; ++nt) {
                            const uint4 q = qs[(nt * G + gr) * 32 + lane];
                            const float4 c = zero[(nt * G + gr) * 4 + j];
                            float z[4] = {c.x, c.y, c.z, c.w};
                            mma16816(z, f[0][0], f[1][0], f[0][1], f[1][1], q.x, q.y);
                            mma16816(z, f[0][2], f[1][2], f[0][3], f[1][3], q.z, q.w);
#pragma unroll
                            for (int e = 0; e < 4; ++e) s[blk][nt][e] = fmaf(z[e], sc[e >> 1], s[blk][nt][e]);
                        }
                    } else {  // fp32 queries: the cached values themselves, with nothing to cancel. The matrix
                              // instruction cuts what does not fit its sum where an addition would round it; in a long
                              // chain that adds up, so a group's products start from zero and are added in fp32 (with
                              // the factors' products below: 26 x 5475 tokens 2.2e-6 off -> 0.3e-6; 141 -> 147 us)
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            const uint32_t s2 = prmt(ksc[x][gr >> 1], 0, gr & 1 ? 0x3232 : 0x1010);
                            expand(kw[x][gr], swap_bytes(kw[x][gr]), s2, minus24(s2), f[x]);
                        }
#pragma unroll
                        for (int nt = 0; nt < NTL; ++nt)
                        {
                            float t[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                            for (int z = QS - 1; z >= 0; --z) {
                                const uint4 q = qs[((nt * G + gr) * QS + z) * 32 + lane];
                                mma16816(t, f[0][0], f[1][0], f[0][1], f[1][1], q.x, q.y);
                                mma16816(t, f[0][2], f[1][2], f[0][3], f[1][3], q.z, q.w);
                            }
#pragma unroll
                            for (int e = 0; e < 4; ++e) s[blk][nt][e] += t[e];
                        }
                    }
                }
            }
            if (edge) {
#pragma unroll
                for (int blk = 0; blk < BLOCKS; ++blk)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const int tt = r + 8 * x, tok = tok0 + 16 * blk + tt;
                        // A value that is not finite would reach rows that do not see it (0 times NaN): its
                        // scale is taken as zero below, and the rows that see the token get their NaN here.
                        bool bad = false;
#pragma unroll
                        for (int gr = 0; gr < G; ++gr)
                            bad |= not_finite16(*reinterpret_cast<const uint16_t *>(buf + blk * BYTES +
                                                                                    value_scale_at<D>(tt, gr)));
#pragma unroll
                        for (int nt = 0; nt < NTL; ++nt)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                float &v = s[blk][nt][2 * x + e];
                                const bool see = tok < hi[nt][e] && tok >= lo[nt][e];
                                v = !see ? -INFINITY : bad ? __int_as_float(0x7fc00000) : v;
                            }
                    }
            }
            // The columns' reference maxima stay where no score of the tile passes one by 2^SLACK, which needs
            // no exchange between lanes; else they are brought up to date.
            bool move = false;
            float top[NTL][2];
#pragma unroll
            for (int nt = 0; nt < NTL; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    top[nt][e] = fmaxf(s[0][nt][e], s[0][nt][2 + e]);
#pragma unroll
                    for (int blk = 1; blk < BLOCKS; ++blk) top[nt][e] = fmaxf(top[nt][e], fmaxf(s[blk][nt][e], s[blk][nt][2 + e]));
                    move |= top[nt][e] > bar[nt][e];
                }
            if (__any_sync(0xffffffffu, move)) {
#pragma unroll
                for (int nt = 0; nt < NTL; ++nt) {
                    float f[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float m = top[nt][e];
                        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
                        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
                        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
                        f[e] = 1.f;
                        if (m > bar[nt][e] - slack) {  // -infinity while there is no maximum
                            const float n = -m * a.scale_log2;
                            f[e] = bar[nt][e] == -INFINITY ? 0.f : exp2_fast(n - neg[nt][e]);
                            neg[nt][e] = n;
                            bar[nt][e] = m + slack;
                        }
                        l[nt][e] *= f[e];
                    }
#pragma unroll
                    for (int gr = 0; gr < G; ++gr)
#pragma unroll
                        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                            for (int e = 0; e < 4; ++e) o[gr][mt][nt][e] *= f[e & 1];
                }
            }
            // factors, and their turn into the second product's operand
#pragma unroll
            for (int blk = 0; blk < BLOCKS; ++blk) {
                uint32_t p[NTL][2][PT];
#pragma unroll
                for (int nt = 0; nt < NTL; ++nt)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const float p0 = exp2_fast(fmaf(s[blk][nt][2 * x], a.scale_log2, neg[nt][0]));
                        const float p1 = exp2_fast(fmaf(s[blk][nt][2 * x + 1], a.scale_log2, neg[nt][1]));
                        l[nt][0] += p0;
                        l[nt][1] += p1;
                        uint32_t sp[PT];
                        split_bf16<PT>(make_float2(p0, p1), sp);
#pragma unroll
                        for (int z = 0; z < PT; ++z) p[nt][x][z] = transpose8x8(sp[z]);
                    }
                const uint8_t *vb = buf + blk * BYTES;
                uint32_t vw[2][G], vsc[2][G];  // pairs j and j + 4
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int pr = j + 4 * x;
                    lds<G>(vw[x], vb + Format<D>::V + pr * D + ((r + 2 * pr) & 7) * (D / 8));
                    lds<G>(vsc[x], vb + Format<D>::VS + pr * (D / 8));
                }
                if (edge) {
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const int tok = tok0 + 16 * blk + 2 * (j + 4 * x);
#pragma unroll
                        for (int gr = 0; gr < G; ++gr) {
                            if (tok >= g.len || not_finite16(vsc[x][gr])) vsc[x][gr] &= 0xffff0000u;
                            if (tok + 1 >= g.len || not_finite16(vsc[x][gr] >> 16)) vsc[x][gr] &= 0xffffu;
                        }
                    }
                }
#pragma unroll
                for (int gr = 0; gr < G; ++gr) {
                    uint32_t f[2][4];
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        // the two tokens' halves of this group side by side, and with their bytes exchanged
                        const uint32_t ev = vw[x][gr >> 1], od = vw[x][G / 2 + (gr >> 1)];
                        expand(prmt(ev, od, gr & 1 ? 0x7632 : 0x5410), prmt(ev, od, gr & 1 ? 0x6723 : 0x4501), vsc[x][gr],
                               minus24(vsc[x][gr]), f[x]);
                    }
                    if constexpr (QS == 1) {  // an accumulator's products apart from one another
#pragma unroll
                        for (int z = PT - 1; z >= 0; --z)
#pragma unroll
                            for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                                for (int nt = 0; nt < NTL; ++nt)
                                    mma16816(o[gr][mt][nt], f[0][2 * mt], f[0][2 * mt + 1], f[1][2 * mt], f[1][2 * mt + 1],
                                             p[nt][0][z], p[nt][1][z]);
                    } else {
#pragma unroll
                        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                            for (int nt = 0; nt < NTL; ++nt) {
                                float t[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                                for (int z = PT - 1; z >= 0; --z)
                                    mma16816(t, f[0][2 * mt], f[0][2 * mt + 1], f[1][2 * mt], f[1][2 * mt + 1], p[nt][0][z],
                                             p[nt][1][z]);
#pragma unroll
                                for (int e = 0; e < 4; ++e) o[gr][mt][nt][e] += t[e];
                            }
                    }
                }
            }
            __syncwarp();  // every lane has read the stage
            copy_next(ring_at + stage * Sm::STAGE);
            idle = false;
            if (++stage == STAGES) stage = 0;
        }

        // the four warps' results of the item, brought to one maximum
#pragma unroll
        for (int nt = 0; nt < NTL; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float x = l[nt][e];
                x += __shfl_xor_sync(0xffffffffu, x, 4);
                x += __shfl_xor_sync(0xffffffffu, x, 8);
                x += __shfl_xor_sync(0xffffffffu, x, 16);
                // no maximum: nothing seen, or scores that are all NaN
                if (r == 0)
                    ml[warp * R + nt * 8 + 2 * j + e] = make_float2(bar[nt][e] == -INFINITY && x == x ? -INFINITY : -neg[nt][e], x);
            }
        __syncthreads();
#pragma unroll
        for (int nt = 0; nt < NTL; ++nt) {
            float f[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float m = -INFINITY;
#pragma unroll
                for (int x = 0; x < WARPS; ++x) m = fmaxf(m, ml[x * R + nt * 8 + 2 * j + e].x);
                f[e] = m == -INFINITY ? 0.f : exp2_fast(-neg[nt][e] - m);
                if (ml[warp * R + nt * 8 + 2 * j + e].x == -INFINITY) f[e] = 0.f;
            }
#pragma unroll
            for (int c = 0; c < D / 64; ++c) {  // 64 channels at a time
#pragma unroll
                for (int gr = 0; gr < 2; ++gr)
#pragma unroll
                    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            sum[(warp * 8 + 2 * j + (e & 1)) * 65 + 32 * gr + 8 * (r >> 1) + (r & 1) + 4 * mt + 2 * (e >> 1)] =
                                o[2 * c + gr][mt][nt][e] * f[e & 1];
                __syncthreads();
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const int row = nt * 8 + 2 * warp + y, rr = g.block * R + row, i = a.by_group(rr);
                    float m = -INFINITY, total_l = 0.f, v0 = 0.f, v1 = 0.f;
#pragma unroll
                    for (int x = 0; x < WARPS; ++x) m = fmaxf(m, ml[x * R + row].x);
#pragma unroll
                    for (int x = 0; x < WARPS; ++x) {
                        if (ml[x * R + row].x != -INFINITY) total_l += ml[x * R + row].y * exp2_fast(ml[x * R + row].x - m);
                        v0 += sum[(x * 8 + 2 * warp + y) * 65 + 2 * lane];
                        v1 += sum[(x * 8 + 2 * warp + y) * 65 + 2 * lane + 1];
                    }
                    if (GROUP && g.piece >= 0) {  // the ring has nothing on its way any more
                        float *to = reinterpret_cast<float *>(smem) + row * D + 64 * c + 2 * lane;
                        to[0] = v0;
                        to[1] = v1;
                        if (lane == 0) reinterpret_cast<float2 *>(smem + R * D * 4)[row] = make_float2(m, total_l);
                    } else if (g.piece >= 0) {
                        const int64_t to = ((int64_t)blockIdx.x * 2 + g.piece) * R + row;
                        *reinterpret_cast<float2 *>(a.part + to * D + 64 * c + 2 * lane) = make_float2(v0, v1);
                        if (lane == 0) a.ml[to] = make_float2(m, total_l);
                    } else if (i < g.n) {
                        const float inv = total_l == 0.f ? 0.f : 1.f / total_l;
                        const int head = g.h * a.group + rr - i * a.group;
                        T *p = static_cast<T *>(a.out) + (g.t0 + i) * a.out_stride + (int64_t)head * D + 64 * c + 2 * lane;
                        if constexpr (QS == 1) *reinterpret_cast<uint32_t *>(p) = pack_bf16(v0 * inv, v1 * inv);
                        else *reinterpret_cast<float2 *>(p) = make_float2(v0 * inv, v1 * inv);
                        if (lane == 0 && a.lse)
                            a.lse[(g.t0 + i) * a.Hq + head] = total_l == 0.f ? -INFINITY : (m + log2f(total_l)) * 0.69314718f;
                    }
                }
                __syncthreads();
            }
        }
    }
    if (__any_sync(0xffffffffu, ld.bad) && lane == 0) atomicOr(a.err, DEVERR_PAGES);
    if constexpr (GROUP) {
        if (!shared_out) return;  // the whole cluster
        const int size = cluster_size(), rank = cluster_rank();
        float2 *mine = reinterpret_cast<float2 *>(smem + R * D * 4);
        if (!at->seg[0].there && threadIdx.x < R) mine[threadIdx.x] = make_float2(-INFINITY, 0.f);
        cluster_sync();
        const int h = w.item % a.c.Hk, block = w.item / a.c.Hk;
        // CTA `rank` has every size-th row from its own on, a warp 32 of a row's channels
        for (int x = warp; rank + size * (x / G) < R; x += WARPS) {
            const int row = rank + size * (x / G), ch = 32 * (x % G) + lane, rr = block * R + row, i = a.by_group(rr);
            if (i >= w.s.n) break;
            const uint32_t ml_at = tc::smem_u32(mine + row), v_at = tc::smem_u32(smem) + (row * D + ch) * 4;
            float pm[MOST_GROUP], m = -INFINITY, l = 0.f, v = 0.f;
#pragma unroll
            for (int p = 0; p < MOST_GROUP; ++p) {
                pm[p] = p < size ? peer_float(ml_at, p) : -INFINITY;
                m = fmaxf(m, pm[p]);
            }
#pragma unroll
            for (int p = 0; p < MOST_GROUP; ++p)
                if (pm[p] != -INFINITY) {
                    const float f = exp2_fast(pm[p] - m);
                    l = fmaf(peer_float(ml_at + 4, p), f, l);
                    v = fmaf(peer_float(v_at, p), f, v);
                }
            const int head = h * a.group + rr - i * a.group;
            Elem<T>::store(static_cast<T *>(a.out) + (w.s.t0 + i) * a.out_stride + (int64_t)head * D + ch, l == 0.f ? 0.f : v / l);
            if (ch == 0 && a.lse) a.lse[(w.s.t0 + i) * a.Hq + head] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718f;
        }
        cluster_sync();  // no CTA leaves while another still reads what it has
    }
}

// Up to eight rows of the item that goes on behind run blockIdx.x, a warp each; where the item has many pieces the
// eight warps share a row's after another. Either way in an order that the sizes alone decide. (A CTA a row: 4096 queries
// over 8192 tokens 406 us instead of 384, in blocks of 256 rows of which few have pieces.)
template <int D, typename T, int R>
__global__ void __launch_bounds__(256) kv4_attn_join_kernel(const __grid_constant__ AttnArgs a) {
    constexpr int V = D / 32, MANY = 12;
    __shared__ float sum[8][D], ls[8];
    dependent_launch();
    const Joint x = a.joint[blockIdx.x];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, row0 = 8 * blockIdx.y;
    const int rows = x.n * a.group - x.block * R - row0;  // from row0 on
    if (x.pieces == 0 || rows <= 0) return;
    // the first piece is its run's second, all others their run's first
    auto at = [&](int p, int row) { return ((int64_t)(blockIdx.x + p) * 2 + (p == 0)) * R + row; };
    auto pieces_of = [&](int row, int first, int step, float &m, float &l, float (&v)[V]) {
        m = -INFINITY;
        for (int p = lane; p < x.pieces; p += 32) m = fmaxf(m, a.ml[at(p, row)].x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        l = 0.f;
#pragma unroll
        for (int e = 0; e < V; ++e) v[e] = 0.f;
#pragma unroll 4
        for (int p = first; p < x.pieces; p += step) {
            const float2 y = a.ml[at(p, row)];
            const float f = y.x == -INFINITY ? 0.f : exp2_fast(y.x - m);
            l = fmaf(y.y, f, l);
            const float *from = a.part + at(p, row) * D + V * lane;
            float w[V];
            if constexpr (V == 4) {
                const float4 z = *reinterpret_cast<const float4 *>(from);
                w[0] = z.x; w[1] = z.y; w[2] = z.z; w[3] = z.w;
            } else {
                const float2 z = *reinterpret_cast<const float2 *>(from);
                w[0] = z.x; w[1] = z.y;
            }
#pragma unroll
            for (int e = 0; e < V; ++e) v[e] = fmaf(w[e], f, v[e]);
        }
    };
    auto put = [&](int row, float m, float l, const float (&v)[V]) {  // channels V lane ..
        const int rr = x.block * R + row, i = a.by_group(rr), head = x.h * a.group + rr - i * a.group;
        const int64_t t = x.t0 + i;
        T *to = static_cast<T *>(a.out) + t * a.out_stride + (int64_t)head * D + V * lane;
        const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
        for (int e = 0; e < V; ++e) Elem<T>::store(to + e, v[e] * inv);
        if (lane == 0 && a.lse) a.lse[t * a.Hq + head] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718f;
    };
    float m, l, v[V];
    if (x.pieces <= MANY) {
        if (warp >= rows || row0 + warp >= R) return;
        pieces_of(row0 + warp, 0, 1, m, l, v);
        put(row0 + warp, m, l, v);
        return;
    }
    for (int r = 0; r < min(min(rows, 8), R - row0); ++r) {
        pieces_of(row0 + r, warp, 8, m, l, v);
#pragma unroll
        for (int e = 0; e < V; ++e) sum[warp][V * lane + e] = v[e];
        if (lane == 0) ls[warp] = l;
        __syncthreads();
        if (warp == 0) {
            l = 0.f;
#pragma unroll
            for (int e = 0; e < V; ++e) v[e] = 0.f;
#pragma unroll
            for (int w = 0; w < 8; ++w) {
                l += ls[w];
#pragma unroll
                for (int e = 0; e < V; ++e) v[e] += sum[w][V * lane + e];
            }
            put(row0 + r, m, l, v);
        }
        __syncthreads();
    }
}

template <int D, typename T, int R> kda_status launch_join(const AttnArgs &a, cudaStream_t s) {
    launch_dependent(kv4_attn_join_kernel<D, T, R>, dim3(a.ctas - 1, (R + 7) / 8), dim3(256), 0, s, a);
    return check_launch("kv4_attn_join_kernel");
}

template kda_status launch_join<128, __nv_bfloat16, 256>(const AttnArgs &a, cudaStream_t s);
template kda_status launch_join<64, __nv_bfloat16, 256>(const AttnArgs &a, cudaStream_t s);

// Blocks of R rows and tiles of an item that these sizes allow, and the CTAs of a cluster where a cluster has one item
// (0: the CTAs have runs). One item a cluster, of as many CTAs as fit the card at once, saves the second kernel (5 us
// a call where launches follow one another) but leaves the SMs as unequal work as the lengths are: taken where even
// the longest item that the block table has room for gives a warp four tiles at most (8 us), and where the clusters come in
// three turns at most: each of them looks for its item among all sequences, so that many more take longer than runs do (8
// key/value heads of 128, 250 tokens a sequence, clusters and runs: 64 sequences 14.4 and 19.4 us, 96 21.2 and 25.0, 128
// 28.2 and 26.1, 256 53.8 and 48.6, 512 125 and 88; 900 tokens: 96 42.8 and 44.5, 192 80.7 and 74.3).
struct FewPlan {
    int64_t blocks, tiles;
    int group;
};
// few_rows: only sequences of at most FEW_ROWS rows are this kernel's (the others went to the one for many rows). A ragged
// batch is then three launches instead of four as a rule, and few empty clusters (3 prompts of up to 598 tokens, 84 over 7
// heads: 83 -> 70 us).
static FewPlan plan_few(const AttnArgs &a, int R, int cap, bool few_rows) {
    FewPlan p;
    p.blocks = a.c.cu ? a.c.T * a.group / R + a.c.B : (int64_t)a.c.B * ((a.group + R - 1) / R);
    if (few_rows) p.blocks = std::min(p.blocks, std::min<int64_t>(a.c.B, a.c.T) * ((FEW_ROWS + R - 1) / R));
    p.tiles = ((int64_t)a.c.cols << a.c.page_shift) / TILE + 1;
    if (a.window > 0) p.tiles = std::min(p.tiles, ((int64_t)a.window + (a.c.cu ? a.c.T : 1)) / TILE + 2);
    p.group = MOST_GROUP;
    while (p.group > 1 && (p.blocks * a.c.Hk * p.group > cap || p.group / 2 * WARPS >= p.tiles)) p.group /= 2;
    if (p.tiles > 4 * WARPS * p.group || p.blocks * a.c.Hk * p.group > 3 * (int64_t)cap) p.group = 0;
    return p;
}

template <int D, typename T, int NTL> static kda_status attn_few(AttnArgs a, cudaStream_t s) {
    using Sm = FewSmem<D, NTL, sizeof(T) == 4 ? 3 : 1>;
    const int cap = a.sms * few_per_sm(D);
    const FewPlan plan = plan_few(a, Sm::R, cap, a.most_rows <= FEW_ROWS);
    if (plan.group > 0) {
        constexpr auto kern = kv4_attn_few_kernel<D, T, NTL, true>;
        if (smem_attr_once<kern>(Sm::BYTES) != cudaSuccess) return check_launch("kv4_attn_few_kernel: shared memory");
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)(plan.blocks * a.c.Hk * plan.group));
        cfg.blockDim = dim3(32 * WARPS);
        cfg.dynamicSmemBytes = Sm::BYTES;
        cfg.stream = s;
        cudaLaunchAttribute at[2];
        at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        at[0].val.programmaticStreamSerializationAllowed = 1;
        at[1].id = cudaLaunchAttributeClusterDimension;
        at[1].val.clusterDim.x = (unsigned)plan.group;
        at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
        cfg.attrs = at;
        cfg.numAttrs = 2;
        cudaLaunchKernelEx(&cfg, kern, a);  // an error is left for check_launch
        return check_launch("kv4_attn_few_kernel");
    }
    constexpr auto kern = kv4_attn_few_kernel<D, T, NTL, false>;
    if (smem_attr_once<kern>(Sm::BYTES) != cudaSuccess) return check_launch("kv4_attn_few_kernel: shared memory");
    a.ctas = ctas_for(plan.blocks, a.c.Hk, plan.tiles, WARPS, cap);
    place_pieces(a, a.part, Sm::R, D);
    launch_dependent(kern, dim3(a.ctas), dim3(32 * WARPS), Sm::BYTES, s, a);
    kda_status st = check_launch("kv4_attn_few_kernel");
    if (st || a.ctas == 1) return st;
    return launch_join<D, T, Sm::R>(a, s);
}

}  // namespace kv4
}  // namespace kda

using namespace kda;

namespace kda {
namespace kv4 {
// The kernels of a call: which it takes, and the workspace that they need.
struct Route {
    bool many, few;  // many first
    int row_tiles;   // of 8 rows, of the kernel for few rows
    size_t bytes;
};
static int sms_here() {
    const int sms = current_sms();
    return sms > 0 ? sms : 152;
}
static Route route(const AttnArgs &a, int D, kda_dtype dtype) {
    Route r = {false, true, 1, 0};
    if (dtype == KDA_BF16) {
        // one new token each: the rows are known; else, with more tokens than sequences, each kernel takes the sequences
        // that suit it, and the second waits for the first, so that they share the workspace
        r.many = a.group > FEW_ROWS || (a.c.cu && a.c.T > a.c.B);
        r.few = a.group <= FEW_ROWS;
        r.row_tiles = !a.c.cu && a.group <= 8 ? 1 : 2;
    }
    const int cap = a.sms * few_per_sm(D);
    if (r.few && plan_few(a, 8 * r.row_tiles, cap, r.many).group == 0) r.bytes = pieces_bytes(cap, 8 * r.row_tiles, D);
    if (r.many) r.bytes = std::max(r.bytes, many_bytes(a.sms, D));
    return r;
}
}  // namespace kv4
}  // namespace kda

extern "C" size_t kda_kv4_attention_workspace_bytes(int B, int64_t T, int Hq, int Hk, int D, int page_size, int table_cols,
                                                    int with_cu_seqlens, int64_t window, kda_dtype dtype) {
    kv4::AttnArgs a = {};
    if (B < 1 || T < 1 || Hq < 1 || Hk < 1 || Hq % Hk || (D != 64 && D != 128) || (dtype != KDA_F32 && dtype != KDA_BF16) ||
        table_cols < 1 || page_size < 16 || page_size > 256 || (page_size & (page_size - 1)) || window < 0)
        return 0;
    static const int64_t some = 0;
    a.c.B = B;
    a.c.T = T;
    a.c.Hk = Hk;
    a.c.cols = table_cols;
    a.c.cu = with_cu_seqlens ? &some : nullptr;  // not looked at
    a.c.page_shift = 4;
    while ((1 << a.c.page_shift) < page_size) ++a.c.page_shift;
    a.group = Hq / Hk;
    a.window = window > 0x7fffff00LL ? 0 : (int)window;
    a.sms = kv4::sms_here();
    return kv4::route(a, D, dtype).bytes;
}

extern "C" kda_status kda_kv4_attention(const void *q, const void *cache, const int32_t *block_table,
                                        const int64_t *lens, const int64_t *cu_seqlens, void *out, float *lse, int B,
                                        int64_t T, int Hq, int Hk, int D, int page_size, int64_t pages, int table_cols,
                                        int64_t table_stride, int64_t q_stride, int64_t out_stride, float scale,
                                        int causal, int64_t window, kda_dtype dtype, void *workspace,
                                        size_t workspace_bytes, kda_stream_t stream) {
    clear_detail();
    kv4::AttnArgs a = {};
    kda_status st = kv4::check_cache(cache, block_table, lens, cu_seqlens, B, T, Hk, D, page_size, pages, table_cols,
                                     table_stride, dtype, a.c);
    if (st) return st;
    if (Hq < 1 || Hq % Hk) return invalid("Hq must be a positive multiple of Hk");
    if (T > 0x7fffff00LL / Hq) return invalid("T*Hq too large");
    if (!(scale >= 1e-30f) || scale > 1e30f) return invalid("scale must be in 1e-30 .. 1e30");
    if (causal != 0 && causal != 1) return invalid("causal must be 0 or 1");
    if (window < 0) return invalid("window must be >= 0");
    if (T == 0) return KDA_OK;
    if ((st = check_ptr(q, "q")) || (st = check_ptr(out, "out"))) return st;
    if (lse && (reinterpret_cast<uintptr_t>(lse) & 3)) return invalid("lse is not 4-byte aligned");
    const int64_t unit = dtype == KDA_BF16 ? 8 : 4;
    if (T > 1 && (q_stride < (int64_t)Hq * D || out_stride < (int64_t)Hq * D))
        return invalid("token strides must be at least Hq*D");
    if (T > 1 && (q_stride % unit || out_stride % unit)) return invalid("token strides must be multiples of 16 bytes");
    if (out == q || out == cache || out == lse || lse == q || lse == cache) return invalid("out and lse must not alias other arguments");
    a.q = q;
    a.out = out;
    a.lse = lse;
    a.q_stride = q_stride;
    a.out_stride = out_stride;
    a.Hq = Hq;
    a.group = Hq / Hk;
    a.by_group = kv4::Div(a.group);
    a.by_hk = kv4::Div(Hk);
    a.causal = causal;
    a.window = window > 0x7fffff00LL ? 0 : (int)window;
    a.scale_log2 = scale * 1.44269504f;
    a.most_rows = 0x7fffffff;
    a.least_rows = 0;
    // the pieces' room and the launches go by one device, the stream's, whichever was current
    if ((st = bind_stream_device(stream))) return st;
    a.sms = kv4::sms_here();
    const kv4::Route r = kv4::route(a, D, dtype);
    if (workspace_bytes < r.bytes) return invalid("workspace too small (kda_kv4_attention_workspace_bytes)");
    if (r.bytes && (st = check_ptr(workspace, "workspace"))) return st;
    a.part = static_cast<float *>(workspace);
    if (!(a.err = device_error_word())) return fail(KDA_ERR_CUDA, "device error word unavailable");
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (dtype == KDA_F32) return D == 128 ? kv4::attn_few<128, float, 1>(a, s) : kv4::attn_few<64, float, 1>(a, s);
    if (r.many) {
        if (r.few) a.least_rows = kv4::FEW_ROWS + 1;
        if ((st = kv4::attn_many(a, D, s)) || !r.few) return st;
        a.least_rows = 0;
        a.most_rows = kv4::FEW_ROWS;
    }
    if (r.row_tiles == 1)
        return D == 128 ? kv4::attn_few<128, __nv_bfloat16, 1>(a, s) : kv4::attn_few<64, __nv_bfloat16, 1>(a, s);
    return D == 128 ? kv4::attn_few<128, __nv_bfloat16, 2>(a, s) : kv4::attn_few<64, __nv_bfloat16, 2>(a, s);
}
