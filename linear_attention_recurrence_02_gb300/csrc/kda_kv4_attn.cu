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
// Each warp is on its own: it takes every fourth tile of 32 tokens of the CTA's run, brings its tiles in
// by bulk copies through a ring of three, and keeps a running maximum and sum (moved only when a score passes the
// maximum by 2^8: the factors stay in range and most tiles rescale nothing). At an item's end the four
// warps' results are joined through shared memory.
#include <algorithm>
#include <string>

#include "kda_fp8.cuh"
#include "kda_kv4_attn.cuh"
#include "kda_prefill.cuh"
#include "kda_tc.cuh"

namespace kda {
namespace kv4 {

constexpr int WARPS = 4, STAGES = 3, TILE = 32;
constexpr long long WAIT_LIMIT_KV4 = 2000000000LL;  // clock cycles (about 1 s)
constexpr float SLACK = 8.f;  // log2 of how far scores may pass the running maximum before it moves

template <int D, int NTL> struct FewSmem {
    static constexpr int R = 8 * NTL, STAGE = 2 * Format<D>::BYTES;
    static constexpr int RING = WARPS * STAGES * STAGE;
    static constexpr int SUM = RING, ML = SUM + WARPS * 8 * (D + 1) * 4, BAR = ML + WARPS * R * 8;
    static constexpr int BYTES = BAR + WARPS * STAGES * 8;
};

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// x as a sum of bf16 numbers, as many as QS: one rounds, three hold all 24 bits of an fp32.
template <int QS> __device__ __forceinline__ void split_bf16(float lo, float hi, uint32_t (&p)[QS]) {
#pragma unroll
    for (int i = 0; i < QS; ++i) {
        p[i] = pack_bf16(lo, hi);
        lo -= __uint_as_float(p[i] << 16);
        hi -= __uint_as_float(p[i] & 0xffff0000u);
    }
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

// A warp's copies: walks the CTA's run ahead of the computing, tile by tile.
template <int D, int R> struct Loader {
    Walk w;
    Segment g;
    int tile;
    bool more;

    __device__ __forceinline__ void start(const AttnArgs &a, const Walk &from, int warp) {
        w = from;
        more = next_segment<R, TILE>(a, w, g);
        tile = g.first + warp;
        settle(a, warp);
    }
    __device__ __forceinline__ void settle(const AttnArgs &a, int warp) {
        while (more && tile >= g.last) {
            more = next_segment<R, TILE>(a, w, g);
            tile = g.first + warp;
        }
    }
    // Lane 0: the copies of the next tile into `dst`; a page outside the cache is flagged and read as page 0.
    __device__ __forceinline__ void issue(const AttnArgs &a, uint8_t *dst, uint64_t *bar) const {
        constexpr int BYTES = Format<D>::BYTES;
        const int sh = a.c.page_shift, in_page = (1 << sh) - 1;
        const int tok = tile * TILE, copies = sh == 4 ? (tok + 16 < g.len ? 2 : 1) : 1;
        const uint32_t bytes = sh == 4 ? BYTES : 2 * BYTES;
        tc::mbar_arrive_expect_tx(bar, bytes * copies);
        for (int i = 0; i < copies; ++i) {
            const int at = tok + 16 * i;
            int page = a.c.table[g.b * a.c.table_stride + (at >> sh)];
            if (page < 0 || page >= a.c.pages) {
                atomicOr(a.err, DEVERR_PAGES);
                page = 0;
            }
            const int64_t block = ((((int64_t)page * a.c.Hk + g.h) << (sh - 4)) + ((at & in_page) >> 4));
            tc::bulk_load(dst + i * BYTES, a.c.data + block * BYTES, bytes, bar);
        }
    }
    __device__ __forceinline__ void advance(const AttnArgs &a, int warp) {
        tile += WARPS;
        settle(a, warp);
    }
};

template <int D, typename T, int NTL>
__global__ void __launch_bounds__(32 * WARPS, 3) kv4_attn_few_kernel(const __grid_constant__ AttnArgs a) {
    using Sm = FewSmem<D, NTL>;
    constexpr int R = Sm::R, G = D / 32, QS = sizeof(T) == 4 ? 3 : 1, BYTES = Format<D>::BYTES;
    extern __shared__ __align__(128) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, j = lane & 3;
    uint8_t *ring = smem + warp * STAGES * Sm::STAGE;
    float *sum = reinterpret_cast<float *>(smem + Sm::SUM);
    float2 *ml = reinterpret_cast<float2 *>(smem + Sm::ML);
    uint64_t *bar = reinterpret_cast<uint64_t *>(smem + Sm::BAR) + warp * STAGES;
    if (lane == 0) {
        for (int i = 0; i < STAGES; ++i) tc::mbar_init(bar + i, 1);
        tc::fence_mbar_init();
    }
    __syncwarp();
    dependent_launch();

    const int64_t total = line_tiles<R, TILE>(a, lane), run = run_length(total, a.ctas, WARPS);
    const int64_t start = blockIdx.x * run;
    if (start >= total) return;  // the whole CTA
    Walk w = walk_at<R, TILE>(a, start, lane);
    w.left = min(run, total - start);
    Loader<D, R> ld;
    ld.start(a, w, warp);
    int issued = 0;
    for (; issued < STAGES && ld.more; ++issued) {
        if (lane == 0) ld.issue(a, ring + issued * Sm::STAGE, bar + issued);
        ld.advance(a, warp);
    }

    int stage = 0, phase = 0, inflight = issued;
    bool ok = true;
    Segment g;
    while (next_segment<R, TILE>(a, w, g)) {
        // this lane's rows as the operand's column r, and its two columns 2j, 2j + 1 of the accumulators
        uint32_t qf[NTL][G][4][QS];
        int hi[NTL][2], lo[NTL][2];
#pragma unroll
        for (int nt = 0; nt < NTL; ++nt) {
            const int rr = g.block * R + nt * 8 + r, i = rr / a.group;
            const bool live = i < g.n;
            const T *p = static_cast<const T *>(a.q) + (g.t0 + i) * a.q_stride +
                         (int64_t)(g.h * a.group + rr - i * a.group) * D + 8 * j;
#pragma unroll
            for (int gr = 0; gr < G; ++gr) {
                if constexpr (QS == 1) {
                    const uint4 v = live ? *reinterpret_cast<const uint4 *>(p + 32 * gr) : make_uint4(0, 0, 0, 0);
                    qf[nt][gr][0][0] = v.x; qf[nt][gr][1][0] = v.y; qf[nt][gr][2][0] = v.z; qf[nt][gr][3][0] = v.w;
                } else {
                    const float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
                    const float4 x = live ? *reinterpret_cast<const float4 *>(p + 32 * gr) : z;
                    const float4 y = live ? *reinterpret_cast<const float4 *>(p + 32 * gr + 4) : z;
                    split_bf16<QS>(x.x, x.y, qf[nt][gr][0]);
                    split_bf16<QS>(x.z, x.w, qf[nt][gr][1]);
                    split_bf16<QS>(y.x, y.y, qf[nt][gr][2]);
                    split_bf16<QS>(y.z, y.w, qf[nt][gr][3]);
                }
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int pos = g.len - g.n + (g.block * R + nt * 8 + 2 * j + e) / a.group;
                hi[nt][e] = a.causal ? min(pos + 1, g.len) : g.len;
                lo[nt][e] = a.window > 0 ? pos - a.window + 1 : 0;
            }
        }
        // tiles between these two ends are seen whole by every row
        const int i0 = g.block * R / a.group, i1 = min(g.n * a.group - 1, g.block * R + R - 1) / a.group;
        const int whole_hi = a.causal ? g.len - g.n + i0 + 1 : g.len;
        const int whole_lo = a.window > 0 ? g.len - g.n + i1 - a.window + 1 : 0;

        float o[G][2][NTL][4], mx[NTL][2], l[NTL][2];
#pragma unroll
        for (int nt = 0; nt < NTL; ++nt) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                mx[nt][e] = -INFINITY;
                l[nt][e] = 0.f;
            }
#pragma unroll
            for (int gr = 0; gr < G; ++gr)
#pragma unroll
                for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[gr][mt][nt][e] = 0.f;
        }

        for (int tile = g.first + warp; tile < g.last; tile += WARPS) {
            const uint8_t *buf = ring + stage * Sm::STAGE;
            if (ok && !__all_sync(0xffffffffu, tc::mbar_wait(bar + stage, phase, WAIT_LIMIT_KV4))) {
                // gave up: the copies in flight land before shared memory goes away, none is started any more
                ok = false;
                for (int i = 0, st = stage, ph = phase; i < inflight; ++i) {
                    tc::mbar_wait(bar + st, ph, WAIT_LIMIT_KV4);
                    if (++st == STAGES) {
                        st = 0;
                        ph ^= 1;
                    }
                }
                if (lane == 0) atomicOr(a.err, DEVERR_TIMEOUT);
            }
            const int tok0 = tile * TILE;
            const bool edge = tok0 + TILE > min(whole_hi, g.len) || tok0 < whole_lo;
            float s[2][NTL][4];
#pragma unroll
            for (int blk = 0; blk < 2; ++blk) {
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
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const uint32_t s2 = prmt(ksc[x][gr >> 1], 0, gr & 1 ? 0x3232 : 0x1010);
                        expand(kw[x][gr], swap_bytes(kw[x][gr]), s2, minus24(s2), f[x]);
                    }
#pragma unroll
                    for (int ks = 0; ks < 2; ++ks)
#pragma unroll
                        for (int nt = 0; nt < NTL; ++nt)
#pragma unroll
                            for (int z = QS - 1; z >= 0; --z)
                                mma16816(s[blk][nt], f[0][2 * ks], f[1][2 * ks], f[0][2 * ks + 1], f[1][2 * ks + 1],
                                         qf[nt][gr][2 * ks][z], qf[nt][gr][2 * ks + 1][z]);
                }
            }
            if (edge) {
#pragma unroll
                for (int blk = 0; blk < 2; ++blk)
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
            // running maxima of the two columns, over the tile's 32 tokens
            bool move = false;
            float top[NTL][2];
#pragma unroll
            for (int nt = 0; nt < NTL; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float m = fmaxf(fmaxf(s[0][nt][e], s[0][nt][2 + e]), fmaxf(s[1][nt][e], s[1][nt][2 + e]));
                    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
                    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
                    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
                    top[nt][e] = m * a.scale_log2;
                    move |= top[nt][e] > mx[nt][e] + SLACK;
                }
            if (__any_sync(0xffffffffu, move)) {
#pragma unroll
                for (int nt = 0; nt < NTL; ++nt) {
                    float f[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float m = fmaxf(mx[nt][e], top[nt][e]);
                        f[e] = m == mx[nt][e] ? 1.f : exp2_fast(mx[nt][e] - m);
                        mx[nt][e] = m;
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
            uint32_t p[2][NTL][2][QS];
#pragma unroll
            for (int nt = 0; nt < NTL; ++nt) {
                const float m0 = mx[nt][0] == -INFINITY ? 0.f : -mx[nt][0], m1 = mx[nt][1] == -INFINITY ? 0.f : -mx[nt][1];
#pragma unroll
                for (int blk = 0; blk < 2; ++blk)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const float p0 = exp2_fast(fmaf(s[blk][nt][2 * x], a.scale_log2, m0));
                        const float p1 = exp2_fast(fmaf(s[blk][nt][2 * x + 1], a.scale_log2, m1));
                        l[nt][0] += p0;
                        l[nt][1] += p1;
                        uint32_t sp[QS];
                        split_bf16<QS>(p0, p1, sp);
#pragma unroll
                        for (int z = 0; z < QS; ++z) p[blk][nt][x][z] = transpose8x8(sp[z]);
                    }
            }
#pragma unroll
            for (int blk = 0; blk < 2; ++blk) {
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
#pragma unroll
                    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                        for (int nt = 0; nt < NTL; ++nt)
#pragma unroll
                            for (int z = QS - 1; z >= 0; --z)
                                mma16816(o[gr][mt][nt], f[0][2 * mt], f[0][2 * mt + 1], f[1][2 * mt], f[1][2 * mt + 1],
                                         p[blk][nt][0][z], p[blk][nt][1][z]);
                }
            }
            __syncwarp();  // every lane has read the stage
            --inflight;
            if (ld.more && ok) {
                if (lane == 0) ld.issue(a, ring + stage * Sm::STAGE, bar + stage);
                ld.advance(a, warp);
                ++inflight;
            }
            if (++stage == STAGES) {
                stage = 0;
                phase ^= 1;
            }
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
                if (x != x) mx[nt][e] = 0.f;  // scores that are all NaN leave no maximum
                if (r == 0) ml[warp * R + nt * 8 + 2 * j + e] = make_float2(mx[nt][e], x);
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
                f[e] = mx[nt][e] == -INFINITY ? 0.f : exp2_fast(mx[nt][e] - m);
            }
#pragma unroll
            for (int gr = 0; gr < G; ++gr)
#pragma unroll
                for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        sum[(warp * 8 + 2 * j + (e & 1)) * (D + 1) + 32 * gr + 8 * (r >> 1) + (r & 1) + 4 * mt +
                            2 * (e >> 1)] = o[gr][mt][nt][e] * f[e & 1];
            __syncthreads();
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const int row = nt * 8 + 2 * warp + y, rr = g.block * R + row, i = rr / a.group;
                float m = -INFINITY, total_l = 0.f;
#pragma unroll
                for (int x = 0; x < WARPS; ++x) m = fmaxf(m, ml[x * R + row].x);
#pragma unroll
                for (int x = 0; x < WARPS; ++x)
                    if (ml[x * R + row].x != -INFINITY) total_l += ml[x * R + row].y * exp2_fast(ml[x * R + row].x - m);
                float v[D / 32];
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    v[c] = 0.f;
                    const int ch = 64 * (c >> 1) + 2 * lane + (c & 1);
#pragma unroll
                    for (int x = 0; x < WARPS; ++x) v[c] += sum[(x * 8 + 2 * warp + y) * (D + 1) + ch];
                }
                if (g.piece >= 0) {
                    const int64_t at = ((int64_t)blockIdx.x * 2 + g.piece) * R + row;
#pragma unroll
                    for (int c = 0; c < D / 64; ++c)
                        *reinterpret_cast<float2 *>(a.part + at * D + 64 * c + 2 * lane) = make_float2(v[2 * c], v[2 * c + 1]);
                    if (lane == 0)
                        *reinterpret_cast<float2 *>(a.part + (int64_t)a.ctas * 2 * R * D + at * 2) = make_float2(m, total_l);
                } else if (i < g.n) {
                    const float inv = total_l == 0.f ? 0.f : 1.f / total_l;
                    const int head = g.h * a.group + rr - i * a.group;
                    T *p = static_cast<T *>(a.out) + (g.t0 + i) * a.out_stride + (int64_t)head * D;
#pragma unroll
                    for (int c = 0; c < D / 64; ++c) {
                        const float x0 = v[2 * c] * inv, x1 = v[2 * c + 1] * inv;
                        if constexpr (QS == 1)
                            *reinterpret_cast<uint32_t *>(p + 64 * c + 2 * lane) = pack_bf16(x0, x1);
                        else
                            *reinterpret_cast<float2 *>(p + 64 * c + 2 * lane) = make_float2(x0, x1);
                    }
                    if (lane == 0 && a.lse)
                        a.lse[(g.t0 + i) * a.Hq + head] = total_l == 0.f ? -INFINITY : (m + log2f(total_l)) * 0.69314718f;
                }
            }
            __syncthreads();
        }
    }
}

// One row of the item that ends run blockIdx.x and goes on in the next, where that is the item's first piece.
template <int D, typename T, int R, int TILE>
__global__ void __launch_bounds__(D) kv4_attn_join_kernel(const __grid_constant__ AttnArgs a, int least) {
    dependent_launch();
    const int lane = threadIdx.x & 31, row = blockIdx.y;
    const int64_t total = line_tiles<R, TILE>(a, lane), run = run_length(total, a.ctas, least);
    const int64_t edge = (blockIdx.x + 1) * run;
    if (edge >= total) return;
    const Walk w = walk_at<R, TILE>(a, edge, lane);
    const int64_t from = edge - w.t, to = from + w.s.tiles;  // the item's tiles
    if (w.t == 0 || from < blockIdx.x * run) return;
    const int block = w.item / a.c.Hk, h = w.item - block * a.c.Hk;
    const int rr = block * R + row, i = rr / a.group;
    if (i >= w.s.n) return;
    const int pieces = (int)((to - 1) / run) - blockIdx.x + 1;
    const float *mlp = a.part + (int64_t)a.ctas * 2 * R * D;
    auto at = [&](int p) { return ((int64_t)(blockIdx.x + p) * 2 + (p == 0)) * R + row; };
    float m = -INFINITY;
    for (int p = lane; p < pieces; p += 32) m = fmaxf(m, mlp[at(p) * 2]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    float l = 0.f, v = 0.f;
#pragma unroll 4
    for (int p = 0; p < pieces; ++p) {
        const float2 x = *reinterpret_cast<const float2 *>(mlp + at(p) * 2);
        const float f = x.x == -INFINITY ? 0.f : exp2_fast(x.x - m);
        l = fmaf(x.y, f, l);
        v = fmaf(a.part[at(p) * D + threadIdx.x], f, v);
    }
    const int head = h * a.group + rr - i * a.group;
    const int64_t t = w.s.t0 + i;
    Elem<T>::store(static_cast<T *>(a.out) + t * a.out_stride + (int64_t)head * D + threadIdx.x, l == 0.f ? 0.f : v / l);
    if (threadIdx.x == 0 && a.lse) a.lse[t * a.Hq + head] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718f;
}

template <int D, typename T, int R, int TILE> kda_status launch_join(const AttnArgs &a, int least, cudaStream_t s) {
    launch_dependent(kv4_attn_join_kernel<D, T, R, TILE>, dim3(a.ctas - 1, R), dim3(D), 0, s, a, least);
    return check_launch("kv4_attn_join_kernel");
}

template <int D, typename T, int NTL> static kda_status attn_few(AttnArgs a, cudaStream_t s) {
    using Sm = FewSmem<D, NTL>;
    constexpr auto kern = kv4_attn_few_kernel<D, T, NTL>;
    if (smem_attr_once<kern>(Sm::BYTES) != cudaSuccess) return check_launch("kv4_attn_few_kernel: shared memory");
    // no more CTAs than the longest line that these sizes allow gives WARPS tiles each
    const int64_t blocks = a.c.T * a.group / Sm::R + a.c.B, tiles = ((int64_t)a.c.cols << a.c.page_shift) / TILE + 1;
    a.ctas = (int)std::min<int64_t>(a.ctas, (blocks * a.c.Hk * tiles + WARPS - 1) / WARPS);
    launch_dependent(kern, dim3(a.ctas), dim3(32 * WARPS), Sm::BYTES, s, a);
    kda_status st = check_launch("kv4_attn_few_kernel");
    if (st || a.ctas == 1) return st;
    return launch_join<D, T, Sm::R, TILE>(a, WARPS, s);
}

static int few_ctas() {
    const int sms = current_sms();
    return 3 * (sms > 0 ? sms : 152);
}

}  // namespace kv4
}  // namespace kda

using namespace kda;

extern "C" size_t kda_kv4_attention_workspace_bytes(int B, int64_t T, int Hq, int Hk, int D, kda_dtype dtype) {
    if (B < 1 || T < 1 || Hq < 1 || Hk < 1 || Hq % Hk || (D != 64 && D != 128) ||
        (dtype != KDA_F32 && dtype != KDA_BF16))
        return 0;
    return (size_t)kv4::few_ctas() * 2 * 16 * (size_t)(D + 2) * sizeof(float);
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
    const size_t need = kda_kv4_attention_workspace_bytes(B, T, Hq, Hk, D, dtype);
    if (workspace_bytes < need) return invalid("workspace too small (kda_kv4_attention_workspace_bytes)");
    if (need && (st = check_ptr(workspace, "workspace"))) return st;
    if ((st = bind_stream_device(stream))) return st;
    if (!(a.err = device_error_word())) return fail(KDA_ERR_CUDA, "device error word unavailable");
    a.q = q;
    a.out = out;
    a.lse = lse;
    a.part = static_cast<float *>(workspace);
    a.q_stride = q_stride;
    a.out_stride = out_stride;
    a.Hq = Hq;
    a.group = Hq / Hk;
    a.causal = causal;
    a.window = window > 0x7fffff00LL ? 0 : (int)window;
    a.scale_log2 = scale * 1.44269504f;
    a.ctas = kv4::few_ctas();
    a.few_rows = 0x7fffffff;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (dtype == KDA_F32) return D == 128 ? kv4::attn_few<128, float, 1>(a, s) : kv4::attn_few<64, float, 1>(a, s);
    if (a.group <= 8 && T == B)
        return D == 128 ? kv4::attn_few<128, __nv_bfloat16, 1>(a, s) : kv4::attn_few<64, __nv_bfloat16, 1>(a, s);
    return D == 128 ? kv4::attn_few<128, __nv_bfloat16, 2>(a, s) : kv4::attn_few<64, __nv_bfloat16, 2>(a, s);
}
