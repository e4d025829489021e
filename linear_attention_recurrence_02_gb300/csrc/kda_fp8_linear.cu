// kda_fp8_linear.cu -- product of 8-bit activations with 8-bit weights, one
// scale per block of 128:
//
//   y[m, n] = sum_k a[m,k] sa[k/128, m] * w[n,k] sw[n/128, k/128]
//
// a and w are e4m3; sa holds one fp32 scale per token and 128 channels (what
// kda_add_rmsnorm_fp8 and kda_gated_rmsnorm_fp8 write), sw one per 128 x 128
// block of the weight. The products of one K block of 128 share their scales,
// so they are summed on the tensor cores (tcgen05 kind::f8f6f4, exact e4m3
// products, fp32 accumulators in TMEM), and the K blocks' sums are joined
// outside it: acc += (sa * sw) * block_sum in fp32 registers.
#include <atomic>
#include <cstring>
#include <string>

#include "kda_common.cuh"
#include "kda_prefill.cuh"
#include "kda_tc.cuh"

namespace kda {
namespace lin {

constexpr int KB = 128;                             // K block: channels per scale
constexpr long long WAIT_LIMIT = 2000000000LL;      // clock cycles (about 1 s)

// D[tmem] (+)= A[smem] B[smem]^T, e4m3 inputs (both K-major), fp32 accumulate
__device__ __forceinline__ void mma_f8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                       uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// instruction descriptor of kind::f8f6f4: e4m3 A and B (format 0), fp32 D, M x N tile
__host__ __device__ constexpr uint32_t idesc_f8(int M, int N) {
    return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// 16 consecutive TMEM columns of the thread's lane
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}

// ---------------------------------------------------------------- waits, clusters
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    __syncwarp();  // .aligned wants the warp's lanes together; some callers come from a lane's own branch
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// address in the cluster's shared window of this CTA's `p` in CTA `rank`
__device__ __forceinline__ uint32_t peer_addr(const void *p, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(tc::smem_u32(p)), "r"(rank));
    return r;
}
__device__ __forceinline__ void arrive_peer(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// The pair's barriers guard TMEM (ordered by the tcgen05 fences) and copies
// (ordered by the barrier's own transaction count) and no plain memory, so
// waits and arrivals stay at their default scope: at cluster scope each one
// waited for the warp's outstanding memory operations (a K block's hand-shakes
// alone took 1700 cycles).
// Once a wait has given up (ok is false) the later ones only look, so that a
// loop of waits has no exit in its middle and ends in bounded time.
__device__ __forceinline__ bool wait_more(uint64_t *bar, uint32_t parity, bool ok) {
    if (tc::mbar_try_wait(bar, parity)) return ok;
    return ok && tc::mbar_wait(bar, parity, WAIT_LIMIT);
}
// One lane of a whole warp. The issuing warps run their loops with all lanes and
// single one out only around the copies and MMAs: under `lane == 0` an MMA took
// 62 cycles to issue, as its descriptors were not in uniform registers.
__device__ __forceinline__ bool elect_one() {
    uint32_t e;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(e));
    return e != 0;
}
// where `yes`, the fp32 value at the place of `p` in the shared memory of the cluster's CTA `rank`, else 0
__device__ __forceinline__ float peer_load_if(bool yes, const float *p, uint32_t rank) {
    float v;
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.u32 q, %2, 0;\n\t"
        "mov.f32 %0, 0f00000000;\n\t"
        "@q ld.shared::cluster.f32 %0, [%1];\n\t}"
        : "=&f"(v)
        : "r"(peer_addr(p, yes ? rank : 0u)), "r"((uint32_t)yes)
        : "memory");
    return v;
}
// wait for the warp's TMEM loads; the loaded registers pass through it, so that no use moves ahead of it
__device__ __forceinline__ void tmem_ld_wait_for(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 :
                 : "memory");
}

// Predicated stores: as branches, a run of them took about 56 cycles each (64 x 12288 x 512: 5.0 us, 3.7 now).
__device__ __forceinline__ void store_raw(bool yes, void *to, uint32_t v) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %0, 0;\n\t@p st.global.b32 [%1], %2;\n\t}"
                 :: "r"((uint32_t)yes), "l"(to), "r"(v) : "memory");
}
__device__ __forceinline__ void store_raw(bool yes, void *to, uint16_t v) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %0, 0;\n\t@p st.global.b16 [%1], %2;\n\t}"
                 :: "r"((uint32_t)yes), "l"(to), "h"(v) : "memory");
}
__device__ __forceinline__ void store_if(bool yes, float *to, float v) { store_raw(yes, to, __float_as_uint(v)); }
__device__ __forceinline__ void store_if(bool yes, __nv_bfloat16 *to, float v) {
    store_raw(yes, to, __bfloat16_as_ushort(__float2bfloat16_rn(v)));
}

// copy of a tile that no other CTA reads: the first to leave L2
__device__ __forceinline__ void tma_load_once(void *dst, const CUtensorMap *map, uint64_t *bar, int x, int y) {
    uint64_t policy;
    asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%3, "
        "%4}], [%2], %5;" ::"r"(tc::smem_u32(dst)),
        "l"(map), "r"(tc::smem_u32(bar)), "r"(x), "r"(y), "l"(policy)
        : "memory");
}

// ---------------------------------------------------------------- few tokens
// A unit is 128 weight rows (the MMA's M axis: TMEM lane = output feature) and
// NT tokens (its N axis). The weights, read once, are what bounds it: a step
// with few tokens still feeds whole 128-row tiles from every SM, as S CTAs of a
// cluster with a run of the K blocks each (SPLIT), or as CTAs that walk several
// units, so that one's first blocks arrive while the one before is stored (128 x
// 36864 x 4096: 25.8 us; while the results' stores were still branches 29.5, and
// 33.3 with a CTA per unit). JW warps join the block
// sums (a thread holds its feature's sums for TPW tokens; the products of the
// token scales with the weight block's come from shared memory), the next
// streams the weight and token tiles through a ring of ST stages, the next issues
// a block's four MMAs into one of AS accumulators, the last two form the
// scales' products of CK blocks at a time. The cluster's partial sums meet in
// shared memory: each CTA adds up its share of the tokens over the S CTAs in
// their order. Two CTAs fit an SM, of 128 tokens one.
// Why 128 tokens: the weight tile is read once where 64 would read it twice, and
// a tile of 256 x 256 would be half empty (100 x 12288 x 8192: 22.0 us, 27.9 at
// 64, 26.5 in the many-token kernel; 128 x 12288 x 4096: 13.0, 15.7 and 16.1).
// A weight tile that one CTA alone reads is marked first to leave L2 (64 x
// 36864 x 4096: 23.4 us, 24.8 without), where the state, the activations and
// the next call's tokens stay.
// A programmatic dependent launch: before the kernel ahead of it on the stream
// has completed it only prefetches weight tiles into L2, which cannot serve a
// stale value; every read and write comes after griddepcontrol.wait.
template <int NT> struct Few {
    static constexpr int JW = NT == 128 ? 8 : 4;      // joining warps: 4 for up to 64 tokens each
    static constexpr int TPW = NT / (JW / 4);         // tokens of a joining warp
    static constexpr int NTHREADS = 32 * (JW + 4), PER_SM = NT == 128 ? 1 : 2;  // CTAs an SM
    static constexpr int STAGE = 128 * KB + NT * KB;  // bytes: weights, then tokens
    static constexpr int ST = NT == 16 || NT == 128 ? 6 : NT == 32 ? 5 : 4;
    static constexpr int AS = 4;                      // accumulators
    static constexpr int COLS = NT * AS;              // TMEM columns (64 to 512)
    static constexpr int CK = 4, CS = 2;              // K blocks of scales per chunk, chunks in flight
    static constexpr int SCALES = ST * STAGE;
    static constexpr int BARS = SCALES + CS * CK * NT * 4;
    static constexpr int SMEM = BARS + (2 * ST + 2 * AS + 2 * CS) * 8 + 16 + 1024;
    static_assert(NT * 128 * 4 <= ST * STAGE, "the partial sums take the ring's place");
};

// Tokens j0, j0 + G, ... below j1 of a feature: the sum of the S CTAs' partial sums (at most P) in the CTAs'
// order, 32 loads on their way at once.
template <int P, int G, typename TO>
__device__ __forceinline__ void add_parts(const float *part, int j0, int j1, int S, bool live, TO *y, int64_t ldy) {
    constexpr int R = 32 / P;
    for (; j0 < j1; j0 += R * G) {
        float v[R][P];
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
            for (int p = 0; p < P; ++p)
                v[i][p] = peer_load_if(p < S && j0 + G * i < j1, part + (j0 + G * i) * 128, (uint32_t)p);
#pragma unroll
        for (int i = 0; i < R; ++i) {
            float sum = v[i][0];
#pragma unroll
            for (int p = 1; p < P; ++p) sum += v[i][p];
            store_if(j0 + G * i < j1 && live, y + (int64_t)(j0 + G * i) * ldy, sum);
        }
    }
}

template <int NT, typename TO, bool SPLIT>
__global__ void __launch_bounds__(Few<NT>::NTHREADS, Few<NT>::PER_SM)
    linear_few_kernel(const __grid_constant__ CUtensorMap tm_w,
                      const __grid_constant__ CUtensorMap tm_a,
                      const float *sa, const float *sw,
                      TO *__restrict__ y, int M, int N, int nkb, int64_t ldy, int mt,
                      int S, unsigned units, unsigned *err) {
    using namespace tc;
    using F = Few<NT>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = smem_raw + ((1024u - ((uint32_t)__cvta_generic_to_shared(smem_raw) & 1023u)) & 1023u);
    uint64_t *full = reinterpret_cast<uint64_t *>(sm + F::BARS), *empty = full + F::ST, *afull = empty + F::ST,
             *aempty = afull + F::AS, *sfull = aempty + F::AS, *sempty = sfull + F::CS;
    uint32_t *s_taddr = reinterpret_cast<uint32_t *>(sempty + F::CS);
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // uniform to the compiler
    // SPLIT: one of the S CTAs of a cluster, which share a unit's K blocks; else a CTA walks units (128 features x
    // NT tokens, the token tiles of a weight tile together)
    const unsigned first = SPLIT ? blockIdx.x / (unsigned)S : blockIdx.x;
    const int r = SPLIT ? (int)(blockIdx.x - first * (unsigned)S) : 0;
    auto feature = [&](unsigned u) { return (int)(u / (unsigned)mt) * 128; };
    auto token = [&](unsigned u) { return (int)(u % (unsigned)mt) * NT; };
    // K blocks of this CTA
    const int k0 = SPLIT ? (int)((int64_t)nkb * r / S) : 0, k1 = SPLIT ? (int)((int64_t)nkb * (r + 1) / S) : nkb;
    if (tid == 0) {
        for (int i = 0; i < F::ST; ++i) {
            mbar_init(full + i, 1);
            mbar_init(empty + i, 1);
        }
        for (int i = 0; i < F::AS; ++i) {
            mbar_init(afull + i, 1);
            mbar_init(aempty + i, F::JW);
        }
        for (int i = 0; i < F::CS; ++i) {
            mbar_init(sfull + i, 2);
            mbar_init(sempty + i, F::JW);
        }
        fence_mbar_init();
    }
    if (warp == F::JW && elect_one()) {
        tma_prefetch_desc(&tm_w);
        tma_prefetch_desc(&tm_a);
        for (int i = 0; i < F::ST && k0 + i < k1; ++i) tma_prefetch_l2_2d(&tm_w, (k0 + i) * KB, feature(first));
    }
    if (warp == F::JW + 1) {
        tmem_alloc(s_taddr, F::COLS);
        tmem_relinquish();
    }
    sync_tc();
    const uint32_t tbase = *s_taddr, sbase = smem_u32(sm);
    asm volatile("griddepcontrol.wait;\n\tgriddepcontrol.launch_dependents;" ::: "memory");
    bool ok = true;
    const int j0w = (warp >> 2) * F::TPW, f = tid & 127;  // a joining thread's first token, its feature
    float acc[F::TPW];
    if (warp < F::JW) {
        const uint32_t trow = tbase + ((uint32_t)(32 * (warp & 3)) << 16) + j0w;
        const float *chunks = reinterpret_cast<const float *>(sm + F::SCALES) + j0w;
        int as = 0, cs = 0;
        uint32_t ph = 0, cph = 0;
        for (unsigned u = first; u < units; u += gridDim.x) {
            const int n0 = feature(u), m0 = token(u);
#pragma unroll
            for (int j = 0; j < F::TPW; ++j) acc[j] = 0.f;
            for (int kb = k0; kb < k1; ++kb) {
                const int ck = (kb - k0) % F::CK;
                if (ck == 0) ok = wait_more(sfull + cs, cph, ok);
                const float *sr = chunks + (cs * F::CK + ck) * NT;
                ok = wait_more(afull + as, ph, ok);
                __syncwarp();
                tc_fence_after();
#pragma unroll
                for (int c = 0; c < F::TPW; c += 16) {
                    uint32_t d[16];
                    tmem_ld16(trow + as * NT + c, d);
                    tmem_ld_wait_for(d);
                    if (c == F::TPW - 16) {  // the accumulator is read: the MMAs may write it again
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(aempty + as);
                    }
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const float4 s = *reinterpret_cast<const float4 *>(sr + c + 4 * q);
                        acc[c + 4 * q] = fmaf(__uint_as_float(d[4 * q]), s.x, acc[c + 4 * q]);
                        acc[c + 4 * q + 1] = fmaf(__uint_as_float(d[4 * q + 1]), s.y, acc[c + 4 * q + 1]);
                        acc[c + 4 * q + 2] = fmaf(__uint_as_float(d[4 * q + 2]), s.z, acc[c + 4 * q + 2]);
                        acc[c + 4 * q + 3] = fmaf(__uint_as_float(d[4 * q + 3]), s.w, acc[c + 4 * q + 3]);
                    }
                }
                if (++as == F::AS) {
                    as = 0;
                    ph ^= 1;
                }
                if (ck == F::CK - 1 || kb == k1 - 1) {  // the chunk's last: its slot may be filled again
                    __syncwarp();
                    if (lane == 0) mbar_arrive(sempty + cs);
                    if (++cs == F::CS) {
                        cs = 0;
                        cph ^= 1;
                    }
                }
            }
            if (!SPLIT) {
                const int live = ok && n0 + f < N ? M - m0 - j0w : 0;
                TO *to = y + (int64_t)(m0 + j0w) * ldy + n0 + f;
#pragma unroll
                for (int j = 0; j < F::TPW; ++j, to += ldy) store_if(j < live, to, acc[j]);
            }
            if (SPLIT) break;
        }
    } else if (warp == F::JW) {
        int st = 0;
        uint32_t ph = 1;  // the ring starts out free
        for (unsigned u = first; u < units; u += gridDim.x) {
            const int n0 = feature(u), m0 = token(u);
            for (int kb = k0; kb < k1; ++kb) {
                ok = wait_more(empty + st, ph, ok);
                __syncwarp();
                if (elect_one()) {
                    uint8_t *d = sm + st * F::STAGE;
                    mbar_arrive_expect_tx(full + st, F::STAGE);
                    if (mt == 1) tma_load_once(d, &tm_w, full + st, kb * KB, n0);
                    else tma_load_2d(d, &tm_w, full + st, kb * KB, n0);
                    tma_load_2d(d + 128 * KB, &tm_a, full + st, kb * KB, m0);
                }
                if (++st == F::ST) {
                    st = 0;
                    ph ^= 1;
                }
            }
            if (SPLIT) break;
        }
        // every copy lands before shared memory is used otherwise or goes away
        for (int i = 0; i < F::ST; ++i) {
            if (--st < 0) {
                st = F::ST - 1;
                ph ^= 1;
            }
            if (!mbar_wait(full + st, ph ^ 1, WAIT_LIMIT)) ok = false;
        }
    } else if (warp == F::JW + 1) {
        int st = 0, as = 0;
        uint32_t ph = 0, aph = 1;  // the accumulators start out free
        const uint64_t a0 = sdesc_sw128(sbase, 16, 1024), b0 = sdesc_sw128(sbase + 128 * KB, 16, 1024);
        // Blocks after which a stage is filled again. The last ones' stages are not released: no one waits for
        // them, and an arrival could come after the CTA has left.
        int64_t refills = (SPLIT ? 1 : (int64_t)((units - first + gridDim.x - 1) / gridDim.x)) * (k1 - k0) - F::ST;
        for (unsigned u = first; u < units; u += gridDim.x) {
            const int n0 = feature(u), m0 = token(u);
            for (int kb = k0; kb < k1; ++kb, --refills) {
                const uint64_t a = a0 + (uint64_t)(st * (F::STAGE / 16)), b = b0 + (uint64_t)(st * (F::STAGE / 16));
                ok = wait_more(full + st, ph, ok);
                ok = wait_more(aempty + as, aph, ok);
                __syncwarp();
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)
                        mma_f8(tbase + as * NT, a + 2 * ks, b + 2 * ks, idesc_f8(128, NT), ks > 0);
                    if (refills > 0) mma_commit(empty + st);
                    mma_commit(afull + as);
                }
                if (++as == F::AS) {
                    as = 0;
                    aph ^= 1;
                }
                if (++st == F::ST) {
                    st = 0;
                    ph ^= 1;
                }
            }
            if (SPLIT) break;
        }
    } else {
        // the scales' products (tokens past the end take the last one's and are not stored)
        float *chunks = reinterpret_cast<float *>(sm + F::SCALES);
        const int t2 = tid - 32 * (F::JW + 2);
        int cs = 0;
        uint32_t cph = 1;
        constexpr int PER = F::CK * NT / 64;  // products of a chunk per lane
        for (unsigned u = first; u < units; u += gridDim.x) {
            const int n0 = feature(u), m0 = token(u);
            const float *swp = sw + (int64_t)(n0 >> 7) * nkb;
            for (int kc = k0; kc < k1; kc += F::CK) {
                float av[PER], wv[PER];
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    const int e = t2 + 64 * i, j = e % NT, kb = kc + e / NT < k1 ? kc + e / NT : k1 - 1;
                    av[i] = ld_plain(sa + (int64_t)kb * M + (m0 + j < M ? m0 + j : M - 1));
                    wv[i] = ld_plain(swp + kb);
                }
                ok = wait_more(sempty + cs, cph, ok);
#pragma unroll
                for (int i = 0; i < PER; ++i) chunks[cs * F::CK * NT + t2 + 64 * i] = av[i] * wv[i];
                __syncwarp();
                if (lane == 0) mbar_arrive(sfull + cs);
                if (++cs == F::CS) {
                    cs = 0;
                    cph ^= 1;
                }
            }
            if (SPLIT) break;
        }
    }
    if (!ok) atomicOr(err, DEVERR_TIMEOUT);
    sync_tc();
    if (warp == F::JW + 1) tmem_dealloc(tbase, F::COLS);
    if (!SPLIT) return;
    // Partial sums [token][feature] in the ring's place; each CTA adds up `per` tokens over the cluster.
    const int n0 = feature(first), m0 = token(first), per = (NT + S - 1) / S;
    float *part = reinterpret_cast<float *>(sm);
    if (warp < F::JW) {
#pragma unroll
        for (int j = 0; j < F::TPW; ++j) part[(j0w + j) * 128 + f] = ok ? acc[j] : __uint_as_float(0x7fffffffu);
    }
    cluster_sync();
    constexpr int G = F::NTHREADS / 128;
    const int j0 = r * per + (tid >> 7), j1 = min(min((r + 1) * per, NT), M - m0);
    TO *to = y + (int64_t)m0 * ldy + n0 + f;
    if (S == 2) add_parts<2, G>(part + f, j0, j1, S, n0 + f < N, to, ldy);
    else if (S <= 4) add_parts<4, G>(part + f, j0, j1, S, n0 + f < N, to, ldy);
    else add_parts<8, G>(part + f, j0, j1, S, n0 + f < N, to, ldy);
    cluster_sync();  // no CTA leaves while another still reads its sums
}

static void few_config(cudaLaunchConfig_t &cfg, cudaLaunchAttribute (&at)[2], unsigned ctas, int threads, int smem,
                       int S, cudaStream_t s) {
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = s;
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)S;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
}

// Clusters of S = 1 to `most` CTAs that run at once on the current device (0: none, or an error). Two CTAs fit an SM,
// but clusters do not always fill the SMs that they have to share: 304 CTAs as clusters of 1 or 2, 296 of 4,
// 276 of 6. The occupancy query counts one CTA per SM for any kernel that allocates TMEM, although two run
// (13.8 of 16 warps active on average at 288 CTAs), so a stand-in of the same shape is asked.
template <int NTHREADS, int PER_SM> __global__ void __launch_bounds__(NTHREADS, PER_SM) few_stand_in() {}
template <int NT> static void few_resident(int (&at_once)[9], int most) {
    using F = Few<NT == 128 ? 128 : 16>;  // of the smaller three, the one with the most shared memory
    static_assert(Few<32>::SMEM <= Few<16>::SMEM && Few<64>::SMEM <= Few<16>::SMEM, "two CTAs of each size fit an SM");
    constexpr auto stand_in = few_stand_in<F::NTHREADS, F::PER_SM>;
    static std::atomic<int> known[9][64];  // value + 1
    int dev = 0;
    const bool found = cudaGetDevice(&dev) == cudaSuccess && dev >= 0 && dev < 64;
    for (int S = 1; S <= most; ++S) {
        int n = found ? known[S][dev].load(std::memory_order_acquire) - 1 : 0;
        if (n < 0) {
            cudaLaunchConfig_t cfg = {};
            cudaLaunchAttribute at[2];
            few_config(cfg, at, (unsigned)S, F::NTHREADS, F::SMEM, S, nullptr);
            cfg.numAttrs = 1;
            if (smem_attr_once<stand_in>(F::SMEM) == cudaSuccess &&
                cudaOccupancyMaxActiveClusters(&n, stand_in, &cfg) == cudaSuccess) {
                known[S][dev].store(n + 1, std::memory_order_release);
            } else {
                cudaGetLastError();
                n = 0;
            }
        }
        at_once[S] = n;
    }
}

// Estimated times in ns choose between kernels and splits of K; their constants are fitted to measurements at
// 8 to 224 weight tiles of 4 to 64 K blocks, which they meet within a tenth. Of 90 sizes drawn over the whole range
// (1 to 800 tokens) 76 run within 7 % of the best kernel and split. The others lose 8 to 23 %: up to 16 weight tiles
// of 12 to 41 K blocks, where six or eight CTAs a tile would be right (8 x 24 x 1984: 3.55 us, 2.96), two tokens
// and 73 to 93 tiles, where none should be split (2 x 11797 x 2768: 10.8 us, 8.8), and rows that straddle 128-byte
// lines (146 x 11144 x 2640: 16.6 us, 14.4 in the many-token kernel; the worst known, with a long K, is
// 182 x 10432 x 11312: 64 us at 64 tokens, 41 there). A call's CTAs take `ctas` and the
// weights' bytes 2.5 ns per 16 KB tile: the longer of the two and some of the shorter.
static int64_t with_weights(int64_t ctas, int N, int nkb) {
    const int64_t bytes = ((int64_t)N + 127) / 128 * nkb * 5 / 2;
    return ctas > bytes ? ctas + bytes * 3 / 20 : bytes + ctas * 3 / 20;
}

// CTAs of a cluster (a split of K) for M x N x K and the time that this takes (S = 0: the kernel cannot run
// here). A call takes FIX and a K block BLOCK, 1.4 times that where two CTAs of 64 tokens share an SM; the
// meeting of the partial sums MEET, 0.7 us more on shared SMs; CTAs that fill the GPU 0.6 to 1.2 us more than a
// few (the next call's cannot set up beside them); and a further wave of clusters a call's time, of units that a
// CTA walks 1.1 us. With 64 tokens or more, rows that straddle 128-byte lines take half as long again where CTAs
// walk units (300 x 30000 x 1040: 28.6 us, 21.5 in the many-token kernel).
// (1 x 12288 x 4096, 96 tiles: 9.6 us at S = 3, 10.8 at 1, 11.2 at 2, 13.5 at 4; 64 x 12288 x 4096: 12.2 us at 2 or
// 3, 13.0 at 1, 17.0 at 4; 64 x 4096 x 8192, 32 tiles: 10.2 us at 4, 19.5 at 1.)
struct FewPlan {
    int64_t units;
    int S, at_once;  // clusters that run at once
    int64_t ns;
};
template <int NT> static FewPlan few_plan(int64_t M, int N, int nkb, bool straddle) {
    constexpr int C = NT == 16 ? 0 : NT == 32 ? 1 : NT == 64 ? 2 : 3;
    constexpr int64_t FIX = C == 0 ? 1800 : C == 1 ? 2000 : C == 2 ? 2150 : 2460;
    constexpr int64_t BLOCK = C == 0 ? 194 : C == 1 ? 208 : C == 2 ? 264 : 281;
    constexpr int64_t MEET[4][9] = {{0, 0, 1100, 1450, 1100, 1500, 1500, 1800, 1800},
                                    {0, 0, 1050, 1400, 1050, 1700, 1700, 2000, 2000},
                                    {0, 0, 1150, 1950, 1300, 2200, 2200, 2300, 2300},
                                    {0, 0, 2300, 2600, 2600, 2800, 2800, 3200, 3200}};
    const int64_t crowd = M < 16 ? 550 + 44 * M : 1240;
    FewPlan p{((M + NT - 1) / NT) * (((int64_t)N + 127) / 128), 0, 0, INT64_MAX};
    int fit[9];
    const int most = nkb < 8 ? nkb : 8;
    few_resident<NT>(fit, most);
    const int sms = fit[1] / Few<NT>::PER_SM;
    for (int S = 1; S <= most; ++S) {
        const int at_once = fit[S];
        if (at_once < 1) continue;
        const int64_t waves = (p.units + at_once - 1) / at_once, resident = p.units < at_once ? p.units : at_once;
        const bool shared = resident * S > sms;  // two CTAs on an SM
        const int64_t meet = MEET[C][S] + (S > 1 && shared ? 700 : 0);
        int64_t block = NT >= 64 && shared ? BLOCK * 14 / 10 : BLOCK;
        if (NT >= 64 && straddle && waves > 1) block += block / 2;
        const int64_t ctas = waves * ((nkb + S - 1) / S) * block + meet + crowd * resident / at_once +
                             (waves - 1) * (S > 1 ? FIX + meet + 1240 : 1100);
        const int64_t t = FIX + with_weights(ctas, N, nkb);
        if (t < p.ns) {
            p.ns = t;
            p.S = S;
            p.at_once = at_once;
        }
    }
    return p;
}

template <int NT, typename TO>
static kda_status launch_few(const CUtensorMap &tw, const CUtensorMap &ta, const float *sa, const float *sw, void *y,
                             int64_t M, int N, int nkb, int64_t ldy, const FewPlan &p, unsigned *err, cudaStream_t s) {
    if (p.S < 1 || smem_attr_once<linear_few_kernel<NT, TO, false>>(Few<NT>::SMEM) != cudaSuccess ||
        smem_attr_once<linear_few_kernel<NT, TO, true>>(Few<NT>::SMEM) != cudaSuccess) {
        cudaGetLastError();
        return fail(KDA_ERR_CUDA, "linear_few_kernel does not fit the device");
    }
    if (p.units * p.S > 0x7fffffffLL) return invalid("M*N too large for one launch");
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[2];
    const int64_t ctas = p.S > 1 ? p.units * p.S : p.units < p.at_once ? p.units : p.at_once;
    few_config(cfg, at, (unsigned)ctas, Few<NT>::NTHREADS, Few<NT>::SMEM, p.S, s);
    cudaLaunchKernelEx(&cfg, p.S > 1 ? linear_few_kernel<NT, TO, true> : linear_few_kernel<NT, TO, false>, tw, ta, sa, sw,
                       static_cast<TO *>(y), (int)M, N, nkb, ldy, (int)((M + NT - 1) / NT), p.S, (unsigned)p.units,
                       err);  // an error is left for check_launch
    return check_launch("linear_few_kernel");
}

// ---------------------------------------------------------------- many tokens
// A pair of CTAs (one cluster, two SMs) owns a 256-token x 256-feature tile:
// the MMAs of cta_group::2 take 128 token rows and half of the 256 weight rows
// from each CTA's shared memory, so every operand byte is copied and read once
// per pair. Each CTA's TMEM holds its 128 tokens (lane = token) in two
// accumulators of 256 columns, one K block each: 512 cycles of MMAs, in which
// the other accumulator has to be read and handed back. Per CTA: warps 0-7 join
// the block sums (warps 0-3 the tile's first 128 features, 4-7 the last; a
// thread holds 128 fp32 sums of one token, and one product of its token's scale
// with the features' scale serves the whole K block), warp 8 copies, warp 9 of
// the even CTA issues the MMAs for both, warps 10 and 11 form the scales'
// products, four K blocks at a time. Persistent: a pair walks tiles, token
// tiles first, so that neighbouring pairs share weight tiles in L2, and the next
// tile's products run while this one's results are stored. Where the tiles would
// leave most pairs idle, 2 or 4 pairs of one cluster take a run of K blocks of
// the same tile each (SPLIT) and exchange their sums at the end.
namespace many {
constexpr int BM = 256, BN = 256;                 // tile of a pair
constexpr int A_BYTES = 128 * KB, W_BYTES = 128 * KB;
constexpr int STAGE = A_BYTES + W_BYTES;          // bytes per CTA: tokens, then weights
constexpr int ST = 5, AS = 2;                      // stages of operands at most, accumulators
constexpr int JW = 8, JC = 128;                   // joining warps, features of each
constexpr int NTHREADS = 32 * (JW + 4);
// Registers a thread: launched with REGS, split so that the joining warps hold their sums and neither
// side spills (208 / 88 and 240 / 24 spill inside the K loop: a third slower).
constexpr int REGS = 168, REGS_JOIN = 216, REGS_ISSUE = 72;
static_assert(JW * REGS_JOIN + 4 * REGS_ISSUE == (JW + 4) * REGS, "the split draws on the launch's registers");
constexpr int CK = 4, CS = 4;                     // K blocks of scales per chunk, chunks in flight
constexpr int CHUNK = CK * 256 * 4;               // [CK][feature half][token] products of the two scales
// Behind the stages the results on their way out: per joining warp one piece of 32 rows of 128 B beside five
// stages, or two beside four (many_stages).
constexpr int PIECE = 4096;
constexpr int SCALES = ST * STAGE + JW * PIECE;
static_assert((ST - 1) * STAGE + JW * 2 * PIECE == SCALES, "a stage is a piece per joining warp");
static_assert(3 * 32768 <= (ST - 1) * STAGE, "a split's partial sums, of 2 or 4 pairs, take the ring's place");
constexpr int BARS = SCALES + CS * CHUNK;
constexpr int SMEM = BARS + (2 * ST + 2 * AS + 2 * CS) * 8 + 16 + 1024;
}  // namespace many

// copy into this CTA's shared memory, completing on a barrier of the pair's even CTA
__device__ __forceinline__ void tma_load_pair(void *dst, const CUtensorMap *map, uint32_t bar, int x, int y) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, "
        "%4}], [%2];" ::"r"(tc::smem_u32(dst)),
        "l"(map), "r"(bar), "r"(x), "r"(y)
        : "memory");
}
__device__ __forceinline__ void mma_f8_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                            uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// arrive on `bar` of both CTAs of the pair (cluster ranks lead and lead + 1) when every MMA issued so far by
// this thread completes
__device__ __forceinline__ void commit_pair(uint64_t *bar, uint32_t lead) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            tc::smem_u32(bar)),
        "h"((uint16_t)(3u << lead))
        : "memory");
}

// (a.lo, a.hi) += (d0, d1) * (s, s) in one instruction
__device__ __forceinline__ void fma2(uint64_t &a, uint32_t d0, uint32_t d1, uint64_t s) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(d0), "r"(d1));
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(a) : "l"(d), "l"(s));
}

// 16 bytes to an address of the cluster's shared window
__device__ __forceinline__ void peer_store16(uint32_t at, float a, float b, float c, float d) {
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(at), "f"(a), "f"(b), "f"(c), "f"(d)
                 : "memory");
}
// (a.lo, a.hi) += (x, y)
__device__ __forceinline__ void add2(uint64_t &a, float x, float y) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(x), "f"(y));
    asm("add.rn.f32x2 %0, %0, %1;" : "+l"(a) : "l"(d));
}

// until at most N of this thread's committed bulk stores have still to read their shared memory
template <int N> __device__ __forceinline__ void bulk_wait_read_but() {
    asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}

// A warp stores `rows` rows of `cols` elements from its staged 128-byte rows (16-byte pieces swizzled by the
// row) to rows of any alignment: 4 bytes a lane, sixteen rows' reads in flight, predicated stores. Where a
// row of 2-byte elements starts between two words, each lane's word is joined from two neighbours' halves and
// the elements at the ends go by themselves. (3000 x 20001 x 464: bf16 63 us, 78 with a branch a row, 131 with
// an element a lane; f32 86. Rows of 20000 elements, which a tensor copy stores: 42 and 58. Rows that start inside
// a 32-byte sector also write that sector in two parts.)
template <typename TO>
__device__ __forceinline__ void store_rows(TO *to, int64_t ld, const uint8_t *from, int rows, int cols) {
    constexpr int B = 16;
    const int lane = threadIdx.x & 31;
    for (int i0 = 0; i0 < rows; i0 += B) {
        uint32_t w[B];
#pragma unroll
        for (int j = 0; j < B; ++j)
            w[j] = *reinterpret_cast<const uint32_t *>(from + (i0 + j) * 128 + (((lane >> 2) ^ (j & 7)) << 4) +
                                                       (lane & 3) * 4);
#pragma unroll
        for (int j = 0; j < B; ++j) {
            const bool live = i0 + j < rows;
            TO *row = to + (i0 + j) * ld;
            if constexpr (sizeof(TO) == 4) {
                store_raw(live && lane < cols, row + lane, w[j]);
            } else {
                const int odd = (int)(reinterpret_cast<uintptr_t>(row) >> 1) & 1, c = 2 * lane + odd;
                const uint32_t up = __shfl_down_sync(0xffffffffu, w[j], 1);
                const uint32_t pair = odd ? __funnelshift_r(w[j], up, 16) : w[j];
                store_raw(live && c + 1 < cols, row + c, pair);
                store_raw(live && c + 1 == cols, row + c, (uint16_t)pair);
                store_raw(live && odd && lane == 0, row, (uint16_t)w[j]);
            }
        }
    }
}

template <typename TO, bool SPLIT>
__global__ void __launch_bounds__(many::NTHREADS, 1)
    linear_many_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_w,
                       const __grid_constant__ CUtensorMap tm_y, const float *sa,
                       const float *sw, TO *__restrict__ y, int M, int N, int nkb, int64_t ldy,
                       unsigned mt, unsigned tile0, unsigned tiles, int by_tma, int S, int stages,
                       unsigned *err) {
    using namespace tc;
    using namespace many;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = smem_raw + ((1024u - ((uint32_t)__cvta_generic_to_shared(smem_raw) & 1023u)) & 1023u);
    uint64_t *full = reinterpret_cast<uint64_t *>(sm + BARS), *empty = full + ST, *afull = empty + ST,
             *aempty = afull + AS, *sfull = aempty + AS, *sempty = sfull + CS;
    uint32_t *s_taddr = reinterpret_cast<uint32_t *>(sempty + CS);
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // uniform to the compiler
    // rank: this CTA in its pair, lead: the cluster rank of the pair's even CTA, sp: the pair in its cluster
    const uint32_t crank = cluster_rank(), rank = crank & 1, lead = crank & ~1u;
    const int sp = SPLIT ? (int)(crank >> 1) : 0;
    const unsigned first = tile0 + (SPLIT ? blockIdx.x / (2u * (unsigned)S) : blockIdx.x >> 1);
    const unsigned npairs = SPLIT ? gridDim.x / (2u * (unsigned)S) : gridDim.x >> 1;
    // K blocks of this pair
    const int kb0 = SPLIT ? (int)((int64_t)nkb * sp / S) : 0, kb1 = SPLIT ? (int)((int64_t)nkb * (sp + 1) / S) : nkb;
    if (tid == 0) {
        for (int i = 0; i < stages; ++i) {
            mbar_init(full + i, 1);  // the even CTA's own arrival; both CTAs' bytes
            mbar_init(empty + i, 1);
        }
        for (int i = 0; i < AS; ++i) {
            mbar_init(afull + i, 1);
            mbar_init(aempty + i, 2 * JW);  // the joining warps of both CTAs
        }
        for (int i = 0; i < CS; ++i) {
            mbar_init(sfull + i, 2);  // the two warps that form scales
            mbar_init(sempty + i, JW);
        }
        fence_mbar_init();
    }
    if (warp == JW + 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(s_taddr)),
                     "r"(AS * BN)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    // A programmatic dependent launch, as the few-token kernel: before the wait only weight tiles move, to L2.
    if (warp == JW && elect_one()) {
        tma_prefetch_desc(&tm_a);
        tma_prefetch_desc(&tm_w);
        for (int kb = kb0; kb < kb0 + stages && kb < kb1; ++kb)
            tma_prefetch_l2_2d(&tm_w, kb * KB, (int)(first / mt) * BN + (int)rank * 128);
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    asm volatile("griddepcontrol.wait;\n\tgriddepcontrol.launch_dependents;" ::: "memory");
    static_assert(AS * BN == 512, "the whole TMEM: its first column is 0");
    constexpr uint32_t tbase = 0;
    const uint32_t sbase = smem_u32(sm);
    bool ok = true;
    if (warp < JW) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_JOIN));
        const int half = warp >> 2;  // features 128 * half of the tile
        const uint32_t trow = tbase + ((uint32_t)(32 * (warp & 3)) << 16) + half * 128;
        const uint32_t rel0 = peer_addr(aempty, lead), rel1 = peer_addr(aempty + 1, lead);
        const int mrow = (int)rank * 128 + 32 * (warp & 3) + lane;
        const float *mine = reinterpret_cast<const float *>(sm + SCALES) + half * 128 + 32 * (warp & 3) + lane;
        const bool two = stages < ST;  // pieces
        uint8_t *out = sm + stages * STAGE + warp * (two ? 2 * PIECE : PIECE);
        int flip = 0;
        int as = 0, cs = 0;
        uint32_t ph = 0, cph = 0;
        for (unsigned tile = first; tile < tiles; tile += npairs) {
            uint64_t acc[JC / 2];  // pairs of fp32
#pragma unroll
            for (int j = 0; j < JC / 2; ++j) acc[j] = 0;
            for (int kb = kb0; kb < kb1; ++kb) {
                const int ck = (kb - kb0) & (CK - 1);
                if (ck == 0) ok = wait_more(sfull + cs, cph, ok);
                const float s0 = mine[cs * (CHUNK / 4) + ck * 256];
                uint64_t s2;
                asm("mov.b64 %0, {%1, %1};" : "=l"(s2) : "f"(s0));
                ok = wait_more(afull + as, ph, ok);
                __syncwarp();
                tc_fence_after();
                // 16 columns at a time, the next 16 on their way while these are joined
                uint32_t d[2][16];
                tmem_ld16(trow + as * BN, d[0]);
                tmem_ld_wait_for(d[0]);
#pragma unroll
                for (int c = 0; c < JC / 16; ++c) {
                    if (c + 1 < JC / 16) tmem_ld16(trow + as * BN + 16 * (c + 1), d[(c + 1) & 1]);
#pragma unroll
                    for (int j = 0; j < 8; ++j) fma2(acc[8 * c + j], d[c & 1][2 * j], d[c & 1][2 * j + 1], s2);
                    if (c + 1 < JC / 16) tmem_ld_wait_for(d[(c + 1) & 1]);
                    if (c + 2 == JC / 16) {  // the accumulator is read: the MMAs may write it again
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) arrive_peer(as ? rel1 : rel0);
                    }
                }
                as ^= 1;
                ph ^= as == 0;
                if (ck == CK - 1 || kb == kb1 - 1) {  // the chunk's last: its slot may be filled again
                    __syncwarp();
                    if (lane == 0) mbar_arrive(sempty + cs);
                    if (++cs == CS) {
                        cs = 0;
                        cph ^= 1;
                    }
                }
            }
            if constexpr (SPLIT) {
                // The pairs' sums meet: each group of 64 features belongs to one pair of the cluster; the
                // others send it theirs, [group][pair][feature / 4][token] in the ring's place, and it adds them
                // to its own in the pairs' order. (One tile per cluster: the rings are free from here on.) Sums of
                // a thread whose waits gave up are sent as NaN, not for the others' to pass as results.
                if (!ok) {
#pragma unroll
                    for (int j = 0; j < JC / 2; ++j) acc[j] = 0x7fffffff7fffffffull;
                }
                cluster_sync();
                const int per = 4 / S, row = 32 * (warp & 3) + lane;  // groups of a pair
                auto val = [&](int j) { return __uint_as_float((uint32_t)(acc[j >> 1] >> (32 * (j & 1)))); };
#pragma unroll
                for (int gi = 0; gi < 2; ++gi) {
                    const int g = 2 * half + gi, o = g / per, slot = (g - o * per) * (S - 1) + (sp < o ? sp : sp - 1);
                    if (o == sp) continue;
                    const uint32_t to = peer_addr(sm, 2u * (uint32_t)o + rank) + (uint32_t)(slot * 32768 + row * 16);
#pragma unroll
                    for (int c = 0; c < 16; ++c)
                        peer_store16(to + c * 2048, val(64 * gi + 4 * c), val(64 * gi + 4 * c + 1),
                                     val(64 * gi + 4 * c + 2), val(64 * gi + 4 * c + 3));
                }
                cluster_sync();
#pragma unroll
                for (int gi = 0; gi < 2; ++gi) {
                    const int g = 2 * half + gi, o = g / per;
                    if (o != sp) continue;
                    const float4 *from = reinterpret_cast<const float4 *>(sm) + (g - o * per) * (S - 1) * 2048 + row;
                    for (int q = 0; q < S - 1; ++q, from += 2048) {
#pragma unroll
                        for (int c = 0; c < 16; ++c) {
                            const float4 x = from[c * 128];
                            add2(acc[32 * gi + 2 * c], x.x, x.y);
                            add2(acc[32 * gi + 2 * c + 1], x.z, x.w);
                        }
                    }
                }
            }
            // The results leave through shared memory, 128 bytes of each of the warp's 32 rows at a time (a
            // row's stores straight from its thread take a cycle per 32 bytes): swizzled 16-byte pieces, then
            // one tensor copy, or whole rows by the warp where y's rows do not suit a tensor map.
            const int mw = (int)(tile % mt) * BM + mrow - lane, n0 = (int)(tile / mt) * BN + half * 128;
            auto at = [&](int j) { return __uint_as_float((uint32_t)(acc[j >> 1] >> (32 * (j & 1)))); };
            if (__all_sync(0xffffffffu, ok) && mw < M) {
                constexpr int V = 16 / (int)sizeof(TO), JR = 8 * V;
#pragma unroll
                for (int r = 0; r < JC / JR; ++r) {
                    const int n = n0 + r * JR;
                    if (n >= N) break;
                    if (SPLIT && (2 * half + r * JR / 64) / (4 / S) != sp) continue;  // another pair's
                    uint8_t *piece = out + flip;
                    if (two) flip ^= PIECE;
                    if (lane == 0) {  // the piece's last copy has read it
                        if (two) bulk_wait_read_but<1>();
                        else bulk_wait_read();
                    }
                    __syncwarp();
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        uint4 raw;
                        TO *e = reinterpret_cast<TO *>(&raw);
#pragma unroll
                        for (int i = 0; i < V; ++i) Elem<TO>::store(e + i, at(r * JR + q * V + i));
                        *reinterpret_cast<uint4 *>(piece + lane * 128 + ((q ^ (lane & 7)) << 4)) = raw;
                    }
                    fence_async_smem();
                    __syncwarp();
                    if (by_tma && (N % V == 0 || n + JR <= N)) {  // the copy would write all of a 16-byte piece
                        if (lane == 0) {
                            tma_store_2d(&tm_y, piece, n, mw);
                            bulk_commit();
                        }
                    } else {
                        store_rows(y + mw * ldy + n, ldy, piece, M - mw < 32 ? M - mw : 32, N - n < JR ? N - n : JR);
                        // an empty group: the wait above counts a group for every piece, and would take this one's
                        // predecessor, whose copy may still read the next piece, for the latest
                        if (lane == 0) bulk_commit();
                    }
                }
            }
        }
        if (lane == 0) bulk_wait_all();
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_ISSUE));
        if (warp == JW) {
            int st = 0;
            uint32_t ph = 1;  // the ring starts out free
            for (unsigned tile = first; tile < tiles; tile += npairs) {
                const int row_a = (int)(tile % mt) * BM + (int)rank * 128;
                const int row_w = (int)(tile / mt) * BN + (int)rank * 128;
                for (int kb = kb0; kb < kb1; ++kb) {
                    ok = wait_more(empty + st, ph, ok);
                    __syncwarp();
                    if (elect_one()) {
                        uint8_t *d = sm + st * STAGE;
                        const uint32_t bar = peer_addr(full + st, lead);
                        if (rank == 0) mbar_arrive_expect_tx(full + st, 2 * STAGE);
                        tma_load_pair(d, &tm_a, bar, kb * KB, row_a);
                        tma_load_pair(d + A_BYTES, &tm_w, bar, kb * KB, row_w);
                    }
                    if (++st == stages) {
                        st = 0;
                        ph ^= 1;
                    }
                }
            }
            // Every copy of both CTAs lands before shared memory goes away (the even CTA's barriers count
            // them): the ring's next phase of each stage is the one that the last copies complete.
            if (rank == 0)
                for (int i = 0; i < stages; ++i) {
                    if (--st < 0) {
                        st = stages - 1;
                        ph ^= 1;
                    }
                    if (!tc::mbar_wait(full + st, ph ^ 1, WAIT_LIMIT)) ok = false;
                }
        } else if (warp == JW + 1) {
            if (rank == 0) {
                int st = 0, as = 0;
                uint32_t ph = 0, aph = 1;  // the accumulators start out free
                const uint64_t a0 = sdesc_sw128(sbase, 16, 1024), b0 = sdesc_sw128(sbase + A_BYTES, 16, 1024);
                // blocks after which a stage is filled again: the last ones' stages are not released, as no one
                // waits for them and an arrival could come after a CTA has left
                int64_t refills = (int64_t)((tiles - first + npairs - 1) / npairs) * (kb1 - kb0) - stages;
                for (unsigned tile = first; tile < tiles; tile += npairs) {
                    for (int kb = kb0; kb < kb1; ++kb, --refills) {
                        const uint64_t a = a0 + (uint64_t)(st * (STAGE / 16)), b = b0 + (uint64_t)(st * (STAGE / 16));
                        ok = wait_more(full + st, ph, ok);
                        ok = wait_more(aempty + as, aph, ok);
                        __syncwarp();
                        tc_fence_after();
                        if (elect_one()) {
#pragma unroll
                            for (int ks = 0; ks < 4; ++ks)
                                mma_f8_pair(tbase + as * BN, a + 2 * ks, b + 2 * ks, idesc_f8(BM, BN), ks > 0);
                            commit_pair(afull + as, lead);
                            if (refills > 0) commit_pair(empty + st, lead);
                        }
                        as ^= 1;
                        aph ^= as == 0;
                        if (++st == stages) {
                            st = 0;
                            ph ^= 1;
                        }
                    }
                }
            }
        } else {
            // the last two warps: the scales' products, two K blocks of a chunk each, CS - 1 chunks ahead of
            // their use (tokens and features past the end take the last ones' and are not stored)
            const int nblk = (N + 127) / 128, w2 = (warp - JW - 2) * 2;
            int cs = 0;
            uint32_t cph = 1;
            for (unsigned tile = first; tile < tiles; tile += npairs) {
                const int m0 = (int)(tile % mt) * BM + (int)rank * 128 + lane, nb = (int)(tile / mt) * 2;
                const float *w0 = sw + (int64_t)nb * nkb, *w1 = nb + 1 < nblk ? w0 + nkb : w0;
                for (int k0 = kb0; k0 < kb1; k0 += CK) {
                    ok = wait_more(sempty + cs, cph, ok);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int kc = k0 + w2 + i < kb1 ? k0 + w2 + i : kb1 - 1;
                        const float *ap = sa + (int64_t)kc * M;
                        float *b = reinterpret_cast<float *>(sm + SCALES) + cs * (CHUNK / 4) + (w2 + i) * 256 + lane;
                        float av[4];
                        const float wa = ld_plain(w0 + kc), wb = ld_plain(w1 + kc);
#pragma unroll
                        for (int q = 0; q < 4; ++q) av[q] = ld_plain(ap + (m0 + 32 * q < M ? m0 + 32 * q : M - 1));
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            b[32 * q] = av[q] * wa;
                            b[128 + 32 * q] = av[q] * wb;
                        }
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(sfull + cs);
                    if (++cs == CS) {
                        cs = 0;
                        cph ^= 1;
                    }
                }
            }
        }
        if (SPLIT) {  // the joining warps' two meetings
            cluster_sync();
            cluster_sync();
        }
    }
    if (!ok) atomicOr(err, DEVERR_TIMEOUT);
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    if (warp == JW + 1)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tbase), "r"(AS * BN) : "memory");
}

// 2-D tiled map over [rows][inner] with a row stride of its own (bytes, a multiple of 16), 128-byte swizzle
static bool row_map(CUtensorMap *m, const void *p, CUtensorMapDataType dt, uint64_t inner, uint64_t rows,
                    uint64_t row_bytes, uint32_t box_inner, uint32_t box_rows) {
    tcp::EncodeTiledFn fn = tcp::encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[2] = {inner, rows}, strides[1] = {row_bytes};
    const cuuint32_t box[2] = {box_inner, box_rows}, es[2] = {1, 1};
    return fn(m, dt, 2, const_cast<void *>(p), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// of a byte matrix [rows][K], box 128 x box_rows
static bool byte_map(CUtensorMap *m, const void *p, int K, int64_t rows, int64_t ld, int box_rows) {
    return row_map(m, p, CU_TENSOR_MAP_DATA_TYPE_UINT8, (uint64_t)K, (uint64_t)rows, (uint64_t)ld, KB,
                   (uint32_t)box_rows);
}

static void many_config(cudaLaunchConfig_t &cfg, cudaLaunchAttribute (&at)[2], unsigned clusters, int S, cudaStream_t s) {
    cfg.gridDim = dim3(clusters * 2u * (unsigned)S);
    cfg.blockDim = dim3(many::NTHREADS);
    cfg.dynamicSmemBytes = many::SMEM;
    cfg.stream = s;
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = 2u * (unsigned)S;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
}

// Clusters of S pairs that run at once on the current device (0: none, or an error), and the kernel
// made ready to launch there.
template <typename TO, bool SPLIT> static int resident_clusters(int S) {
    static std::atomic<int> known[3][64];  // value + 1
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev > 63) return 0;
    std::atomic<int> &slot = known[S >> 1][dev];
    int n = slot.load(std::memory_order_acquire);
    if (n > 0) return n - 1;
    // the register split only adds up for the launch register count it was made for
    cudaFuncAttributes fa;
    if (cudaFuncGetAttributes(&fa, linear_many_kernel<TO, SPLIT>) != cudaSuccess || fa.numRegs != many::REGS ||
        smem_attr_once<linear_many_kernel<TO, SPLIT>>(many::SMEM) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[2];
    many_config(cfg, at, 1, S, nullptr);
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, linear_many_kernel<TO, SPLIT>, &cfg) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    slot.store(n + 1, std::memory_order_release);
    return n;
}

// How the CTA pairs take a product's tiles: `whole` of them in turn, one pair each, then the rest one per
// cluster with its K blocks split over S pairs.
struct ManyPlan {
    int64_t whole, tiles;
    int S;
    int64_t ns;  // estimated time
};

// 350 ns a K block, 1 us a tile, 3.5 us a launch and 1.2 us more for one that fills the GPU; a split takes 3 or
// 5.5 us (2 or 4 pairs) for the meeting of the partial sums, and pays for tiles that would leave most pairs idle,
// be it all of them or a last wave's, when K is long. (512 x 4096 x 12288, 32 tiles: 25 us at S = 2, 35 whole;
// 240 x 3800 x 12288, 15 tiles: 19 us at 4, 22.5 at 2, 34.5 whole; 2560 x 2250 x 8192: 45.5 and 51.3.)
template <typename TO> static ManyPlan many_plan(int64_t M, int N, int nkb) {
    ManyPlan p{0, 0, 1, INT64_MAX};
    p.tiles = ((M + many::BM - 1) / many::BM) * (((int64_t)N + many::BN - 1) / many::BN);
    const int pairs = resident_clusters<TO, false>(1);
    if (pairs < 1) return p;
    const int64_t wave = (int64_t)nkb * 350 + 1000, full = p.tiles / pairs, rest = p.tiles % pairs;
    p.whole = p.tiles;
    p.ns = with_weights((full + (rest ? 1 : 0)) * wave, N, nkb) + 3500 + (full ? 1200 : 1200 * rest / pairs);
    for (int S = 2; S <= 4 && S <= nkb && rest && rest * S <= pairs; S *= 2) {
        const int64_t t = with_weights(full * wave + (int64_t)((nkb + S - 1) / S) * 350, N, nkb) +
                          (full ? 4700 : 1200 * rest * S / pairs) + 4500 + (S == 2 ? 3000 : 5500);
        if (t < p.ns && rest <= resident_clusters<TO, true>(S)) p = ManyPlan{p.tiles - rest, p.tiles, S, t};
    }
    return p;
}

// Four stages and two pieces where a pair has tiles after its first and short ones: results leave beside the next
// tile's K blocks (4864 x 4096 x 512: 14.6 us, 15.7 with one piece; x 2048: 32.6 and 33.1; 3000 x 20000 x 464:
// 42.7 and 46.2). Else five and one, for weights that come from memory (128 x 12288 x 4096: 16.2 us, 17.2 with
// four; 182 x 10432 x 11312: 40.8 and 42.4; 4096 x 4096 x 12288 the same).
static int many_stages(bool more_tiles, int nkb) { return more_tiles && nkb <= 16 ? many::ST - 1 : many::ST; }

template <typename TO>
static kda_status launch_many(const CUtensorMap &ta, const CUtensorMap &tw, const float *sa, const float *sw, void *y,
                              int64_t M, int N, int K, int64_t ldy, const ManyPlan &p, unsigned *err, cudaStream_t s) {
    if (p.tiles > 0x7fffffffLL) return invalid("M*N too large for one launch");
    // y's rows suit a tensor map where their stride is a multiple of 16 bytes
    const int by_tma = (ldy * sizeof(TO)) % 16 == 0 && ldy < (1LL << 36);
    CUtensorMap ty;
    memset(&ty, 0, sizeof(ty));
    if (by_tma && !row_map(&ty, y, sizeof(TO) == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32,
                           (uint64_t)N, (uint64_t)M, (uint64_t)ldy * sizeof(TO), 128 / sizeof(TO), 32))
        return fail(KDA_ERR_CUDA, "cuTensorMapEncodeTiled failed");
    const unsigned mt = (unsigned)((M + many::BM - 1) / many::BM);
    const int nkb = (K + KB - 1) / KB;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[2];
    auto go = [&](auto kern, int64_t tile0, int64_t tiles, int64_t most, int S) {
        many_config(cfg, at, (unsigned)(tiles - tile0 < most ? tiles - tile0 : most), S, s);
        cudaLaunchKernelEx(&cfg, kern, ta, tw, ty, sa, sw, static_cast<TO *>(y), (int)M, N, nkb, ldy, mt,
                           (unsigned)tile0, (unsigned)tiles, by_tma, S, many_stages(tiles - tile0 > most, nkb),
                           err);  // an error is left for check_launch
    };
    if (p.whole > 0) go(linear_many_kernel<TO, false>, 0, p.whole, resident_clusters<TO, false>(1), 1);
    if (p.whole < p.tiles) go(linear_many_kernel<TO, true>, p.whole, p.tiles, p.tiles - p.whole, p.S);
    return check_launch("linear_many_kernel");
}

template <typename TO>
static kda_status run_linear(const void *a, const float *sa, const void *w, const float *sw, void *y, int64_t M,
                             int N, int K, int64_t lda, int64_t ldw, int64_t ldy, unsigned *err, cudaStream_t s) {
    // Up to 64 tokens a weight tile is read once and its bytes bound the call: the few-token kernel. With
    // more, whichever is estimated fastest: that kernel, 64 or 128 tokens at a time, or the many-token one.
    int nt = M <= 16 ? 16 : M <= 32 ? 32 : 64;
    const int nkb = (K + KB - 1) / KB;
    // Rows of contiguous operands straddle 128-byte lines by K. The strides themselves stay out of the choice: it
    // sets the order of the sums, and a matrix has the same bits whole and as a slice of wider rows.
    const bool straddle = K % 128 != 0;
    FewPlan p = nt == 16   ? few_plan<16>(M, N, nkb, straddle)
                : nt == 32 ? few_plan<32>(M, N, nkb, straddle)
                           : few_plan<64>(M, N, nkb, straddle);
    if (M > 64) {
        const FewPlan p128 = few_plan<128>(M, N, nkb, straddle);
        if (p128.ns < p.ns) {
            p = p128;
            nt = 128;
        }
        const ManyPlan plan = many_plan<TO>(M, N, nkb);
        if (plan.ns < p.ns) {
            CUtensorMap ta, tw;
            if (!byte_map(&ta, a, K, M, lda, 128) || !byte_map(&tw, w, K, N, ldw, 128))
                return fail(KDA_ERR_CUDA, "cuTensorMapEncodeTiled failed");
            return launch_many<TO>(ta, tw, sa, sw, y, M, N, K, ldy, plan, err, s);
        }
    }
    CUtensorMap tw, ta;
    if (!byte_map(&tw, w, K, N, ldw, 128) || !byte_map(&ta, a, K, M, lda, nt))
        return fail(KDA_ERR_CUDA, "cuTensorMapEncodeTiled failed");
    switch (nt) {
    case 16: return launch_few<16, TO>(tw, ta, sa, sw, y, M, N, nkb, ldy, p, err, s);
    case 32: return launch_few<32, TO>(tw, ta, sa, sw, y, M, N, nkb, ldy, p, err, s);
    case 64: return launch_few<64, TO>(tw, ta, sa, sw, y, M, N, nkb, ldy, p, err, s);
    default: return launch_few<128, TO>(tw, ta, sa, sw, y, M, N, nkb, ldy, p, err, s);
    }
}

}  // namespace lin
}  // namespace kda

using namespace kda;

extern "C" kda_status kda_fp8_linear(const void *a, const float *a_scales, const void *w, const float *w_scales,
                                     void *y, int64_t M, int N, int K, int64_t lda, int64_t ldw, int64_t ldy,
                                     kda_dtype out_dtype, kda_stream_t stream) {
    clear_detail();
    if (M < 0 || M > 0x7fffff00LL) return invalid("M must be in 0..2^31-256");
    if (N < 1 || N > 0x7fffff00) return invalid("N must be in 1..2^31-256");
    if (K < 16 || K % 16 != 0 || K > 0x7fffff00) return invalid("K must be a positive multiple of 16");
    if (lda < K || lda % 16 != 0 || ldw < K || ldw % 16 != 0) return invalid("lda and ldw must be multiples of 16, at least K");
    if (lda >= (1LL << 40) || ldw >= (1LL << 40)) return invalid("lda and ldw must be below 2^40");
    if (ldy < N) return invalid("ldy must be at least N");
    if (out_dtype != KDA_F32 && out_dtype != KDA_BF16) return invalid("out_dtype must be KDA_F32 or KDA_BF16");
    if (M == 0) return KDA_OK;
    kda_status st;
    if ((st = check_ptr(a, "a")) || (st = check_ptr(a_scales, "a_scales")) || (st = check_ptr(w, "w")) ||
        (st = check_ptr(w_scales, "w_scales")) || (st = check_ptr(y, "y")))
        return st;
    if (y == a || y == w || y == a_scales || y == w_scales) return invalid("y must not alias another argument");
    if ((st = bind_stream_device(stream))) return st;
    unsigned *err = device_error_word();
    if (err == nullptr) return fail(KDA_ERR_CUDA, "device error word unavailable");
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (out_dtype == KDA_BF16)
        return lin::run_linear<__nv_bfloat16>(a, a_scales, w, w_scales, y, M, N, K, lda, ldw, ldy, err, s);
    return lin::run_linear<float>(a, a_scales, w, w_scales, y, M, N, K, lda, ldw, ldy, err, s);
}
