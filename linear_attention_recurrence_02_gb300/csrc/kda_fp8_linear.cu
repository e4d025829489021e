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

// ---------------------------------------------------------------- few tokens
// A CTA owns 128 weight rows (the MMA's M axis: TMEM lane = output feature)
// and NT tokens (its N axis), so that a step with few tokens still feeds whole
// 128-row tiles: the weights, read once, are what bounds it. Warp 0 streams
// the weight and token tiles of each K block through a ring of ST stages,
// warp 1 issues the block's four MMAs into one of AS accumulator stages, and
// warps 2-5 join the block sums: each multiplies the block's token scales by
// the weight block's scale once, and then has one fused multiply-add per
// feature and token.
template <int NT> struct Few {
    static constexpr int STAGE = 128 * KB + NT * KB;  // bytes: weights, then tokens
    static constexpr int ST = NT <= 32 ? 10 : NT <= 64 ? 8 : 6;
    static constexpr int AS = NT <= 64 ? 4 : 2;       // accumulator stages
    static constexpr int COLS = NT * AS;              // TMEM columns (64, 128, 256, 256)
    static constexpr int SBUF = ST * STAGE;           // scale rows: 4 warps x 2 x NT floats
    static constexpr int BARS = SBUF + 4 * 2 * NT * 4;
    static constexpr int SMEM = BARS + (2 * ST + 2 * AS) * 8 + 16 + 1024;
    static constexpr int NTHREADS = 192;
};

template <int NT, typename TO>
__global__ void __launch_bounds__(192) linear_few_kernel(const __grid_constant__ CUtensorMap tm_w,
                                                         const __grid_constant__ CUtensorMap tm_a,
                                                         const float *__restrict__ sa, const float *__restrict__ sw,
                                                         TO *__restrict__ y, int64_t M, int N, int nkb, int64_t ldy,
                                                         int mt, unsigned *err) {
    using namespace tc;
    using F = Few<NT>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = smem_raw + ((1024u - ((uint32_t)__cvta_generic_to_shared(smem_raw) & 1023u)) & 1023u);
    uint64_t *full = reinterpret_cast<uint64_t *>(sm + F::BARS), *empty = full + F::ST, *afull = empty + F::ST,
             *aempty = afull + F::AS;
    uint32_t *s_taddr = reinterpret_cast<uint32_t *>(aempty + F::AS);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int nt = blockIdx.x / mt;
    const int64_t m0 = (int64_t)(blockIdx.x % mt) * NT;
    const int n0 = nt * 128;
    if (tid == 0) {
        for (int i = 0; i < F::ST; ++i) {
            mbar_init(full + i, 1);
            mbar_init(empty + i, 1);
        }
        for (int i = 0; i < F::AS; ++i) {
            mbar_init(afull + i, 1);
            mbar_init(aempty + i, 4);
        }
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(s_taddr, F::COLS);
        tmem_relinquish();
    }
    sync_tc();
    const uint32_t tbase = *s_taddr, sbase = smem_u32(sm);
    bool ok = true;
    float acc[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[j] = 0.f;
    if (warp == 0) {
        if (lane == 0) {
            int kb = 0;
            for (; kb < nkb && ok; ++kb) {
                const int st = kb % F::ST;
                if (kb >= F::ST) ok = mbar_wait(empty + st, (kb / F::ST - 1) & 1, WAIT_LIMIT);
                if (!ok) break;
                uint8_t *d = sm + st * F::STAGE;
                mbar_arrive_expect_tx(full + st, F::STAGE);
                tma_load_2d(d, &tm_w, full + st, kb * KB, n0);
                tma_load_2d(d + 128 * KB, &tm_a, full + st, kb * KB, (int)m0);
            }
            // every copy issued has landed before shared memory goes away
            for (int i = kb > F::ST ? kb - F::ST : 0; i < kb; ++i)
                ok = mbar_wait(full + i % F::ST, (i / F::ST) & 1, WAIT_LIMIT) && ok;
        }
        __syncwarp();
    } else if (warp == 1) {
        if (lane == 0) {
            for (int kb = 0; kb < nkb; ++kb) {
                const int st = kb % F::ST, as = kb % F::AS;
                if (kb >= F::AS) ok = mbar_wait(aempty + as, (kb / F::AS - 1) & 1, WAIT_LIMIT);
                ok = ok && mbar_wait(full + st, (kb / F::ST) & 1, WAIT_LIMIT);
                if (!ok) break;
                tc_fence_after();
                const uint32_t a = sbase + st * F::STAGE, b = a + 128 * KB;
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
                    mma_f8(tbase + as * NT, sdesc_sw128(a + ks * 32, 16, 1024), sdesc_sw128(b + ks * 32, 16, 1024),
                           idesc_f8(128, NT), ks > 0);
                mma_commit(empty + st);
                mma_commit(afull + as);
            }
        }
        __syncwarp();
    } else {
        const int ew = warp - 2;
        const uint32_t trow = tbase + ((uint32_t)(32 * (warp & 3)) << 16);
        float *srow = reinterpret_cast<float *>(sm + F::SBUF) + ew * 2 * NT;
        const float *swp = sw + (int64_t)nt * nkb;
        constexpr int L = NT < 32 ? 1 : NT / 32;
        float sv[L];  // this lane's token scales of the coming K block
        auto fetch = [&](int kb) {
            const float ws = __ldg(swp + kb);
#pragma unroll
            for (int i = 0; i < L; ++i) {
                const int j = lane + 32 * i;
                sv[i] = j < NT && m0 + j < M ? ws * __ldg(sa + (int64_t)kb * M + m0 + j) : 0.f;
            }
        };
        fetch(0);
        for (int kb = 0; kb < nkb; ++kb) {
            const int as = kb % F::AS;
            float *sr = srow + (kb & 1) * NT;
#pragma unroll
            for (int i = 0; i < L; ++i)
                if (lane + 32 * i < NT) sr[lane + 32 * i] = sv[i];
            if (kb + 1 < nkb) fetch(kb + 1);
            __syncwarp();
            ok = mbar_wait(afull + as, (kb / F::AS) & 1, WAIT_LIMIT);
            if (__any_sync(0xffffffffu, !ok)) {
                ok = false;
                break;
            }
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < NT; c += 16) {
                uint32_t d[16];
                tmem_ld16(trow + as * NT + c, d);
                tmem_ld_wait();
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const float4 s = *reinterpret_cast<const float4 *>(sr + c + 4 * q);
                    acc[c + 4 * q] = fmaf(__uint_as_float(d[4 * q]), s.x, acc[c + 4 * q]);
                    acc[c + 4 * q + 1] = fmaf(__uint_as_float(d[4 * q + 1]), s.y, acc[c + 4 * q + 1]);
                    acc[c + 4 * q + 2] = fmaf(__uint_as_float(d[4 * q + 2]), s.z, acc[c + 4 * q + 2]);
                    acc[c + 4 * q + 3] = fmaf(__uint_as_float(d[4 * q + 3]), s.w, acc[c + 4 * q + 3]);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(aempty + as);
        }
        const int n = n0 + 32 * (warp & 3) + lane;
        if (ok && n < N) {
#pragma unroll
            for (int j = 0; j < NT; ++j)
                if (m0 + j < M) Elem<TO>::store(y + (m0 + j) * ldy + n, acc[j]);
        }
    }
    if (!ok && lane == 0) atomicOr(err, DEVERR_TIMEOUT);
    sync_tc();
    if (warp == 1) tmem_dealloc(tbase, F::COLS);
}

template <int NT, typename TO>
static kda_status launch_few(const CUtensorMap &tw, const CUtensorMap &ta, const float *sa, const float *sw, void *y,
                             int64_t M, int N, int K, int64_t ldy, unsigned *err, cudaStream_t s) {
    using F = Few<NT>;
    if (smem_attr_once<linear_few_kernel<NT, TO>>(F::SMEM) != cudaSuccess)
        return check_launch("linear_few_kernel (shared memory attribute)");
    const int64_t mt = (M + NT - 1) / NT, grid = mt * ((N + 127) / 128);
    if (grid > 0x7fffffffLL) return invalid("M*N too large for one launch");
    linear_few_kernel<NT, TO><<<(unsigned)grid, F::NTHREADS, F::SMEM, s>>>(
        tw, ta, sa, sw, static_cast<TO *>(y), M, N, (K + KB - 1) / KB, ldy, (int)mt, err);
    return check_launch("linear_few_kernel");
}

// map of a row-major [rows][K] byte matrix with row stride ld, box 128 x box_rows, 128-byte swizzle
static bool byte_map(CUtensorMap *m, const void *p, int K, int64_t rows, int64_t ld, int box_rows) {
    return tcp::make_map_ld(m, p, CU_TENSOR_MAP_DATA_TYPE_UINT8, (uint64_t)K, (uint64_t)rows, (uint64_t)ld, KB,
                            (uint32_t)box_rows, CU_TENSOR_MAP_SWIZZLE_128B);
}

template <typename TO>
static kda_status run_linear(const void *a, const float *sa, const void *w, const float *sw, void *y, int64_t M,
                             int N, int K, int64_t lda, int64_t ldw, int64_t ldy, unsigned *err, cudaStream_t s) {
    const int nt = M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : 128;
    CUtensorMap tw, ta;
    if (!byte_map(&tw, w, K, N, ldw, 128) || !byte_map(&ta, a, K, M, lda, nt))
        return fail(KDA_ERR_CUDA, "cuTensorMapEncodeTiled failed");
    switch (nt) {
    case 16: return launch_few<16, TO>(tw, ta, sa, sw, y, M, N, K, ldy, err, s);
    case 32: return launch_few<32, TO>(tw, ta, sa, sw, y, M, N, K, ldy, err, s);
    case 64: return launch_few<64, TO>(tw, ta, sa, sw, y, M, N, K, ldy, err, s);
    default: return launch_few<128, TO>(tw, ta, sa, sw, y, M, N, K, ldy, err, s);
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
