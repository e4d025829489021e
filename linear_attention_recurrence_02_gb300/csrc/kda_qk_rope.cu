// kda_qk_rope.cu -- RMSNorm of every query and key head and the rotation by their position, in one pass
// (kda_qk_norm_rope).
//
//   y = x / sqrt(mean x^2 + eps) * w;  then pair i of the first R channels turns by position * freq_i
//
// Bound by memory: each element is read and written once. A row (token, head) is D / 8 lanes of eight
// channels, so the sum of squares is a shuffle reduction and a channel's partner R/2 further on is a
// lane's shuffle away. A CTA owns one token and some or all of its heads: the R/2 sines and cosines are
// formed once per CTA, while the rows' loads are in flight.
//
// Angles: a position's turn is position * freq / 2 pi modulo 1. freq / 2 pi modulo 1 is kept as a 64-bit
// fraction (2^-64 turns a unit), so the product with an integer position wraps around exactly: the angle
// of position 2^31 is as good as that of position 1, and its upper 32 bits (2^-32 turns, 1.5e-9 radians)
// go to the sine and cosine in half turns.
#include <string>

#include "kda_fp8.cuh"
#include "kda_prefill.cuh"

namespace kda {

struct RopeArgs {
    const void *q, *k;
    void *q_out, *k_out;
    const float *q_weight, *k_weight;
    const int64_t *positions;
    const double *freq;
    int64_t q_stride, k_stride, qo_stride, ko_stride;
    int Hq, Hk, half;  // half = R / 2 pairs
    float eps;
};

// UP rows a thread: row (blockIdx.y * UP + u) * (blockDim.x / LPR) + threadIdx.x / LPR of the token's Hq + Hk.
template <int D, typename T, bool INTER, int UP>
__global__ void __launch_bounds__(512) qk_norm_rope_kernel(const RopeArgs a) {
    constexpr int LPR = D / 8;
    __shared__ float2 turn[D / 2];  // (cos, sin) of each pair
    const int64_t t = blockIdx.x;
    const int rows = blockDim.x / LPR, ln = threadIdx.x % LPR, c0 = 8 * ln;
    const int first = blockIdx.y * UP * rows + threadIdx.x / LPR;
    dependent_launch();
    Raw8<T> raw[UP];
#pragma unroll
    for (int u = 0; u < UP; ++u) {
        const int r = first + u * rows;
        if (r < a.Hq) load8(static_cast<const T *>(a.q) + t * a.q_stride + (int64_t)r * D + c0, raw[u]);
        else if (r < a.Hq + a.Hk) load8(static_cast<const T *>(a.k) + t * a.k_stride + (int64_t)(r - a.Hq) * D + c0, raw[u]);
    }
    if (a.half > 0) {
        const int64_t pos = a.positions[t];
        for (int i = threadIdx.x; i < a.half; i += blockDim.x) {
            double f = a.freq[i] * 0.15915494309189533577;  // turns a position
            f -= rint(f);
            const uint64_t phase = (uint64_t)pos * (uint64_t)__double2ll_rn(f * 0x1p64);
            float x = (float)(int32_t)(phase >> 32) * 0x1p-31f;  // half turns in [-1, 1)
            if (!(f == f)) x = __int_as_float(0x7fc00000);
            float sn, cs;
            sincospif(x, &sn, &cs);
            turn[i] = make_float2(cs, sn);
        }
        __syncthreads();
    }
#pragma unroll
    for (int u = 0; u < UP; ++u) {
        const int r = first + u * rows;
        const bool live = r < a.Hq + a.Hk, is_q = r < a.Hq;
        float x[8];
        if (live) {
            unpack8(raw[u], x);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = 0.f;
        }
        const float *w = is_q ? a.q_weight : a.k_weight;
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if (live && w) {
            const float inv = rms_inv(fmaf(ss, 1.0f / D, a.eps));
            const float4 w0 = ld_plain(reinterpret_cast<const float4 *>(w + c0)),
                         w1 = ld_plain(reinterpret_cast<const float4 *>(w + c0) + 1);
            const float wv[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = x[i] * inv * wv[i];
        }
        if constexpr (INTER) {  // pairs of neighbouring channels
            if (c0 < 2 * a.half) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 cs = turn[4 * ln + i];
                    const float p = x[2 * i], q = x[2 * i + 1];
                    x[2 * i] = p * cs.x - q * cs.y;
                    x[2 * i + 1] = q * cs.x + p * cs.y;
                }
            }
        } else {  // channel i with channel i + R/2
            const int step = a.half / 8, at = ln < step ? ln + step : ln < 2 * step ? ln - step : ln;
            float other[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) other[i] = __shfl_sync(0xffffffffu, x[i], at, LPR);
            if (c0 < 2 * a.half) {
                const int p0 = ln < step ? c0 : c0 - a.half;
                const float sign = ln < step ? -1.f : 1.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float2 cs = turn[p0 + i];
                    x[i] = x[i] * cs.x + sign * other[i] * cs.y;
                }
            }
        }
        if (!live) continue;
        if (is_q) store8(static_cast<T *>(a.q_out) + t * a.qo_stride + (int64_t)r * D + c0, x);
        else store8(static_cast<T *>(a.k_out) + t * a.ko_stride + (int64_t)(r - a.Hq) * D + c0, x);
    }
}

template <int D, typename T, bool INTER>
static kda_status launch_rope(const RopeArgs &a, int64_t T_, cudaStream_t s) {
    // Many tokens: a CTA takes a whole token with up to four rows a thread, so that a thread has that many
    // loads in flight and the angles are formed once. Few tokens: one row a thread, for latency.
    constexpr int LPR = D / 8, MOST = 512 / LPR;
    const int all = a.Hq + a.Hk;
    int up = 1, rows = 0;
    if (T_ > 2 * current_sms()) {
        up = all <= MOST ? 1 : all <= 2 * MOST ? 2 : 4;
        if (all > 16 && up < 2) up = 2;
    }
    const int cap = up == 1 ? 256 / LPR : MOST;
    rows = (all + up - 1) / up;
    if (rows > cap) rows = cap;
    const int nt = (rows * LPR + 31) / 32 * 32;
    rows = nt / LPR;
    const unsigned ny = (unsigned)((all + up * rows - 1) / (up * rows));
    const dim3 grid((unsigned)T_, ny);
    if (up == 1) launch_dependent(qk_norm_rope_kernel<D, T, INTER, 1>, grid, dim3(nt), 0, s, a);
    else if (up == 2) launch_dependent(qk_norm_rope_kernel<D, T, INTER, 2>, grid, dim3(nt), 0, s, a);
    else launch_dependent(qk_norm_rope_kernel<D, T, INTER, 4>, grid, dim3(nt), 0, s, a);
    return check_launch("qk_norm_rope_kernel");
}

template <typename T, bool INTER>
static kda_status dispatch_rope(int D, const RopeArgs &a, int64_t T_, cudaStream_t s) {
    switch (D) {
    case 16: return launch_rope<16, T, INTER>(a, T_, s);
    case 32: return launch_rope<32, T, INTER>(a, T_, s);
    case 64: return launch_rope<64, T, INTER>(a, T_, s);
    default: return launch_rope<128, T, INTER>(a, T_, s);
    }
}

}  // namespace kda

using namespace kda;

extern "C" kda_status kda_qk_norm_rope(const void *q, const void *k, void *q_out, void *k_out, const float *q_weight,
                                       const float *k_weight, const int64_t *positions, const double *inv_freq,
                                       int64_t T, int Hq, int Hk, int D, int R, int64_t q_stride, int64_t k_stride,
                                       int64_t q_out_stride, int64_t k_out_stride, int interleaved, float eps,
                                       kda_dtype dtype, kda_stream_t stream) {
    clear_detail();
    if (T < 0 || T > 0x7fffffffLL) return invalid("T must be in 0 .. 2^31 - 1");
    if (Hq < 1 || Hk < 0) return invalid("Hq must be >= 1 and Hk >= 0");
    if (!valid_head_dim(D)) return invalid("D must be one of 16, 32, 64, 128");
    if (Hq > 32768 || Hk > 32768) return invalid("Hq and Hk must be at most 32768");
    if (R < 0 || R > D || R % 16) return invalid("R must be a multiple of 16 in 0..D");
    if (interleaved != 0 && interleaved != 1) return invalid("interleaved must be 0 or 1");
    if (dtype != KDA_F32 && dtype != KDA_BF16) return invalid("dtype must be KDA_F32 or KDA_BF16");
    if (!(eps >= 0.f)) return invalid("eps must be >= 0");
    if (T == 0) return KDA_OK;
    kda_status st;
    if ((st = check_ptr(q, "q")) || (st = check_ptr(q_out, "q_out")) ||
        (Hk > 0 && ((st = check_ptr(k, "k")) || (st = check_ptr(k_out, "k_out")))) ||
        (q_weight && (st = check_ptr(q_weight, "q_weight"))) || (k_weight && (st = check_ptr(k_weight, "k_weight"))) ||
        (R > 0 && ((st = check_ptr(positions, "positions")) || (st = check_ptr(inv_freq, "inv_freq")))))
        return st;
    const int64_t unit = dtype == KDA_BF16 ? 8 : 4;
    if (T > 1 && (q_stride % unit || q_out_stride % unit || (Hk > 0 && (k_stride % unit || k_out_stride % unit))))
        return invalid("token strides must be multiples of 16 bytes");
    if (T > 1 && (q_stride < (int64_t)Hq * D || q_out_stride < (int64_t)Hq * D ||
                  (Hk > 0 && (k_stride < (int64_t)Hk * D || k_out_stride < (int64_t)Hk * D))))
        return invalid("token strides must be at least the heads times D");
    if ((q_out == q && q_out_stride != q_stride && T > 1) || (Hk > 0 && k_out == k && k_out_stride != k_stride && T > 1))
        return invalid("in place, the strides must agree");
    if (Hk > 0 && (q_out == k_out || q_out == k || k_out == q))
        return invalid("q_out may alias only q, k_out only k");
    if ((st = bind_stream_device(stream))) return st;
    const RopeArgs a = {q, k, q_out, k_out, q_weight, k_weight, positions, inv_freq, q_stride, k_stride, q_out_stride,
                        k_out_stride, Hq, Hk, R / 2, eps};
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (dtype == KDA_BF16)
        return interleaved ? dispatch_rope<__nv_bfloat16, true>(D, a, T, s) : dispatch_rope<__nv_bfloat16, false>(D, a, T, s);
    return interleaved ? dispatch_rope<float, true>(D, a, T, s) : dispatch_rope<float, false>(D, a, T, s);
}
