// kda_qk_rope.cu -- RMSNorm of every query and key head and the rotation by their position, in one pass
// (kda_qk_norm_rope).
//
//   y = x / sqrt(mean x^2 + eps) * w;  then pair i of the first R channels turns by position * freq_i
//
// Bound by memory: each element is read and written once (in bf16 the issue slots come close behind). A row (token,
// head) is D / 8 lanes of eight channels, both channels of a pair in one lane, so the sum of squares is a shuffle
// reduction and the rotation needs none. A CTA owns one token, or several where they have few rows, and some or all of
// their heads: the R/2 sines and cosines of each are formed once per CTA, while the rows' loads are in flight.
//
// Angles: a position's turn is position * freq / 2 pi modulo 1. freq / 2 pi modulo 1 is formed as a 64-bit
// fraction (2^-64 turns a unit), so the product with an integer position wraps around exactly: the angle
// of position 2^31 is as good as that of position 1. Its upper 32 bits go to the sine and cosine as an fp32 number of
// half turns in [-1, 1], off by at most 2^-25 of one: 9.4e-8 radians.
#include <algorithm>
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

// (cos, sin) of pair i at position pos. The frequency's mantissa (53 bits) times 2^64 / 2 pi, shifted by its
// exponent, is the fraction of a turn in units of 2^-64, off by less than the frequency in radians: in integers,
// because this card has few units for 64-bit floating point (8192 tokens' angles took 5 us of them).
__device__ __forceinline__ float2 turn_of(const RopeArgs &a, int64_t pos, int i) {
    const uint64_t bits = (uint64_t)__double_as_longlong(a.freq[i]);
    const int e = (int)(bits >> 52) & 0x7ff;
    const uint64_t m = (bits & 0xfffffffffffffull) | (e ? 1ull << 52 : 0), C = 0x28be60db9391054aull;  // 2^64 / 2 pi
    const uint64_t hi = __umul64hi(m, C), lo = m * C;
    const int down = 1075 - max(e, 1);  // the value is m 2^-down
    uint64_t unit = down <= 0 ? (down > -64 ? lo << -down : 0)
                  : down < 64 ? (lo >> down) | (hi << (64 - down)) : down < 128 ? hi >> (down - 64) : 0;
    if (bits >> 63) unit = 0 - unit;
    const uint64_t phase = (uint64_t)pos * unit;
    float x = (float)(int32_t)(phase >> 32) * 0x1p-31f;  // half turns in [-1, 1]
    if (e == 0x7ff) x = __int_as_float(0x7fc00000);
    float sn, cs;
    sincospif(x, &sn, &cs);
    return make_float2(cs, sn);
}

// A row is D / 8 lanes of two vectors of four channels. Lane ln has pairs 4 ln .. 4 ln + 3, so that both channels of a
// pair are its own and its angles are the same in every row: neighbouring channels as pairs, eight channels from 8 ln
// on; channels i and i + R/2, four from 4 ln on and the four R/2 behind. Lanes past the pairs share out the channels that
// do not turn. (With eight neighbouring channels a lane throughout, partners came by eight shuffles and the angles
// from shared memory for every row: 8192 tokens, 64 + 8 heads of 128 in bf16, 102 us.)
struct Lane {
    int a, b;     // the two vectors' first channels
    bool turns;
};
template <bool INTER> __device__ __forceinline__ Lane lane_of(int ln, int half) {
    const bool turns = 4 * ln < half;
    if (INTER) return {8 * ln, 8 * ln + 4, turns};
    return turns ? Lane{4 * ln, half + 4 * ln, true} : Lane{8 * ln, 8 * ln + 4, false};
}

template <typename T> struct Raw4x2;
template <> struct Raw4x2<__nv_bfloat16> { uint2 a, b; };
template <> struct Raw4x2<float> { float4 a, b; };
template <typename T> __device__ __forceinline__ void load_row(const T *row, const Lane &l, Raw4x2<T> &r) {
    using V = decltype(r.a);
    r.a = __ldcs(reinterpret_cast<const V *>(row + l.a));
    r.b = __ldcs(reinterpret_cast<const V *>(row + l.b));
}
__device__ __forceinline__ void unpack(const Raw4x2<__nv_bfloat16> &r, float2 (&x)[4]) {
    const uint32_t w[4] = {r.a.x, r.a.y, r.b.x, r.b.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}
__device__ __forceinline__ void unpack(const Raw4x2<float> &r, float2 (&x)[4]) {
    x[0] = make_float2(r.a.x, r.a.y);
    x[1] = make_float2(r.a.z, r.a.w);
    x[2] = make_float2(r.b.x, r.b.y);
    x[3] = make_float2(r.b.z, r.b.w);
}
__device__ __forceinline__ void store_row(__nv_bfloat16 *row, const Lane &l, const float2 (&x)[4]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(x[i].x, x[i].y);
        memcpy(&w[i], &v, 4);
    }
    __stcs(reinterpret_cast<uint2 *>(row + l.a), make_uint2(w[0], w[1]));
    __stcs(reinterpret_cast<uint2 *>(row + l.b), make_uint2(w[2], w[3]));
}
__device__ __forceinline__ void store_row(float *row, const Lane &l, const float2 (&x)[4]) {
    __stcs(reinterpret_cast<float4 *>(row + l.a), make_float4(x[0].x, x[0].y, x[1].x, x[1].y));
    __stcs(reinterpret_cast<float4 *>(row + l.b), make_float4(x[2].x, x[2].y, x[3].x, x[3].y));
}

// The norm (with `w`, the row's weights in shared memory, or none) and the turn of a row; all lanes call.
template <int D, bool INTER>
__device__ __forceinline__ void norm_and_turn(float2 (&x)[4], const float *w, const Lane &l, const float2 (&cs)[4], float eps) {
    float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < 4; ++i) s2 = __ffma2_rn(x[i], x[i], s2);
    float ss = s2.x + s2.y;
#pragma unroll
    for (int o = D / 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (w) {  // rows of q and of k may share a warp, one of them without weights
        const float inv = rms_inv(fmaf(ss, 1.0f / D, eps));
        const float4 wa = *reinterpret_cast<const float4 *>(w + l.a), wb = *reinterpret_cast<const float4 *>(w + l.b);
        const float2 wv[4] = {make_float2(wa.x, wa.y), make_float2(wa.z, wa.w), make_float2(wb.x, wb.y), make_float2(wb.z, wb.w)};
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = __fmul2_rn(__fmul2_rn(x[i], make_float2(inv, inv)), wv[i]);
    }
    if (!l.turns) return;
    if (INTER) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            x[i] = make_float2(x[i].x * cs[i].x - x[i].y * cs[i].y, x[i].y * cs[i].x + x[i].x * cs[i].y);
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float2 c = make_float2(cs[2 * i].x, cs[2 * i + 1].x), s = make_float2(cs[2 * i].y, cs[2 * i + 1].y);
            const float2 p = x[i], q = x[2 + i];
            x[i] = __ffma2_rn(p, c, __fmul2_rn(q, make_float2(-s.x, -s.y)));
            x[2 + i] = __ffma2_rn(q, c, __fmul2_rn(p, s));
        }
    }
}

// A CTA has `tokens` tokens, `slots` rows of D / 8 lanes for each, and each lane UP rows of its token: the token's
// rows (queries' heads, then keys') (blockIdx.y * UP + u) * slots + its slot. ONE: a single token, with no division before
// the loads. 8192 tokens, 64 + 8 heads of 128 in bf16: 59 us, 5.1 TB/s (with the division 71; with 40 registers 67,
// with 59 as the compiler likes it 61, and 54 instead of 45 for 4096 tokens of 96 + 8 heads; tokens streamed through
// shared memory by persistent CTAs 71: the rows' arithmetic needs more warps than that leaves; several tokens one after
// another in a CTA, the next one's rows loaded ahead, 62; lanes of two 16-byte vectors, half as many, 65). What bounds it
// is issue slots (73 % used; ALU 45 %) and a CTA's chain of loads, angles, barrier and stores with the warps that
// registers allow: fp32 rows, twice the bytes behind each angle, move at 6.5 TB/s.
template <int D, typename T, bool INTER, int UP, bool ONE>
__global__ void __maxnreg__(sizeof(T) == 2 ? 48 : 64) qk_norm_rope_kernel(const RopeArgs a, int64_t T_, int many, int slots) {
    constexpr int LPR = D / 8;
    extern __shared__ __align__(16) float2 turn[];  // [tokens][half] (cos, sin)
    __shared__ __align__(16) float w[2][D];
    const int tokens = ONE ? 1 : many;
    const int ln = threadIdx.x % LPR, group = threadIdx.x / LPR, tk = ONE ? 0 : group / slots, slot = group - tk * slots;
    const int64_t t0 = (int64_t)blockIdx.x * tokens, t = t0 + tk;
    const int first = blockIdx.y * UP * slots + slot, all = ONE ? a.Hq + a.Hk : tk < tokens && t < T_ ? a.Hq + a.Hk : 0;
    const Lane l = lane_of<INTER>(ln, a.half);
    dependent_launch();
    Raw4x2<T> raw[UP];
#pragma unroll
    for (int u = 0; u < UP; ++u) {
        const int r = first + u * slots;
        if (r >= all) continue;
        if (r < a.Hq) load_row(static_cast<const T *>(a.q) + t * a.q_stride + (int64_t)r * D, l, raw[u]);
        else load_row(static_cast<const T *>(a.k) + t * a.k_stride + (int64_t)(r - a.Hq) * D, l, raw[u]);
    }
    for (int i = threadIdx.x; i < tokens * a.half; i += blockDim.x) {
        const int k = ONE ? 0 : i / a.half;
        if (ONE || t0 + k < T_) turn[i] = turn_of(a, a.positions[t0 + k], i - k * a.half);
    }
    for (int i = threadIdx.x; i < 2 * D; i += blockDim.x) {
        const float *from = i < D ? a.q_weight : a.k_weight;
        if (from) w[i / D][i % D] = ld_plain(from + i % D);
    }
    __syncthreads();
    float2 cs[4] = {};
    if (l.turns && all) {
#pragma unroll
        for (int i = 0; i < 4; ++i) cs[i] = turn[tk * a.half + 4 * ln + i];
    }
#pragma unroll
    for (int u = 0; u < UP; ++u) {
        const int r = first + u * slots;
        const bool live = r < all, is_q = r < a.Hq;
        float2 x[4] = {};
        if (live) unpack(raw[u], x);
        norm_and_turn<D, INTER>(x, (is_q ? a.q_weight : a.k_weight) ? w[is_q ? 0 : 1] : nullptr, l, cs, a.eps);
        if (!live) continue;
        if (is_q) store_row(static_cast<T *>(a.q_out) + t * a.qo_stride + (int64_t)r * D, l, x);
        else store_row(static_cast<T *>(a.k_out) + t * a.ko_stride + (int64_t)(r - a.Hq) * D, l, x);
    }
}

template <int D, typename T, bool INTER>
static kda_status launch_rope(const RopeArgs &a, int64_t T_, cudaStream_t s) {
    // Many tokens: up to four rows a lane, so that each has that many loads in flight and the angles are formed once a
    // token, and several tokens a CTA where they have few rows. Few tokens: one row a lane, for latency.
    constexpr int LPR = D / 8, MOST = 512 / LPR;
    const int all = a.Hq + a.Hk;
    const int up = T_ <= 2 * current_sms() || all <= 2 ? 1 : all <= 4 ? 2 : 4;
    const int slots = std::min((all + up - 1) / up, up == 1 ? 256 / LPR : MOST);
    const int tokens = T_ <= 2 * current_sms() ? 1 : std::max(1, 256 / (slots * LPR));
    const int nt = (tokens * slots * LPR + 31) / 32 * 32;
    const dim3 grid((unsigned)((T_ + tokens - 1) / tokens), (unsigned)((all + up * slots - 1) / (up * slots)));
    const size_t smem = (size_t)tokens * a.half * sizeof(float2);
    auto go = [&](auto kern) { launch_dependent(kern, grid, dim3(nt), smem, s, a, T_, tokens, slots); };
    if (up == 1) tokens == 1 ? go(qk_norm_rope_kernel<D, T, INTER, 1, true>) : go(qk_norm_rope_kernel<D, T, INTER, 1, false>);
    else if (up == 2) go(qk_norm_rope_kernel<D, T, INTER, 2, false>);
    else tokens == 1 ? go(qk_norm_rope_kernel<D, T, INTER, 4, true>) : go(qk_norm_rope_kernel<D, T, INTER, 4, false>);
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
