// kda_fp8_norm.cu -- RMSNorms whose output leaves in 8 bits: e4m3 codes with
// one fp32 scale for each token and block of 128 channels, the operand of
// kda_fp8_linear.
//
//   kda_add_rmsnorm_fp8    h = x + residual, y = h / sqrt(mean h^2 + eps) * w
//   kda_gated_rmsnorm_fp8  the output epilogue of kda_gated_rmsnorm
//                          ("为什么 Kimi K3 敢把 KV Cache 扔掉？一篇讲透 GPT-2 到 K3 的
//                          架构进化", section 6: the gate that scales the output's features)
//
// Both are bound by HBM: every input element is read once, every output
// written once. A thread owns 8 consecutive channels, so the 128 channels of
// a scale lie in 16 neighbouring lanes and the block's maximum is four
// shuffles; the row never leaves the registers between its sum of squares
// and its codes.
//
// Both are programmatic dependent launches that wait for the kernel before
// them first thing, then let the kernel behind them start: a kda_fp8_linear
// that reads their output sets itself up and prefetches its weights meanwhile.
#include <string>

#include "kda_fp8.cuh"
#include "kda_prefill.cuh"

namespace kda {

// ---------------------------------------------------------------- residual add + RMSNorm
// A row of N channels is held by blockDim.x threads, VPT vectors of 8
// channels each (vector c * blockDim.x + t: neighbouring lanes hold
// neighbouring channels); blockDim.y rows per CTA. The sum of squares is a
// shuffle reduction per warp, then one over the row's warps, in a fixed
// order: the same inputs give the same bits. The norm takes the fp32 sum
// x + residual itself, not its rounding to sum_out's type.
template <typename TX, typename TR, bool RES, int VPT>
__global__ void __launch_bounds__(1024) add_rmsnorm_fp8_kernel(const TX *x, const TR *res,
                                                               const float *w, TR *sum_out,
                                                               uint8_t *__restrict__ y, float *__restrict__ scales,
                                                               int64_t T, int N, float inv_n, float eps) {
    __shared__ float red[32];
    const int nv = N / 8, lane = threadIdx.x & 31;
    const int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    const bool live = t < T;
    const int64_t row = t * (int64_t)N;
    float h[VPT][8];
    float ss = 0.f;
    dependent_launch();
    Raw8<TX> rx[VPT];
    Raw8<TR> rr[VPT];
#pragma unroll
    for (int c = 0; c < VPT; ++c) {
        const int v = c * blockDim.x + threadIdx.x;
        if (live && v < nv) {
            load8(x + row + 8 * v, rx[c]);
            if constexpr (RES) load8(res + row + 8 * v, rr[c]);
        }
    }
#pragma unroll
    for (int c = 0; c < VPT; ++c) {
        const int v = c * blockDim.x + threadIdx.x;
        const bool in = live && v < nv;
        if (in) {
            unpack8(rx[c], h[c]);
            if constexpr (RES) {
                float r[8];
                unpack8(rr[c], r);
#pragma unroll
                for (int i = 0; i < 8; ++i) h[c][i] += r[i];
            }
            if (sum_out) store8(sum_out + row + 8 * v, h[c]);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (!in) h[c][i] = 0.f;
            ss = fmaf(h[c][i], h[c][i], ss);
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const int wpr = blockDim.x / 32;  // warps per row; wpr * blockDim.y <= 32
    if (wpr > 1) {
        if (lane == 0) red[threadIdx.y * wpr + threadIdx.x / 32] = ss;
        __syncthreads();
        ss = lane < wpr ? red[threadIdx.y * wpr + lane] : 0.f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    }
    const float inv = rms_inv(fmaf(ss, inv_n, eps));
#pragma unroll
    for (int c = 0; c < VPT; ++c) {
        const int v = c * blockDim.x + threadIdx.x;
        const bool in = live && v < nv;
        if (in) {
            float wv[8];
            const float4 w0 = ld_plain(reinterpret_cast<const float4 *>(w + 8 * v));
            const float4 w1 = ld_plain(reinterpret_cast<const float4 *>(w + 8 * v) + 1);
            wv[0] = w0.x; wv[1] = w0.y; wv[2] = w0.z; wv[3] = w0.w;
            wv[4] = w1.x; wv[5] = w1.y; wv[6] = w1.z; wv[7] = w1.w;
#pragma unroll
            for (int i = 0; i < 8; ++i) h[c][i] = h[c][i] * inv * wv[i];
        }
        const float m = block_amax(h[c]);
        if (in) {
            __stcs(reinterpret_cast<uint2 *>(y + row + 8 * v), codes8(h[c], block_inv(m)));
            if ((v & 15) == 0) scales[(int64_t)(v >> 4) * T + t] = block_scale(m);
        }
    }
}

template <typename TX, typename TR, bool RES>
static kda_status launch_add(const void *x, const void *res, const float *w, void *sum_out, void *y, float *scales,
                             int64_t T, int N, float eps, cudaStream_t s) {
    // Many rows: about 256 threads a row (512 where an input is fp32, whose vectors take twice the
    // registers), so that an SM has several rows in flight and one row's reductions hide behind another's
    // loads. Few rows: as many threads a row as it has vectors, for latency. (8192 x 8192 bf16: 72 us at
    // four vectors a thread, 82 at two, 90 at one; fp32: 137 at four, 127 at two. 4096 x 4096 bf16: 21.5
    // at four, 20.6 at two.)
    const int nv = N / 8, sms = current_sms();
    const int most = T <= 2 * sms ? 1024 : sizeof(TX) + (RES ? sizeof(TR) : 0) > 4 ? 512 : 256;
    const int vpt = nv <= most ? 1 : nv <= 2 * most ? 2 : 4;
    const int nt = ((nv + vpt - 1) / vpt + 31) / 32 * 32;
    const int rows = nt >= 128 ? 1 : 128 / nt;
    const int64_t blocks = (T + rows - 1) / rows;
    if (blocks > 0x7fffffffLL) return invalid("T too large for one launch");
    auto go = [&](auto kern) {
        launch_dependent(kern, dim3((unsigned)blocks), dim3((unsigned)nt, (unsigned)rows), 0, s, static_cast<const TX *>(x),
                         static_cast<const TR *>(res), w, static_cast<TR *>(sum_out), static_cast<uint8_t *>(y),
                         scales, T, N, 1.0f / (float)N, eps);
    };
    if (vpt == 1) go(add_rmsnorm_fp8_kernel<TX, TR, RES, 1>);
    else if (vpt == 2) go(add_rmsnorm_fp8_kernel<TX, TR, RES, 2>);
    else go(add_rmsnorm_fp8_kernel<TX, TR, RES, 4>);
    return check_launch("add_rmsnorm_fp8_kernel");
}

template <typename TX>
static kda_status dispatch_add(bool res_bf16, const void *x, const void *res, const float *w, void *sum_out, void *y,
                               float *scales, int64_t T, int N, float eps, cudaStream_t s) {
    if (res_bf16)
        return res ? launch_add<TX, __nv_bfloat16, true>(x, res, w, sum_out, y, scales, T, N, eps, s)
                   : launch_add<TX, __nv_bfloat16, false>(x, res, w, sum_out, y, scales, T, N, eps, s);
    return res ? launch_add<TX, float, true>(x, res, w, sum_out, y, scales, T, N, eps, s)
               : launch_add<TX, float, false>(x, res, w, sum_out, y, scales, T, N, eps, s);
}

// ---------------------------------------------------------------- gated RMSNorm
// Eight lanes own one (token, block of 128 channels), 16 channels each, so a
// head is D / 16 lanes and a shuffle reduction has at most three steps. Issue
// slots bound the bf16 form, so the per-element work is kept short: products
// two at a time (f32x2), the gate's activation by the hardware exponential
// and reciprocal without their handling of denormals (a few ulp, far below the
// 2^-4 step of e4m3; a gate below about -87 closes fully), three-way maxima.
// 4096 x 96 heads x 128, bf16: 40.1 us (41.1 without the bound to ten blocks
// an SM; 41.2 with blocks of 256 threads, 50.3 with 64). The bound suits that
// form: bf16 SiLU takes 43.2 us with it and 41.5 without, fp32 74.7 and 70.5 (a
// few registers spill), fp32 SiLU 71.5 and 71.4. When it took 41.4 us, a
// persistent grid that loads a unit ahead took 44.1 at best, and 8 channels a
// lane with one product at a time 56.5.
constexpr int GATED_NT = 128;
__device__ __forceinline__ float sigmoid_fast(float z) {
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(z * -1.4426950408889634f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
    return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

template <int D, typename T, int ACT>
__global__ void __launch_bounds__(GATED_NT, 10) gated_rmsnorm_fp8_kernel(const T *o, const T *gate,
                                                                const float *w, uint8_t *__restrict__ y,
                                                                float *__restrict__ scales, int64_t Ttot, int C,
                                                                int nb, float eps) {
    const int ln = threadIdx.x & 7;
    const int64_t unit = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 3;  // t * nb + b
    const int64_t t = unit / nb;
    const int b = (int)(unit - t * nb), c = b * QBLOCK + 16 * ln;  // the lane's first channel of the token
    const bool in = t < Ttot && c < C;
    const int64_t at = t * C + c;
    dependent_launch();
    Raw8<T> ro[2], rg[2];
    if (in) {
        load8(o + at, ro[0]);
        load8(o + at + 8, ro[1]);
        load8(gate + at, rg[0]);
        load8(gate + at + 8, rg[1]);
    }
    const int j = (16 * ln) % D;
    float2 v[8], ss = make_float2(0.f, 0.f);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        float f[8];
        if (in) {
            unpack8(ro[q], f);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[4 * q + i] = make_float2(f[2 * i], f[2 * i + 1]);
            ss = __ffma2_rn(v[4 * q + i], v[4 * q + i], ss);
        }
    }
    float sum = ss.x + ss.y;
#pragma unroll
    for (int m = D / 32; m > 0; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
    const float inv = rms_inv(fmaf(sum, 1.0f / (float)D, eps));
    float m = QAMAX_MIN;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        float z[8];
        if (in) {
            unpack8(rg[q], z);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) z[i] = 0.f;
        }
        const float4 w0 = ld_plain(reinterpret_cast<const float4 *>(w + j + 8 * q)),
                     w1 = ld_plain(reinterpret_cast<const float4 *>(w + j + 8 * q) + 1);
        const float2 wv[4] = {make_float2(w0.x, w0.y), make_float2(w0.z, w0.w), make_float2(w1.x, w1.y),
                              make_float2(w1.z, w1.w)};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float2 g = make_float2(sigmoid_fast(z[2 * i]), sigmoid_fast(z[2 * i + 1]));
            if (ACT == KDA_ACT_SILU) g = __fmul2_rn(g, make_float2(z[2 * i], z[2 * i + 1]));
            float2 &x = v[4 * q + i];
            x = __fmul2_rn(__fmul2_rn(x, __fmul2_rn(wv[i], make_float2(inv, inv))), g);
            m = max3(m, fabsf(x.x), fabsf(x.y));
        }
    }
#pragma unroll
    for (int k = 4; k > 0; k >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, k));
    if (in) {
        const float bi = block_inv(m);
        uint32_t code[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 p = __fmul2_rn(v[2 * i], make_float2(bi, bi)), r = __fmul2_rn(v[2 * i + 1], make_float2(bi, bi));
            code[i] = __nv_cvt_float2_to_fp8x2(p, __NV_SATFINITE, __NV_E4M3) |
                      ((uint32_t)__nv_cvt_float2_to_fp8x2(r, __NV_SATFINITE, __NV_E4M3) << 16);
        }
        __stcs(reinterpret_cast<uint4 *>(y + at), make_uint4(code[0], code[1], code[2], code[3]));
        if (ln == 0) scales[(int64_t)b * Ttot + t] = block_scale(m);
    }
}

template <typename T, int ACT>
static kda_status dispatch_gated(int D, const void *o, const void *gate, const float *w, void *y, float *scales,
                                 int64_t Ttot, int H, float eps, cudaStream_t s) {
    const int C = H * D, nb = (C + QBLOCK - 1) / QBLOCK;
    const int64_t blocks = (Ttot * nb + GATED_NT / 8 - 1) / (GATED_NT / 8);
    if (blocks > 0x7fffffffLL) return invalid("T*H*D too large for one launch");
    auto go = [&](auto kern) {
        launch_dependent(kern, dim3((unsigned)blocks), dim3(GATED_NT), 0, s, static_cast<const T *>(o), static_cast<const T *>(gate),
                         w, static_cast<uint8_t *>(y), scales, Ttot, C, nb, eps);
    };
    switch (D) {
    case 16: go(gated_rmsnorm_fp8_kernel<16, T, ACT>); break;
    case 32: go(gated_rmsnorm_fp8_kernel<32, T, ACT>); break;
    case 64: go(gated_rmsnorm_fp8_kernel<64, T, ACT>); break;
    default: go(gated_rmsnorm_fp8_kernel<128, T, ACT>); break;
    }
    return check_launch("gated_rmsnorm_fp8_kernel");
}

}  // namespace kda

using namespace kda;

extern "C" kda_status kda_add_rmsnorm_fp8(const void *x, const void *residual, const float *weight, void *sum_out,
                                          void *y, float *scales, int64_t T, int N, kda_dtype dtype,
                                          kda_dtype res_dtype, float eps, kda_stream_t stream) {
    clear_detail();
    if (T < 0) return invalid("T must be >= 0");
    if (N < 16 || N % 16 != 0 || N > 32768) return invalid("N must be a multiple of 16 in 16..32768");
    if (dtype != KDA_F32 && dtype != KDA_BF16) return invalid("dtype must be KDA_F32 or KDA_BF16");
    if (res_dtype != KDA_F32 && res_dtype != KDA_BF16) return invalid("res_dtype must be KDA_F32 or KDA_BF16");
    if (!(eps >= 0.f)) return invalid("eps must be >= 0");
    if (T == 0) return KDA_OK;
    kda_status st;
    if ((st = check_ptr(x, "x")) || (st = check_ptr(weight, "weight")) || (st = check_ptr(y, "y")) ||
        (st = check_ptr(scales, "scales")) || (residual && (st = check_ptr(residual, "residual"))) ||
        (sum_out && (st = check_ptr(sum_out, "sum_out"))))
        return st;
    if (sum_out == x && sum_out && dtype != res_dtype)
        return invalid("sum_out may be x only where both have the same type");
    if (y == x || y == residual || y == sum_out || y == scales || y == weight)
        return invalid("y must not alias another argument");
    if (scales == x || scales == residual || scales == sum_out || scales == weight || sum_out == weight)
        return invalid("scales and sum_out must not alias other arguments");
    if ((st = bind_stream_device(stream))) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (dtype == KDA_BF16)
        return dispatch_add<__nv_bfloat16>(res_dtype == KDA_BF16, x, residual, weight, sum_out, y, scales, T, N, eps, s);
    return dispatch_add<float>(res_dtype == KDA_BF16, x, residual, weight, sum_out, y, scales, T, N, eps, s);
}

extern "C" kda_status kda_gated_rmsnorm_fp8(const void *o, const void *gate, const float *weight, void *y,
                                            float *scales, int64_t T, int H, int D, kda_dtype dtype,
                                            kda_gate_act act, float eps, kda_stream_t stream) {
    clear_detail();
    if (T < 0) return invalid("T must be >= 0");
    if (H < 1) return invalid("H must be >= 1");
    if (!valid_head_dim(D)) return invalid("D must be one of 16, 32, 64, 128");
    if ((long long)H * D > 0x7fffff00LL) return invalid("H*D too large");
    if (dtype != KDA_F32 && dtype != KDA_BF16) return invalid("dtype must be KDA_F32 or KDA_BF16");
    if (act != KDA_ACT_SIGMOID && act != KDA_ACT_SILU) return invalid("act must be KDA_ACT_SIGMOID or KDA_ACT_SILU");
    if (!(eps >= 0.f)) return invalid("eps must be >= 0");
    if (T == 0) return KDA_OK;
    kda_status st;
    if ((st = check_ptr(o, "o")) || (st = check_ptr(gate, "gate")) || (st = check_ptr(weight, "weight")) ||
        (st = check_ptr(y, "y")) || (st = check_ptr(scales, "scales")))
        return st;
    if (y == o || y == gate || y == scales || y == weight || scales == o || scales == gate || scales == weight)
        return invalid("y and scales must not alias other arguments");
    if ((st = bind_stream_device(stream))) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (dtype == KDA_BF16)
        return act == KDA_ACT_SILU
                   ? dispatch_gated<__nv_bfloat16, KDA_ACT_SILU>(D, o, gate, weight, y, scales, T, H, eps, s)
                   : dispatch_gated<__nv_bfloat16, KDA_ACT_SIGMOID>(D, o, gate, weight, y, scales, T, H, eps, s);
    return act == KDA_ACT_SILU ? dispatch_gated<float, KDA_ACT_SILU>(D, o, gate, weight, y, scales, T, H, eps, s)
                               : dispatch_gated<float, KDA_ACT_SIGMOID>(D, o, gate, weight, y, scales, T, H, eps, s);
}
