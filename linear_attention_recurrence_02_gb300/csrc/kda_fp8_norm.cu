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
#include <string>

#include "kda_fp8.cuh"

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
                                                               const float *__restrict__ w, TR *sum_out,
                                                               uint8_t *__restrict__ y, float *__restrict__ scales,
                                                               int64_t T, int N, float eps) {
    __shared__ float red[32];
    const int nv = N / 8, lane = threadIdx.x & 31;
    const int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    const bool live = t < T;
    const int64_t row = t * (int64_t)N;
    float h[VPT][8];
    float ss = 0.f;
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
    const float inv = rms_inv(ss / (float)N + eps);
#pragma unroll
    for (int c = 0; c < VPT; ++c) {
        const int v = c * blockDim.x + threadIdx.x;
        const bool in = live && v < nv;
        if (in) {
            float wv[8];
            const float4 w0 = __ldg(reinterpret_cast<const float4 *>(w + 8 * v));
            const float4 w1 = __ldg(reinterpret_cast<const float4 *>(w + 8 * v) + 1);
            wv[0] = w0.x; wv[1] = w0.y; wv[2] = w0.z; wv[3] = w0.w;
            wv[4] = w1.x; wv[5] = w1.y; wv[6] = w1.z; wv[7] = w1.w;
#pragma unroll
            for (int i = 0; i < 8; ++i) h[c][i] = h[c][i] * inv * wv[i];
        }
        const float m = block_amax(h[c]);
        if (in) {
            __stcs(reinterpret_cast<uint2 *>(y + row + 8 * v), codes8(h[c], QMAX / m));
            if ((v & 15) == 0) scales[(int64_t)(v >> 4) * T + t] = m / QMAX;
        }
    }
}

template <typename TX, typename TR, bool RES>
static kda_status launch_add(const void *x, const void *res, const float *w, void *sum_out, void *y, float *scales,
                             int64_t T, int N, float eps, cudaStream_t s) {
    const int nv = N / 8;
    const int vpt = nv <= 1024 ? 1 : nv <= 2048 ? 2 : 4;
    const int nt = ((nv + vpt - 1) / vpt + 31) / 32 * 32;
    const int rows = nt >= 128 ? 1 : 128 / nt;
    const int64_t blocks = (T + rows - 1) / rows;
    if (blocks > 0x7fffffffLL) return invalid("T too large for one launch");
    const dim3 grid((unsigned)blocks), block((unsigned)nt, (unsigned)rows);
    auto go = [&](auto kern) {
        kern<<<grid, block, 0, s>>>(static_cast<const TX *>(x), static_cast<const TR *>(res), w,
                                    static_cast<TR *>(sum_out), static_cast<uint8_t *>(y), scales, T, N, eps);
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
// A half-warp owns one (token, block of 128 channels): 128 / D whole heads,
// D / 8 lanes each. The gate's activation is taken with the fast exponential
// and division (a few ulp, far below the 2^-4 step of e4m3).
template <int D, typename T, int ACT>
__global__ void __launch_bounds__(256) gated_rmsnorm_fp8_kernel(const T *__restrict__ o, const T *__restrict__ gate,
                                                                const float *__restrict__ w, uint8_t *__restrict__ y,
                                                                float *__restrict__ scales, int64_t Ttot, int C,
                                                                int nb, float eps) {
    const int ln = threadIdx.x & 15;
    const int64_t unit = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 4;  // t * nb + b
    const int64_t t = unit / nb;
    const int b = (int)(unit - t * nb), c = b * QBLOCK + 8 * ln;  // the lane's first channel of the token
    const bool in = t < Ttot && c < C;
    const int64_t at = t * C + c;
    float ov[8], gv[8], ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ov[i] = gv[i] = 0.f;
    if (in) {
        Raw8<T> ro, rg;
        load8(o + at, ro);
        load8(gate + at, rg);
        unpack8(ro, ov);
        unpack8(rg, gv);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(ov[i], ov[i], ss);
#pragma unroll
    for (int m = D / 16; m > 0; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
    const float inv = rms_inv(ss / (float)D + eps);
    const int j = (8 * ln) % D;
    const float4 w0 = __ldg(reinterpret_cast<const float4 *>(w + j)), w1 = __ldg(reinterpret_cast<const float4 *>(w + j) + 1);
    const float wv[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float sg = __fdividef(1.0f, 1.0f + __expf(-gv[i]));
        ov[i] = ov[i] * (wv[i] * inv) * (ACT == KDA_ACT_SILU ? gv[i] * sg : sg);
    }
    const float m = block_amax(ov);
    if (in) {
        __stcs(reinterpret_cast<uint2 *>(y + at), codes8(ov, QMAX / m));
        if (ln == 0) scales[(int64_t)b * Ttot + t] = m / QMAX;
    }
}

template <typename T, int ACT>
static kda_status dispatch_gated(int D, const void *o, const void *gate, const float *w, void *y, float *scales,
                                 int64_t Ttot, int H, float eps, cudaStream_t s) {
    const int C = H * D, nb = (C + QBLOCK - 1) / QBLOCK;
    const int64_t blocks = (Ttot * nb + 15) / 16;
    if (blocks > 0x7fffffffLL) return invalid("T*H*D too large for one launch");
    auto go = [&](auto kern) {
        kern<<<(unsigned)blocks, 256, 0, s>>>(static_cast<const T *>(o), static_cast<const T *>(gate), w,
                                              static_cast<uint8_t *>(y), scales, Ttot, C, nb, eps);
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
