// kda_proj.cu -- the layer's way out in one call: attention output, gated
// RMSNorm in 8 bits, output projection.
//
// kda_shortconv_decode_step_proj and kda_chunk_prefill_proj run the decode
// step or the prefill into a workspace, kda_gated_rmsnorm_fp8 over its output
// and kda_fp8_linear with the projection's weight. The codes and scales
// between the last two stay in the workspace (at decode sizes, in L2). Every
// argument is checked before the first launch; the norm and the product are
// dependent launches, so the product's weights are on their way into L2 while
// the norm runs.
#include <string>

#include "kda_common.cuh"

namespace kda {

static size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }

// Workspace of the way out: the attention output (sized for fp32, so that one
// size serves both types), its codes and its scales.
struct ProjWs {
    uint8_t *o, *codes;
    float *scales;
};
static size_t proj_layout(int64_t T, int H, int D, uint8_t *base, ProjWs *ws) {
    const size_t e = (size_t)T * H * D, nb = ((size_t)H * D + 127) / 128;
    const size_t o = up256(e * 4), codes = up256(e), scales = up256(nb * (size_t)T * 4);
    if (ws) {
        ws->o = base;
        ws->codes = base + o;
        ws->scales = reinterpret_cast<float *>(base + o + codes);
    }
    return o + codes + scales;
}

// The checks of what the two later calls take; the first call checks its own.
static kda_status check_proj(const void *out_gate, const float *norm_weight, const void *proj, const float *proj_scales,
                             const void *y, int64_t T, int H, int D, int Nout, kda_dtype dtype, kda_gate_act act,
                             float norm_eps, const void *workspace, size_t have, size_t need) {
    if (H < 1) return invalid("H must be >= 1");
    if (!valid_head_dim(D)) return invalid("D must be one of 16, 32, 64, 128");
    if ((long long)H * D > 0x7fffff00LL) return invalid("H*D too large");
    if (T < 0 || T > 0x7fffff00LL) return invalid("the number of tokens must be in 0..2^31-256");
    if (Nout < 1 || Nout > 0x7fffff00) return invalid("Nout must be in 1..2^31-256");
    if (dtype != KDA_F32 && dtype != KDA_BF16) return invalid("dtype must be KDA_F32 or KDA_BF16");
    if (act != KDA_ACT_SIGMOID && act != KDA_ACT_SILU) return invalid("act must be KDA_ACT_SIGMOID or KDA_ACT_SILU");
    if (!(norm_eps >= 0.f)) return invalid("norm_eps must be >= 0");
    if (have < need) return invalid("workspace too small");
    kda_status st;
    if (need && (st = check_ptr(workspace, "workspace"))) return st;
    if (T == 0) return KDA_OK;
    if ((st = check_ptr(out_gate, "out_gate")) || (st = check_ptr(norm_weight, "norm_weight")) ||
        (st = check_ptr(proj, "proj")) || (st = check_ptr(proj_scales, "proj_scales")) || (st = check_ptr(y, "y")))
        return st;
    if (y == out_gate || y == norm_weight || y == proj || y == proj_scales || y == workspace)
        return invalid("y must not alias another argument");
    return KDA_OK;
}

static kda_status way_out(const ProjWs &ws, const void *out_gate, const float *norm_weight, const void *proj,
                          const float *proj_scales, void *y, int64_t T, int H, int D, int Nout, kda_dtype dtype,
                          kda_gate_act act, float norm_eps, kda_stream_t stream) {
    kda_status st = kda_gated_rmsnorm_fp8(ws.o, out_gate, norm_weight, ws.codes, ws.scales, T, H, D, dtype, act,
                                          norm_eps, stream);
    if (st != KDA_OK) return st;
    const int64_t K = (int64_t)H * D;
    return kda_fp8_linear(ws.codes, ws.scales, proj, proj_scales, y, T, Nout, (int)K, K, K, Nout, dtype, stream);
}

}  // namespace kda

using namespace kda;

extern "C" size_t kda_shortconv_decode_step_proj_workspace_bytes(int B, int H, int D) {
    if (B <= 0 || H < 1 || D < 1) return 0;
    return proj_layout(B, H, D, nullptr, nullptr);
}

extern "C" kda_status kda_shortconv_decode_step_proj(const void *x, void *ring, const float *w, const float *g,
                                                     const float *beta, float *state, const void *out_gate,
                                                     const float *norm_weight, const void *proj,
                                                     const float *proj_scales, void *y, int B, int H, int D, int Nout,
                                                     kda_dtype dtype, kda_gate gate, kda_gate_act act, float l2_eps,
                                                     float norm_eps, unsigned flags, void *workspace,
                                                     size_t workspace_bytes, kda_stream_t stream) {
    clear_detail();
    if (B < 0) return invalid("B must be >= 0");
    const size_t need = kda_shortconv_decode_step_proj_workspace_bytes(B, H, D);
    kda_status st = check_proj(out_gate, norm_weight, proj, proj_scales, y, B, H, D, Nout, dtype, act, norm_eps,
                               workspace, workspace_bytes, need);
    if (st != KDA_OK) return st;
    if (B > 0 && (y == x || y == ring || y == w || y == state || y == g || y == beta))
        return invalid("y must not alias another argument");
    ProjWs ws{};
    proj_layout(B, H, D, static_cast<uint8_t *>(workspace), &ws);
    st = kda_shortconv_decode_step_ex(x, ring, w, g, beta, state, ws.o, B, H, D, dtype, gate, l2_eps, flags, stream);
    if (st != KDA_OK || B == 0) return st;
    return way_out(ws, out_gate, norm_weight, proj, proj_scales, y, B, H, D, Nout, dtype, act, norm_eps, stream);
}

extern "C" size_t kda_chunk_prefill_proj_workspace_bytes(int64_t total_tokens, int num_seqs, int H, int D, int C) {
    if (total_tokens < 0 || num_seqs < 1 || H < 1 || D < 1 || C < 1) return 0;
    return up256(kda_chunk_prefill_workspace_bytes(total_tokens, num_seqs, H, D, C)) +
           proj_layout(total_tokens, H, D, nullptr, nullptr);
}

extern "C" kda_status kda_chunk_prefill_proj(const void *q, const void *k, const void *v, const float *g,
                                             const float *beta, const float *initial_state, float *final_state,
                                             const int64_t *cu_seqlens, int N, int64_t T, int H, int D, int C,
                                             kda_dtype dtype, kda_gate gate, float l2_eps, const void *out_gate,
                                             const float *norm_weight, kda_gate_act act, float norm_eps,
                                             const void *proj, const float *proj_scales, void *y, int Nout,
                                             void *workspace, size_t workspace_bytes, kda_stream_t stream) {
    clear_detail();
    if (N < 1) return invalid("N must be >= 1");
    if (C < 1 || C > 64) return invalid("C must be in 1..64");
    kda_status st = check_proj(out_gate, norm_weight, proj, proj_scales, y, T, H, D, Nout, dtype, act, norm_eps,
                               workspace, workspace_bytes, kda_chunk_prefill_proj_workspace_bytes(T, N, H, D, C));
    if (st != KDA_OK) return st;
    if (T > 0 && (y == q || y == k || y == v || y == g || y == beta || y == initial_state || y == final_state))
        return invalid("y must not alias another argument");
    const size_t pre = kda_chunk_prefill_workspace_bytes(T, N, H, D, C);
    uint8_t *base = static_cast<uint8_t *>(workspace);
    ProjWs ws{};
    proj_layout(T, H, D, base + up256(pre), &ws);
    st = kda_chunk_prefill_gated(q, k, v, g, beta, initial_state, final_state, ws.o, cu_seqlens, N, T, H, D, C, dtype,
                                 gate, l2_eps, pre ? base : nullptr, pre, stream);
    if (st != KDA_OK || T == 0) return st;
    return way_out(ws, out_gate, norm_weight, proj, proj_scales, y, T, H, D, Nout, dtype, act, norm_eps, stream);
}
