"""GPU tests of a layer's run in 8 bits: residual norm -> q/k/v projection ->
short conv + recurrence -> gated norm -> output projection, for a prompt and
then token by token, through the separate calls and through the one-call ways
out (kda_chunk_prefill_proj, kda_shortconv_decode_step_proj).

Each stage is held to its fp64 statement on what the stage before it really
gave, so a stage's rounding is counted once and the tolerances are those of
the single operators."""
import numpy as np
import pytest

import oracle
from linear_attention_recurrence_02_gb300 import synth
from tests import _fp8
from tests._util import assert_close, cuda_or_skip, ensure_built, to_dev, to_np

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    torch = cuda_or_skip()
    ensure_built()
    from linear_attention_recurrence_02_gb300 import kda
    return torch, kda


def _weight(torch, gen, N, K):
    """Codes and 128 x 128 block scales of a weight of about unit gain."""
    w = (torch.randn((N, K), generator=gen, device="cuda") * 110).clamp(-448, 448).to(torch.float8_e4m3fn)
    s = torch.exp(0.3 * torch.randn((_fp8.nblocks(N), _fp8.nblocks(K)), generator=gen, device="cuda"))
    return w, s / (110 * K ** 0.5)


class _Layer:
    """The weights of one layer and the calls of its two halves."""

    def __init__(self, torch, kda, seed, hidden, H, D, dtype):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.torch, self.kda, self.hidden, self.H, self.D, self.dt = torch, kda, hidden, H, D, dtype
        self.norm_in = torch.rand(hidden, generator=g, device="cuda") + 0.5
        self.w_in, self.s_in = _weight(torch, g, 3 * H * D, hidden)
        self.w_gate, self.s_gate = _weight(torch, g, H * D, hidden)
        self.taps = torch.randn((3, H, D, 4), generator=g, device="cuda") * 0.5
        self.norm_out = torch.rand(D, generator=g, device="cuda") + 0.5
        self.w_out, self.s_out = _weight(torch, g, hidden, H * D)

    def inward(self, x, residual):
        """Returns the new residual stream, the conv's input [T,3,H,D] and the output gate [T,H,D], checked."""
        torch, kda, T = self.torch, self.kda, x.shape[0]
        q = torch.empty((T, self.hidden), dtype=torch.float8_e4m3fn, device="cuda")
        s = torch.empty((_fp8.nblocks(self.hidden), T), device="cuda")
        r = torch.empty_like(residual)
        kda.kda_add_rmsnorm_fp8(x, self.norm_in, q, s, residual=residual, sum_out=r)
        proj = torch.empty((T, 3 * self.H * self.D), dtype=self.dt, device="cuda")
        gate = torch.empty((T, self.H * self.D), dtype=self.dt, device="cuda")
        kda.kda_fp8_linear(q, s, self.w_in, self.s_in, proj)
        kda.kda_fp8_linear(q, s, self.w_gate, self.s_gate, gate)
        _, ref = _fp8.add_rmsnorm(to_np(x), to_np(residual), to_np(self.norm_in), 1e-6)
        _fp8.check_codes(ref, _fp8.codes_to_np(q), to_np(s), _fp8.add_norm_steps(self.hidden), "norm in")
        for y, w, sw in ((proj, self.w_in, self.s_in), (gate, self.w_gate, self.s_gate)):
            _fp8.check_linear(to_np(y), _fp8.codes_to_np(q), to_np(s), _fp8.codes_to_np(w), to_np(sw),
                              self.dt == torch.bfloat16, "projection in")
        return r, proj.view(T, 3, self.H, self.D), gate.view(T, self.H, self.D)

    def outward(self, o, gate):
        """Gated norm and output projection by their own calls, checked."""
        torch, kda, T = self.torch, self.kda, o.shape[0]
        K = self.H * self.D
        q = torch.empty((T, self.H, self.D), dtype=torch.float8_e4m3fn, device="cuda")
        s = torch.empty((_fp8.nblocks(K), T), device="cuda")
        y = torch.empty((T, self.hidden), dtype=self.dt, device="cuda")
        kda.kda_gated_rmsnorm_fp8(o, gate, self.norm_out, q, s)
        kda.kda_fp8_linear(q.view(T, K), s, self.w_out, self.s_out, y)
        ref = oracle.gated_rmsnorm(to_np(o), to_np(gate), to_np(self.norm_out)).reshape(T, K)
        _fp8.check_codes(ref, _fp8.codes_to_np(q).reshape(T, K), to_np(s),
                         _fp8.gated_steps(float(gate.abs().max())), "norm out")
        _fp8.check_linear(to_np(y), _fp8.codes_to_np(q).reshape(T, K), to_np(s), _fp8.codes_to_np(self.w_out),
                          to_np(self.s_out), self.dt == torch.bfloat16, "projection out")
        return y


@pytest.mark.parametrize("H,D,hidden,bf16", [(5, 64, 272, False), (4, 128, 640, True), (3, 16, 128, True)])
def test_layer_prompt_then_tokens(env, H, D, hidden, bf16):
    """A packed batch of two prompts (70 and 3 tokens), then two tokens of each: every stage against its fp64
    statement, the one-call ways out against the separate calls bit by bit."""
    torch, kda = env
    dt = torch.bfloat16 if bf16 else torch.float32
    layer = _Layer(torch, kda, 7 + D, hidden, H, D, dt)
    cu = np.array([0, 70, 73], dtype=np.int64)
    T, N = 73, 2
    g = torch.Generator(device="cuda").manual_seed(9)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    _, x, gate = layer.inward(rnd(T, hidden).to(dt), 2 * rnd(T, hidden))
    gg, beta = -torch.nn.functional.softplus(rnd(T, H, D)), torch.sigmoid(rnd(T, H))
    dcu = torch.from_numpy(cu).cuda()
    yc, ring = torch.empty((3, T, H, D), dtype=dt, device="cuda"), torch.empty((N, 3, H, 3, D), dtype=dt, device="cuda")
    kda.kda_shortconv_prefill(x, layer.taps, yc, ring_out=ring, cu_seqlens=dcu)
    state, st2 = torch.empty((N, H, D, D), device="cuda"), torch.empty((N, H, D, D), device="cuda")
    o = torch.empty((T, H, D), dtype=dt, device="cuda")
    kda.kda_chunk_prefill(yc[0], yc[1], yc[2], gg, beta, o, final_state=state, cu_seqlens=dcu)
    ro, rs = oracle.recurrence(to_np(yc[0]), to_np(yc[1]), to_np(yc[2]), to_np(gg), to_np(beta), cu_seqlens=cu)
    assert_close(to_np(o), ro, bf16, (1,), "prefill")
    assert_close(to_np(state), rs, bf16, (0, 1), "state")
    y = layer.outward(o, gate)
    y2 = torch.empty_like(y)
    kda.kda_chunk_prefill_proj(yc[0], yc[1], yc[2], gg, beta, gate, layer.norm_out, layer.w_out, layer.s_out, y2,
                               final_state=st2, cu_seqlens=dcu)
    assert torch.equal(y, y2) and torch.equal(state, st2)

    for step in range(2):
        _, x, gate = layer.inward(rnd(N, hidden).to(dt), 2 * rnd(N, hidden))
        gg, beta = -torch.nn.functional.softplus(rnd(N, H, D)), torch.sigmoid(rnd(N, H))
        ring2, st2 = ring.clone(), state.clone()
        ry, _ = oracle.shortconv_step(to_np(x), to_np(ring), to_np(layer.taps))
        ro, rs = oracle.decode_step(ry[:, 0], ry[:, 1], ry[:, 2], to_np(gg), to_np(beta), to_np(state))
        o = torch.empty((N, H, D), dtype=dt, device="cuda")
        kda.kda_shortconv_decode_step(x, ring, layer.taps, gg, beta, state, o)
        assert_close(to_np(o), ro, bf16, (0, 1), f"step {step}")
        assert_close(to_np(state), rs, bf16, (0, 1), f"state after step {step}")
        y = layer.outward(o, gate)
        y2 = torch.empty_like(y)
        kda.kda_shortconv_decode_step_proj(x, ring2, layer.taps, gg, beta, st2, gate, layer.norm_out, layer.w_out,
                                           layer.s_out, y2)
        assert torch.equal(y, y2) and torch.equal(state, st2) and torch.equal(ring, ring2)
    kda.kda_sync_status()


@pytest.mark.parametrize("gate_form", ["head", "none"])
def test_decode_proj_gate_forms_in_a_graph(env, gate_form):
    """Captured with a workspace of its own and replayed: three steps give the states, rings and outputs of
    direct calls."""
    torch, kda = env
    B, H, D, hidden = 6, 4, 128, 384
    layer = _Layer(torch, kda, 3, hidden, H, D, torch.bfloat16)
    d = synth.decode_inputs(31, B, H, D, True, s0_std=0.3)
    e = synth.epilogue_inputs(32, B, H, D, True)
    bf, f32 = torch.bfloat16, torch.float32
    x, beta, gate = to_dev(d["x"], bf, torch), to_dev(d["beta"], f32, torch), to_dev(e["gate"], bf, torch)
    g = to_dev(np.ascontiguousarray(d["g"][..., 0]), f32, torch) if gate_form == "head" else None

    def buffers():
        return to_dev(d["ring"], bf, torch), to_dev(d["s0"], f32, torch), torch.zeros((B, hidden), dtype=bf, device="cuda")

    def step(ring, st, y, ws):
        kda.kda_shortconv_decode_step_proj(x, ring, layer.taps, g, beta, st, gate, layer.norm_out, layer.w_out,
                                           layer.s_out, y, gate=gate_form, workspace=ws)

    need = kda.kda_shortconv_decode_step_proj_workspace_bytes(B, H, D)
    ws1, ws2 = (torch.empty(need, dtype=torch.uint8, device="cuda") for _ in range(2))
    direct, replayed = buffers(), buffers()
    for _ in range(3):
        step(*direct, ws1)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    warm = buffers()
    step(*warm, ws2)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step(*replayed, ws2)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(direct, replayed):
        assert torch.equal(a, b)


def test_proj_calls_refuse_bad_tensors(env):
    torch, kda = env
    layer = _Layer(torch, kda, 4, 256, 2, 64, torch.float32)
    B, H, D = 3, 2, 64
    z = lambda *s: torch.zeros(s, device="cuda")  # noqa: E731
    args = lambda **k: [k.get(n, v) for n, v in dict(  # noqa: E731
        x=z(B, 3, H, D), ring=z(B, 3, H, 3, D), w=layer.taps, g=z(B, H, D), beta=z(B, H), state=z(B, H, D, D),
        gate=z(B, H, D), nw=layer.norm_out, proj=layer.w_out, ps=layer.s_out, y=z(B, 256)).items()]
    with pytest.raises(ValueError, match="shape"):
        kda.kda_shortconv_decode_step_proj(*args(y=z(B, 255)))
    with pytest.raises(TypeError, match="float8"):
        kda.kda_shortconv_decode_step_proj(*args(proj=layer.w_out.float()))
    with pytest.raises(TypeError, match="inputs' dtype"):
        kda.kda_shortconv_decode_step_proj(*args(y=z(B, 256).bfloat16()))
    with pytest.raises(ValueError, match="device"):
        kda.kda_shortconv_decode_step_proj(*args(ps=layer.s_out.cpu()))
    with pytest.raises(kda.KdaError, match="workspace too small"):
        kda.kda_shortconv_decode_step_proj(*args(), workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    kda.kda_shortconv_decode_step_proj(*args())
    kda.kda_sync_status()
