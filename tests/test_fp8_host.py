"""Host-side checks of the 8-bit operators: refusals of the C ABI and of the
binding (no GPU, no launch), and the fp64 statements the GPU tests compare with."""
import numpy as np
import pytest

from tests import _fp8
from tests._util import ensure_built


@pytest.fixture(scope="module")
def kda():
    ensure_built()
    from linear_attention_recurrence_02_gb300 import kda as mod
    mod.lib()
    return mod


def _refused(kda, st, detail):
    assert st == kda.KDA_ERR_INVALID_ARG
    assert detail in kda.lib().kda_last_error_detail().decode()


@pytest.mark.parametrize("case,detail", [
    (dict(T=-1), "T must be"),
    (dict(N=0), "N must be"),
    (dict(N=1032), "N must be"),
    (dict(N=32784), "N must be"),
    (dict(dtype=5), "dtype must be"),
    (dict(rdtype=-1), "res_dtype must be"),
    (dict(eps=-1e-6), "eps must be"),
    (dict(eps=float("nan")), "eps must be"),
    (dict(x=None), "x is NULL"),
    (dict(w=0x30008), "weight is not 16-byte aligned"),
    (dict(y=None), "y is NULL"),
    (dict(scales=0x60004), "scales is not 16-byte aligned"),
    (dict(res=0x20002), "residual is not 16-byte aligned"),
    (dict(so=0x40001), "sum_out is not 16-byte aligned"),
    (dict(so=0x10000, dtype=1, rdtype=0), "sum_out may be x only"),
    (dict(y=0x10000), "y must not alias"),
    (dict(y=0x40000), "y must not alias"),
    (dict(scales=0x20000), "must not alias"),
    (dict(so=0x30000), "must not alias"),
])
def test_add_rmsnorm_refusals(kda, case, detail):
    a = dict(x=0x10000, res=0x20000, w=0x30000, so=0x40000, y=0x50000, scales=0x60000, T=3, N=1024, dtype=1,
             rdtype=1, eps=1e-6)
    a.update(case)
    _refused(kda, kda.lib().kda_add_rmsnorm_fp8(a["x"], a["res"], a["w"], a["so"], a["y"], a["scales"], a["T"],
                                                a["N"], a["dtype"], a["rdtype"], a["eps"], None), detail)


@pytest.mark.parametrize("case,detail", [
    (dict(T=-1), "T must be"),
    (dict(H=0), "H must be"),
    (dict(D=48), "D must be"),
    (dict(H=1 << 28), "H*D too large"),
    (dict(dtype=2), "dtype must be"),
    (dict(act=2), "act must be"),
    (dict(eps=-1.0), "eps must be"),
    (dict(gate=None), "gate is NULL"),
    (dict(o=0x10004), "o is not 16-byte aligned"),
    (dict(y=0x10000), "must not alias"),
    (dict(scales=0x20000), "must not alias"),
])
def test_gated_rmsnorm_fp8_refusals(kda, case, detail):
    a = dict(o=0x10000, gate=0x20000, w=0x30000, y=0x40000, scales=0x50000, T=3, H=4, D=128, dtype=1, act=0,
             eps=1e-6)
    a.update(case)
    _refused(kda, kda.lib().kda_gated_rmsnorm_fp8(a["o"], a["gate"], a["w"], a["y"], a["scales"], a["T"], a["H"],
                                                  a["D"], a["dtype"], a["act"], a["eps"], None), detail)


@pytest.mark.parametrize("case,detail", [
    (dict(M=-1), "M must be"),
    (dict(M=1 << 31), "M must be"),
    (dict(N=0), "N must be"),
    (dict(K=0), "K must be"),
    (dict(K=24), "K must be"),
    (dict(lda=112), "lda and ldw"),
    (dict(lda=136), "lda and ldw"),
    (dict(ldw=1000), "lda and ldw"),
    (dict(lda=1 << 41), "below 2^40"),
    (dict(ldy=99), "ldy must be"),
    (dict(out=3), "out_dtype must be"),
    (dict(a=None), "a is NULL"),
    (dict(sw=0x40008), "w_scales is not 16-byte aligned"),
    (dict(y=0x10000), "y must not alias"),
])
def test_fp8_linear_refusals(kda, case, detail):
    a = dict(a=0x10000, sa=0x20000, w=0x30000, sw=0x40000, y=0x50000, M=5, N=100, K=128, lda=128, ldw=128, ldy=100,
             out=1)
    a.update(case)
    _refused(kda, kda.lib().kda_fp8_linear(a["a"], a["sa"], a["w"], a["sw"], a["y"], a["M"], a["N"], a["K"],
                                           a["lda"], a["ldw"], a["ldy"], a["out"], None), detail)


def test_no_tokens_is_a_noop_without_cuda(kda):
    L = kda.lib()
    assert L.kda_add_rmsnorm_fp8(None, None, None, None, None, None, 0, 1024, 1, 1, 1e-6, None) == kda.KDA_OK
    assert L.kda_gated_rmsnorm_fp8(None, None, None, None, None, 0, 4, 128, 1, 0, 1e-6, None) == kda.KDA_OK
    assert L.kda_fp8_linear(None, None, None, None, None, 0, 100, 128, 128, 128, 100, 1, None) == kda.KDA_OK


def test_binding_refuses_before_the_library(kda):
    """Shapes, types and devices are refused from the tensors themselves (here on the CPU)."""
    import torch
    f8 = torch.float8_e4m3fn
    x, w = torch.zeros(3, 256), torch.ones(256)
    y, s = torch.zeros(3, 256, dtype=f8), torch.zeros(2, 3)
    with pytest.raises(ValueError, match="shape"):
        kda.kda_add_rmsnorm_fp8(x, w, y, torch.zeros(3, 2))
    with pytest.raises(ValueError, match="shape"):
        kda.kda_add_rmsnorm_fp8(x, w, y, s, residual=torch.zeros(2, 256))
    with pytest.raises(TypeError, match="float8"):
        kda.kda_add_rmsnorm_fp8(x, w, torch.zeros(3, 256), s)
    with pytest.raises(TypeError, match="float32"):
        kda.kda_add_rmsnorm_fp8(x, w.double(), y, s)
    with pytest.raises(TypeError, match="residual's dtype"):
        kda.kda_add_rmsnorm_fp8(x, w, y, s, residual=x, sum_out=x.bfloat16())
    with pytest.raises(TypeError, match="unsupported dtype"):
        kda.kda_add_rmsnorm_fp8(x.half(), w, y, s)
    with pytest.raises(ValueError, match="shape"):
        kda.kda_gated_rmsnorm_fp8(torch.zeros(3, 2, 128), torch.zeros(3, 2, 64), torch.ones(128),
                                  torch.zeros(3, 2, 128, dtype=f8), s)
    with pytest.raises(ValueError, match="act must be"):
        kda.kda_gated_rmsnorm_fp8(torch.zeros(3, 2, 128), torch.zeros(3, 2, 128), torch.ones(128),
                                  torch.zeros(3, 2, 128, dtype=f8), s, act="relu")
    with pytest.raises(TypeError, match="gate must have"):
        kda.kda_gated_rmsnorm_fp8(torch.zeros(3, 2, 128), torch.zeros(3, 2, 128).bfloat16(), torch.ones(128),
                                  torch.zeros(3, 2, 128, dtype=f8), s)
    a, b = torch.zeros(3, 256, dtype=f8), torch.zeros(5, 256, dtype=f8)
    with pytest.raises(ValueError, match="shape"):
        kda.kda_fp8_linear(a, s, b, torch.zeros(1, 2), torch.zeros(3, 6))
    with pytest.raises(ValueError, match="shape"):
        kda.kda_fp8_linear(a, s.t(), b, torch.zeros(1, 2), torch.zeros(3, 5))
    with pytest.raises(TypeError, match="float8"):
        kda.kda_fp8_linear(a.float(), s, b, torch.zeros(1, 2), torch.zeros(3, 5))
    with pytest.raises(ValueError, match="CUDA"):
        kda.kda_fp8_linear(a, s, b, torch.zeros(1, 2), torch.zeros(3, 5))


def test_e4m3_table_is_torchs():
    import torch
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn)
    assert np.array_equal(t.float().numpy().astype(np.float64), _fp8.E4M3, equal_nan=True)


def test_fp64_statements():
    """The comparison values themselves: a row norm of one, a block's largest code at 448, and a product
    against the plain matrix product of the dequantised operands."""
    rng = np.random.default_rng(0)
    x = rng.normal(size=(4, 272))
    _, y = _fp8.add_rmsnorm(x, None, np.ones(272), 0.0)
    assert np.allclose((y * y).mean(-1), 1.0)
    s = _fp8.block_scales(y)
    assert s.shape == (3, 4)
    assert np.allclose(np.abs(y / _fp8.per_channel(s, 272))[:, 256:].max(-1), 448.0)
    assert np.all(_fp8.block_scales(np.zeros((2, 16))) == 2.0 ** -96 / 448)
    a, w = rng.normal(size=(3, 144)), rng.normal(size=(130, 144))
    sa, sw = rng.uniform(0.5, 2, (2, 3)), rng.uniform(0.5, 2, (2, 2))
    full = (a * _fp8.per_channel(sa, 144)) @ (w * np.repeat(np.repeat(sw, 128, 0)[:130], 128, 1)[:, :144]).T
    assert np.allclose(_fp8.linear(a, sa, w, sw)[0], full)


_DECODE_PROJ = dict(x=0x10000, ring=0x20000, w=0x30000, g=0x40000, beta=0x50000, state=0x60000, og=0x70000,
                    nw=0x80000, proj=0x90000, ps=0xa0000, y=0xb0000, B=2, H=3, D=128, Nout=100, dtype=1, gate=0, act=0,
                    l2=1e-6, eps=1e-6, flags=0, ws=0xc0000, wsz=1 << 20)


@pytest.mark.parametrize("case,detail", [
    (dict(B=-1), "B must be"),
    (dict(H=0), "H must be"),
    (dict(D=40), "D must be"),
    (dict(Nout=0), "Nout must be"),
    (dict(dtype=4), "dtype must be"),
    (dict(act=3), "act must be"),
    (dict(eps=-1.0), "norm_eps must be"),
    (dict(wsz=100), "workspace too small"),
    (dict(ws=None), "workspace is NULL"),
    (dict(og=None), "out_gate is NULL"),
    (dict(ps=0xa0004), "proj_scales is not 16-byte aligned"),
    (dict(y=0x10000), "y must not alias"),
    (dict(y=0x90000), "y must not alias"),
    (dict(flags=2), "flags"),
    (dict(gate=9), "gate must be"),
    (dict(beta=None), "beta is NULL"),
])
def test_decode_proj_refusals(kda, case, detail):
    """Refused before the first launch, the later calls' arguments as well as the step's own."""
    a = dict(_DECODE_PROJ)
    a.update(case)
    _refused(kda, kda.lib().kda_shortconv_decode_step_proj(
        a["x"], a["ring"], a["w"], a["g"], a["beta"], a["state"], a["og"], a["nw"], a["proj"], a["ps"], a["y"], a["B"],
        a["H"], a["D"], a["Nout"], a["dtype"], a["gate"], a["act"], a["l2"], a["eps"], a["flags"], a["ws"], a["wsz"],
        None), detail)


@pytest.mark.parametrize("case,detail", [
    (dict(N=0), "N must be"),
    (dict(T=-1), "tokens must be"),
    (dict(C=65), "C must be"),
    (dict(Nout=0), "Nout must be"),
    (dict(act=-1), "act must be"),
    (dict(wsz=1000), "workspace too small"),
    (dict(proj=None), "proj is NULL"),
    (dict(nw=0x80008), "norm_weight is not 16-byte aligned"),
    (dict(y=0x10000), "y must not alias"),
    (dict(N=2), "cu_seqlens is NULL"),
    (dict(k=None), "k is NULL"),
])
def test_prefill_proj_refusals(kda, case, detail):
    a = dict(q=0x10000, k=0x20000, v=0x30000, g=0x40000, beta=0x50000, N=1, T=10, H=3, D=128, C=64, dtype=1, gate=0,
             og=0x70000, nw=0x80000, act=0, proj=0x90000, ps=0xa0000, y=0xb0000, Nout=100, ws=0xc0000, wsz=1 << 20)
    a.update(case)
    _refused(kda, kda.lib().kda_chunk_prefill_proj(
        a["q"], a["k"], a["v"], a["g"], a["beta"], None, None, None, a["N"], a["T"], a["H"], a["D"], a["C"], a["dtype"],
        a["gate"], 1e-6, a["og"], a["nw"], a["act"], 1e-6, a["proj"], a["ps"], a["y"], a["Nout"], a["ws"], a["wsz"],
        None), detail)


def test_proj_workspace_sizes(kda):
    """The output in fp32, its codes and its scales, each rounded up to 256 bytes, and the prefill's own."""
    up = lambda n: (n + 255) // 256 * 256  # noqa: E731
    want = up(5 * 3 * 64 * 4) + up(5 * 3 * 64) + up(2 * 5 * 4)
    assert kda.kda_shortconv_decode_step_proj_workspace_bytes(5, 3, 64) == want
    assert kda.kda_shortconv_decode_step_proj_workspace_bytes(0, 3, 64) == 0
    assert kda.kda_chunk_prefill_proj_workspace_bytes(5, 1, 3, 64, 64) == want
    assert kda.kda_chunk_prefill_proj_workspace_bytes(5, 8, 3, 64, 64) == want + 256
    L = kda.lib()
    assert L.kda_shortconv_decode_step_proj(*[None] * 11, 0, 3, 128, 100, 1, 0, 0, 1e-6, 1e-6, 0, None, 0,
                                            None) == kda.KDA_OK


def test_binding_refuses_wrong_types_of_arguments(kda):
    """Arguments that are no tensors raise, a wrong number of them too, and nothing is called."""
    import torch
    f8 = torch.float8_e4m3fn
    x, w = torch.zeros(3, 256), torch.ones(256)
    y, s = torch.zeros(3, 256, dtype=f8), torch.zeros(2, 3)
    with pytest.raises(AttributeError):
        kda.kda_add_rmsnorm_fp8([[1.0]], w, y, s)
    with pytest.raises(TypeError):
        kda.kda_add_rmsnorm_fp8(x.cuda() if torch.cuda.is_available() else x, w)
    with pytest.raises(ValueError, match="CUDA"):
        kda.kda_add_rmsnorm_fp8(x, w, y, s)
    with pytest.raises(ValueError, match="CUDA"):
        kda.kda_gated_rmsnorm_fp8(torch.zeros(3, 2, 128), torch.zeros(3, 2, 128), torch.ones(128),
                                  torch.zeros(3, 2, 128, dtype=f8), s)
    calls = kda._fastcall()
    with pytest.raises(TypeError, match="number of arguments"):
        calls.linear(1, 2)
    with pytest.raises(ValueError, match="shape"):
        kda.kda_gated_rmsnorm_fp8(x, x, w, y, s)
    with pytest.raises(ValueError, match="shape"):
        kda.kda_fp8_linear(torch.zeros(256, dtype=f8), s, torch.zeros(5, 256, dtype=f8), torch.zeros(1, 2),
                           torch.zeros(3, 5))
