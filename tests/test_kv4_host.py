"""Host-side checks of the softmax-attention layers' calls that need no GPU: what the C ABI refuses before any CUDA
call, what the binding refuses before the library, the sizes, and the plain forms that the GPU tests compare with."""
import ctypes

import numpy as np
import pytest

from tests import _kv4 as ref
from tests._util import ensure_built
from tests.test_binding_host import _Dev, _Stream

torch = pytest.importorskip("torch")
BF, F32, F64, I64, I32, U8 = (torch.bfloat16, torch.float32, torch.float64, torch.int64, torch.int32, torch.uint8)


@pytest.fixture(scope="module")
def kda():
    ensure_built()
    from linear_attention_recurrence_02_gb300 import kda as mod
    mod.lib()
    return mod


def _p(x):
    return None if x is None else ctypes.c_void_p(x)


def _rope(kda, **k):
    a = dict(q=0x10000, k=0x20000, q_out=0x30000, k_out=0x40000, qw=0x50000, kw=0x60000, pos=0x70000, freq=0x80000,
             T=3, Hq=4, Hk=2, D=128, R=64, qs=512, ks=256, qos=512, kos=256, inter=0, eps=1e-6, dtype=1)
    a.update(k)
    ptrs = [_p(a[n]) for n in ("q", "k", "q_out", "k_out", "qw", "kw", "pos", "freq")]
    return kda.lib().kda_qk_norm_rope(*ptrs, a["T"], a["Hq"], a["Hk"], a["D"], a["R"], a["qs"], a["ks"], a["qos"],
                                      a["kos"], a["inter"], a["eps"], a["dtype"], None)


def _cache_call(kda, name, **k):
    a = dict(cache=0x100000, table=0x200000, lens=0x300000, cu=0x400000, k=0x500000, v=0x600000, B=2, T=5, Hk=2, D=128,
             page=64, pages=9, cols=4, ts=4, ks=256, vs=256, dtype=1)
    a.update(k)
    order = ("k", "v", "cache", "table", "lens", "cu") if name == "kda_kv4_append" else \
        ("cache", "table", "lens", "cu", "k", "v")
    return getattr(kda.lib(), name)(*[_p(a[n]) for n in order], a["B"], a["T"], a["Hk"], a["D"], a["page"], a["pages"],
                                    a["cols"], a["ts"], a["ks"], a["vs"], a["dtype"], None)


def _attention(kda, **k):
    a = dict(q=0x10000, cache=0x100000, table=0x200000, lens=0x300000, cu=0x400000, out=0x500000, lse=0x600000, B=2, T=5,
             Hq=4, Hk=2, D=128, page=64, pages=9, cols=4, ts=4, qs=512, os=512, scale=0.1, causal=1, window=0, dtype=1,
             ws=0x700000, size=1 << 30)
    a.update(k)
    return kda.lib().kda_kv4_attention(*[_p(a[n]) for n in ("q", "cache", "table", "lens", "cu", "out", "lse")], a["B"],
                                       a["T"], a["Hq"], a["Hk"], a["D"], a["page"], a["pages"], a["cols"], a["ts"],
                                       a["qs"], a["os"], a["scale"], a["causal"], a["window"], a["dtype"], _p(a["ws"]),
                                       a["size"], None)


@pytest.mark.parametrize("case,detail", [
    (dict(T=-1), "T must be"), (dict(Hq=0), "Hq must be"), (dict(Hk=-1), "Hk"), (dict(D=48), "D must be"),
    (dict(D=256), "D must be"), (dict(R=130), "R must be"), (dict(R=24), "R must be"), (dict(R=-16), "R must be"),
    (dict(inter=2), "interleaved"), (dict(dtype=2), "dtype"), (dict(eps=-1.0), "eps"), (dict(eps=float("nan")), "eps"),
    (dict(q=None), "q is NULL"), (dict(k=None), "k is NULL"), (dict(q_out=0x30008), "q_out is not 16-byte aligned"),
    (dict(pos=None), "positions is NULL"), (dict(freq=None), "inv_freq is NULL"), (dict(qs=516), "multiples of 16"),
    (dict(qs=504), "at least the heads"), (dict(kos=248), "at least the heads"), (dict(q_out=0x10000, qos=520), "in place"),
    (dict(q_out=0x40000), "may alias only"), (dict(k_out=0x10000), "may alias only"), (dict(kw=0x60004), "k_weight"),
])
def test_norm_rope_refuses(kda, case, detail):
    assert _rope(kda, **case) == kda.KDA_ERR_INVALID_ARG
    assert detail in kda.lib().kda_last_error_detail().decode()


def test_norm_rope_without_tokens_is_a_no_op(kda):
    assert _rope(kda, T=0, q=None, pos=None) == kda.KDA_OK


_SHARED = [
    (dict(B=-1), "B must be"), (dict(T=-1), "T must be"), (dict(Hk=0), "Hk must be"), (dict(D=32), "D must be"),
    (dict(D=96), "D must be"), (dict(dtype=5), "dtype"), (dict(page=48), "page_size"), (dict(page=8), "page_size"),
    (dict(page=512), "page_size"), (dict(pages=0), "pages"), (dict(pages=1 << 31), "pages"), (dict(cols=0), "columns"),
    (dict(cols=(1 << 31) // 64), "columns"), (dict(ts=3), "table_stride"), (dict(cu=None), "one token for each"),
    (dict(B=0), "without a sequence"), (dict(cache=None), "cache is NULL"), (dict(cache=0x100008), "cache is not 16"),
    (dict(table=None), "block_table is NULL"), (dict(lens=0x300008), "lens is not 16"), (dict(cu=0x400004), "cu_seqlens"),
    (dict(T=1 << 31), "T must be"), (dict(B=(1 << 30) + 1), "B must be"), (dict(Hk=32769, Hq=32769), "Hk must be"),
]


@pytest.mark.parametrize("case,detail", _SHARED + [
    (dict(k=None), "k is NULL"), (dict(v=0x600008), "v is not 16"), (dict(ks=248), "at least Hk*D"),
    (dict(vs=260), "multiples of 16"), (dict(dtype=0, ks=258), "multiples of 16"), (dict(k=0x100000), "alias"),
])
@pytest.mark.parametrize("name", ["kda_kv4_append", "kda_kv4_read"])
def test_cache_calls_refuse(kda, name, case, detail):
    assert _cache_call(kda, name, **case) == kda.KDA_ERR_INVALID_ARG
    assert detail in kda.lib().kda_last_error_detail().decode()


def test_read_refuses_one_tensor_for_both(kda):
    assert _cache_call(kda, "kda_kv4_read", v=0x500000) == kda.KDA_ERR_INVALID_ARG


@pytest.mark.parametrize("case,detail", _SHARED + [
    (dict(Hq=3), "multiple of Hk"), (dict(Hq=0), "multiple of Hk"), (dict(T=1 << 30), "T*Hq"), (dict(scale=0.0), "scale"),
    (dict(scale=float("nan")), "scale"), (dict(scale=float("inf")), "scale"), (dict(scale=-1.0), "scale"),
    (dict(causal=2), "causal"), (dict(window=-1), "window"), (dict(q=None), "q is NULL"), (dict(out=0x500004), "out is not 16"),
    (dict(lse=0x600002), "lse"), (dict(qs=504), "at least Hq*D"), (dict(os=516), "multiples of 16"),
    (dict(out=0x10000), "alias"), (dict(lse=0x500000), "alias"), (dict(size=1 << 10), "workspace too small"),
    (dict(ws=None), "workspace is NULL"), (dict(ws=0x700008), "workspace is not 16"),
])
def test_attention_refuses(kda, case, detail):
    assert _attention(kda, **case) == kda.KDA_ERR_INVALID_ARG
    assert detail in kda.lib().kda_last_error_detail().decode()


def test_calls_without_tokens_are_no_ops(kda):
    for name in ("kda_kv4_append", "kda_kv4_read"):
        assert _cache_call(kda, name, T=0, B=0, cu=None, k=None, v=None, cache=None) == kda.KDA_OK
        assert _cache_call(kda, name, T=0, k=None, v=None) == kda.KDA_OK
    assert _attention(kda, T=0, q=None, ws=None, size=0) == kda.KDA_OK


def test_sizes(kda):
    assert kda.kda_kv4_cache_bytes(10, 8, 64, 128) == 10 * 8 * 4 * 18 * 128
    assert np.prod(kda.kda_kv4_cache_shape(10, 8, 64, 128)) == kda.kda_kv4_cache_bytes(10, 8, 64, 128)
    assert kda.kda_kv4_cache_bytes(10, 8, 40, 128) == 0 and kda.kda_kv4_cache_bytes(-1, 8, 64, 128) == 0
    size = kda.kda_kv4_attention_workspace_bytes
    assert size(64, 64, 96, 8, 128, 64, 128, False, BF) > 0 and size(64, 64, 8, 8, 64, 64, 1000, False, F32) > 0
    assert size(1, 1, 32, 8, 128, 64, 64, False, BF) == 0  # short enough for one item a cluster
    assert size(1, 4000, 32, 8, 128, 64, 64, True, BF) > size(64, 64, 96, 8, 128, 64, 128, False, BF)
    assert size(0, 1, 8, 8, 128, 64, 9, False, BF) == 0 and size(1, 1, 8, 3, 128, 64, 9, False, BF) == 0
    assert size(1, 1, 8, 8, 32, 64, 9, False, BF) == 0 and size(1, 1, 8, 8, 64, 48, 9, False, BF) == 0


# ---------------------------------------------------------------- the binding
_T = _Dev


def _args(**k):
    a = dict(q=_T(2, 4, 128, dtype=BF), k=_T(2, 2, 128, dtype=BF), v=_T(2, 2, 128, dtype=BF), out=_T(2, 4, 128, dtype=BF),
             cache=_T(9, 2, 4, 18 * 128, dtype=U8), table=_T(2, 4, dtype=I32), lens=_T(2, dtype=I64), cu=None, stream=None,
             lse=None, workspace=None)
    a.update(k)
    return a


def _append(kda, **k):
    a = _args(**k)
    kda.kda_kv4_append(a["k"], a["v"], a["cache"], a["table"], a["lens"], cu_seqlens=a["cu"], stream=a["stream"])


def _read(kda, **k):
    a = _args(**k)
    kda.kda_kv4_read(a["cache"], a["table"], a["lens"], a["k"], a["v"], cu_seqlens=a["cu"], stream=a["stream"])


def _attend(kda, **k):
    a = _args(**k)
    kda.kda_kv4_attention(a["q"], a["cache"], a["table"], a["lens"], a["out"], cu_seqlens=a["cu"], lse=a["lse"],
                          workspace=a["workspace"], stream=a["stream"])


class _Strided(_T):
    def __init__(self, *shape, strides, **k):
        super().__init__(*shape, **k)
        self._strides = strides

    def stride(self):
        return self._strides

    def is_contiguous(self):
        return False


_BAD = [
    (dict(cache=_T(9, 2, 4, 18 * 64, dtype=U8)), ValueError), (dict(cache=_T(9, 2, 4, 18 * 128, dtype=F32)), TypeError),
    (dict(cache=_T(9, 2, 4 * 18 * 128, dtype=U8)), ValueError), (dict(table=_T(3, 4, dtype=I32)), ValueError),
    (dict(table=_T(2, 4, dtype=I64)), TypeError), (dict(table=_Strided(2, 4, dtype=I32, strides=(1, 2))), ValueError),
    (dict(lens=_T(2, dtype=I32)), TypeError), (dict(cu=_T(2, dtype=I64)), ValueError), (dict(cu=_T(3, dtype=I32)), TypeError),
    (dict(lens=_T(2, dtype=I64, device="cuda:1")), ValueError), (dict(table=_T(2, 4, dtype=I32, device="cuda:1")), ValueError),
    (dict(stream=_Stream(1)), ValueError),
]
_ROWS = [
    (dict(k=_T(2, 3, 128, dtype=BF)), ValueError), (dict(v=_T(2, 2, 64, dtype=BF)), ValueError),
    (dict(v=_T(2, 2, 128, dtype=F32)), TypeError), (dict(k=_T(2, 2, 128, dtype=torch.float16), v=_T(2, 2, 128, dtype=torch.float16)), TypeError),
    (dict(v=_T(2, 2, 128, dtype=BF, device="cuda:1")), ValueError),
    (dict(k=_Strided(2, 2, 128, dtype=BF, strides=(512, 256, 1))), ValueError),
    (dict(k=_Strided(2, 2, 128, dtype=BF, strides=(512, 128, 2))), ValueError),
]
_QUERIES = [
    (dict(out=_T(2, 3, 128, dtype=BF)), ValueError), (dict(out=_T(2, 4, 128, dtype=F32)), TypeError),
    (dict(lse=_T(2, 3)), ValueError), (dict(lse=_T(2, 4, dtype=BF)), TypeError),
    (dict(workspace=_T(1 << 20)), TypeError), (dict(workspace=_T(1 << 28, dtype=U8, device="cuda:1")), ValueError),
    (dict(q=_Strided(2, 4, 128, dtype=BF, strides=(128, 256, 1))), ValueError),
]


@pytest.mark.parametrize("call,bad,error", [(c, b, e) for c in (_append, _read) for b, e in _BAD + _ROWS] +
                         [(_attend, b, e) for b, e in _BAD + _QUERIES])
def test_binding_refuses(kda, call, bad, error):
    with pytest.raises(error):
        call(kda, **bad)


def _norm(kda, **k):
    a = dict(q=_T(3, 4, 64, dtype=BF), k=_T(3, 2, 64, dtype=BF), qo=_T(3, 4, 64, dtype=BF), ko=_T(3, 2, 64, dtype=BF),
             pos=_T(3, dtype=I64), freq=_T(16, dtype=F64), qw=_T(64), kw=_T(64), stream=None)
    a.update(k)
    kda.kda_qk_norm_rope(a["q"], a["k"], a["qo"], a["ko"], a["pos"], a["freq"], q_weight=a["qw"], k_weight=a["kw"],
                         stream=a["stream"])


@pytest.mark.parametrize("bad,error", [
    (dict(k=None), ValueError), (dict(pos=None), ValueError), (dict(qo=_T(3, 4, 32, dtype=BF)), ValueError),
    (dict(ko=_T(3, 3, 64, dtype=BF)), ValueError), (dict(k=_T(2, 2, 64, dtype=BF)), ValueError),
    (dict(pos=_T(4, dtype=I64)), ValueError), (dict(pos=_T(3, dtype=I32)), TypeError), (dict(freq=_T(16)), TypeError),
    (dict(qw=_T(32)), ValueError), (dict(kw=_T(64, dtype=BF)), TypeError), (dict(qo=_T(3, 4, 64)), TypeError),
    (dict(q=_T(3, 4, 64, dtype=torch.float16), k=None, ko=None, qo=_T(3, 4, 64, dtype=torch.float16)), TypeError),
    (dict(ko=_T(3, 2, 64, dtype=BF, device="cuda:1")), ValueError), (dict(stream=_Stream(1)), ValueError),
    (dict(q=_Strided(3, 4, 64, dtype=BF, strides=(512, 128, 1))), ValueError),
])
def test_norm_rope_binding_refuses(kda, bad, error):
    with pytest.raises(error):
        _norm(kda, **bad)


def test_calls_without_tokens_reach_the_library(kda):
    """Which then returns before CUDA; with the tensors' device current, and a stream of theirs named."""
    s, none = _Stream(0), dict(k=_T(0, 2, 128, dtype=BF), v=_T(0, 2, 128, dtype=BF), q=_T(0, 4, 128, dtype=BF),
                               out=_T(0, 4, 128, dtype=BF), cu=_T(3, dtype=I64))
    _append(kda, stream=s, **none)
    _read(kda, stream=s, **none)
    _attend(kda, stream=s, **none)
    _attend(kda, stream=s, lse=_T(0, 4), workspace=_T(1 << 28, dtype=U8), **none)
    _norm(kda, q=_T(0, 4, 64), k=None, qo=_T(0, 4, 64), ko=None, kw=None, pos=None, freq=None, stream=s)


def test_wrong_sizes_reach_the_library_and_come_back_as_errors(kda):
    with pytest.raises(kda.KdaError, match="page_size"):
        _append(kda, cache=_T(9, 2, 3, 18 * 128, dtype=U8), stream=_Stream(0))
    with pytest.raises(kda.KdaError, match="multiple of Hk"):
        _attend(kda, q=_T(2, 5, 128, dtype=BF), out=_T(2, 5, 128, dtype=BF), stream=_Stream(0))
    with pytest.raises(kda.KdaError, match="R must be"):
        _norm(kda, freq=_T(12, dtype=F64), stream=_Stream(0))


# ---------------------------------------------------------------- the plain forms
def test_plain_cache_holds_what_it_was_given():
    rng = np.random.default_rng(0)
    for D in (64, 128):
        block, ks, vs = np.full(18 * D, 255, np.uint8), rng.normal(size=(16, D)), rng.normal(size=(16, D))
        for t in range(16):
            ref.put(block, t, ks[t], vs[t])
        for t in range(16):
            k, v = ref.get(block, t, D)
            assert np.array_equal(k, ref.held(ks[t])) and np.array_equal(v, ref.held(vs[t]))
        cached = ref.tokens(block.reshape(1, 1, 1, -1), np.zeros((1, 1), int), 0, 16)
        assert np.array_equal(cached[0][:, 0], ref.held(ks)) and np.array_equal(cached[1][:, 0], ref.held(vs))


def test_held_values_are_bf16_numbers_within_half_a_step():
    x = np.random.default_rng(1).normal(size=(500, 64)) * np.exp(np.random.default_rng(2).normal(size=(500, 1)) * 5)
    codes, s = ref.quantise(x)
    y = ref.held(x)
    assert np.array_equal(ref.bf16_values(ref.bf16_bits(y.astype(np.float32))), y)
    step = np.repeat(s, 32, -1)
    assert np.all(np.abs(x - y) <= step / 2 * (1 + 1e-12)) and codes.min() >= 1 and codes.max() <= 15
    amax = np.abs(x).reshape(500, 2, 32).max(-1)
    assert np.all(7 * s >= amax) and np.all(7 * s <= amax * (1 + 2.0 ** -4))
    assert np.all((s / 2.0 ** (np.floor(np.log2(s)) - 4)) % 1 == 0)  # five bits


def test_plain_rotation_agrees_with_cosine_and_sine():
    x = np.random.default_rng(3).normal(size=(4, 2, 32))
    freq = 100.0 ** (-np.arange(8) / 8)
    for inter in (False, True):
        y = ref.norm_rope(x, None, [0, 1, 5, -3], freq, 1e-6, inter)
        assert np.array_equal(y[0], x[0])
        a, b = (x[2, 1, 6], x[2, 1, 7]) if inter else (x[2, 1, 3], x[2, 1, 11])
        got = (y[2, 1, 6], y[2, 1, 7]) if inter else (y[2, 1, 3], y[2, 1, 11])
        t = 5 * freq[3]
        assert np.allclose(got, (a * np.cos(t) - b * np.sin(t), b * np.cos(t) + a * np.sin(t)), atol=1e-14)
        assert np.allclose(np.linalg.norm(y, axis=-1), np.linalg.norm(x, axis=-1))


def test_plain_attention_of_one_token_is_its_value():
    rng = np.random.default_rng(4)
    k, v, q = rng.normal(size=(1, 1, 8)), rng.normal(size=(1, 1, 8)), rng.normal(size=(2, 2, 8))
    out, lse, _, _ = ref.attention(q, k, v, [-1, 0], 0.5, True, 0)
    assert np.array_equal(out[0], np.zeros((2, 8))) and np.all(lse[0] == -np.inf)
    assert np.allclose(out[1], v[0, 0]) and np.allclose(lse[1], 0.5 * q[1] @ k[0, 0])
