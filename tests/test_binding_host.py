"""Host-side checks of the Python binding that need no GPU: what it allocates, on which stream, and what it
refuses, with stand-ins for device tensors, streams and the library."""
import contextlib

import numpy as np
import pytest

from tests._util import ensure_built

torch = pytest.importorskip("torch")
F8, BF, F32 = torch.float8_e4m3fn, torch.bfloat16, torch.float32


class _Dev:
    """A device tensor's attributes without the device."""
    is_cuda = True

    def __init__(self, *shape, dtype=F32, device="cuda:0"):
        self.shape, self.dtype, self.device = shape, dtype, torch.device(device)

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 1 << 20

    def get_device(self):
        return self.device.index

    def numel(self):
        return int(np.prod(self.shape))

    def element_size(self):
        return self.dtype.itemsize

    def stride(self):
        return tuple(int(np.prod(self.shape[i + 1:])) for i in range(len(self.shape)))


class _Stream:
    cuda_stream = 77

    def __init__(self, index=0):
        self.device, self.device_index = torch.device("cuda", index), index


class _Library:
    """Answers the workspace questions from the real library and takes every call as successful."""

    def __init__(self, real):
        self.real, self.calls = real, []

    def __getattr__(self, name):
        if name.endswith("workspace_bytes"):
            return getattr(self.real, name)

        def call(*args):
            self.calls.append((name, args))
            return 0
        return call


@pytest.fixture
def env(monkeypatch):
    """The binding over _Library; `env.made` lists (bytes, stream that was current) of each allocation."""
    ensure_built()
    from linear_attention_recurrence_02_gb300 import kda
    kda._fastcall()  # over the real library
    fake, state = _Library(kda.lib()), {"current": None}
    made = []

    @contextlib.contextmanager
    def stream_context(s):
        before, state["current"] = state["current"], s if s is not None else state["current"]
        yield
        state["current"] = before

    def empty(n, dtype=None, device=None):
        made.append((n, state["current"]))
        return _Dev(n, dtype=torch.uint8)

    class Host:  # what torch.from_numpy gives: its copy to the device is an allocation as well
        def to(self, device):
            return empty(4, device=device)

    monkeypatch.setattr(kda, "lib", lambda: fake)
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch, "from_numpy", lambda a: Host())
    monkeypatch.setattr(torch.cuda, "stream", stream_context)
    monkeypatch.setattr(torch.cuda, "device", lambda d: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: type("Default", (), {"cuda_stream": 0})())
    fake.made, fake.kda = made, kda
    return fake


def _decode(kda, B=4, H=2, D=64, hidden=256, dt=BF, **k):
    a = dict(x=_Dev(B, 3, H, D, dtype=dt), ring=_Dev(B, 3, H, 3, D, dtype=dt), w=_Dev(3, H, D, 4), g=_Dev(B, H, D),
             beta=_Dev(B, H), state=_Dev(B, H, D, D), out_gate=_Dev(B, H, D, dtype=dt), norm_weight=_Dev(D),
             proj=_Dev(hidden, H * D, dtype=F8), proj_scales=_Dev(2, 1), y=_Dev(B, hidden, dtype=dt))
    a.update(k)
    kda.kda_shortconv_decode_step_proj(**a)


def _prefill(kda, T=100, H=2, D=64, hidden=256, dt=BF, **k):
    a = dict(q=_Dev(T, H, D, dtype=dt), k=_Dev(T, H, D, dtype=dt), v=_Dev(T, H, D, dtype=dt), g=_Dev(T, H, D),
             beta=_Dev(T, H), out_gate=_Dev(T, H, D, dtype=dt), norm_weight=_Dev(D),
             proj=_Dev(hidden, H * D, dtype=F8), proj_scales=_Dev(2, 1), y=_Dev(T, hidden, dtype=dt))
    a.update(k)
    kda.kda_chunk_prefill_proj(**a)


def _old_prefill(name, T=40000, H=2, D=128, **k):
    def call(kda, **extra):
        a = dict(q=_Dev(T, H, D, dtype=BF), k=_Dev(T, H, D, dtype=BF), v=_Dev(T, H, D, dtype=BF), g=_Dev(T, H, D),
                 beta=_Dev(T, H), out=_Dev(T, H, D, dtype=BF))
        a.update(k)
        a.update(extra)
        getattr(kda, name)(**a)
    return call


_ALLOCATING = {
    "decode_proj": (_decode, 1),
    "prefill_proj": (_prefill, 1),
    "prefill": (_old_prefill("kda_chunk_prefill", cu_seqlens=_Dev(4, dtype=torch.int64)), 1),
    "prefill_gated": (_old_prefill("kda_chunk_prefill_gated", cu_seqlens=_Dev(4, dtype=torch.int64)), 1),
    "prefill_epi": (_old_prefill("kda_chunk_prefill_epi", out_gate=_Dev(40000, 2, 128, dtype=BF),
                                 norm_weight=_Dev(128), cu_seqlens=_Dev(4, dtype=torch.int64)), 1),
    "prefill_scan": (_old_prefill("kda_chunk_prefill_scan", segments=4), 1),
    "prefill_split": (_old_prefill("kda_chunk_prefill_split", cu_seqlens=np.array([0, 39000, 40000])), 2),
}


@pytest.mark.parametrize("which", sorted(_ALLOCATING))
def test_own_memory_belongs_to_the_calls_stream(env, which):
    """Memory that a binding allocates for a call on a given stream is allocated with that stream current: the
    caching allocator then hands it out again only in that stream's order. Without a stream it is the current
    one's."""
    call, allocations = _ALLOCATING[which]
    s = _Stream()
    call(env.kda, stream=s)
    assert [cur for _, cur in env.made] == [s] * allocations and all(n > 0 for n, _ in env.made)
    assert env.calls and env.calls[-1][1][-1] == s.cuda_stream
    env.made.clear()
    call(env.kda)
    assert [cur for _, cur in env.made] == [None] * allocations
    assert env.calls[-1][1][-1] == 0


def test_a_given_workspace_is_used_as_it_is(env):
    need = env.real.kda_shortconv_decode_step_proj_workspace_bytes(4, 2, 64)
    _decode(env.kda, workspace=_Dev(need, dtype=torch.uint8), stream=_Stream())
    assert env.made == [] and env.calls[-1][1][-2] == need


@pytest.mark.parametrize("bad,error", [
    (dict(ring=_Dev(4, 3, 2, 3, 64)), TypeError),
    (dict(w=_Dev(3, 2, 64, 4, dtype=BF)), TypeError),
    (dict(g=_Dev(4, 2, 64, dtype=BF)), TypeError),
    (dict(beta=_Dev(4, 2, dtype=torch.float64)), TypeError),
    (dict(state=_Dev(4, 2, 64, 64, dtype=BF)), TypeError),
    (dict(out_gate=_Dev(4, 2, 64)), TypeError),
    (dict(x=_Dev(4, 3, 2, 64, dtype=torch.float16)), TypeError),
    (dict(state=_Dev(4, 2, 64, 64, device="cuda:1")), ValueError),
    (dict(ring=_Dev(4, 3, 2, 3, 64, dtype=BF, device="cuda:1")), ValueError),
    (dict(beta=_Dev(4, 2, device="cuda:1")), ValueError),
    (dict(workspace=_Dev(1 << 20, dtype=torch.uint8, device="cuda:1")), ValueError),
])
def test_decode_proj_refuses_types_and_devices(env, bad, error):
    """Nothing reaches the library, which could not tell the types apart."""
    with pytest.raises(error):
        _decode(env.kda, **bad)
    assert env.calls == [] and env.made == []


@pytest.mark.parametrize("bad,error", [
    (dict(k=_Dev(100, 2, 64)), TypeError),
    (dict(v=_Dev(100, 2, 64, dtype=torch.float16)), TypeError),
    (dict(g=_Dev(100, 2, 64, dtype=BF)), TypeError),
    (dict(beta=_Dev(100, 2, dtype=BF)), TypeError),
    (dict(initial_state=_Dev(1, 2, 64, 64, dtype=BF)), TypeError),
    (dict(final_state=_Dev(1, 2, 64, 64, dtype=BF)), TypeError),
    (dict(cu_seqlens=_Dev(2, dtype=torch.int32)), TypeError),
    (dict(v=_Dev(100, 2, 64, dtype=BF, device="cuda:1")), ValueError),
    (dict(final_state=_Dev(1, 2, 64, 64, device="cuda:1")), ValueError),
    (dict(cu_seqlens=_Dev(2, dtype=torch.int64, device="cuda:1")), ValueError),
    (dict(workspace=_Dev(1 << 24, dtype=torch.uint8, device="cuda:1")), ValueError),
])
def test_prefill_proj_refuses_types_and_devices(env, bad, error):
    with pytest.raises(error):
        _prefill(env.kda, **bad)
    assert env.calls == [] and env.made == []


def test_one_call_ways_out_take_what_they_document(env):
    """Optional tensors absent and present, every gate form, fp32 and bf16."""
    for dt in (BF, F32):
        _decode(env.kda, dt=dt)
        _decode(env.kda, dt=dt, g=_Dev(4, 2), gate="head")
        _decode(env.kda, dt=dt, g=None, gate="none")
        _prefill(env.kda, dt=dt)
        _prefill(env.kda, dt=dt, g=None, gate="none", initial_state=_Dev(1, 2, 64, 64), final_state=_Dev(1, 2, 64, 64),
                 cu_seqlens=_Dev(2, dtype=torch.int64))
    assert len(env.calls) == 10


def test_streams_of_another_device_are_refused(env):
    """By the one-call ways out and by the three operators (no tokens: the library then returns before CUDA)."""
    for call in (_decode, _prefill):
        with pytest.raises(ValueError, match="stream"):
            call(env.kda, stream=_Stream(1))
    assert env.calls == [] and env.made == []
    kda = env.kda

    def add(stream):
        kda.kda_add_rmsnorm_fp8(_Dev(0, 256), _Dev(256), _Dev(0, 256, dtype=F8), _Dev(2, 0), stream=stream)

    def gated(stream):
        kda.kda_gated_rmsnorm_fp8(_Dev(0, 2, 128), _Dev(0, 2, 128), _Dev(128), _Dev(0, 2, 128, dtype=F8), _Dev(2, 0),
                                  stream=stream)

    def linear(stream):
        kda.kda_fp8_linear(_Dev(0, 256, dtype=F8), _Dev(2, 0), _Dev(100, 256, dtype=F8), _Dev(1, 2), _Dev(0, 100),
                           stream=stream)

    class Handle:  # a stream that does not say where it is
        cuda_stream = 78

    for call in (add, gated, linear):
        call(_Stream(0))
        call(Handle())
        with pytest.raises(ValueError, match="stream must be on the tensors' device"):
            call(_Stream(1))
        with pytest.raises(AttributeError):
            call(object())
