"""GPU tests of the memory that a call allocates for itself: with `stream=` and no workspace, what the current
stream allocates and fills right after the call (and what it was still using before) stays apart from it."""
import numpy as np
import pytest

from tests._util import cuda_or_skip, ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    torch = cuda_or_skip()
    ensure_built()
    from linear_attention_recurrence_02_gb300 import kda
    return torch, kda


def _weight(torch, gen, N, K):
    w = (torch.randn((N, K), generator=gen, device="cuda") * 110).clamp(-448, 448).to(torch.float8_e4m3fn)
    return w, torch.rand(((N + 127) // 128, (K + 127) // 128), generator=gen, device="cuda") / 1000


def _decode_proj(torch, kda, gen):
    B, H, D, hidden, bf = 64, 8, 128, 512, torch.bfloat16
    r = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    x, ring, taps = r(B, 3, H, D).to(bf), r(B, 3, H, 3, D).to(bf), r(3, H, D, 4) / 2
    g, beta = -torch.nn.functional.softplus(r(B, H, D)), torch.sigmoid(r(B, H))
    state, gate, nw, (w, ws) = r(B, H, D, D) / 4, r(B, H, D).to(bf), r(D).abs(), _weight(torch, gen, hidden, H * D)
    size = kda.kda_shortconv_decode_step_proj_workspace_bytes(B, H, D)

    def call(**k):
        rg, st, y = ring.clone(), state.clone(), torch.zeros((B, hidden), dtype=bf, device="cuda")
        torch.cuda.synchronize()
        return lambda: kda.kda_shortconv_decode_step_proj(x, rg, taps, g, beta, st, gate, nw, w, ws, y, **k), (rg, st, y)
    return call, size


def _prompt(torch, gen, T, H, D):
    r = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    bf = torch.bfloat16
    return (r(T, H, D).to(bf), r(T, H, D).to(bf), r(T, H, D).to(bf), -torch.nn.functional.softplus(r(T, H, D)),
            torch.sigmoid(r(T, H)))


def _prefill_proj(torch, kda, gen):
    T, H, D, hidden, bf = 1000, 8, 128, 512, torch.bfloat16
    ins, gate, nw = _prompt(torch, gen, T, H, D), torch.randn((T, H, D), generator=gen, device="cuda").to(bf), \
        torch.rand(D, generator=gen, device="cuda")
    w, ws = _weight(torch, gen, hidden, H * D)
    cu = torch.tensor([0, 300, 301, T], device="cuda")
    size = kda.kda_chunk_prefill_proj_workspace_bytes(T, 3, H, D, 64)

    def call(**k):
        y, st = torch.zeros((T, hidden), dtype=bf, device="cuda"), torch.zeros((3, H, D, D), device="cuda")
        torch.cuda.synchronize()
        return lambda: kda.kda_chunk_prefill_proj(*ins, gate, nw, w, ws, y, final_state=st, cu_seqlens=cu, **k), (y, st)
    return call, size


def _scan(torch, kda, gen):
    T, H, D = 4096, 2, 128
    ins = _prompt(torch, gen, T, H, D)
    size = kda.kda_chunk_prefill_scan_workspace_bytes(T, H, D, 64, 8)

    def call(**k):
        o, st = torch.zeros((T, H, D), dtype=torch.bfloat16, device="cuda"), torch.zeros((H, D, D), device="cuda")
        torch.cuda.synchronize()
        return lambda: kda.kda_chunk_prefill_scan(*ins, o, 8, final_state=st, **k), (o, st)
    return call, size


def _split(torch, kda, gen):
    T, H, D = 6000, 2, 128
    ins = _prompt(torch, gen, T, H, D)
    cu = np.array([0, 100, 5900, T], dtype=np.int64)
    size = 1 << 22

    def call(**k):
        o, st = torch.zeros((T, H, D), dtype=torch.bfloat16, device="cuda"), torch.zeros((3, H, D, D), device="cuda")
        torch.cuda.synchronize()
        return lambda: kda.kda_chunk_prefill_split(*ins, o, cu, final_state=st, **k), (o, st)
    return call, size


@pytest.mark.parametrize("make", [_decode_proj, _prefill_proj, _scan, _split])
def test_own_workspace_on_another_stream(env, make):
    """The call waits behind other work on its stream while the current stream allocates and fills blocks of the
    workspace's size; the result has the bits of a call made alone."""
    torch, kda = env
    call, size = make(torch, kda, torch.Generator(device="cuda").manual_seed(17))
    go, want = call()
    go()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        go, got = call(stream=side)
        blocks = [torch.empty(size, dtype=torch.uint8, device="cuda").fill_(255) for _ in range(2)]
        del blocks  # freed while the fills may still run
        with torch.cuda.stream(side):
            torch.cuda._sleep(4_000_000)  # cycles, about 2 ms
        go()
        after = [torch.empty(size, dtype=torch.uint8, device="cuda").fill_(255) for _ in range(4)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        for t in after:
            assert bool((t == 255).all())
    kda.kda_sync_status()


def test_ways_out_without_tokens(env):
    """No sequences at a decode step and no tokens of a prompt: nothing is launched but the states' passage."""
    torch, kda = env
    H, D, hidden, bf = 4, 128, 256, torch.bfloat16
    w, ws = _weight(torch, torch.Generator(device="cuda").manual_seed(1), hidden, H * D)
    z = lambda *s, dt=torch.float32: torch.zeros(s, dtype=dt, device="cuda")  # noqa: E731
    nw = torch.ones(D, device="cuda")
    kda.kda_shortconv_decode_step_proj(z(0, 3, H, D, dt=bf), z(0, 3, H, 3, D, dt=bf), z(3, H, D, 4), z(0, H, D), z(0, H),
                                       z(0, H, D, D), z(0, H, D, dt=bf), nw, w, ws, z(0, hidden, dt=bf))
    none = [z(0, H, D, dt=bf)] * 3 + [z(0, H, D), z(0, H), z(0, H, D, dt=bf), nw, w, ws, z(0, hidden, dt=bf)]
    for n, cu in ((1, None), (3, torch.zeros(4, dtype=torch.int64, device="cuda"))):
        s0 = torch.randn((n, H, D, D), device="cuda")
        s1 = torch.full_like(s0, float("nan"))
        for k in ({}, {"stream": torch.cuda.Stream()}):
            torch.cuda.synchronize()
            kda.kda_chunk_prefill_proj(*none, initial_state=s0, final_state=s1, cu_seqlens=cu, **k)
            torch.cuda.synchronize()
            assert torch.equal(s0, s1)
    kda.kda_sync_status()
