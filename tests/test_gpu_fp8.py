"""GPU tests of the 8-bit operators (kda_add_rmsnorm_fp8, kda_gated_rmsnorm_fp8,
kda_fp8_linear) against fp64 statements of the same formulas, element by
element; the tolerances are counted in tests/_fp8.py."""
import numpy as np
import pytest

import oracle
from tests import _fp8
from tests._util import cuda_or_skip, ensure_built, to_np

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    torch = cuda_or_skip()
    ensure_built()
    from linear_attention_recurrence_02_gb300 import kda
    return torch, kda


def _gen(torch, seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _dt(torch, name):
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


# ---------------------------------------------------------------- residual add + RMSNorm
def _add_case(torch, seed, T, N, dtype, res):
    g = _gen(torch, seed)
    x = torch.randn((T, N), generator=g, device="cuda").to(_dt(torch, dtype))
    r = None if res == "none" else (3 * torch.randn((T, N), generator=g, device="cuda")).to(_dt(torch, res))
    w = torch.rand(N, generator=g, device="cuda") + 0.5
    return x, r, w


def _add_out(torch, T, N, guard=2):
    """Codes and scales with `guard` rows behind the last token that must keep their bytes."""
    y = torch.full((T + guard, N), 77, dtype=torch.uint8, device="cuda")
    s = torch.full((_fp8.nblocks(N) * T + 8,), -5.0, device="cuda")
    return y, s, y[:T].view(torch.float8_e4m3fn), s[:_fp8.nblocks(N) * T].view(_fp8.nblocks(N), T)


@pytest.mark.parametrize("T,N", [(1, 16), (3, 112), (1, 128), (7, 144), (2, 1040), (5, 4096), (1, 8192), (3, 8208),
                                 (2, 16400), (2, 32768), (130, 272)])
@pytest.mark.parametrize("dtype,res", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16"), ("f32", "none")])
def test_add_rmsnorm(env, T, N, dtype, res):
    torch, kda = env
    x, r, w = _add_case(torch, 1000 * T + N, T, N, dtype, res)
    yb, sb, y, s = _add_out(torch, T, N)
    so = torch.empty_like(x if r is None else r)
    kda.kda_add_rmsnorm_fp8(x, w, y, s, residual=r, sum_out=so)
    h, ref = _fp8.add_rmsnorm(to_np(x), None if r is None else to_np(r), to_np(w), 1e-6)
    _fp8.check_codes(ref, _fp8.codes_to_np(y), to_np(s), _fp8.add_norm_steps(N), f"{T}x{N}")
    half = 2.0 ** -8 if so.dtype == torch.bfloat16 else _fp8.U  # one rounding of the sum (two into bf16)
    assert np.all(np.abs(to_np(so) - h) <= np.abs(h) * (half + 2 * _fp8.U))
    assert bool((yb[T:] == 77).all()) and bool((sb[s.numel():] == -5.0).all())


def test_add_rmsnorm_without_sum_and_in_place(env):
    """sum_out may be absent, the residual itself, or x of the same type; codes and scales are the same bits."""
    torch, kda = env
    T, N = 9, 2048
    x, r, w = _add_case(torch, 3, T, N, "bf16", "bf16")
    outs = []
    for how in ("none", "own", "residual", "x"):
        xi, ri = x.clone(), r.clone()
        _, _, y, s = _add_out(torch, T, N)
        so = {"none": None, "own": torch.empty_like(r), "residual": ri, "x": xi}[how]
        kda.kda_add_rmsnorm_fp8(xi, w, y, s, residual=ri, sum_out=so)
        outs.append((y.view(torch.uint8).clone(), s.clone(), so))
    for y, s, so in outs[1:]:
        assert torch.equal(y, outs[0][0]) and torch.equal(s, outs[0][1]) and torch.equal(so, outs[1][2])


def test_add_rmsnorm_zero_rows_and_small_blocks(env):
    """A row of zeros with eps = 0, a block of zeros inside a row, and a block so small that its scale is
    the floor's."""
    torch, kda = env
    x = torch.randn((4, 384), generator=_gen(torch, 5), device="cuda")
    x[1] = 0
    x[2, 128:256] = 0
    w = torch.ones(384, device="cuda")
    w[256:] = 1e-36
    _, _, y, s = _add_out(torch, 4, 384)
    kda.kda_add_rmsnorm_fp8(x, w, y, s, eps=0.0)
    c, sc = _fp8.codes_to_np(y), to_np(s)
    floor = np.float32(2.0 ** -96) / np.float32(448)
    assert np.all(c[1] == 0) and np.all(sc[:, 1] == floor)
    assert np.all(c[2, 128:256] == 0) and sc[1, 2] == floor
    assert np.all(sc[2] == floor)
    _, ref = _fp8.add_rmsnorm(to_np(x), None, to_np(w), 0.0)
    assert np.all(np.abs(c[:, 256:] * floor - ref[:, 256:]) <= 2.0 ** -10 * floor + np.abs(ref[:, 256:]) * 0.0626)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_add_rmsnorm_non_finite(env, bad):
    """A NaN makes its whole row NaN codes (its norm is NaN); with an infinity the other channels are
    finite / inf = 0 and its own is NaN. Other rows are untouched."""
    torch, kda = env
    x = torch.randn((3, 256), generator=_gen(torch, 6), device="cuda")
    clean = x.clone()
    x[1, 7] = bad
    w = torch.ones(256, device="cuda")
    _, _, y, s = _add_out(torch, 3, 256)
    _, _, y2, s2 = _add_out(torch, 3, 256)
    kda.kda_add_rmsnorm_fp8(x, w, y, s)
    kda.kda_add_rmsnorm_fp8(clean, w, y2, s2)
    c = _fp8.codes_to_np(y)
    if np.isnan(bad):
        assert np.all(np.isnan(c[1]))
    else:
        assert np.isnan(c[1, 7]) and np.all(np.delete(c[1], 7) == 0)
    for row in (0, 2):
        assert np.array_equal(c[row], _fp8.codes_to_np(y2)[row]) and torch.equal(s[:, row], s2[:, row])


def test_add_rmsnorm_offsets_past_32_bits(env):
    """140,000 x 32,768 elements (4.6e9): the last rows, whose offsets pass 32 bits."""
    torch, kda = env
    T, N = 140_000, 32_768
    x = torch.zeros((T, N), dtype=torch.bfloat16, device="cuda")
    x[-3:] = torch.randn((3, N), generator=_gen(torch, 8), device="cuda").bfloat16()
    w = torch.rand(N, generator=_gen(torch, 9), device="cuda") + 0.5
    y = torch.empty((T, N), dtype=torch.float8_e4m3fn, device="cuda")
    s = torch.empty((N // 128, T), device="cuda")
    kda.kda_add_rmsnorm_fp8(x, w, y, s)
    _, ref = _fp8.add_rmsnorm(to_np(x[-3:]), None, to_np(w), 1e-6)
    _fp8.check_codes(ref, _fp8.codes_to_np(y[-3:]), to_np(s[:, -3:]), _fp8.add_norm_steps(N))
    assert not bool(y[70_000].view(torch.uint8).any())


# ---------------------------------------------------------------- gated RMSNorm
@pytest.mark.parametrize("T,H,D", [(1, 1, 16), (1, 1, 128), (5, 3, 16), (37, 5, 64), (4, 9, 32), (33, 8, 16),
                                   (7, 96, 128), (3, 2, 128)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("act", ["sigmoid", "silu"])
def test_gated_rmsnorm_fp8(env, T, H, D, dtype, act):
    torch, kda = env
    g = _gen(torch, T * 100 + H * 10 + D)
    o = torch.randn((T, H, D), generator=g, device="cuda") * torch.exp(torch.randn((T, H, 1), generator=g,
                                                                                  device="cuda"))
    o, z = o.to(_dt(torch, dtype)), (2 * torch.randn((T, H, D), generator=g, device="cuda")).to(_dt(torch, dtype))
    w = torch.rand(D, generator=g, device="cuda") + 0.5
    if T > 2:
        o[2, 0] = 0
    yb, sb, y, s = _add_out(torch, T, H * D)
    kda.kda_gated_rmsnorm_fp8(o, z, w, y.view(T, H, D), s, act=act)
    ref = oracle.gated_rmsnorm(to_np(o), to_np(z), to_np(w), act=act).reshape(T, H * D)
    _fp8.check_codes(ref, _fp8.codes_to_np(y), to_np(s), _fp8.gated_steps(float(z.abs().max())), f"{T}x{H}x{D}")
    assert bool((yb[T:] == 77).all()) and bool((sb[s.numel():] == -5.0).all())


def test_gated_rmsnorm_fp8_extreme_gates(env):
    """Gates that close (-1e4: zeros) and open (1e4) and a NaN gate, which stays in its own channel."""
    torch, kda = env
    o = torch.randn((2, 2, 128), generator=_gen(torch, 4), device="cuda")
    z = torch.full((2, 2, 128), 1e4, device="cuda")
    z[0, 0] = -1e4
    z[1, 1, 5] = float("nan")
    w = torch.ones(128, device="cuda")
    _, _, y, s = _add_out(torch, 2, 256)
    kda.kda_gated_rmsnorm_fp8(o, z, w, y.view(2, 2, 128), s)
    c = _fp8.codes_to_np(y).reshape(2, 2, 128)
    assert np.all(c[0, 0] == 0)
    assert np.isnan(c[1, 1, 5]) and np.isfinite(np.delete(c[1, 1], 5)).all()
    assert np.abs(np.delete(c[1, 1], 5)).max() == 448


# ---------------------------------------------------------------- linear
def _lin_case(torch, seed, M, N, K):
    g = _gen(torch, seed)
    f8 = torch.float8_e4m3fn
    a = (torch.randn((M, K), generator=g, device="cuda") * 120).clamp(-448, 448).to(f8)
    w = (torch.randn((N, K), generator=g, device="cuda") * 110).clamp(-448, 448).to(f8)
    kb = _fp8.nblocks(K)
    sa = torch.exp(torch.randn((kb, M), generator=g, device="cuda")) / 100
    sw = torch.exp(torch.randn((_fp8.nblocks(N), kb), generator=g, device="cuda")) / 100
    return a, sa, w, sw


def _lin_check(torch, y, a, sa, w, sw, what=""):
    _fp8.check_linear(to_np(y), _fp8.codes_to_np(a), to_np(sa), _fp8.codes_to_np(w), to_np(sw),
                      y.dtype == torch.bfloat16, what)


LINEAR_SHAPES = [(1, 1, 16), (1, 128, 128), (2, 7, 144), (16, 130, 256), (17, 96, 1040), (33, 1000, 272),
                 (64, 256, 2048), (65, 129, 128), (128, 384, 640), (129, 257, 400), (300, 520, 1168), (777, 1000, 1040),
                 (1, 640, 12288), (513, 1153, 512)]


@pytest.mark.parametrize("M,N,K", LINEAR_SHAPES)
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_linear(env, M, N, K, out):
    torch, kda = env
    a, sa, w, sw = _lin_case(torch, M + N + K, M, N, K)
    y = torch.full((M, N), float("nan"), dtype=_dt(torch, out), device="cuda")
    kda.kda_fp8_linear(a, sa, w, sw, y)
    kda.kda_sync_status()
    _lin_check(torch, y, a, sa, w, sw, f"{M}x{N}x{K}")
    again = torch.empty_like(y)
    kda.kda_fp8_linear(a, sa, w, sw, again)
    assert torch.equal(y, again)  # the same inputs give the same bits


@pytest.mark.parametrize("M", [3, 40, 200, 600])
def test_linear_row_strides(env, M):
    """Operands and result as slices of wider rows: what lies between the rows is not read into the result
    (it holds NaN codes) nor written."""
    torch, kda = env
    N, K = 200, 400
    a, sa, w, sw = _lin_case(torch, 20, M, N, K)
    big_a = torch.full((M, K + 48), 0x7f, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    big_w = torch.full((N, K + 112), 0x7f, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    big_a.view(torch.uint8)[:, 16:16 + K] = a.view(torch.uint8)
    big_w.view(torch.uint8)[:, 32:32 + K] = w.view(torch.uint8)
    for dt in (torch.bfloat16, torch.float32):
        for off, ld in ((8, N + 24), (0, N + 3)):
            big_y = torch.full((M, ld), -7.0, dtype=dt, device="cuda")
            y = big_y[:, off:off + N]
            kda.kda_fp8_linear(big_a[:, 16:16 + K], sa, big_w[:, 32:32 + K], sw, y)
            _lin_check(torch, y, a, sa, w, sw, f"{M} {dt} {off}")
            assert bool((big_y[:, :off] == -7.0).all()) and bool((big_y[:, off + N:] == -7.0).all())


def test_linear_refuses_rows_it_cannot_copy(env):
    torch, kda = env
    a, sa, w, sw = _lin_case(torch, 21, 4, 32, 64)
    wide = torch.zeros((4, 72), dtype=torch.float8_e4m3fn, device="cuda")
    y = torch.zeros((4, 32), device="cuda")
    with pytest.raises(kda.KdaError, match="multiples of 16"):
        kda.kda_fp8_linear(wide[:, :64], sa, w, sw, y)
    with pytest.raises(ValueError, match="contiguous"):
        kda.kda_fp8_linear(a, sa, w, sw, torch.zeros((32, 4), device="cuda").t())
    with pytest.raises(kda.KdaError, match="aligned"):
        kda.kda_fp8_linear(torch.zeros((4, 160), dtype=torch.float8_e4m3fn, device="cuda")[:, 8:72], sa, w, sw, y)


@pytest.mark.parametrize("M", [5, 200])
def test_linear_non_finite_stays_in_its_row(env, M):
    """A NaN code and an infinite scale reach their own token's outputs and no other's."""
    torch, kda = env
    N, K = 150, 304
    a, sa, w, sw = _lin_case(torch, 22, M, N, K)
    y0, y = torch.empty((M, N), device="cuda"), torch.empty((M, N), device="cuda")
    kda.kda_fp8_linear(a, sa, w, sw, y0)
    a2, sa2 = a.clone(), sa.clone()
    a2.view(torch.uint8)[1, 290] = 0x7f
    sa2[0, 3] = float("inf")
    kda.kda_fp8_linear(a2, sa2, w, sw, y)
    assert bool(torch.isnan(y[1]).all()) and not bool(torch.isfinite(y[3]).any())
    keep = [i for i in range(M) if i not in (1, 3)]
    assert torch.equal(y[keep], y0[keep])


def test_linear_offsets_past_32_bits(env):
    """66,000 x 36,864 results (2.4e9): rows at both ends and in the middle of the tensor."""
    torch, kda = env
    M, N, K = 66_000, 36_864, 48
    a, sa, w, sw = _lin_case(torch, 23, M, N, K)
    y = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    kda.kda_fp8_linear(a, sa, w, sw, y)
    for r in (slice(0, 2), slice(58_254, 58_256), slice(M - 2, M)):
        _lin_check(torch, y[r], a[r], sa[:, r], w, sw, str(r))


def test_linear_zero_tokens(env):
    torch, kda = env
    _, _, w, sw = _lin_case(torch, 24, 1, 64, 128)
    f8 = torch.float8_e4m3fn
    kda.kda_fp8_linear(torch.empty((0, 128), dtype=f8, device="cuda"), torch.empty((1, 0), device="cuda"), w, sw,
                       torch.empty((0, 64), device="cuda"))
    kda.kda_sync_status()


# ---------------------------------------------------------------- streams and graphs
@pytest.mark.parametrize("M", [2, 48, 600])
def test_fp8_chain_on_a_side_stream_and_in_a_graph(env, M):
    """norm -> linear on a stream of its own, then captured and replayed twice on new inputs: the same bits
    as direct calls on the default stream."""
    torch, kda = env
    N, K = 264, 1040
    x, r, nw = _add_case(torch, 31, M, K, "bf16", "f32")
    _, _, w, sw = _lin_case(torch, 32, 1, N, K)
    q = torch.empty((M, K), dtype=torch.float8_e4m3fn, device="cuda")
    s, y = torch.empty((_fp8.nblocks(K), M), device="cuda"), torch.empty((M, N), device="cuda")

    def chain():
        kda.kda_add_rmsnorm_fp8(x, nw, q, s, residual=r)
        kda.kda_fp8_linear(q, s, w, sw, y)

    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    chain()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        chain()
    for k in range(2):
        x.copy_(torch.randn((M, K), generator=_gen(torch, 40 + k), device="cuda"))
        chain()
        direct = y.clone()
        y.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            chain()
        side.synchronize()
        assert torch.equal(y, direct)
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, direct)


def test_linear_two_streams_at_once(env):
    """Calls that overlap on two streams share nothing: the bits of calls made alone."""
    torch, kda = env
    cases = [_lin_case(torch, 50 + i, m, 700, 4096) for i, m in enumerate((3, 64, 300))]
    alone = []
    for c in cases:
        y = torch.empty((c[0].shape[0], 700), device="cuda")
        kda.kda_fp8_linear(*c, y)
        alone.append(y)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = [[torch.empty_like(y) for _ in range(4)] for y in alone]
    for k in range(4):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                kda.kda_fp8_linear(*cases[i], outs[i][k])
    torch.cuda.synchronize()
    for i in range(3):
        for k in range(4):
            assert torch.equal(outs[i][k], alone[i])


@pytest.mark.parametrize("M,N,K", [(130, 520, 4112), (20, 300, 2064), (64, 96, 4096), (2600, 2600, 272), (2600, 2601, 128),
                                   (1000, 640, 3600)])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_linear_splits_and_several_tiles(env, M, N, K, out):
    """K split over a cluster with uneven runs and several token tiles, and CTA pairs that take more than one
    tile; a sample of rows from every tile, and the same bits twice."""
    torch, kda = env
    a, sa, w, sw = _lin_case(torch, 70 + M, M, N, K)
    y = torch.full((M, N), float("nan"), dtype=_dt(torch, out), device="cuda")
    kda.kda_fp8_linear(a, sa, w, sw, y)
    kda.kda_sync_status()
    assert bool(torch.isfinite(y).all())
    rows = torch.arange(0, M, 1 if M < 200 else 13, device="cuda")
    _lin_check(torch, y[rows], a.view(torch.uint8)[rows].view(a.dtype), sa[:, rows], w, sw, f"{M}x{N}x{K}")
    again = torch.empty_like(y)
    kda.kda_fp8_linear(a, sa, w, sw, again)
    assert torch.equal(y, again)


def test_norms_zero_tokens(env):
    torch, kda = env
    f8 = torch.float8_e4m3fn
    e = lambda *s, dt=torch.float32: torch.empty(s, dtype=dt, device="cuda")  # noqa: E731
    kda.kda_add_rmsnorm_fp8(e(0, 256), e(256), e(0, 256, dt=f8), e(2, 0))
    kda.kda_gated_rmsnorm_fp8(e(0, 3, 64), e(0, 3, 64), e(64), e(0, 3, 64, dt=f8), e(2, 0))
    kda.kda_sync_status()


def test_calls_on_a_given_stream_follow_it(env):
    """stream= names the stream: work queued on it ahead of the call is seen, without any other order."""
    torch, kda = env
    M, N, K = 40, 300, 1040
    _, sa, w, sw = _lin_case(torch, 91, M, N, K)
    x, r, nw = _add_case(torch, 92, M, K, "f32", "f32")
    q, s = torch.empty((M, K), dtype=torch.float8_e4m3fn, device="cuda"), torch.empty_like(sa)
    want, got = torch.empty((M, N), device="cuda"), torch.empty((M, N), device="cuda")
    kda.kda_add_rmsnorm_fp8(x, nw, q, s, residual=r)
    kda.kda_fp8_linear(q, s, w, sw, want)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    x2, q2, s2 = torch.zeros_like(x), torch.zeros_like(q), torch.zeros_like(s)
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        for _ in range(20):
            x2.copy_(x)
    kda.kda_add_rmsnorm_fp8(x2, nw, q2, s2, residual=r, stream=st)
    kda.kda_fp8_linear(q2, s2, w, sw, got, stream=st)
    st.synchronize()
    assert torch.equal(got, want)


def test_linear_behind_a_kernel_that_rewrites_its_operands(env):
    """The product is launched while the kernel before it still runs: operands (the weight as well) that
    this kernel writes are read only when it has finished."""
    torch, kda = env
    for M in (16, 600):
        N, K = 512, 2048
        a, sa, w, sw = _lin_case(torch, 95 + M, M, N, K)
        want, got = torch.empty((M, N), device="cuda"), torch.empty((M, N), device="cuda")
        kda.kda_fp8_linear(a, sa, w, sw, want)
        a2, w2 = torch.zeros_like(a.view(torch.uint8)), torch.zeros_like(w.view(torch.uint8))
        sa2, sw2 = torch.zeros_like(sa), torch.zeros_like(sw)
        for _ in range(5):
            for t in (a2, w2, sa2, sw2):
                t.zero_()
            kda.kda_fp8_linear(a2.view(a.dtype), sa2, w2.view(w.dtype), sw2, got)
            sa2.copy_(sa)
            sw2.copy_(sw)
            a2.copy_(a.view(torch.uint8))
            w2.copy_(w.view(torch.uint8))
            kda.kda_fp8_linear(a2.view(a.dtype), sa2, w2.view(w.dtype), sw2, got)
            assert torch.equal(got, want)


def test_capture_with_forked_streams(env):
    """Captured with the two norms on a stream of their own between event waits, a copy ahead of them: the
    replay gives the bits of direct calls."""
    torch, kda = env
    M, N, K = 40, 260, 1024
    _, sa, w, sw = _lin_case(torch, 101, M, N, K)
    x, r, nw = _add_case(torch, 102, M, K, "bf16", "bf16")
    src = x.clone()
    q, s = torch.empty((M, K), dtype=torch.float8_e4m3fn, device="cuda"), torch.empty_like(sa)
    y, z = torch.empty((M, N), device="cuda"), torch.empty((M, N), device="cuda")
    og, gw = torch.randn((M, 8, 128), device="cuda").bfloat16(), torch.ones(128, device="cuda")
    q2, s2 = torch.empty((M, 8, 128), dtype=torch.float8_e4m3fn, device="cuda"), torch.empty_like(sa)
    side = torch.cuda.Stream()

    def work():
        x.copy_(src)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            kda.kda_gated_rmsnorm_fp8(x.view(M, 8, 128), og, gw, q2, s2)
        kda.kda_add_rmsnorm_fp8(x, nw, q, s, residual=r)
        kda.kda_fp8_linear(q, s, w, sw, y)
        torch.cuda.current_stream().wait_stream(side)
        kda.kda_fp8_linear(q2.view(M, K), s2, w, sw, z)

    work()
    torch.cuda.synchronize()
    want = y.clone(), z.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        work()
    for _ in range(3):
        y.zero_()
        z.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[0]) and torch.equal(z, want[1])


def test_linear_result_feeds_the_next_calls_input(env):
    """Ten products in a row, each reading what the one before wrote (through the norm), without any
    synchronisation, against the same calls made one at a time."""
    torch, kda = env
    for M in (1, 30, 300):
        K = 512
        w, sw = _lin_case(torch, 110 + M, 1, K, K)[2:]
        nw = torch.ones(K, device="cuda")
        start = torch.randn((M, K), generator=_gen(torch, M), device="cuda")
        q, s = torch.empty((M, K), dtype=torch.float8_e4m3fn, device="cuda"), torch.empty((4, M), device="cuda")

        def chain(wait):
            h = start.clone()
            for _ in range(10):
                kda.kda_add_rmsnorm_fp8(h, nw, q, s)
                if wait:
                    torch.cuda.synchronize()
                kda.kda_fp8_linear(q, s, w, sw, h)
                if wait:
                    torch.cuda.synchronize()
            return h

        assert torch.equal(chain(False), chain(True))


@pytest.mark.parametrize("M,N,K", [(500, 4000, 4112), (250, 3800, 12304), (385, 3970, 4096),
                                   (2560, 2250, 8192)])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_linear_pairs_that_share_a_tile(env, M, N, K, out):
    """Few tiles and a long K: two or four CTA pairs take a run of K blocks each (uneven ones among them) and
    exchange their sums; ragged tokens, features and channels, a result whose rows are a slice. The last size
    has a full wave of whole tiles ahead of the shared ones."""
    torch, kda = env
    a, sa, w, sw = _lin_case(torch, 130 + M, M, N, K)
    ld = N + (24 if out == "bf16" else 5)  # whole 16-byte rows, and rows that are not
    big = torch.full((M + 1, ld), -3.0, dtype=_dt(torch, out), device="cuda")
    y = big[:M, :N]
    kda.kda_fp8_linear(a, sa, w, sw, y)
    kda.kda_sync_status()
    rows = torch.arange(0, M, 7 if M < 600 else 41, device="cuda")
    _lin_check(torch, y[rows], a.view(torch.uint8)[rows].view(a.dtype), sa[:, rows], w, sw, f"{M}x{N}x{K}")
    assert bool(torch.isfinite(y).all()) and bool((big[:M, N:] == -3.0).all()) and bool((big[M:] == -3.0).all())
    again = torch.empty((M, N), dtype=y.dtype, device="cuda")
    for _ in range(3):
        kda.kda_fp8_linear(a, sa, w, sw, again)
        assert torch.equal(y, again)


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("M,N,off,ld", [(700, 1001, 0, 1001), (700, 1002, 0, 1002), (700, 1000, 8, 1031),
                                        (700, 1003, 8, 1040), (700, 260, 0, 263), (700, 961, 0, 963),
                                        (1500, 2001, 0, 2001), (1500, 2002, 0, 2002), (1530, 2000, 8, 2031),
                                        (1509, 2003, 8, 2040), (1500, 1985, 8, 1994), (1500, 2047, 0, 2048),
                                        (2600, 2603, 0, 2608)])
def test_linear_rows_of_any_alignment(env, M, N, off, ld, out):
    """Rows of the result at every alignment that the element size allows, whole and partial tiles: each
    element, and what lies beside it."""
    torch, kda = env
    K = 256
    a, sa, w, sw = _lin_case(torch, 150 + N, M, N, K)
    big = torch.full((M + 2, ld), -9.0, dtype=_dt(torch, out), device="cuda")
    y = big[:M, off:off + N]
    kda.kda_fp8_linear(a, sa, w, sw, y)
    _lin_check(torch, y, a, sa, w, sw, f"{N} {off} {ld}")
    assert bool((big[:M, :off] == -9.0).all()) and bool((big[:M, off + N:] == -9.0).all())
    assert bool((big[M:] == -9.0).all())


@pytest.mark.parametrize("K", [2048, 2064])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_linear_several_tiles_a_pair(env, K, out):
    """More tiles than CTA pairs at 16 and 17 K blocks: results that leave beside the next tile, and ahead of it."""
    torch, kda = env
    M, N = 2600, 2312
    a, sa, w, sw = _lin_case(torch, 160 + K, M, N, K)
    y = torch.full((M, N), float("nan"), dtype=_dt(torch, out), device="cuda")
    kda.kda_fp8_linear(a, sa, w, sw, y)
    assert bool(torch.isfinite(y).all())
    rows = torch.arange(0, M, 13, device="cuda")
    _lin_check(torch, y[rows], a.view(torch.uint8)[rows].view(a.dtype), sa[:, rows], w, sw, f"{M}x{N}x{K}")
    again = torch.empty_like(y)
    kda.kda_fp8_linear(a, sa, w, sw, again)
    assert torch.equal(y, again)


@pytest.mark.parametrize("M,N,K", [(66, 28677, 528), (100, 40000, 144), (128, 20000, 1040), (128, 1000, 4112), (101, 4001, 8208),
                                   (127, 12288, 272), (250, 4100, 4112), (1000, 330, 4880), (48, 40010, 272),
                                   (9, 41000, 144)])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_linear_some_tokens(env, M, N, K, out):
    """64 and 128 tokens at a time, split and unsplit, CTAs that walk several units: a sample of columns, what
    lies beside the result, and the same bits twice."""
    torch, kda = env
    a, sa, w, sw = _lin_case(torch, 180 + M, M, N, K)
    big = torch.full((M + 1, N + 3), -9.0, dtype=_dt(torch, out), device="cuda")
    y = big[:M, :N]
    kda.kda_fp8_linear(a, sa, w, sw, y)
    kda.kda_sync_status()
    assert bool((big[:M, N:] == -9.0).all()) and bool((big[M:] == -9.0).all())
    assert bool(torch.isfinite(y).all())
    # whole blocks of 128 features from the start, the middle and the end
    nb = _fp8.nblocks(N)
    blocks = sorted({0, 1 % nb, nb // 2, nb - 2 if nb > 1 else 0, nb - 1})
    for b in blocks:
        n0, n1 = 128 * b, min(128 * b + 128, N)
        _lin_check(torch, y[:, n0:n1], a, sa, w.view(torch.uint8)[n0:n1].view(w.dtype), sw[b:b + 1], f"{M}x{N}x{K} at {n0}")
    again = torch.empty_like(y)
    kda.kda_fp8_linear(a, sa, w, sw, again)
    assert torch.equal(y, again)
