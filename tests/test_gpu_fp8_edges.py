"""GPU tests of kda_fp8_linear where its parts meet: results that leave through two alternating pieces of shared
memory. Bounds as counted in tests/_fp8.py, evaluated in fp64 on the GPU."""
import pytest

from tests import _fp8
from tests._util import cuda_or_skip, ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    torch = cuda_or_skip()
    ensure_built()
    from linear_attention_recurrence_02_gb300 import kda
    return torch, kda


def _case(torch, seed, M, N, K):
    g = torch.Generator(device="cuda").manual_seed(seed)
    a = (torch.randn((M, K), generator=g, device="cuda") * 120).clamp(-448, 448).to(torch.float8_e4m3fn)
    w = (torch.randn((N, K), generator=g, device="cuda") * 110).clamp(-448, 448).to(torch.float8_e4m3fn)
    kb = _fp8.nblocks(K)
    sa = torch.exp(torch.randn((kb, M), generator=g, device="cuda")) / 100
    sw = torch.exp(torch.randn((_fp8.nblocks(N), kb), generator=g, device="cuda")) / 100
    return a, sa, w, sw


def _bound(torch, a, sa, w, sw):
    """The product and the bound of tests/_fp8.py's check_linear without its bf16 term, in fp64."""
    K, N = a.shape[1], w.shape[0]
    y = mag = 0.0
    rows = torch.arange(N, device="cuda") // _fp8.BLOCK
    for b in range(_fp8.nblocks(K)):
        c = slice(b * _fp8.BLOCK, (b + 1) * _fp8.BLOCK)
        ab, wb = a[:, c].double(), w[:, c].double()
        s = sa[b].double()[:, None] * sw[rows, b].double()[None, :]
        y, mag = y + (ab @ wb.t()) * s, mag + (ab.abs() @ wb.abs().t()) * s
    return y, mag * (2 * 128 + 2 + _fp8.nblocks(K)) * _fp8.U + 1e-37


@pytest.mark.parametrize("M,N,K", [(19_800, 2603, 16), (19_800, 2635, 16), (19_800, 2635, 144), (20_011, 587, 528)])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_linear_ragged_columns_of_many_token_tiles(env, M, N, K, out):
    """More token tiles than CTA pairs, so that a pair stores two tiles of the last columns one after the other, of
    which the last piece goes by ordinary stores between tensor copies: every element, several times."""
    torch, kda = env
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[out]
    a, sa, w, sw = _case(torch, N + K, M, N, K)
    ref, tol = _bound(torch, a, sa, w, sw)
    if out == "bf16":
        tol = tol + ref.abs() * 2.0 ** -8
    ld = (N + 7) // 8 * 8
    big = torch.empty((M, ld), dtype=dt, device="cuda")
    for k in range(6):
        big.fill_(-9.0 - k)
        kda.kda_fp8_linear(a, sa, w, sw, big[:, :N])
        assert bool(((big[:, :N].double() - ref).abs() <= tol).all())
        assert bool((big[:, N:] == -9.0 - k).all())
    kda.kda_sync_status()


def test_linear_shared_tiles_back_to_back(env):
    """Tiles shared by two and four CTA pairs, forty calls without a wait in between: the same bits each time."""
    torch, kda = env
    for M, N, K in ((500, 4000, 4112), (250, 3800, 12304)):
        a, sa, w, sw = _case(torch, M, M, N, K)
        outs = [torch.full((M, N), float("nan"), device="cuda") for _ in range(40)]
        for y in outs:
            kda.kda_fp8_linear(a, sa, w, sw, y)
        ref, tol = _bound(torch, a, sa, w, sw)
        assert bool(((outs[0].double() - ref).abs() <= tol).all())
        for y in outs[1:]:
            assert torch.equal(y, outs[0])
    kda.kda_sync_status()


@pytest.mark.parametrize("M,N,K,ld", [(48, 39_680, 6912, 6928), (96, 21_760, 6656, 6672), (128, 19_968, 5376, 5392),
                                      (128, 19_968, 5360, 5376), (300, 30_000, 1024, 1040), (33, 700, 400, 512),
                                      (500, 4000, 4096, 4112)])
def test_linear_bits_do_not_depend_on_strides(env, M, N, K, ld):
    """Contiguous operands and slices of wider rows, results whole and as a slice, in fp32 and rounded to bf16."""
    torch, kda = env
    a, sa, w, sw = _case(torch, M + K, M, N, K)
    wide = [torch.zeros((t.shape[0], ld), dtype=torch.uint8, device="cuda").view(t.dtype) for t in (a, w)]
    for t, b in zip((a, w), wide):
        b.view(torch.uint8)[:, :K] = t.view(torch.uint8)
    want = torch.empty((M, N), device="cuda")
    kda.kda_fp8_linear(a, sa, w, sw, want)
    for x, z in ((wide[0], w), (a, wide[1]), wide):
        for dt in (torch.float32, torch.bfloat16):
            for ldy in (N, N + 5):
                y = torch.empty((M, ldy), dtype=dt, device="cuda")[:, :N]
                kda.kda_fp8_linear(x[:, :K], sa, z[:, :K], sw, y)
                assert torch.equal(y, want.to(dt))


def test_scales_and_weights_written_by_the_kernel_ahead(env):
    """What a product writes is the next norm's weight and the next product's scales of both kinds, buffers used
    again at once with other values and no wait in between: the bits of the same calls made one at a time."""
    torch, kda = env
    K, f8 = 512, torch.float8_e4m3fn
    gen = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn((24, K), generator=gen, device="cuda")
    a, sa, w, sw = _case(torch, 6, 6, K, 256)  # six rows of products: the weights of six rounds
    d, sd, v, sv = _case(torch, 7, 300, 640, K)
    og = torch.randn((24, 4, 128), generator=gen, device="cuda")

    def rounds(wait):
        weight = torch.zeros((1, K), device="cuda")  # one buffer for every round's weight and scales
        q, s = torch.zeros((24, K), dtype=f8, device="cuda"), torch.zeros((4, 24), device="cuda")
        y = torch.zeros((24, 640), device="cuda")
        out = []

        def call(fn, *args, **k):
            fn(*args, **k)
            if wait:
                torch.cuda.synchronize()

        for i in range(6):
            call(kda.kda_fp8_linear, a[i:i + 1], sa[:, i:i + 1].contiguous(), w, sw, weight)
            call(kda.kda_add_rmsnorm_fp8, x, weight[0], q, s)
            out += [q.view(torch.uint8).clone(), s.clone()]
            call(kda.kda_fp8_linear, a[i:i + 1], sa[:, i:i + 1].contiguous(), w, sw, weight)
            call(kda.kda_gated_rmsnorm_fp8, x.view(24, 4, 128), og, weight[0, :128], q.view(24, 4, 128), s)
            call(kda.kda_fp8_linear, q, s, v, sv, y)  # scales from the norm just ahead
            out += [q.view(torch.uint8).clone(), y.clone()]
            call(kda.kda_fp8_linear, a[i:i + 1], sa[:, i:i + 1].contiguous(), w, sw, weight)
            call(kda.kda_fp8_linear, q, s, v, weight[0, :20].view(5, 4), y)  # a weight's scales from a product
            out.append(y.clone())
            z = torch.zeros((128, 640), device="cuda")
            call(kda.kda_fp8_linear, a[i:i + 1], sa[:, i:i + 1].contiguous(), w, sw, weight)
            call(kda.kda_fp8_linear, d[:128], weight.view(4, 128), v, sv, z)  # and a token's
            out.append(z)
        return out

    for _ in range(5):
        for got, want in zip(rounds(False), rounds(True)):
            assert torch.equal(got, want)
    kda.kda_sync_status()
