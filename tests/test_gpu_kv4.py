"""GPU tests of the softmax-attention layers' operators against plain 64-bit forms: the head norms with the position
rotation, the 4-bit cache (bytes equal, values exact) and attention over it, one by one and as a layer's run.

Tolerances. A rounding to type t is off by at most u = finfo(t).eps / 2 of the value. A rotated, normalised value is
one rounding of a form of about ten fp32 operations (the root's, the reciprocal's and the sine's included). An attention output is off by the
rounding of each softmax factor to bf16 (2^-8 of sum p |v|; none with fp32 inputs), its own rounding, and what the
fp32 sums leave: scores of D products of size c are off by at most D 2^-23 c, which moves factors and their sum by
as much each, and sums over L tokens by at most (L + 64) 2^-23 of their terms.
"""
import numpy as np
import pytest

from tests import _kv4 as ref
from tests._util import cuda_or_skip, ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    torch = cuda_or_skip()
    ensure_built()
    from linear_attention_recurrence_02_gb300 import kda
    return torch, kda


def np64(t):
    return t.detach().double().cpu().numpy()


def half_step(torch, dt):
    return torch.finfo(dt).eps / 2


# ---------------------------------------------------------------- norms and rotation
@pytest.mark.parametrize("T,Hq,Hk,D,R,inter,dt,weights", [
    (1, 1, 1, 16, 16, False, "bfloat16", True),
    (1, 96, 8, 128, 128, False, "bfloat16", True),
    (3, 5, 2, 32, 32, True, "float32", True),
    (7, 3, 1, 64, 32, False, "float32", True),
    (5, 9, 3, 128, 64, True, "bfloat16", True),
    (400, 6, 2, 64, 64, False, "bfloat16", True),
    (500, 40, 8, 128, 128, False, "float32", True),
    (333, 17, 0, 128, 96, False, "bfloat16", True),
    (2, 300, 4, 128, 128, True, "bfloat16", True),
    (9, 4, 4, 128, 0, False, "float32", True),
    (9, 4, 4, 128, 128, False, "float32", False),
    (350, 130, 3, 16, 16, True, "float32", False),
])
def test_norm_rope(env, T, Hq, Hk, D, R, inter, dt, weights):
    torch, kda = env
    dt = getattr(torch, dt)
    gen = torch.Generator(device="cuda").manual_seed(T + Hq + D + R)
    wide = (torch.randn((T, (Hq + 2 * Hk) * D + 8), generator=gen, device="cuda") *
            torch.exp(torch.randn((T, 1), generator=gen, device="cuda"))).to(dt)
    q = wide[:, :Hq * D].unflatten(1, (Hq, D))
    k = wide[:, Hq * D:(Hq + Hk) * D].unflatten(1, (Hk, D)) if Hk else None
    qw, kw = (torch.rand(D, generator=gen, device="cuda") + 0.5 for _ in range(2)) if weights else (None, None)
    pos = torch.randint(-5000, 1 << 33, (T,), generator=gen, device="cuda")
    freq = 10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64, device="cuda") / max(R, 1)) if R else None
    qo, ko = torch.empty((T, Hq, D), dtype=dt, device="cuda"), torch.empty((T, Hk, D), dtype=dt, device="cuda") if Hk else None
    kda.kda_qk_norm_rope(q, k, qo, ko, pos if R else None, freq, q_weight=qw, k_weight=kw, interleaved=inter)
    kda.kda_sync_status()
    u = half_step(torch, dt)
    for x, w, y in ((q, qw, qo), (k, kw, ko)):
        if x is None:
            continue
        wn = None if w is None else np64(w)
        want = ref.norm_rope(np64(x), wn, pos.cpu().numpy(), None if freq is None else np64(freq), 1e-6, inter)
        plain = np.abs(ref.norm_rope(np64(x), wn, [0] * T, None, 1e-6, inter))
        # a turned channel has terms of both channels of its pair: their sizes are bounded by the row's largest
        tol = u * np.abs(want) + 16 * 2.0 ** -24 * 2 * plain.max(-1, keepdims=True) + 1e-30
        assert np.all(np.abs(np64(y) - want) <= tol)


def test_norm_rope_in_place_and_strided_out(env):
    torch, kda = env
    T, Hq, Hk, D = 37, 6, 2, 128
    gen = torch.Generator(device="cuda").manual_seed(3)
    wide = torch.randn((T, (Hq + 2 * Hk) * D), generator=gen, device="cuda").to(torch.bfloat16)
    view = lambda w: (w[:, :Hq * D].unflatten(1, (Hq, D)), w[:, Hq * D:(Hq + Hk) * D].unflatten(1, (Hk, D)))  # noqa: E731
    pos, freq = torch.arange(T, device="cuda"), torch.rand(D // 2, dtype=torch.float64, device="cuda", generator=gen)
    w = torch.rand(D, generator=gen, device="cuda")
    q, k = view(wide)
    qo, ko = torch.empty((T, Hq, D), dtype=q.dtype, device="cuda"), torch.empty((T, Hk, D), dtype=q.dtype, device="cuda")
    kda.kda_qk_norm_rope(q, k, qo, ko, pos, freq, q_weight=w, k_weight=w)
    other = wide.clone()
    q2, k2 = view(other)
    kda.kda_qk_norm_rope(q2, k2, q2, k2, pos, freq, q_weight=w, k_weight=w)
    assert torch.equal(q2, qo) and torch.equal(k2, ko)
    assert torch.equal(other[:, (Hq + Hk) * D:], wide[:, (Hq + Hk) * D:])


def test_norm_rope_zero_rows_and_nan_rows_stay_apart(env):
    torch, kda = env
    q = torch.randn((4, 2, 64), device="cuda")
    q[1, 0] = 0
    q[2, 1, 5] = float("nan")
    qo = torch.empty_like(q)
    kda.kda_qk_norm_rope(q, None, qo, None, None, None, q_weight=torch.ones(64, device="cuda"), eps=0.0)
    assert torch.equal(qo[1, 0], torch.zeros(64, device="cuda"))
    assert bool(qo[2, 1].isnan().all()) and not bool(qo.flatten(0, 1)[[0, 1, 2, 3, 4, 6, 7]].isnan().any())


@pytest.mark.parametrize("which", ["q", "k"])
@pytest.mark.parametrize("T", [3, 1300])
def test_norm_rope_with_one_weight(env, which, T):
    """Only the queries or only the keys are normed, though their rows share warps."""
    torch, kda = env
    gen = torch.Generator(device="cuda").manual_seed(8)
    q, k = (torch.randn((T, h, 32), generator=gen, device="cuda") for h in (3, 2))
    w = torch.rand(32, generator=gen, device="cuda")
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    kda.kda_qk_norm_rope(q, k, qo, ko, None, None, **{which + "_weight": w})
    for x, y, n in ((q, qo, "q"), (k, ko, "k")):
        want = ref.norm_rope(np64(x), np64(w) if n == which else None, [0] * T, None, 1e-6, False)
        assert np.all(np.abs(np64(y) - want) <= 2.0 ** -20 * np.abs(want))


@pytest.mark.parametrize("Hq,Hk,D,R,dt,inter", [(64, 8, 128, 128, "bfloat16", False), (3, 1, 64, 32, "float32", True),
                                                (40, 0, 128, 64, "float32", False), (5, 4, 16, 16, "bfloat16", True)])
def test_norm_rope_many_tokens(env, Hq, Hk, D, R, dt, inter):
    """The form for many tokens gives each token what a call on it alone gives."""
    torch, kda = env
    dt = getattr(torch, dt)
    gen = torch.Generator(device="cuda").manual_seed(Hq)
    T = 4 * 2 * torch.cuda.get_device_properties(0).multi_processor_count + 5
    wide = torch.randn((T, (Hq + Hk) * D + 16), generator=gen, device="cuda").to(dt)
    q = wide[:, :Hq * D].unflatten(1, (Hq, D))
    k = wide[:, Hq * D:(Hq + Hk) * D].unflatten(1, (Hk, D)) if Hk else None
    w, pos = torch.rand(D, generator=gen, device="cuda"), torch.randint(0, 1 << 20, (T,), generator=gen, device="cuda")
    freq = 10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64, device="cuda") / R)
    qo, ko = torch.empty((T, Hq, D), dtype=dt, device="cuda"), torch.empty((T, Hk, D), dtype=dt, device="cuda") if Hk else None
    kda.kda_qk_norm_rope(q, k, qo, ko, pos, freq, q_weight=w, k_weight=w, interleaved=inter)
    kda.kda_sync_status()
    q1, k1 = torch.empty_like(qo), None if ko is None else torch.empty_like(ko)
    for a in range(0, T, 100):
        s = slice(a, min(a + 100, T))
        kda.kda_qk_norm_rope(q[s], None if k is None else k[s], q1[s], None if k is None else k1[s], pos[s], freq, q_weight=w,
                             k_weight=w, interleaved=inter)
    assert torch.equal(qo, q1) and (k is None or torch.equal(ko, k1))
    wide2 = wide.clone()  # in place, too
    q2 = wide2[:, :Hq * D].unflatten(1, (Hq, D))
    k2 = wide2[:, Hq * D:(Hq + Hk) * D].unflatten(1, (Hk, D)) if Hk else None
    kda.kda_qk_norm_rope(q2, k2, q2, k2, pos, freq, q_weight=w, k_weight=w, interleaved=inter)
    assert torch.equal(q2, qo) and (k is None or torch.equal(k2, ko)) and torch.equal(wide2[:, -16:], wide[:, -16:])


# ---------------------------------------------------------------- the cache
def _layout(torch, rng, lens, page, spare=2, cols=None):
    """A block table over shuffled pages whose unused entries are pages that do not exist."""
    used = [-(-n // page) for n in lens]
    cols = max(max(used, default=0), 1) if cols is None else cols
    order = rng.permutation(sum(used) + spare)
    table, at = np.full((len(lens), cols), -77, np.int32), 0
    for b, n in enumerate(used):
        table[b, :n] = order[at:at + n]
        at += n
    return table, sum(used) + spare


def _dev(torch, a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


_SEQS = {  # lengths once the new tokens are in, and new tokens (None: one each)
    "steps": ([1, 17, 64, 0, 33, 130], None),
    "prompts": ([5, 64, 0, 100, 49], [5, 31, 0, 1, 49]),
    "one": ([1], None),
}


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("which,dt", [("steps", "bfloat16"), ("prompts", "float32"), ("one", "float32")])
def test_append_and_read(env, D, page, which, dt):
    """Bytes of the whole cache as the plain form leaves them: new tokens in, all else untouched; what is read
    back is what those bytes stand for; rows behind the last sequence stay as they are."""
    torch, kda = env
    dt = getattr(torch, dt)
    lens, new = _SEQS[which]
    counts = [1] * len(lens) if new is None else new
    rng = np.random.default_rng(D + page)
    Hk = 3
    table, pages = _layout(torch, rng, lens, page)
    extra = 0 if new is None else 4
    T = sum(counts) + extra
    wide = _dev(torch, rng.normal(size=(T, 2 * Hk * D)) * np.exp(rng.normal(size=(T, 1)))).to(dt)
    wide[0, :32] = 0                       # a group of zeros
    wide[0, Hk * D:Hk * D + 32] = torch.arange(-16, 16, device="cuda") / 4  # ties between codes
    k, v = wide[:, :Hk * D].unflatten(1, (Hk, D)), wide[:, Hk * D:].unflatten(1, (Hk, D))
    before = rng.integers(0, 256, size=(pages, Hk, page // 16, 18 * D)).astype(np.uint8)
    cache = _dev(torch, before)
    cu = None if new is None else np.concatenate([[0], np.cumsum(counts)])
    args = (_dev(torch, table), _dev(torch, np.array(lens, np.int64)))
    kda.kda_kv4_append(k, v, cache, *args, cu_seqlens=None if cu is None else _dev(torch, cu))
    kda.kda_sync_status()
    want, kn, vn, t = before.copy(), np64(k), np64(v), 0
    for b, (n, m) in enumerate(zip(lens, counts)):
        for i in range(m):
            p = n - m + i
            if p >= 0:
                for h in range(Hk):
                    ref.put(want[table[b, p // page], h, p % page // 16], p % 16, kn[t, h], vn[t, h])
            t += 1
    assert np.array_equal(cache.cpu().numpy(), want)

    for odt in (torch.float32, torch.bfloat16):
        ko, vo = (torch.full((T, Hk, D), 7.0, dtype=odt, device="cuda") for _ in range(2))
        kda.kda_kv4_read(cache, *args, ko, vo, cu_seqlens=None if cu is None else _dev(torch, cu))
        kda.kda_sync_status()
        t = 0
        for n, m in zip(lens, counts):
            for i in range(m):
                got, wk = (np64(ko[t]), np64(vo[t])), (ref.held(kn[t]), ref.held(vn[t]))
                if n - m + i < 0:
                    wk = (np.full((Hk, D), 7.0),) * 2
                assert np.array_equal(got[0], wk[0]) and np.array_equal(got[1], wk[1])
                t += 1
        assert bool((ko[t:] == 7).all()) and bool((vo[t:] == 7).all())


def test_append_many_tokens(env):
    """The form with several heads a thread (many tokens) writes the same bytes as one token at a time does."""
    torch, kda = env
    Hk, D, page, n = 6, 128, 32, 21000
    rng = np.random.default_rng(1)
    gen = torch.Generator(device="cuda").manual_seed(1)
    table, pages = _layout(torch, rng, [n], page)
    k, v = (torch.randn((n, Hk, D), generator=gen, device="cuda").to(torch.bfloat16) for _ in range(2))
    cache = torch.zeros((pages, Hk, page // 16, 18 * D), dtype=torch.uint8, device="cuda")
    tb, lens = _dev(torch, table), torch.tensor([n], device="cuda")
    kda.kda_kv4_append(k, v, cache, tb, lens, cu_seqlens=torch.tensor([0, n], device="cuda"))
    ko, vo = torch.empty_like(k), torch.empty_like(k)
    kda.kda_kv4_read(cache, tb, lens, ko, vo, cu_seqlens=torch.tensor([0, n], device="cuda"))
    for at in (0, 1, 15, 16, 4097, n - 1):
        one = torch.zeros_like(cache)
        kda.kda_kv4_append(k[at:at + 1], v[at:at + 1], one, tb, torch.tensor([at + 1], device="cuda"))
        pg = table[0, at // page]
        blk = one[pg, :, at % page // 16]
        same = cache[pg, :, at % page // 16]
        assert bool(((blk == 0) | (blk == same)).all()) and int((blk != 0).sum()) > 9 * D * Hk // 10
        for x, y in ((k, ko), (v, vo)):
            assert np.array_equal(ref.held(np64(x[at])), np64(y[at]))
    kda.kda_sync_status()


def test_quantising_edges(env):
    """Values next to a border between two codes or scales, the largest and smallest fp32, and groups that are not
    finite, which read back as NaN without touching their neighbours."""
    torch, kda = env
    D = 64
    rng = np.random.default_rng(5)
    x = rng.normal(size=(200, 1, D)).astype(np.float32)
    for i in range(60):  # scales of five bits, values on and beside the halves between codes
        s = (16 + i % 16) / 16 * 2.0 ** rng.integers(-8, 8)
        half = (rng.integers(-7, 7, 32) + 0.5) * s
        half[0] = 7 * s
        x[i, 0, :32] = half
        x[i, 0, 32:] = np.nextafter(half.astype(np.float32), np.float32(rng.choice([-1e9, 1e9])))
    for i in range(60, 100):  # largest values on and just beside 7 times a scale
        s = np.float32((16 + i % 16) / 16 * 2.0 ** rng.integers(-8, 8))
        x[i, 0, 5] = np.nextafter(7 * s, np.float32([0, 0, 1e9][i % 3])) if i % 3 else 7 * s
    x[100] *= 2.0 ** 120
    x[101] = 3.4e38
    x[102] *= 2.0 ** -120
    x[103] = 1e-44
    x[104, 0, 3], x[105, 0, 40], x[106, 0, :] = np.nan, np.inf, -np.inf
    x[107] = -0.0
    n = x.shape[0]
    table, pages = _layout(torch, rng, [n], 16)
    cache = torch.zeros((pages, 1, 1, 18 * D), dtype=torch.uint8, device="cuda")
    tb, lens, cu = _dev(torch, table), torch.tensor([n], device="cuda"), torch.tensor([0, n], device="cuda")
    k = _dev(torch, x)
    kda.kda_kv4_append(k, -k, cache, tb, lens, cu_seqlens=cu)
    ko, vo = torch.empty_like(k), torch.empty_like(k)
    kda.kda_kv4_read(cache, tb, lens, ko, vo, cu_seqlens=cu)
    kda.kda_sync_status()
    assert np.array_equal(np64(ko), ref.held(x.astype(np.float64)), equal_nan=True)
    assert np.array_equal(np64(vo), ref.held(-x.astype(np.float64)), equal_nan=True)


def test_quantising_every_bf16_quotient(env):
    """Every bf16 significand against every scale of five bits, of both signs, at the sizes where codes differ, with
    scales near both ends of their range too."""
    torch, kda = env
    D = 128
    rows = []
    for S in range(16, 32):
        for up in (0, -90, 110):
            x = np.array([X * 2.0 ** a for a in range(-7, 1) for X in range(128, 256) if X * 2.0 ** a <= 7 * S])
            x = np.concatenate([x, -x]) * 2.0 ** (up - 6)
            x = np.pad(x, (0, -len(x) % 31)).reshape(-1, 31)
            rows.append(np.concatenate([np.full((len(x), 1), 7 * S * 2.0 ** (up - 6)), x], 1))
    x = np.concatenate(rows)
    x = np.concatenate([x, np.zeros((-len(x) % 4, 32))]).reshape(-1, 1, D)
    k = _dev(torch, x).to(torch.bfloat16)
    assert np.array_equal(np64(k), x)
    big = torch.full_like(k[:3], torch.finfo(torch.bfloat16).max)
    big[1] = 2.0 ** -133
    big[2, 0, 5], big[2, 0, 40] = float("nan"), float("inf")
    k = torch.cat([k, big])
    n = k.shape[0]
    table, pages = _layout(torch, np.random.default_rng(2), [n], 64)
    cache = torch.zeros((pages, 1, 4, 18 * D), dtype=torch.uint8, device="cuda")
    tb, lens, cu = _dev(torch, table), torch.tensor([n], device="cuda"), torch.tensor([0, n], device="cuda")
    kda.kda_kv4_append(k, -k, cache, tb, lens, cu_seqlens=cu)
    ko, vo = torch.empty_like(k), torch.empty_like(k)
    kda.kda_kv4_read(cache, tb, lens, ko, vo, cu_seqlens=cu)
    kda.kda_sync_status()
    assert np.array_equal(np64(ko), ref.held(np64(k)), equal_nan=True)
    assert np.array_equal(np64(vo), ref.held(-np64(k)), equal_nan=True)


# ---------------------------------------------------------------- attention
def _filled(torch, kda, rng, lens, page, Hk, D, cols=None):
    """A cache with random tokens for every sequence; what the pages hold behind a sequence's end has NaN scales."""
    table, pages = _layout(torch, rng, lens, page, cols=cols)
    cache = torch.full((pages, Hk, page // 16, 18 * D), 255, dtype=torch.uint8, device="cuda")
    tb, lt = _dev(torch, table), _dev(torch, np.array(lens, np.int64))
    n = sum(lens)
    if n:
        k, v = (_dev(torch, rng.normal(size=(n, Hk, D))).to(torch.bfloat16) for _ in range(2))
        kda.kda_kv4_append(k, v, cache, tb, lt, cu_seqlens=_dev(torch, np.concatenate([[0], np.cumsum(lens)])))
    kda.kda_sync_status()
    return cache, tb, lt, table


def _check(torch, got, lse, q, cache, table, lens, new, scale, causal, window):
    host, t = cache.cpu().numpy(), 0
    D, bf = q.shape[-1], q.dtype == torch.bfloat16
    for b, (n, m) in enumerate(zip(lens, new)):
        k, v = ref.tokens(host, table, b, n)
        qn = np64(q[t:t + m])
        out, ls, terms, size = ref.attention(qn, k, v, [n - m + i for i in range(m)], scale, causal, window)
        ds = (D + 8) * 2.0 ** -23 * size + 2.0 ** -20
        rest = (2 * ds + (n + 64) * 2.0 ** -23)[..., None]
        tol = (2.0 ** -8 if bf else 0.0) * terms + half_step(torch, q.dtype) * np.abs(out) + rest * 1.1 * terms + 1e-30
        assert np.all(np.abs(np64(got[t:t + m]) - out) <= tol), (b, n, m)
        l = np64(lse[t:t + m])
        seen = np.isfinite(ls)
        assert np.array_equal(seen, np.isfinite(l)) and np.all(l[~seen] == -np.inf)
        assert np.all(np.abs(l[seen] - ls[seen]) <= ds[seen] + (n + 64) * 2.0 ** -23 + 2.0 ** -21 * np.abs(ls[seen]))
        t += m


@pytest.mark.parametrize("lens,new,Hq,Hk,D,page,dt,causal,window", [
    ([1], None, 1, 1, 128, 16, "bfloat16", True, 0),
    ([1, 0, 2, 31, 32, 33, 127, 500], None, 8, 2, 128, 64, "bfloat16", True, 0),
    ([1, 0, 2, 31, 32, 33, 127, 500], None, 6, 2, 64, 16, "float32", True, 0),
    ([300, 17, 1000], None, 24, 2, 128, 32, "bfloat16", True, 0),       # twelve rows a head
    ([300, 17, 1000], None, 16, 1, 64, 128, "bfloat16", True, 100),
    ([700, 65], None, 40, 1, 128, 256, "bfloat16", True, 0),            # more rows than a block
    ([40, 9, 0, 130], [7, 9, 0, 3], 6, 3, 128, 16, "bfloat16", True, 0),
    ([40, 9, 0, 130], [7, 9, 0, 3], 6, 3, 64, 32, "float32", True, 5),
    ([257, 64, 3], [100, 1, 3], 4, 2, 128, 64, "bfloat16", True, 33),
    ([257, 64, 3], [100, 1, 3], 4, 2, 128, 64, "float32", False, 0),
    ([90, 5, 0], [11, 20, 4], 4, 4, 64, 16, "bfloat16", False, 0),      # an encoder's states of other lengths
    ([600], [600], 3, 1, 128, 64, "bfloat16", True, 0),                 # a whole prompt
    ([600, 50], [600, 50], 4, 2, 64, 64, "bfloat16", True, 128),
    ([333, 1], [333, 1], 2, 2, 64, 64, "float32", True, 0),
    ([3000], [130], 16, 2, 128, 64, "bfloat16", True, 0),
    ([5, 3], [9, 3], 4, 2, 128, 16, "bfloat16", True, 0),               # more new tokens than the cache counts
])
def test_attention(env, lens, new, Hq, Hk, D, page, dt, causal, window):
    torch, kda = env
    dt = getattr(torch, dt)
    rng = np.random.default_rng(len(lens) + Hq + D + page)
    cache, tb, lt, table = _filled(torch, kda, rng, lens, page, Hk, D)
    counts = [1] * len(lens) if new is None else new
    extra = 0 if new is None else 3
    T = sum(counts) + extra
    q = _dev(torch, 2 * rng.normal(size=(T, Hq, D))).to(dt)
    out, lse = torch.full_like(q, 7.0), torch.full((T, Hq), 7.0, device="cuda")
    cu = None if new is None else _dev(torch, np.concatenate([[0], np.cumsum(counts)]))
    kda.kda_kv4_attention(q, cache, tb, lt, out, cu_seqlens=cu, causal=causal, window=window, lse=lse)
    kda.kda_sync_status()
    _check(torch, out, lse, q, cache, table, lens, counts, D ** -0.5, causal, window)
    if extra:
        assert bool((out[-extra:] == 7).all()) and bool((lse[-extra:] == 7).all())
    again = torch.empty_like(out)
    kda.kda_kv4_attention(q, cache, tb, lt, again, cu_seqlens=cu, causal=causal, window=window)
    assert torch.equal(again[:T - extra], out[:T - extra])  # the same bits, without lse too


@pytest.mark.parametrize("lens,Hq,Hk,dt,window,cols", [
    ([3000, 1, 0, 77], 8, 2, "bfloat16", 0, 400),   # a table with room for more than a cluster takes at once
    ([3000, 1, 0, 77], 12, 1, "bfloat16", 200, 400),
    ([2500, 640], 4, 4, "float32", 0, 300),
    ([1030, 5, 0, 65, 64], 8, 8, "bfloat16", 0, 20),
    ([1030, 5, 0, 65, 64], 32, 2, "float32", 300, 20),
])
def test_attention_of_one_token_however_the_work_is_cut(env, lens, Hq, Hk, dt, window, cols):
    """Lines of tiles cut into runs, and items shared by the CTAs of a cluster: the block table's width decides."""
    torch, kda = env
    dt = getattr(torch, dt)
    rng = np.random.default_rng(cols + Hq)
    cache, tb, lt, table = _filled(torch, kda, rng, lens, 64, Hk, 128, cols=cols)
    B = len(lens)
    q = _dev(torch, 2 * rng.normal(size=(B, Hq, 128))).to(dt)
    for width in (cols, max(-(-n // 64) for n in lens)):
        out, lse = torch.full_like(q, 7.0), torch.full((B, Hq), 7.0, device="cuda")
        kda.kda_kv4_attention(q, cache, tb[:, :width], lt, out, window=window, lse=lse)
        kda.kda_sync_status()
        _check(torch, out, lse, q, cache, table, lens, [1] * B, 128 ** -0.5, True, window)


@pytest.mark.parametrize("Hq,Hk,new,dt", [(8, 2, None, "bfloat16"), (12, 1, None, "bfloat16"), (4, 2, 5, "float32"),
                                          (8, 2, 40, "bfloat16"), (40, 1, None, "bfloat16")])
def test_attention_many_sequences(env, Hq, Hk, new, dt):
    """More sequences than a warp has lanes, short and long ones mixed, and a table wider than any of them needs."""
    torch, kda = env
    dt = getattr(torch, dt)
    rng = np.random.default_rng(Hq)
    B, D, page = 75, 64, 32
    lens = [int(x) for x in rng.integers(0, 90, B)]
    lens[3], lens[40], lens[41] = 900, 0, 700
    counts = [1] * B if new is None else [int(min(x, rng.integers(0, new + 1))) for x in lens]
    cache, tb, lt, table = _filled(torch, kda, rng, lens, page, Hk, D, cols=64)
    q = _dev(torch, rng.normal(size=(sum(counts), Hq, D))).to(dt)
    out, lse = torch.empty_like(q), torch.empty((sum(counts), Hq), device="cuda")
    cu = None if new is None else _dev(torch, np.concatenate([[0], np.cumsum(counts)]))
    kda.kda_kv4_attention(q, cache, tb, lt, out, cu_seqlens=cu, lse=lse)
    kda.kda_sync_status()
    _check(torch, out, lse, q, cache, table, lens, counts, D ** -0.5, True, 0)


@pytest.mark.parametrize("lens,new,Hq,D,window", [
    ([6000], [1], 20, 128, 0),           # one row tile, its tokens shared by as many CTAs as there are
    ([6000, 0, 9], [1, 0, 1], 32, 64, 1500),
    ([5000], [9], 24, 128, 0),           # two row tiles
    ([4000, 77], [3, 2], 48, 64, 0),
])
def test_attention_of_many_pieces(env, lens, new, Hq, D, window):
    """Few blocks of many rows over long sequences: an item in more pieces than a warp joins by itself."""
    torch, kda = env
    rng = np.random.default_rng(Hq + D)
    cache, tb, lt, table = _filled(torch, kda, rng, lens, 128, 1, D)
    q = _dev(torch, 2 * rng.normal(size=(sum(new), Hq, D))).to(torch.bfloat16)
    out, lse = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device="cuda")
    cu = _dev(torch, np.concatenate([[0], np.cumsum(new)]))
    kda.kda_kv4_attention(q, cache, tb, lt, out, cu_seqlens=cu, window=window, lse=lse)
    kda.kda_sync_status()
    _check(torch, out, lse, q, cache, table, lens, new, D ** -0.5, True, window)


def _against_64_bits(torch, kda, B, L, Hq, Hk, D, dt, cols, seed):
    """Relative root-mean-square error of one new token's attention for each of B sequences of about L, positive values."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    lens = [L - 37 * b for b in range(B)]
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), device="cuda")
    table, pages = _layout(torch, np.random.default_rng(seed), lens, 64, cols=cols)
    cache, tb, lt = (torch.zeros((pages, Hk, 4, 18 * D), dtype=torch.uint8, device="cuda"), _dev(torch, table),
                     torch.tensor(lens, device="cuda"))
    k, v = (torch.randn((sum(lens), Hk, D), generator=gen, device="cuda") for _ in range(2))
    kda.kda_kv4_append(k, v.abs(), cache, tb, lt, cu_seqlens=cu)
    kda.kda_kv4_read(cache, tb, lt, k, v, cu_seqlens=cu)
    q = torch.randn((B, Hq, D), generator=gen, device="cuda").to(dt)
    out = torch.empty_like(q)
    kda.kda_kv4_attention(q, cache, tb, lt, out)
    kda.kda_sync_status()
    far = size = 0.0
    for b in range(B):
        kb, vb = (x[cu[b]:cu[b + 1]].double().repeat_interleave(Hq // Hk, 1).transpose(0, 1) for x in (k, v))
        p = torch.softmax(torch.einsum("hd,hjd->hj", q[b].double(), kb) * D ** -0.5, -1)
        want = torch.einsum("hj,hjd->hd", p, vb)
        far += float((out[b].double() - want).pow(2).sum())
        size += float(want.pow(2).sum())
    return (far / size) ** 0.5


@pytest.mark.parametrize("B,L,cols", [(26, 5475, 200), (2, 1000, 20)])
def test_long_fp32_sums_do_not_drift(env, B, L, cols):
    """Values of one sign, over which the cutting of a chain of matrix products would add up. Scores of up to 8 are off by
    some 2^-24 of themselves a step of a short chain, the exponential by 2^-22, and sums that round walk at random: 2^-21 in
    all, twice that allowed."""
    torch, kda = env
    assert _against_64_bits(torch, kda, B, L, 7, 7, 128, torch.float32, cols, 61) <= 2.0 ** -20


def test_short_bf16_items_lose_the_outputs_rounding_only(env):
    """Factors in two terms are off by 2^-16 at most, the output by its rounding: 2^-8 / sqrt(3) of the lower end of an
    octave, at most."""
    torch, kda = env
    for seed in range(4):
        assert _against_64_bits(torch, kda, 1, 4000, 20, 5, 64, torch.bfloat16, 63, seed) <= 2.0 ** -8 / 3 ** 0.5 + 2.0 ** -14


def test_two_graphs_share_a_workspace(env):
    """Captured calls of different sizes that use one workspace in turn, its bytes arbitrary before."""
    torch, kda = env
    rng = np.random.default_rng(51)
    size, calls = 0, []
    for lens, new, Hq, Hk in (([3000, 40], [1, 1], 8, 1), ([700, 1500], [100, 3], 16, 2), ([2600], [1], 40, 1)):
        cache, tb, lt, table = _filled(torch, kda, rng, lens, 64, Hk, 128, cols=200)
        q = _dev(torch, 2 * rng.normal(size=(sum(new), Hq, 128))).to(torch.bfloat16)
        cu = None if new == [1] * len(lens) else _dev(torch, np.concatenate([[0], np.cumsum(new)]))
        out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
        calls.append((q, cache, tb, lt, out, cu, lse, table, lens, new))
        size = max(size, kda.kda_kv4_attention_workspace_bytes(len(lens), sum(new), Hq, Hk, 128, 64, tb.shape[1],
                                                               cu is not None, torch.bfloat16))
    ws, graphs = torch.full((size,), 255, dtype=torch.uint8, device="cuda"), []
    for q, cache, tb, lt, out, cu, lse, *_ in calls:
        graphs.append(torch.cuda.CUDAGraph())
        kda.kda_kv4_attention(q, cache, tb, lt, out, cu_seqlens=cu, lse=lse, workspace=ws)
        torch.cuda.synchronize()
        with torch.cuda.graph(graphs[-1]):
            kda.kda_kv4_attention(q, cache, tb, lt, out, cu_seqlens=cu, lse=lse, workspace=ws)
    for c in calls:
        c[4].fill_(7.0)
    for g in graphs + graphs[::-1]:
        g.replay()
    kda.kda_sync_status()
    for q, cache, tb, lt, out, cu, lse, table, lens, new in calls:
        _check(torch, out, lse, q, cache, table, lens, new, 128 ** -0.5, True, 0)


@pytest.mark.parametrize("Hq,new,dt", [(2, 1, "bfloat16"), (4, 40, "bfloat16"), (2, 3, "float32")])
def test_attention_strides_and_scale(env, Hq, new, dt):
    torch, kda = env
    dt = getattr(torch, dt)
    rng = np.random.default_rng(9)
    lens, D, Hk = [200, 77], 128, 2
    cache, tb, lt, table = _filled(torch, kda, rng, lens, 64, Hk, D)
    T = 2 * new
    wide = _dev(torch, rng.normal(size=(T, (Hq + 4) * D))).to(dt)
    q = wide[:, 2 * D:(Hq + 2) * D].unflatten(1, (Hq, D))
    into = torch.full((T, (Hq + 1) * D), 5.0, dtype=dt, device="cuda")
    out = into[:, :Hq * D].unflatten(1, (Hq, D))
    lse = torch.empty((T, Hq), device="cuda")
    wide_table = torch.full((2, tb.shape[1] + 3), -1, dtype=torch.int32, device="cuda")
    wide_table[:, :tb.shape[1]] = tb
    cu = torch.tensor([0, new, T], device="cuda")
    kda.kda_kv4_attention(q, cache, wide_table[:, :tb.shape[1]], lt, out, cu_seqlens=cu, scale=0.3, lse=lse)
    kda.kda_sync_status()
    _check(torch, out, lse, q, cache, table, lens, [new, new], 0.3, True, 0)
    assert bool((into[:, Hq * D:] == 5).all())


@pytest.mark.parametrize("Hq,new,dt,what", [(2, 6, "bfloat16", "k"), (2, 6, "bfloat16", "v"), (2, 6, "float32", "v"),
                                            (4, 70, "bfloat16", "k"), (4, 70, "bfloat16", "v"), (2, 6, "float32", "k")])
def test_values_that_are_not_finite_reach_only_those_who_see_them(env, Hq, new, dt, what):
    """A token with NaN keys or values in the middle of the new ones: queries before it are as if it were not there,
    queries from it on are NaN (in the channels of its group at least)."""
    torch, kda = env
    dt = getattr(torch, dt)
    rng = np.random.default_rng(11)
    D, n, at = 128, 150, 150 - new + new // 2
    lens, Hk = [n], 2
    table, pages = _layout(torch, rng, lens, 32)
    cache = torch.zeros((pages, Hk, 2, 18 * D), dtype=torch.uint8, device="cuda")
    tb, lt, cu = _dev(torch, table), torch.tensor([n], device="cuda"), torch.tensor([0, n], device="cuda")
    k, v = (_dev(torch, rng.normal(size=(n, Hk, D))).to(dt) for _ in range(2))
    q = _dev(torch, rng.normal(size=(new, Hq, D))).to(dt)
    res = []
    for bad in (False, True):
        if bad:
            (k if what == "k" else v)[at, 1, 40] = float("nan")
        kda.kda_kv4_append(k, v, cache, tb, lt, cu_seqlens=cu)
        out = torch.empty_like(q)
        kda.kda_kv4_attention(q, cache, tb, lt, out, cu_seqlens=torch.tensor([0, new], device="cuda"))
        res.append(out)
    kda.kda_sync_status()
    good, got = res
    first = at - (n - new)
    heads = Hq // Hk
    assert torch.equal(got[:, :heads], good[:, :heads]) and torch.equal(got[:first], good[:first])
    assert bool(got[first:, heads:, 32:64].isnan().all())


def test_bad_pages_and_lengths_are_reported(env):
    """Pages and lengths outside the cache are found by the kernels' own checks: nothing outside is touched, the
    status says so, other sequences are as they should be."""
    torch, kda = env
    rng = np.random.default_rng(13)
    D, Hk, page, lens = 64, 2, 16, [20, 40, 30]
    cache, tb, lt, table = _filled(torch, kda, rng, lens, page, Hk, D)
    bad = tb.clone()
    bad[1, 1] = cache.shape[0]
    k = torch.randn((3, Hk, D), device="cuda")
    q = torch.randn((3, 4, D), device="cuda")
    out, lse = torch.empty_like(q), torch.empty((3, 4), device="cuda")
    kda.kda_kv4_attention(q, cache, bad, lt, out, lse=lse)
    with pytest.raises(kda.KdaError) as e:
        kda.kda_sync_status()
    assert e.value.status == kda.KDA_ERR_DEVICE_CHECK
    _check(torch, out[[0]], lse[[0]], q[[0]], cache, table, [20], [1], D ** -0.5, True, 0)
    before = cache.clone()
    bad = tb.clone()
    bad[:, :] = -1
    kda.kda_kv4_append(k, k, cache, bad, lt)
    with pytest.raises(kda.KdaError):
        kda.kda_sync_status()
    assert torch.equal(before, cache)
    for lengths in ([20, 49, 30], [20, -3, 30]):  # past the table's columns, negative
        kda.kda_kv4_attention(q, cache, tb, torch.tensor(lengths, device="cuda"), out, lse=lse)
        with pytest.raises(kda.KdaError):
            kda.kda_sync_status()
        _check(torch, out[[0]], lse[[0]], q[[0]], cache, table, [20], [1], D ** -0.5, True, 0)
    for cu in ([0, 2, 1, 3], [0, 1, 2, 9], [-1, 1, 2, 3]):
        kda.kda_kv4_attention(q, cache, tb, lt, out, cu_seqlens=torch.tensor(cu, device="cuda"))
        with pytest.raises(kda.KdaError):
            kda.kda_sync_status()
    kda.kda_sync_status()


def test_no_tokens_and_no_sequences(env):
    torch, kda = env
    cache = torch.zeros((1, 2, 1, 18 * 64), dtype=torch.uint8, device="cuda")
    none = torch.empty((0, 4, 64), device="cuda")
    kv = torch.empty((0, 2, 64), device="cuda")
    table, lens = torch.zeros((0, 1), dtype=torch.int32, device="cuda"), torch.zeros(0, dtype=torch.int64, device="cuda")
    kda.kda_kv4_append(kv, kv, cache, table, lens)
    kda.kda_kv4_read(cache, table, lens, kv, kv.clone())
    kda.kda_kv4_attention(none, cache, table, lens, none.clone())
    kda.kda_qk_norm_rope(none, kv, none.clone(), kv.clone(), None, None)
    kda.kda_sync_status()


# ---------------------------------------------------------------- streams, graphs, a layer's run
def _layer(torch, kda, gen, Hq, Hk, D, dt, page, steps, prompt):
    """Prompts and decode steps of two sequences through norm + rotation, cache and attention; the outputs and what
    went in, as a program would run them."""
    r = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    qw, kw = r(D).abs() + 0.5, r(D).abs() + 0.5
    freq = 10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64, device="cuda") / D)
    total = [p + steps for p in prompt]
    cols = max(-(-n // page) for n in total)
    table = torch.arange(2 * cols, dtype=torch.int32, device="cuda").view(cols, 2).t().contiguous()
    cache = torch.full((2 * cols, Hk, page // 16, 18 * D), 255, dtype=torch.uint8, device="cuda")
    calls = []
    for s in range(steps + 1):
        n = prompt if s == 0 else [1, 1]
        T = sum(n)
        x = r(T, (Hq + 2 * Hk) * D).to(dt)
        lens = torch.tensor([p + s for p in prompt], device="cuda")
        pos = torch.cat([torch.arange(p + s - m, p + s, device="cuda") for p, m in zip(prompt, n)])
        cu = None if s else torch.tensor([0, n[0], T], device="cuda")
        calls.append((x, lens, pos, cu, torch.empty((T, Hq, D), dtype=dt, device="cuda"),
                      torch.empty((T, Hk, D), dtype=dt, device="cuda"), torch.empty((T, Hq, D), dtype=dt, device="cuda"), n))

    def step(c, stream=None):
        x, lens, pos, cu, q, k, out, _ = c
        qv, kv, v = (x[:, a * D:b * D].unflatten(1, (b - a, D)) for a, b in ((0, Hq), (Hq, Hq + Hk), (Hq + Hk, Hq + 2 * Hk)))
        kda.kda_qk_norm_rope(qv, kv, q, k, pos, freq, q_weight=qw, k_weight=kw, stream=stream)
        kda.kda_kv4_append(k, v, cache, table, lens, cu_seqlens=cu, stream=stream)
        kda.kda_kv4_attention(q, cache, table, lens, out, cu_seqlens=cu, stream=stream)

    def check():
        host = cache.cpu().numpy()
        tb = table.cpu().numpy()
        for c in calls:
            x, lens, pos, cu, q, k, out, n = c
            want_q = ref.norm_rope(np64(x[:, :Hq * D].unflatten(1, (Hq, D))), np64(qw), pos.cpu().numpy(), np64(freq), 1e-6, False)
            assert np.all(np.abs(np64(q) - want_q) <= half_step(torch, dt) * np.abs(want_q) + 1e-5 * np.abs(want_q).max())
            t = 0
            for b, m in enumerate(n):
                L = int(lens[b])
                kk, vv = ref.tokens(host, tb, b, L)
                o, _, terms, size = ref.attention(np64(q[t:t + m]), kk, vv, [L - m + i for i in range(m)], D ** -0.5, True, 0)
                rest = (2 * (D + 8) * 2.0 ** -23 * size + 2.0 ** -19 + (L + 64) * 2.0 ** -23)[..., None]
                tol = (2.0 ** -8 if dt == torch.bfloat16 else 0) * terms + half_step(torch, dt) * np.abs(o) + 1.1 * rest * terms
                assert np.all(np.abs(np64(out[t:t + m]) - o) <= tol)
                t += m
    return calls, step, check


@pytest.mark.parametrize("Hq,Hk,D,dt,page", [(6, 2, 128, "bfloat16", 16), (4, 4, 64, "float32", 64), (24, 2, 64, "bfloat16", 32)])
def test_a_layers_run(env, Hq, Hk, D, dt, page):
    """Prompts, then single tokens, each behind the other without a synchronisation; on another stream the same bits."""
    torch, kda = env
    make = lambda: _layer(torch, kda, torch.Generator(device="cuda").manual_seed(2), Hq, Hk, D, getattr(torch, dt), page, 5, [37, 90])  # noqa: E731
    calls, step, check = make()
    for c in calls:
        step(c)
    kda.kda_sync_status()
    check()
    again, step2, _ = make()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for c in again:
        step2(c, side)
    side.synchronize()
    for c, d in zip(calls, again):
        assert torch.equal(c[6], d[6])


def test_a_captured_step_replays_with_longer_sequences(env):
    """A decode step captured once: lengths, positions and inputs are read from device memory at each replay."""
    torch, kda = env
    Hq, Hk, D, dt, page = 8, 2, 128, torch.bfloat16, 32
    calls, step, check = _layer(torch, kda, torch.Generator(device="cuda").manual_seed(4), Hq, Hk, D, dt, page, 6, [61, 3])
    step(calls[0])
    x, lens, pos, cu, q, k, out, n = [t.clone() if hasattr(t, "clone") else t for t in calls[1]]
    c = (x, lens, pos, None, q, k, out, n)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(c)  # outside the capture first
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(c)
    for d in calls[1:]:
        x.copy_(d[0])
        lens.copy_(d[1])
        pos.copy_(d[2])
        graph.replay()
        d[4].copy_(q)
        d[5].copy_(k)
        d[6].copy_(out)
    kda.kda_sync_status()
    check()


def test_a_layers_way_out(env):
    """Attention, then the library's own 8-bit way out (gated norm and product) on its output."""
    torch, kda = env
    rng = np.random.default_rng(21)
    lens, Hq, Hk, D, hidden = [70, 33], 4, 2, 128, 256
    cache, tb, lt, _ = _filled(torch, kda, rng, lens, 32, Hk, D)
    q = _dev(torch, rng.normal(size=(2, Hq, D))).to(torch.bfloat16)
    out = torch.empty_like(q)
    gate, w = _dev(torch, rng.normal(size=(2, Hq, D))).to(torch.bfloat16), torch.ones(D, device="cuda")
    codes, scales = torch.empty((2, Hq, D), dtype=torch.float8_e4m3fn, device="cuda"), torch.empty((Hq, 2), device="cuda")
    wq = _dev(torch, rng.normal(size=(hidden, Hq * D)) * 50).to(torch.float8_e4m3fn)
    ws = torch.full((2, Hq), 1e-3, device="cuda")
    y = torch.empty((2, hidden), device="cuda")
    kda.kda_kv4_attention(q, cache, tb, lt, out)
    kda.kda_gated_rmsnorm_fp8(out, gate, w, codes, scales)
    kda.kda_fp8_linear(codes.view(2, -1), scales, wq, ws, y)
    kda.kda_sync_status()
    a = np64(codes.float()).reshape(2, Hq, D) * np64(scales).T[:, :, None]
    o = np64(out)
    want = o / np.sqrt((o ** 2).mean(-1, keepdims=True) + 1e-6) / (1 + np.exp(-np64(gate)))
    assert np.all(np.abs(a - want) <= 2.0 ** -4 * np.abs(want) + 2.0 ** -9 * np.abs(want).max(-1, keepdims=True))
    prod = a.reshape(2, -1) @ (np64(wq.float()) * 1e-3).T
    size = np.abs(a.reshape(2, -1)) @ np.abs(np64(wq.float()) * 1e-3).T
    assert np.all(np.abs(np64(y) - prod) <= 1e-4 * size)


def test_calls_side_by_side(env):
    """Two calls at once on two streams, each with a workspace of its own."""
    torch, kda = env
    rng = np.random.default_rng(31)
    lens, Hq, Hk, D = [2000, 900], 16, 2, 128
    cache, tb, lt, table = _filled(torch, kda, rng, lens, 64, Hk, D, cols=200)
    qs = [_dev(torch, rng.normal(size=(2, Hq, D))).to(torch.bfloat16) for _ in range(2)]
    size = kda.kda_kv4_attention_workspace_bytes(2, 2, Hq, Hk, D, 64, tb.shape[1], False, torch.bfloat16)
    assert size > 0
    spaces = [torch.full((size,), 255, dtype=torch.uint8, device="cuda") for _ in range(2)]
    streams, outs = [torch.cuda.Stream() for _ in range(2)], [torch.empty_like(q) for q in qs]
    lses = [torch.empty((2, Hq), device="cuda") for _ in qs]
    torch.cuda.synchronize()
    for _ in range(3):
        for q, ws, s, o, l in zip(qs, spaces, streams, outs, lses):
            kda.kda_kv4_attention(q, cache, tb, lt, o, lse=l, workspace=ws, stream=s)
    torch.cuda.synchronize()
    kda.kda_sync_status()
    for q, o, l in zip(qs, outs, lses):
        _check(torch, o, l, q, cache, table, lens, [1, 1], D ** -0.5, True, 0)


def test_offsets_past_32_bits(env):
    """A cache of more than 4 GiB: the last pages are reached."""
    torch, kda = env
    Hk, D, page = 8, 128, 256
    per = kda.kda_kv4_cache_bytes(1, Hk, page, D)
    pages = (5 << 30) // per
    cache = torch.zeros((pages, Hk, page // 16, 18 * D), dtype=torch.uint8, device="cuda")
    rng = np.random.default_rng(41)
    table = torch.tensor([[pages - 1, pages - 3], [2, pages // 2]], dtype=torch.int32, device="cuda")
    lens, n = [300, 280], 580
    lt, cu = torch.tensor(lens, device="cuda"), torch.tensor([0, 300, n], device="cuda")
    k, v = (_dev(torch, rng.normal(size=(n, Hk, D))).to(torch.bfloat16) for _ in range(2))
    kda.kda_kv4_append(k, v, cache, table, lt, cu_seqlens=cu)
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    kda.kda_kv4_read(cache, table, lt, ko, vo, cu_seqlens=cu)
    kda.kda_sync_status()
    assert np.array_equal(np64(ko), ref.held(np64(k))) and np.array_equal(np64(vo), ref.held(np64(v)))
    q = _dev(torch, rng.normal(size=(2, 8, D))).to(torch.bfloat16)
    out = torch.empty_like(q)
    kda.kda_kv4_attention(q, cache, table, lt, out)
    t = 0
    for b, L in enumerate(lens):
        o, _, terms, _ = ref.attention(np64(q[b:b + 1]), np64(ko[t:t + L]), np64(vo[t:t + L]), [L - 1], D ** -0.5, True, 0)
        assert np.all(np.abs(np64(out[b:b + 1]) - o) <= 2.0 ** -8 * (terms + np.abs(o)) + 1e-3 * terms)
        t += L
