"""GPU tests of the 4-bit cache's calls at what their first tests did not reach: how exact the softmax factors are in
every form of the attention, bad lengths and offsets wherever they stand, and long lines of work.

Tolerances as in test_gpu_kv4, but a softmax factor is off by at most 2^-16 of itself, what two bf16 terms leave,
whatever the form that a call takes (2^-8 there, half a step of bf16).
"""
import ctypes
import subprocess

import numpy as np
import pytest

from tests import _kv4 as ref
from tests.test_gpu_kv4 import _check, _dev, _filled, env, half_step, np64  # noqa: F401

pytestmark = pytest.mark.gpu


def _check_tightly(torch, got, q, cache, table, lens, new, scale):
    host, t, D = cache.cpu().numpy(), 0, q.shape[-1]
    for b, (n, m) in enumerate(zip(lens, new)):
        k, v = ref.tokens(host, table, b, n)
        out, _, terms, size = ref.attention(np64(q[t:t + m]), k, v, [n - m + i for i in range(m)], scale, True, 0)
        ds = (D + 8) * 2.0 ** -23 * size + 2.0 ** -20
        rest = (2 * ds + (n + 64) * 2.0 ** -23)[..., None]
        tol = 2.0 ** -16 * terms + half_step(torch, q.dtype) * np.abs(out) + rest * 1.1 * terms + 1e-30
        assert np.all(np.abs(np64(got[t:t + m]) - out) <= tol), (b, n, m)
        t += m


_FORMS = [
    ([20, 33, 9], None, 8, 2, 128, 4),             # an item a cluster
    ([20, 130, 9], None, 8, 2, 128, 1000),         # runs, eight rows a block
    ([20, 130, 9], None, 24, 2, 64, 1000),         # sixteen
    ([70, 33, 9], None, 24, 2, 128, 1000),
    ([40, 21, 80], [3, 1, 2], 8, 2, 128, 1000),    # runs behind the kernel for many rows
    ([40, 21, 30], [9, 1, 20], 8, 2, 128, 1000),   # up to 128 rows: one row tile
    ([24, 140], None, 40, 1, 64, 4),
    ([20, 130], None, 40, 2, 128, 1000),           # two blocks of sixteen
    ([70, 33, 9], None, 34, 2, 64, 4),
    ([40, 21, 80], [8, 1, 5], 8, 2, 128, 4),
    ([90, 70, 12], [2, 3, 9], 20, 2, 64, 1000),    # 20, 30 and 90 rows
    ([60, 150], [50, 40], 8, 2, 128, 4),           # two row tiles
    ([45, 300], [33, 70], 12, 2, 64, 1000),
]


def _sized(torch, kda, rng, lens, page, Hk, D, cols, size):
    """As _filled, with token t's values size[t] as large; a size of 0 leaves it zeros."""
    cache, tb, lt, table = _filled(torch, kda, rng, lens, page, Hk, D, cols=cols)
    k, v = (rng.normal(size=(sum(lens), Hk, D)) for _ in range(2))
    kda.kda_kv4_append(_dev(torch, k).float(), _dev(torch, v * size[:, None, None]).float(), cache, tb, lt,
                       cu_seqlens=_dev(torch, np.concatenate([[0], np.cumsum(lens)])))
    return cache, tb, lt, table


_SIZES = {"even": lambda rng, n: np.ones(n),
          "uneven": lambda rng, n: np.where(rng.random(n) < 0.02, rng.choice([0.0, 1e-9, 300.0, 1e30], n), 1.0)}


@pytest.mark.parametrize("size", list(_SIZES))
@pytest.mark.parametrize("lens,new,Hq,Hk,D,cols", _FORMS)
def test_factors_are_as_exact_in_every_form(env, lens, new, Hq, Hk, D, cols, size):  # noqa: F811
    """Few tokens of near-equal weight and values of both signs: an output far below its terms shows what the factors
    lost, which the output's own rounding hides elsewhere."""
    torch, kda = env
    rng = np.random.default_rng(Hq + D + cols)
    cache, tb, lt, table = _sized(torch, kda, rng, lens, 16, Hk, D, max(cols, -(-max(lens) // 16)),
                                  _SIZES[size](rng, sum(lens)))
    counts = [1] * len(lens) if new is None else new
    q = _dev(torch, 0.5 * rng.normal(size=(sum(counts), Hq, D))).to(torch.bfloat16)
    out = torch.empty_like(q)
    cu = None if new is None else _dev(torch, np.concatenate([[0], np.cumsum(counts)]))
    kda.kda_kv4_attention(q, cache, tb, lt, out, cu_seqlens=cu)
    kda.kda_sync_status()
    _check_tightly(torch, out, q, cache, table, lens, counts, D ** -0.5)


_LINE = """
#include "kda_kv4_attn.cuh"
using namespace kda::kv4;
__global__ void line(AttnArgs a, int64_t *out) {
    const int64_t many = sequence_tiles<256, 128, 3>(a, 0, threadIdx.x, false), few = line_tiles<16, 64>(a, threadIdx.x);
    if (threadIdx.x == 0) out[0] = many, out[1] = few;
}
extern "C" int tiles_of(const int64_t *lens, const int64_t *cu, int64_t T, int group, int Hk, int cols, int causal,
                        int window, int64_t *out) {
    AttnArgs a = {};
    a.c.lens = lens, a.c.cu = cu, a.c.T = T, a.c.B = 1, a.c.Hk = Hk, a.c.cols = cols, a.c.page_shift = 8;
    a.group = group, a.by_group = Div(group), a.causal = causal, a.window = window, a.most_rows = 0x7fffffff;
    line<<<1, 32>>>(a, out);
    return (int)cudaDeviceSynchronize();
}
"""


def _compiled(where, name, source):
    """A small library of kernels that include the library's own headers."""
    from linear_attention_recurrence_02_gb300 import build
    (where / (name + ".cu")).write_text(source)
    subprocess.run([build._nvcc(), "-O2", "-std=c++17", "--expt-relaxed-constexpr", "-Xcompiler", "-fPIC", *build.ARCH, "-I",
                    build.INCLUDE, "-I", build.CSRC, "-shared", "-o", str(where / (name + ".so")),
                    str(where / (name + ".cu"))], check=True)
    return ctypes.CDLL(str(where / (name + ".so")))


@pytest.fixture(scope="module")
def tiles_of(env, tmp_path_factory):  # noqa: F811
    fn = _compiled(tmp_path_factory.mktemp("line"), "line", _LINE).tiles_of
    p, i = ctypes.c_void_p, ctypes.c_int
    fn.argtypes, fn.restype = [p, p, ctypes.c_int64, i, i, i, i, i, p], i
    return fn


@pytest.mark.parametrize("n,length,group,Hk,causal,window", [
    (1000, 3000, 4, 2, True, 0), (77, 5000, 16, 3, False, 0), (3000, 3000, 8, 1, True, 700),
    (1_500_000, 1_500_000, 64, 1, True, 0),     # 2.2e9 tiles
    (1 << 20, 1 << 20, 128, 1, False, 0), (4_200_000, 4_200_000, 8, 1, True, 0), (1_500_000, 8_000_000, 64, 4, True, 5000),
])
def test_long_lines_of_work_are_counted(env, tiles_of, n, length, group, Hk, causal, window):  # noqa: F811
    """The tiles that the kernels cut into runs, at sizes whose product passes 32 bits (and would take minutes to run)."""
    torch, _ = env
    lens, cu, out = torch.tensor([length], device="cuda"), torch.tensor([0, n], device="cuda"), torch.zeros(2, dtype=torch.int64, device="cuda")
    torch.cuda.synchronize()
    assert tiles_of(lens.data_ptr(), cu.data_ptr(), n, group, Hk, -(-length // 256), causal, window, out.data_ptr()) == 0
    row = np.arange(0, n * group, 256)
    hi = length - n + np.minimum(row + 255, n * group - 1) // group + 1 if causal else np.full(len(row), length)
    lo = np.maximum(length - n + row // group - window + 1, 0) if window else np.zeros(len(row), int)
    many = int((np.maximum(-(-hi // 128) - lo // 128, 1) + 3).sum()) * Hk
    first = max(length - n - window + 1, 0) // 64 if window else 0
    few = -(-n * group // 16) * Hk * (-(-length // 64) - first)
    assert out.tolist() == [many, few]


def _reported(kda):
    with pytest.raises(kda.KdaError) as e:
        kda.kda_sync_status()
    assert e.value.status == kda.KDA_ERR_DEVICE_CHECK
    kda.kda_sync_status()  # and cleared


@pytest.mark.parametrize("where", [40, 63])
@pytest.mark.parametrize("cols,Hq,dt", [(4, 4, "bfloat16"), (4, 2, "float32"), (1000, 4, "bfloat16"), (4, 40, "bfloat16")])
@pytest.mark.parametrize("what", ["long", "negative", "offsets", "past"])
def test_bad_lengths_far_down_the_batch_are_reported(env, where, cols, Hq, dt, what):  # noqa: F811
    """More sequences than a warp has lanes, a bad one behind the first 32: in the cluster form, in runs, in the
    kernel for many rows."""
    torch, kda = env
    B, Hk, D = 64, 2, 64
    rng = np.random.default_rng(where + cols)
    lens = [int(x) for x in rng.integers(1, 60, B)]
    cache, tb, lt, _ = _filled(torch, kda, rng, lens, 16, Hk, D, cols=cols)
    q = _dev(torch, rng.normal(size=(B, Hq, D))).to(getattr(torch, dt))
    good, out = torch.empty_like(q), torch.full_like(q, 7.0)
    cu = torch.arange(B + 1, device="cuda") if what in ("offsets", "past") else None
    kda.kda_kv4_attention(q, cache, tb, lt, good, cu_seqlens=cu)
    kda.kda_sync_status()
    bad = lt.clone()
    clean = [b for b in range(B) if b != where]
    if what == "long":
        bad[where] = 16 * cols + 1
    elif what == "negative":
        bad[where] = -1
    elif what == "past":  # ends behind the call's rows (the last one); starts before them (another)
        if where == B - 1:
            cu[B] = B + 1
        else:
            cu[where] = -3
            clean.remove(where - 1)
    else:
        cu[where] = where - 4  # the sequence before ends before it starts, this one overlaps those before it
        clean = [b for b in range(B) if not where - 4 <= b <= where]
    kda.kda_kv4_attention(q, cache, tb, bad if cu is None else lt, out, cu_seqlens=cu)
    _reported(kda)
    assert torch.equal(out[clean], good[clean])


def test_empty_sequences_with_bad_lengths_are_reported(env):  # noqa: F811
    """Sequences without new tokens that no block of rows belongs to, the last ones of the batch."""
    torch, kda = env
    rng = np.random.default_rng(3)
    B, D = 70, 64
    lens = [int(x) for x in rng.integers(1, 60, B)]
    for new, Hq in ((1, 2), (30, 2), (1, 40)):
        cache, tb, lt, _ = _filled(torch, kda, rng, lens, 16, 1, D, cols=4)
        q = _dev(torch, rng.normal(size=(new, Hq, D))).to(torch.bfloat16)
        good, out = torch.empty_like(q), torch.empty_like(q)
        cu = torch.full((B + 1,), new, device="cuda")
        cu[0] = 0
        kda.kda_kv4_attention(q, cache, tb, lt, good, cu_seqlens=cu)
        kda.kda_sync_status()
        lt[B - 1] = -1
        kda.kda_kv4_attention(q, cache, tb, lt, out, cu_seqlens=cu)
        _reported(kda)
        assert torch.equal(out, good)


@pytest.mark.parametrize("Hq,new", [(4, 1), (4, 40), (40, 1), (6, 3)])
def test_pages_outside_the_cache_are_reported_in_every_form(env, Hq, new):  # noqa: F811
    torch, kda = env
    rng = np.random.default_rng(Hq + new)
    lens, D, Hk = [50, 200, 90], 128, 2
    cache, tb, lt, _ = _filled(torch, kda, rng, lens, 32, Hk, D)
    q = _dev(torch, rng.normal(size=(3 * new, Hq, D))).to(torch.bfloat16)
    cu = torch.arange(0, 3 * new + 1, new, device="cuda")
    good, out, before = torch.empty_like(q), torch.empty_like(q), cache.clone()
    kda.kda_kv4_attention(q, cache, tb, lt, good, cu_seqlens=cu)
    kda.kda_sync_status()
    for page in (cache.shape[0], -1, 1 << 30):
        bad = tb.clone()
        bad[1, 3] = page
        kda.kda_kv4_attention(q, cache, bad, lt, out, cu_seqlens=cu)
        _reported(kda)
        assert torch.equal(out[:new], good[:new]) and torch.equal(out[2 * new:], good[2 * new:])
    assert torch.equal(cache, before)


_BAD_SEQUENCES = {  # lens, cu_seqlens (None: one new token each), tokens of the call; which of its tokens may be written
    "past the rows": ([9], [0, 3], 2, []),
    "before the rows": ([9, 9], [-2, 1, 3], 3, [1, 2]),
    "falling": ([9, 9, 9], [0, 2, 1, 3], 3, [0, 1, 2]),
    "falling behind all rows": ([9, 9, 9], [0, 3, 5, 2], 3, [0, 1, 2]),
    "empty, past the rows": ([9, 9, 9], [0, 1, 3, 4], 3, [0, 1, 2]),
    "negative length": ([9, -4, 9], None, 3, [0, 2]),
    "long": ([9, 49, 9], None, 3, [0, 2]),
    "long, several": ([9, 50, 9], [0, 1, 3, 5], 5, [0, 3, 4]),
    "far": ([9, 1 << 40, 9], [0, 1, 3, 5], 5, [0, 3, 4]),
    "lowest": ([9, -(1 << 63), 9], [0, 1, 3, 5], 5, [0, 3, 4]),
    "negative length of an empty one": ([9, -1, 9], [0, 1, 1, 3], 3, [0, 1, 2]),
    "long one of an empty one": ([9, 4000, 9], [0, 1, 1, 3], 3, [0, 1, 2]),
    "far down": ([9] * 600 + [-1], None, 601, list(range(600))),
    "far down, empty": ([9] * 600 + [-1], [0, 3] + [3] * 600, 3, [0, 1, 2]),
}


@pytest.mark.parametrize("name", list(_BAD_SEQUENCES))
@pytest.mark.parametrize("Hk", [2, 70])
def test_append_and_read_report_bad_sequences(env, name, Hk):  # noqa: F811
    """Nothing is written or read for a sequence whose offsets or length cannot be, and the status says so, whether or
    not one of the call's tokens is its."""
    torch, kda = env
    lens, cu, T, may = _BAD_SEQUENCES[name]
    B, D, page, cols = len(lens), 64, 16, 3
    table = _dev(torch, np.arange(B * cols, dtype=np.int32).reshape(B, cols))
    before = torch.randint(0, 256, (B * cols, Hk, 1, 18 * D), dtype=torch.uint8, device="cuda",
                           generator=torch.Generator(device="cuda").manual_seed(1))
    cache, lt = before.clone(), torch.tensor(lens, device="cuda")
    ct = None if cu is None else torch.tensor(cu, device="cuda")
    k = torch.randn((T, Hk, D), device="cuda")
    kda.kda_kv4_append(k, k, cache, table, lt, cu_seqlens=ct)
    _reported(kda)
    ok = set()  # the pages that a token which may be written can go to
    seq = range(B) if cu is None else [max((b for b in range(B) if cu[b] <= t), default=0) for t in range(T)]
    for t in may:
        ok.update(range(cols * seq[t], cols * seq[t] + cols))
    for p in (cache != before).flatten(1).any(1).nonzero().flatten().tolist():
        assert p in ok, (p, name)
    ko, vo = torch.full_like(k, 7.0), torch.full_like(k, 7.0)
    kda.kda_kv4_read(cache, table, lt, ko, vo, cu_seqlens=ct)
    _reported(kda)
    for t in range(T):
        if t not in may:
            assert bool((ko[t] == 7).all()) and bool((vo[t] == 7).all()), t


def test_append_and_read_leave_padding_alone(env):  # noqa: F811
    """Sequences of length 0, empty ones and more new tokens than a sequence counts are not errors."""
    torch, kda = env
    table = torch.arange(6, dtype=torch.int32, device="cuda").view(3, 2)
    cache = torch.zeros((6, 1, 1, 18 * 64), dtype=torch.uint8, device="cuda")
    k = torch.randn((9, 1, 64), device="cuda")
    for lens, cu in (([0, 0, 32], [0, 3, 3, 5]), ([2, 0, 1], [0, 4, 4, 9]), ([5, 32, 0], [0, 0, 0, 0])):
        lt, ct = torch.tensor(lens, device="cuda"), torch.tensor(cu, device="cuda")
        kda.kda_kv4_append(k, k, cache, table, lt, cu_seqlens=ct)
        kda.kda_kv4_read(cache, table, lt, k.clone(), k.clone(), cu_seqlens=ct)
    kda.kda_kv4_append(k[:3], k[:3], cache, table, torch.tensor([0, 32, 0], device="cuda"))
    kda.kda_sync_status()


_WAIT = """
#include "kda_common.cuh"
#include "kda_tc.cuh"
using namespace kda::tc;
template <int NS> __device__ void one(uint64_t *bar, long long limit, long long *out) {
    const long long t0 = clock64();
    out[0] = mbar_wait_lean<NS>(bar, 0, limit);
    out[1] = clock64() - t0;
    mbar_arrive(bar);
    out[2] = mbar_wait_lean<NS>(bar, 0, limit);
}
__global__ void wait_twice(long long limit, long long *out) {
    __shared__ uint64_t bar[2];
    if (threadIdx.x == 0) {
        mbar_init(bar, 1);
        mbar_init(bar + 1, 1);
        fence_mbar_init();
        one<0>(bar, limit, out);
        one<100>(bar + 1, limit, out + 3);
    }
}
extern "C" int waits(long long limit, long long *out) {
    wait_twice<<<1, 32>>>(limit, out);
    return (int)cudaDeviceSynchronize();
}
"""


def test_a_wait_that_nothing_ends_gives_up_by_the_clock(env, tmp_path):  # noqa: F811
    """After its limit in clock cycles and at most 64 tries more, however long the hardware suspends a try; one whose
    barrier has completed does not wait."""
    torch, _ = env
    fn = _compiled(tmp_path, "wait", _WAIT).waits
    fn.argtypes, fn.restype = [ctypes.c_longlong, ctypes.c_void_p], ctypes.c_int
    out = torch.zeros(6, dtype=torch.int64, device="cuda")
    torch.cuda.synchronize()
    for limit in (1_000_000, 20_000_000):
        assert fn(limit, out.data_ptr()) == 0
        for gave, cycles, ended in (out[:3].tolist(), out[3:].tolist()):
            assert gave == 0 and ended == 1 and limit <= cycles < 2 * limit + 20_000_000


def test_a_large_batch_of_short_sequences(env):  # noqa: F811
    """More items than clusters take in a few turns: runs over a narrow block table."""
    torch, kda = env
    B, Hq, Hk, D, rng = 260, 8, 4, 64, np.random.default_rng(12)
    lens = [int(x) for x in rng.integers(0, 40, B)]
    cache, tb, lt, table = _filled(torch, kda, rng, lens, 16, Hk, D, cols=3)
    assert kda.kda_kv4_attention_workspace_bytes(2 * B, 2 * B, Hq, Hk, D, 16, 3, False, torch.bfloat16) > 0
    for dt in (torch.bfloat16, torch.float32):
        q = _dev(torch, rng.normal(size=(2 * B, Hq, D))).to(dt)
        out, lse = torch.empty_like(q), torch.empty((2 * B, Hq), device="cuda")
        kda.kda_kv4_attention(q, cache, tb.repeat(2, 1), lt.repeat(2), out, lse=lse)
        kda.kda_sync_status()
        _check(torch, out, lse, q, cache, np.tile(table, (2, 1)), lens + lens, [1] * (2 * B), D ** -0.5, True, 0)
