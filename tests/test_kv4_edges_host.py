"""Host-side checks of the 4-bit cache's attention that need no GPU: which device a workspace's size is of."""
import ctypes

import pytest

from tests.test_binding_host import _Dev, _Stream
from tests.test_kv4_host import BF, I32, I64, U8, kda, torch  # noqa: F401


@pytest.fixture
def on_device_0(kda):  # noqa: F811
    """The extension over stand-ins for the current device (0) and its streams."""
    ext, lib = kda._fastcall(), kda.lib()
    fns = [ctypes.cast(f, ctypes.c_void_p).value for f in (
        lib.kda_add_rmsnorm_fp8, lib.kda_gated_rmsnorm_fp8, lib.kda_fp8_linear, lib.kda_qk_norm_rope, lib.kda_kv4_append,
        lib.kda_kv4_read, lib.kda_kv4_attention, lib.kda_kv4_attention_workspace_bytes)]
    types = (torch.float32, torch.bfloat16, torch.float8_e4m3fn, torch.float64, torch.int64, torch.int32, torch.uint8)
    ext.setup(*fns, *types, lambda: 0, lambda d: 0)
    yield ext
    ext.setup(*fns, *types, torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream)


def test_a_workspace_is_sized_on_the_tensors_device(kda, on_device_0):  # noqa: F811
    """A stream of another device is found by its handle; the workspace's size depends on the device all the same: the
    binding is told (-1) to make the tensors' device current first."""
    def call(index):
        d = f"cuda:{index}"
        return on_device_0.kv4_attention(
            _Dev(64, 96, 128, dtype=BF, device=d), _Dev(9, 8, 4, 18 * 128, dtype=U8, device=d),
            _Dev(64, 128, dtype=I32, device=d), _Dev(64, dtype=I64, device=d), _Dev(64, 96, 128, dtype=BF, device=d), None, None,
            True, 0, None, None, _Stream(index))
    need = kda.kda_kv4_attention_workspace_bytes(64, 64, 96, 8, 128, 64, 128, False, BF)
    assert need > 1 and call(0) == -need
    assert call(1) == -1


def test_many_short_sequences_are_cut_into_runs(kda):  # noqa: F811
    """Clusters, which need no workspace, as long as they come in a few turns; runs, which do, for more sequences."""
    size = kda.kda_kv4_attention_workspace_bytes
    for dt in (BF, torch.float32):
        assert size(1, 1, 32, 8, 128, 64, 4, False, dt) == 0 and size(64, 64, 32, 8, 128, 64, 4, False, dt) == 0
        assert size(512, 512, 32, 8, 128, 64, 4, False, dt) > 0 and size(512, 512, 32, 1, 128, 64, 4, True, dt) > 0


def test_sizes_of_caches_that_the_calls_would_refuse(kda):  # noqa: F811
    """No bytes, and no shape: rounded down to whole blocks, a page of 40 tokens would be one of 32 that the caller's
    block table knows nothing of."""
    for args in ((10, 8, 40, 128), (10, 8, 8, 128), (10, 8, 512, 128), (10, 8, 48, 64), (10, 8, 64, 32), (10, 8, 64, 96),
                 (10, 0, 64, 128), (10, 32769, 64, 128), (-1, 8, 64, 128), (1 << 31, 8, 64, 128)):
        assert kda.kda_kv4_cache_bytes(*args) == 0
        with pytest.raises(ValueError):
            kda.kda_kv4_cache_shape(*args)
    for page in (16, 32, 64, 128, 256):
        assert kda.kda_kv4_cache_shape(3, 2, page, 64) == (3, 2, page // 16, 18 * 64)
        assert kda.kda_kv4_cache_bytes(3, 2, page, 64) == 3 * 2 * page // 16 * 18 * 64
    assert kda.kda_kv4_cache_bytes(0, 8, 64, 128) == 0
