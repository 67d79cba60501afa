"""Host-only test of the expert layer's workspace query."""
import pytest

import int8_gemm_gemv_b200 as bsq
from int8_gemm_gemv_b200 import build

A = [0x7F0000000000 + 0x100000 * i for i in range(10)]  # fake, never dereferenced device addresses


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


def test_moe_workspace_bytes_match_the_device():
    """The sums of shared tiles grow with the SMs of the current device; 0
    where there is no device, and the layer then reports the CUDA failure
    instead of launching."""
    torch = pytest.importorskip("torch")
    shapes = ((1, 128, 128, 1), (4, 256, 128, 2), (16, 65536, 65536, 16))
    if torch.cuda.is_available():
        sums = torch.cuda.get_device_properties(0).multi_processor_count * 2 * 128 * 16 * 4
        for t, h, i, k in shapes:
            assert 0 <= bsq.fp8_moe_workspace_bytes(t, h, i, k) - sums - t * k * (2 * i + i // 16) - h // 16 < 1024
        return
    assert [bsq.fp8_moe_workspace_bytes(*s) for s in shapes] == [0, 0, 0]
    n0 = bsq.debug_launch_count()
    assert bsq.lib().fp8_moe_blockscaled(*A, 1 << 40, 4, 256, 128, 8, 2, 1, None) == bsq.BSQ_ERR_CUDA
    assert bsq.debug_launch_count() == n0
