"""Host-only tests of the block-FP8 feed-forward entry points: every refusal
happens before any CUDA call and launches nothing."""
import pytest

import int8_gemm_gemv_b200 as bsq
from int8_gemm_gemv_b200 import build

A = [0x7F0000000000 + 0x100000 * i for i in range(12)]  # fake, never dereferenced device addresses
ODD = A[0] + 1
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


@pytest.fixture(autouse=True)
def launches_nothing():
    n0 = bsq.debug_launch_count()
    yield
    assert bsq.debug_launch_count() == n0


def rms(x=A[0], residual=A[1], gain=A[2], eps=1e-6, residual_out=A[3], q=A[4], scale=A[5], group=128, m=4, k=256):
    return bsq.lib().rmsnorm_residual_quant_fp8(x, residual, gain, eps, residual_out, q, scale, group, m, k, None)


@pytest.mark.parametrize("kw,status", [
    (dict(m=-1), 1), (dict(k=0), 1), (dict(k=24), 1), (dict(group=64), 1), (dict(group=-1), 1),
    (dict(group=128, k=144), 1), (dict(eps=-1e-6), 1), (dict(eps=NAN), 1), (dict(eps=INF), 1),
    (dict(x=None), 1), (dict(gain=None), 1), (dict(q=None), 1), (dict(scale=None), 1),
    (dict(x=ODD), 2), (dict(residual=A[1] + 2), 2), (dict(gain=ODD), 2), (dict(residual_out=A[3] + 8), 2),
    (dict(q=A[4] + 4), 2), (dict(scale=A[5] + 2), 2), (dict(k=65536 + 128), 3),
    (dict(m=0), 0), (dict(m=0, x=None, gain=None, q=None, scale=None), 0),
])
def test_rmsnorm_refusals(kw, status):
    assert rms(**kw) == status


@pytest.mark.parametrize("fn", ["quant_act_fp8_per128", "silu_mul_quant_fp8_per128"])
def test_activation_quantiser_refusals(fn):
    f = getattr(bsq.lib(), fn)
    assert f(A[0], A[1], A[2], -1, 128, None) == bsq.BSQ_ERR_INVALID_ARG
    assert f(A[0], A[1], A[2], 1, 0, None) == bsq.BSQ_ERR_INVALID_ARG
    assert f(A[0], A[1], A[2], 1, 192, None) == bsq.BSQ_ERR_INVALID_ARG
    assert f(A[0], A[1], A[2], 1, -128, None) == bsq.BSQ_ERR_INVALID_ARG
    for i in range(3):
        args = [A[0], A[1], A[2]]
        args[i] = None
        assert f(*args, 1, 128, None) == bsq.BSQ_ERR_INVALID_ARG
        args[i] = A[i] + (2 if i == 2 else 8)
        assert f(*args, 1, 128, None) == bsq.BSQ_ERR_MISALIGNED
    assert f(None, None, None, 0, 128, None) == bsq.BSQ_OK


def test_gemm_refusals():
    f = bsq.lib().fp8_gemm_blockscaled
    ok = [A[0], A[1], A[2], A[3], A[4]]
    for m, n, k in [(-1, 8, 128), (8, -1, 128), (8, 8, 0), (8, 8, -128), (8, 8, 24)]:
        assert f(*ok, m, n, k, None) == bsq.BSQ_ERR_INVALID_ARG, (m, n, k)
    assert f(*ok, 8, 8, 144, None) == bsq.BSQ_ERR_UNSUPPORTED
    for i, off in enumerate([8, 2, 8, 2, 2]):
        args = list(ok)
        args[i] = None
        assert f(*args, 8, 8, 128, None) == bsq.BSQ_ERR_INVALID_ARG
        args[i] = A[i] + off
        assert f(*args, 8, 8, 128, None) == bsq.BSQ_ERR_MISALIGNED
    assert f(None, None, None, None, None, 0, 8, 128, None) == bsq.BSQ_OK
    assert f(None, None, None, None, None, 8, 0, 128, None) == bsq.BSQ_OK


def moe(ptr=None, ws_bytes=1 << 40, tokens=4, hidden=256, inter=128, experts=8, topk=2, renorm=1):
    p = list(A[:10])
    for i, v in (ptr or {}).items():
        p[i] = v
    return bsq.lib().fp8_moe_blockscaled(*p, ws_bytes, tokens, hidden, inter, experts, topk, renorm, None)


@pytest.mark.parametrize("kw,status", [
    (dict(tokens=-1), 1), (dict(tokens=17), 1), (dict(experts=0), 1), (dict(experts=-1), 1), (dict(topk=0), 1),
    (dict(topk=9), 1), (dict(hidden=0), 1), (dict(hidden=24), 1), (dict(inter=-128), 1), (dict(inter=40), 1),
    (dict(renorm=2), 1), (dict(hidden=144), 3), (dict(inter=192), 3), (dict(experts=64, topk=17), 3),
    (dict(experts=513), 3), (dict(experts=512, inter=1 << 21), 3), (dict(experts=512, hidden=1 << 22), 3),
    (dict(tokens=0), 0),
])
def test_moe_refusals(kw, status):
    assert moe(**kw) == status


@pytest.mark.parametrize("i", range(10))
def test_moe_pointer_refusals(i):
    if i not in (7, 8):  # topk_ids and topk_weights may be NULL
        assert moe({i: None}) == bsq.BSQ_ERR_INVALID_ARG
    assert moe({i: A[i] + 2}) == bsq.BSQ_ERR_MISALIGNED
    if i in (0, 2, 4, 6, 9):
        assert moe({i: A[i] + 8}) == bsq.BSQ_ERR_MISALIGNED


def test_moe_workspace_query_refuses_bad_shapes():
    f = bsq.fp8_moe_workspace_bytes
    for bad in [(-1, 256, 128, 2), (17, 256, 128, 2), (4, 250, 128, 2), (4, 256, 130, 2), (4, 256, 128, 0),
                (4, 256, 128, 17), (4, 65536 + 128, 128, 2), (4, 256, 65536 + 128, 2)]:
        assert f(*bad) == 0


def test_binding_refuses_host_and_strided_tensors():
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        bsq.quant_act_fp8_per128(x, A[1], A[2], 4, 128, stream=0)
    with pytest.raises(bsq.BsqError) as e:
        bsq.fp8_gemm_blockscaled(A[0], A[1], A[2], A[3], A[4], 8, 8, 144, stream=0)
    assert e.value.status == bsq.BSQ_ERR_UNSUPPORTED
