"""GPU tests of what the block-FP8 feed-forward operators make of values that
are not finite: inputs have to be finite, but a model that has diverged must
show it, not go on with rows of zeros."""
import pytest
import torch

import int8_gemm_gemv_b200 as bsq
from test_gpu_block_ffn import DEV, Ffn, Moe, activations, poisoned

pytestmark = pytest.mark.gpu
NAN, INF, HUGE = float("nan"), float("inf"), 2.0**126


@pytest.fixture(autouse=True)
def _no_timeouts():
    yield
    assert bsq.debug_take_timeouts() == 0


def norm(x, residual, gain, group):
    m, k = x.shape
    q, s = poisoned((m, k), torch.uint8), torch.zeros((m, k // group) if group else (m,), device=DEV)
    q.zero_()
    bsq.rmsnorm_residual_quant_fp8(x, residual, gain, 1e-6, None, q, s, group, m, k)
    return q, s.view(m, -1)


def is_nan_code(q):
    return (q & 0x7F) == 0x7F


# a warp per row with one and two units per lane; a CTA per row with one, two and four units per thread
WIDTHS = [(3, 256), (5, 1024), (6, 1408), (700, 5120), (3, 20480), (3, 40960)]


@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("bad", [NAN, INF, -INF, HUGE])
@pytest.mark.parametrize("m,k", WIDTHS)
def test_norm_of_a_row_without_a_finite_sum(m, k, bad, group):
    """NaN, an infinity, or a value whose square overflows, in x or in the
    residual: NaN throughout the row's codes and scales, other rows untouched."""
    gain = activations(1, k, 1)[0]
    x, r = activations(m, k, 2), activations(m, k, 3)
    q0, s0 = norm(x, r, gain, group)
    x[1, k - 3] = bad
    r[2, 5] = bad
    q, s = norm(x, r, gain, group)
    assert s[1:3].isnan().all() and is_nan_code(q[1:3]).all()
    rest = torch.arange(m, device=DEV)
    rest = rest[(rest != 1) & (rest != 2)]
    assert torch.equal(q[rest], q0[rest]) and torch.equal(s[rest], s0[rest])


@pytest.mark.parametrize("m,k", WIDTHS)
def test_norm_with_nan_in_the_gain(m, k):
    """Only the groups that hold the column."""
    gain, x = activations(1, k, 1)[0], activations(m, k, 2)
    q0, s0 = norm(x, None, gain, 128)
    gain[130] = NAN
    q, s = norm(x, None, gain, 128)
    assert s[:, 1].isnan().all() and is_nan_code(q[:, 128:256]).all()
    other = torch.arange(k // 128, device=DEV) != 1
    assert torch.equal(s[:, other], s0[:, other])
    assert torch.equal(q.view(m, -1, 128)[:, other], q0.view(m, -1, 128)[:, other])


@pytest.mark.parametrize("m", [3, 4000])
def test_silu_of_nan(m):
    """One and two units per lane; NaN in the gate or in the up projection,
    anywhere in a group, gives NaN to that group's codes and scale."""
    k = 4096
    x = activations(m, 2 * k, 4)
    q0, s0 = poisoned((m, k), torch.uint8), poisoned((m, k // 128), torch.float32)
    bsq.silu_mul_quant_fp8_per128(x, q0, s0, m, k)
    x[1, 128 * 3 + 77] = NAN
    x[2, k + 128 * 7] = NAN
    q, s = poisoned((m, k), torch.uint8), torch.zeros((m, k // 128), device=DEV)
    q.zero_()
    bsq.silu_mul_quant_fp8_per128(x, q, s, m, k)
    hit = torch.zeros((m, k // 128), dtype=torch.bool, device=DEV)
    hit[1, 3] = hit[2, 7] = True
    assert s[hit].isnan().all() and is_nan_code(q.view(m, -1, 128)[hit]).all()
    assert torch.equal(s[~hit], s0[~hit]) and torch.equal(q.view(m, -1, 128)[~hit], q0.view(m, -1, 128)[~hit])


@pytest.mark.parametrize("m", [3, 4000])
def test_quantiser_of_nan(m):
    k = 4096
    x = activations(m, k, 4)
    x[1, 128 * 3 + 77] = NAN
    q, s = torch.zeros((m, k), dtype=torch.uint8, device=DEV), torch.zeros((m, k // 128), device=DEV)
    bsq.quant_act_fp8_per128(x, q, s, m, k)
    hit = torch.zeros((m, k // 128), dtype=torch.bool, device=DEV)
    hit[1, 3] = True
    assert s[hit].isnan().all() and is_nan_code(q.view(m, -1, 128)[hit]).all()
    assert torch.isfinite(s[~hit]).all() and not is_nan_code(q.view(m, -1, 128)[~hit]).any()


@pytest.mark.parametrize("m", [3, 300])
def test_a_diverged_token_stays_visible_through_the_chain(m):
    f = Ffn(m, 1024, 640)
    f.x[1, 100] = NAN
    f()
    bad = f.out.isnan()
    assert bad[1].all()
    bad[1] = False
    assert not bad.any()


def test_a_diverged_token_stays_visible_through_the_expert_layer():
    m = Moe(4, 256, 256, 5, 2, 1, seed=2)
    m()
    good = m.out[:4].clone()
    m.x[2, 9] = NAN
    m()
    assert m.out[2].isnan().all()
    for t in (0, 1, 3):
        assert torch.equal(m.out[t].view(torch.int16), good[t].view(torch.int16))
