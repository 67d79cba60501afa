"""GPU tests that a row of the block-FP8 feed-forward's producers gives the
same bits alone and in a batch of any size, whichever form of the kernel the
batch selects."""
import pytest
import torch

import int8_gemm_gemv_b200 as bsq
from test_gpu_block_ffn import DEV, activations, poisoned

pytestmark = pytest.mark.gpu


def rows_of(call, x, m, k, groups):
    """The call on the first m rows of x; nothing is written behind them."""
    q, s = poisoned((m + 1, k), torch.uint8), poisoned((m + 1, groups), torch.float32)
    call(x[:m], q, s, m)
    assert (q[m] == 0xFF).all() and s[m].isnan().all()
    return q[:m], s[:m]


# K on both sides of every bound at which the rows per CTA or the units per thread change
@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("k", [256, 512, 640, 1024, 1152, 2560, 2688, 5120, 6144, 6272, 16384, 16512, 32768, 33024])
def test_norm_of_a_row_does_not_depend_on_the_batch(k, group):
    most = 2000 if k <= 6272 else 400
    x, r = activations(most, k, 1), activations(most, k, 2)
    gain = activations(1, k, 3)[0]

    def call(x, q, s, m):
        bsq.rmsnorm_residual_quant_fp8(x, r, gain, 1e-6, None, q, s, group, m, k)

    groups = k // group if group else 1
    q, s = rows_of(call, x, most, k, groups)
    for m in (1, 3, 149, 300, 395):
        q1, s1 = rows_of(call, x, m, k, groups)
        assert torch.equal(q1, q[:m]) and torch.equal(s1, s[:m]), m


# m * k / 16 units on both sides of the bound between one unit per lane and two, also where the last CTA's second
# unit, or its first, is out of range
@pytest.mark.parametrize("k", [128, 640, 5120])
def test_quantisers_of_a_row_do_not_depend_on_the_batch(k):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    bound = sms * 2048 * 3 * 16 // k  # rows
    most = bound + 70
    x = activations(most, 2 * k, 4)
    for width, call in ((k, lambda x, q, s, m: bsq.quant_act_fp8_per128(x, q, s, m, k)),
                        (2 * k, lambda x, q, s, m: bsq.silu_mul_quant_fp8_per128(x, q, s, m, k))):
        y = x.view(-1, width)
        whole = rows_of(call, y, most, k, k // 128)
        for m in (bound + 1, bound + 7, bound + 33, bound - 1, 5):
            part = rows_of(call, y, m, k, k // 128)
            assert torch.equal(part[0], whole[0][:m]) and torch.equal(part[1], whole[1][:m]), (width, m)


@pytest.mark.parametrize("k", [128, 1024, 1152, 5120, 16384, 65536])
def test_error_of_the_quantised_values(k):
    """The scale is amax|y| / 448 rounded once, so it shows the error of y:
    within 2^-19 of itself for the norm, 2^-20 for SiLU (|g| <= 87).

    Norm: a square and its addition 16 times in a unit, five additions over 32
    units, at most 4 + 5 over those sums, half of it after the root: 15 x 2^-24;
    division and eps half a rounding each, rsqrt 2 ulp, two products: 22 x 2^-24.
    SiLU: exp 2 ulp, 1 + z half an ulp, the reciprocal one, three products half
    each: 5 x 2^-23.  (A gate below -87, where exp loses bits, gives a y near
    2^-120 here, never a group's largest; above 87 1 + z is 1 either way.)"""
    m = 64
    x, gain = activations(m, k, 5), activations(1, k, 6)[0]
    for group in (0, 128):
        q, s = poisoned((m, k), torch.uint8), poisoned((m, k // group if group else 1), torch.float32)
        bsq.rmsnorm_residual_quant_fp8(x, None, gain, 1e-6, None, q, s, group, m, k)
        y = x.double() / torch.sqrt((x.double()**2).mean(1, keepdim=True) + 1e-6) * gain.double()
        want = y.abs().view(m, -1, group or k).amax(-1) / 448
        assert ((s.double() - want).abs() <= (2.0**-19 + 2.0**-23) * want).all(), (k, group)
    x = activations(m, 2 * k, 7)
    q, s = poisoned((m, k), torch.uint8), poisoned((m, k // 128), torch.float32)
    bsq.silu_mul_quant_fp8_per128(x, q, s, m, k)
    g, u = x.double().split(k, dim=1)
    want = (g * torch.sigmoid(g) * u).abs().view(m, -1, 128).amax(-1) / 448
    assert ((s.double() - want).abs() <= (2.0**-20 + 2.0**-23) * want).all(), k
