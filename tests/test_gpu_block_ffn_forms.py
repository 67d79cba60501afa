"""GPU tests of the block-FP8 feed-forward operators by form: every size is
chosen by the rule that selects a kernel's form, and compared with the 64-bit
definition (or, where codes are exact, with the oracle)."""
import numpy as np
import pytest
import torch

import int8_gemm_gemv_b200 as bsq
import oracle
from test_gpu_block_ffn import (DEV, F8, Moe, U32, activations, check_codes, check_gemm, codes, dequant_a, dequant_w, gen,
                                norm_exact, norm_rel, poisoned, run_gemm, scales)

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _no_timeouts():
    yield
    assert bsq.debug_take_timeouts() == 0


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def many_rows(m, n):
    """Whether the product runs on CTA pairs: more than 64 rows, and more tiles of 128 x 32 than SMs."""
    return m > 64 and -(-n // 128) * -(-m // 32) > sms()


# --------------------------------------------------- product, CTA pairs ---

@pytest.mark.parametrize("k", [128, 256, 384, 640, 1408, 5120, 17408])
def test_pair_depths(k):
    assert many_rows(1100, 640)
    run_gemm(1100, 640, k, seed=k)


@pytest.mark.parametrize("m,n", [(1300, 577), (1300, 584), (1300, 639), (1300, 641), (1300, 648), (1300, 1001),
                                 (5000, 1), (5000, 7), (5000, 8), (5000, 64), (5000, 100), (5000, 130)])
def test_pair_columns(m, n):
    """Rows stored by TMA, and rows of an odd length stored one by one; tiles that end inside a scale block."""
    assert many_rows(m, n)
    run_gemm(m, n, 384, seed=n)


@pytest.mark.parametrize("m", [1153, 1279, 1281, 1407, 1535, 1537, 4737])
def test_pair_rows(m):
    """The last tile with 1 to 256 rows; several tiles to a CTA pair."""
    n = 2112 if m > 4096 else 520
    assert many_rows(m, n)
    run_gemm(m, n, 512, seed=m)


def test_pair_exact_sums():
    """Small integers and power-of-two scales: the correctly rounded value, whatever the order."""
    m, n, k = 1100, 640, 1024
    assert many_rows(m, n)
    g = gen(11)
    a = torch.randint(-4, 5, (m, k), device=DEV, generator=g).float().to(F8).view(torch.uint8)
    w = torch.randint(-4, 5, (n, k), device=DEV, generator=g).float().to(F8).view(torch.uint8)
    sa = 2.0 ** torch.randint(-2, 3, (m, k // 128), device=DEV, generator=g).float()
    sw = 2.0 ** torch.randint(-2, 3, (n // 128, k // 128), device=DEV, generator=g).float()
    out = poisoned((m, n), torch.bfloat16)
    bsq.fp8_gemm_blockscaled(a, sa, w, sw, out, m, n, k)
    assert torch.equal(out, (dequant_a(a, sa) @ dequant_w(w, sw).t()).float().bfloat16())


@pytest.mark.parametrize("blocks", [4, 5])
def test_pair_scales_are_per_block(blocks):
    """One K block and one N block at a time carry a non-zero scale (K blocks in fours, and one more)."""
    m, n, k = 1100, 640, 128 * blocks
    assert many_rows(m, n)
    a, w = codes((m, k), 20), codes((n, k), 21)
    for kb in range(blocks):
        for nb in range(n // 128):
            sa, sw = torch.zeros(m, blocks, device=DEV), torch.zeros(n // 128, blocks, device=DEV)
            sa[:, kb] = 1 + torch.arange(m, device=DEV) / 64
            sw[nb, kb] = 0.5
            out = poisoned((m, n), torch.bfloat16)
            bsq.fp8_gemm_blockscaled(a, sa, w, sw, out, m, n, k)
            check_gemm(out, a, sa, w, sw, (kb, nb))
            other = torch.ones(n, dtype=torch.bool, device=DEV)
            other[128 * nb:128 * nb + 128] = False
            assert (out[:, other] == 0).all()


@pytest.mark.parametrize("m,n", [(1, 640), (16, 640), (40, 640), (1100, 640), (1300, 577)])
@pytest.mark.parametrize("k", [512, 640, 2048])
@pytest.mark.parametrize("off_a,off_w", [(1, 0), (0, 1), (3, 2)])
def test_product_with_scales_on_4_byte_addresses(m, n, k, off_a, off_w):
    """Scale matrices that start one to three floats past a 16-byte boundary."""
    a, w = codes((m, k), 1), codes((n, k), 2)
    sa = scales((m * (k // 128) + off_a,), 3)[off_a:].view(m, k // 128)
    sw = scales((-(-n // 128) * (k // 128) + off_w,), 4)[off_w:].view(-1, k // 128)
    assert sa.data_ptr() % 16 == 4 * off_a and sw.data_ptr() % 16 == 4 * off_w
    out = poisoned((m + 1, n), torch.bfloat16)
    bsq.fp8_gemm_blockscaled(a, sa, w, sw, out, m, n, k)
    check_gemm(out[:m], a, sa, w, sw, (m, n, k))
    assert out[m].isnan().all()


# ------------------------------------------- producers, two units a lane ---

def two_units(m, k):
    return m * k // 16 >= sms() * 2048 * 3


# the last CTA holds 512 units where all are in range; these leave it a part of its first or second 256
@pytest.mark.parametrize("m,k", [(23000, 640), (7700, 1920), (1003, 17408), (120001, 128)])
def test_quantiser_two_units(m, k):
    assert two_units(m, k) and m * k // 16 % 512
    x = activations(m, k, 1)
    q, s = poisoned((m + 1, k), torch.uint8), poisoned((m + 1, k // 128), torch.float32)
    bsq.quant_act_fp8_per128(x, q, s, m, k)
    assert (q[m] == 0xFF).all() and s[m].isnan().all()
    for rows in (slice(0, 150), slice(m // 2, m // 2 + 150), slice(m - 150, m)):
        oq, os_ = oracle.quant_rowwise_fp8(x[rows].view(torch.int16).cpu().numpy().view(np.uint16).reshape(-1, 128))
        assert np.array_equal(q[rows].cpu().numpy().reshape(-1, 128), oq)
        assert np.array_equal(s[rows].cpu().numpy().reshape(-1), os_)
    check_codes(q[:m], s[:m], x.double(), 128, 0.0, (m, k))


@pytest.mark.parametrize("m,k", [(23000, 640), (7700, 1920), (1003, 17408), (120001, 128)])
def test_silu_two_units(m, k):
    assert two_units(m, k) and m * k // 16 % 512
    x = activations(m, 2 * k, 2)
    q, s = poisoned((m + 1, k), torch.uint8), poisoned((m + 1, k // 128), torch.float32)
    bsq.silu_mul_quant_fp8_per128(x, q, s, m, k)
    g, u = x.double().split(k, dim=1)
    check_codes(q[:m], s[:m], g * torch.sigmoid(g) * u, 128, 6 * U32, (m, k))
    assert (q[m] == 0xFF).all() and s[m].isnan().all()


@pytest.mark.parametrize("group", [128, 0])
@pytest.mark.parametrize("residual", [True, False])
@pytest.mark.parametrize("m,k", [(600, 5120), (2100, 2688), (700, 4224), (200, 16384), (5, 20480), (4, 40960), (3, 65536)])
def test_norm_two_and_four_units(m, k, residual, group):
    """A CTA per row with two units per thread (the long prefill's form) and, beyond K = 32768, four."""
    assert (k // 16 > 160 and m * (k // 16) > 1024 * sms()) or k // 16 > 1024
    x, r = activations(m, k, 3), activations(m, k, 4)
    gain = (1 + 0.2 * torch.randn(k, device=DEV, generator=gen(5))).bfloat16()
    h = (x.float() + r.float()).bfloat16() if residual else x
    out = poisoned((m, k), torch.bfloat16) if residual else None
    q = poisoned((m + 1, k), torch.uint8)
    s = poisoned((m + 1, k // group) if group else (m + 1,), torch.float32)
    bsq.rmsnorm_residual_quant_fp8(x, r if residual else None, gain, 1e-6, out, q, s, group, m, k)
    if residual:
        assert torch.equal(out.view(torch.int16), h.view(torch.int16))
    check_codes(q[:m], s[:m], norm_exact(h, gain, 1e-6), group, norm_rel(k), (m, k, residual, group))
    assert (q[m] == 0xFF).all() and s[m].isnan().all()


# ------------------------------------------ expert layer, choice by rounds ---

@pytest.mark.parametrize("renorm", [0, 1])
@pytest.mark.parametrize("e,topk", [(64, 8), (300, 8), (512, 16)])
def test_moe_routing_corners_by_rounds(e, topk, renorm):
    """The corners of the choice of experts where it is made by rounds of a maximum: beyond 2^15 tokens x experts^2."""
    t = 16
    assert t * e * e > 1 << 15
    l = torch.randn(t, e, device=DEV, generator=gen(1))
    l[0] = -torch.inf  # nothing may be chosen
    l[1] = 0.0  # all tie: the lowest indices
    l[2, 5:] = -torch.inf  # fewer candidates than choices
    l[3, 7] = torch.nan  # counts as -inf
    l[3, 9] = torch.inf  # certain
    l[4] = -0.0
    l[4, 30] = 0.0  # equals -0
    l[5, 3] = 90.0  # others' weights underflow
    l[6] = torch.finfo(torch.float32).min  # masks of the type's lowest value
    l[6, 11] = 1.0
    l[7] = torch.nan
    l[8] = torch.inf  # all certain
    l[9] = l[9].round()  # many ties
    l[10] = -l[10].abs().round()
    l[11, ::32] = 7.0  # ties among one lane's experts
    l[12, 1::2] = -torch.inf
    l[13, e - 3:] = 50.0  # the last experts
    l[14, 32:] = torch.nan
    l[15] = torch.arange(e, device=DEV) * 1e-3
    m = Moe(t, 256, 128, e, topk, renorm, seed=5, logits=l)
    m()
    m.check((e, renorm))
    assert (m.out[0] == 0).all() and (m.out[7] == 0).all()
