"""GPU tests of the block-FP8 feed-forward operators against plain 64-bit
implementations of their definitions.

Tolerances count roundings: half a step is 2^-8 (BF16), 2^-11 (FP16), 2^-24
(FP32) of a value, and half the E4M3 step at it.  A sum of n FP32 terms in any
order is off by less than n * 2^-23 times the sum of their magnitudes, also
where each addition truncates."""
import numpy as np
import pytest
import torch

import int8_gemm_gemv_b200 as bsq
import oracle

pytestmark = pytest.mark.gpu
DEV = "cuda"
F8 = torch.float8_e4m3fn
U32 = 2.0**-23


@pytest.fixture(autouse=True)
def _no_timeouts():
    yield
    assert bsq.debug_take_timeouts() == 0


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def activations(m, k, seed):
    g = gen(seed)
    x = torch.randn(m, k, device=DEV, generator=g) * (1 + 19 * (torch.rand(k, device=DEV, generator=g) < 0.01))
    return x.bfloat16()


def codes(shape, seed):
    """Every finite E4M3 code, each as likely as another."""
    q = torch.randint(0, 254, shape, device=DEV, dtype=torch.int32, generator=gen(seed))
    return torch.where(q >= 127, q + 1, q).to(torch.uint8)  # 0x7F and 0xFF are NaN


def scales(shape, seed):
    return torch.rand(shape, device=DEV, generator=gen(seed)) * 1e-3 + 1e-5


def poisoned(shape, dtype):
    t = torch.empty(shape, dtype=dtype, device=DEV)
    t.view(torch.uint8).fill_(0xFF)
    return t


def e4m3(q):
    return q.view(F8).double()


def half_step(v):
    """Half the E4M3 step at each value."""
    _, ex = torch.frexp(v.abs())
    return torch.ldexp(torch.ones_like(v), (ex - 1).clamp(min=-6, max=8) - 4)


def check_codes(q, s, y, group, rel, what):
    """q, s against the exact rows y: s = amax / 448 and q the code nearest
    y / s, where y carries a relative error of at most `rel`."""
    m, k = y.shape
    g = group or k
    ex = y.abs().view(m, k // g, g).amax(-1) / 448
    s = s.double().view(m, k // g)
    assert torch.isfinite(s).all(), what
    # s: the error of y, one division
    assert ((s - ex).abs() <= (rel + U32) * ex + 2.0**-149).all(), what
    v = (y.view(m, k // g, g) / torch.where(s == 0, 1, s)[..., None]).view(m, k)
    got = e4m3(q)
    assert torch.isfinite(got).all(), what
    # q: half a step (values up to 448 (1 + rel) saturate), the error of y, one division
    tol = half_step(v) + 2 * (rel + U32) * v.abs()
    bad = (got - v).abs() > tol
    assert not bad.any(), (what, int(bad.sum()), got[bad][:4], v[bad][:4])
    assert (got[(s == 0).repeat_interleave(g, 1)] == 0).all(), what


# ------------------------------------------------------ quant per 128 ---

@pytest.mark.parametrize("m,k", [(1, 128), (3, 256), (16, 5120), (129, 1408), (1000, 128), (7, 17408), (513, 640)])
def test_quant_act_codes_are_the_oracles(m, k):
    x = activations(m, k, 1)
    if m > 2:
        x[1, :128] = 0
        x[2, 128 % k:] = torch.finfo(torch.bfloat16).max
        x[2, 5] = -1e-38
    q, s = poisoned((m + 1, k), torch.uint8), poisoned((m + 1, k // 128), torch.float32)
    bsq.quant_act_fp8_per128(x, q, s, m, k)
    oq, os_ = oracle.quant_rowwise_fp8(x.view(torch.int16).cpu().numpy().view(np.uint16).reshape(-1, 128))
    assert np.array_equal(q[:m].cpu().numpy().reshape(-1, 128), oq)
    assert np.array_equal(s[:m].cpu().numpy().reshape(-1), os_)
    assert (q[m] == 0xFF).all() and s[m].isnan().all()  # nothing behind the last row


def test_quant_act_on_code_boundaries():
    """Values at, and one BF16 step either side of, every boundary between two
    codes, for every BF16 mantissa of amax: ties and near-ties."""
    codes_up = torch.arange(0x7F, dtype=torch.uint8).view(F8).double()  # 0 .. 448
    mid = (codes_up[1:] + codes_up[:-1]) / 2  # 126 of them
    top = (1 + torch.arange(128) / 128).double()
    amax = torch.cat([top * 2.0**e for e in (-125, -60, -52, 0, 7, 66, 127)])
    x = (amax[:, None] * mid / 448).bfloat16()
    x = torch.cat([x, torch.zeros(len(amax), 1), amax[:, None]], 1).bfloat16()
    x = torch.cat([torch.where(x.view(torch.int16) + d >= 0, x.view(torch.int16) + d, 0).view(torch.bfloat16)
                   for d in (-1, 0, 1)])
    x[:, 127] = amax.bfloat16().repeat(3)
    x[:, :126:2] *= -1
    assert torch.equal(x.abs().amax(1).double(), amax.repeat(3))
    q, s = poisoned(x.shape, torch.uint8), poisoned((len(x),), torch.float32)
    bsq.quant_act_fp8_per128(x.to(DEV), q, s, len(x), 128)
    oq, os_ = oracle.quant_rowwise_fp8(x.view(torch.int16).numpy().view(np.uint16))
    assert np.array_equal(s.cpu().numpy(), os_)
    assert np.array_equal(q.cpu().numpy(), oq)


# ---------------------------------------------------------- silu * mul ---

@pytest.mark.parametrize("m,k", [(1, 128), (5, 17408), (64, 1408), (333, 256), (3, 512)])
def test_silu_mul_quant(m, k):
    x = activations(m, 2 * k, 2)
    if m > 2:
        x[0, :128] = 0  # a zero gate: an all-zero group
        x[1, 3] = -90.0  # exp(90) is finite, exp(-g) of the next is not
        x[1, 4] = -300.0
        x[2, 7] = 300.0
    q, s = poisoned((m + 1, k), torch.uint8), poisoned((m + 1, k // 128), torch.float32)
    bsq.silu_mul_quant_fp8_per128(x, q, s, m, k)
    g, u = x.double().split(k, dim=1)
    # exp: 2 ulp; 1 + e, the quotient and the product: half an ulp each (and one more for a fast quotient)
    check_codes(q[:m], s[:m], g * torch.sigmoid(g) * u, 128, 6 * U32, (m, k))
    assert (q[m] == 0xFF).all() and s[m].isnan().all()


# ------------------------------------------------------------- rmsnorm ---

def norm_exact(h, gain, eps):
    h = h.double()
    return h / torch.sqrt((h * h).mean(1, keepdim=True) + eps) * gain.double()


# the sum of k squares (all positive) is off by at most k * 2^-23 of itself in the worst order, its root by half
# of that; the kernels add at most k / 32 terms in a row and then 64, so this bounds every shape here
def norm_rel(k):
    return (k // 32 + 64) * U32 / 2 + 5 * U32


@pytest.mark.parametrize("group", [128, 0])
@pytest.mark.parametrize("residual", ["none", "kept", "dropped", "into_residual", "into_x"])
@pytest.mark.parametrize("m,k", [(1, 128), (2, 256), (5, 5120), (33, 1408), (300, 640)])
def test_rmsnorm(m, k, residual, group):
    x, r = activations(m, k, 3), activations(m, k, 4)
    gain = (1 + 0.2 * torch.randn(k, device=DEV, generator=gen(5))).bfloat16()
    if m > 2:
        x[1] = 0
        r[1] = 0
    h = x if residual == "none" else (x.float() + r.float()).bfloat16()
    h = h.clone()
    out = {"none": None, "dropped": None, "kept": poisoned((m, k), torch.bfloat16), "into_residual": r,
           "into_x": x}[residual]
    q = poisoned((m + 1, k), torch.uint8)
    s = poisoned((m + 1, k // group) if group else (m + 1,), torch.float32)
    bsq.rmsnorm_residual_quant_fp8(x, None if residual == "none" else r, gain, 1e-6, out, q, s, group, m, k)
    torch.cuda.synchronize()
    if out is not None:
        assert torch.equal(out.view(torch.int16), h.view(torch.int16))
    check_codes(q[:m], s[:m], norm_exact(h, gain, 1e-6), group, norm_rel(k), (m, k, residual, group))
    assert (q[m] == 0xFF).all() and s[m].isnan().all()


@pytest.mark.parametrize("k", [16, 48, 112, 4112, 8208, 20000, 65536])
def test_rmsnorm_rows_of_any_width(k):
    m = 9
    x, r = activations(m, k, 6), activations(m, k, 7)
    gain = (1 + 0.2 * torch.randn(k, device=DEV, generator=gen(8))).bfloat16()
    h = (x.float() + r.float()).bfloat16()
    for group in (0, 128) if k % 128 == 0 else (0,):
        res = r.clone()
        q = poisoned((m, k), torch.uint8)
        s = poisoned((m, k // group) if group else (m,), torch.float32)
        bsq.rmsnorm_residual_quant_fp8(x, res, gain, 1e-5, res, q, s, group, m, k)
        torch.cuda.synchronize()
        assert torch.equal(res.view(torch.int16), h.view(torch.int16))
        check_codes(q, s, norm_exact(h, gain, 1e-5), group, norm_rel(k), (k, group))


def test_rmsnorm_zero_row_without_eps():
    x = torch.zeros(2, 256, dtype=torch.bfloat16, device=DEV)
    x[1, 0] = 3
    gain = torch.ones(256, dtype=torch.bfloat16, device=DEV)
    q, s = poisoned((2, 256), torch.uint8), poisoned((2, 2), torch.float32)
    bsq.rmsnorm_residual_quant_fp8(x, None, gain, 0.0, None, q, s, 128, 2, 256)
    assert (q[0] == 0).all() and (s[0] == 0).all()
    check_codes(q[1:], s[1:], norm_exact(x[1:], gain, 0.0), 128, norm_rel(256), "one spike")


@pytest.mark.parametrize("group", [128, 0])
def test_rmsnorm_rows_whose_squares_vanish(group):
    """eps alone under the root: h^2 is below FP32's range, h and y are not."""
    x = (activations(3, 1024, 9).float() * 1e-25).bfloat16()
    gain = torch.ones(1024, dtype=torch.bfloat16, device=DEV)
    q, s = poisoned((3, 1024), torch.uint8), poisoned((3, 8) if group else (3,), torch.float32)
    bsq.rmsnorm_residual_quant_fp8(x, None, gain, 1e-6, None, q, s, group, 3, 1024)
    check_codes(q, s, norm_exact(x, gain, 1e-6), group, norm_rel(1024), group)


# ------------------------------------------------- offsets past 32 bits ---

def test_rows_past_two_to_the_31_elements():
    """A row's result does not depend on where it lies."""
    m, k, last = 131200, 16384, 3
    x = torch.zeros(m, k, dtype=torch.bfloat16, device=DEV)
    assert x.numel() > 2**31
    x[-last:] = activations(last, k, 10)
    gain = activations(1, k, 11)[0]
    for groups, call in ((k // 128, lambda x, q, s, m: bsq.quant_act_fp8_per128(x, q, s, m, k)),
                         (1, lambda x, q, s, m: bsq.rmsnorm_residual_quant_fp8(x, None, gain, 1e-6, None, q, s, 0, m,
                                                                               k)),
                         (k // 256, lambda x, q, s, m: bsq.silu_mul_quant_fp8_per128(x, q, s, m, k // 2))):
        width = k // 2 if groups == k // 256 else k
        q, s = poisoned((m, width), torch.uint8), poisoned((m, groups), torch.float32)
        call(x, q, s, m)
        q1, s1 = poisoned((last, width), torch.uint8), poisoned((last, groups), torch.float32)
        call(x[-last:], q1, s1, last)
        assert torch.equal(q[-last:], q1) and torch.equal(s[-last:], s1)
        assert not (q[:-last].any() or s[:-last].any())


@pytest.mark.parametrize("n", [16400, 16401])
def test_gemm_output_past_two_to_the_31_elements(n):
    m, k, last = 131200, 256, 3
    a, sa = torch.zeros(m, k, dtype=torch.uint8, device=DEV), scales((m, k // 128), 12)
    a[-last:] = codes((last, k), 13)
    w, sw = codes((n, k), 14), scales(((n + 127) // 128, k // 128), 15)
    out = poisoned((m, n), torch.bfloat16)
    assert out.numel() > 2**31
    bsq.fp8_gemm_blockscaled(a, sa, w, sw, out, m, n, k)
    check_gemm(out[-last:], a[-last:], sa[-last:], w, sw, n)
    assert not out[:-last].any()


# ---------------------------------------------------------------- GEMM ---

def dequant_a(a, sa):
    return (e4m3(a).unflatten(-1, (-1, 128)) * sa.double()[..., None]).flatten(-2)


def dequant_w(w, sw):
    n = w.shape[-2]
    return (e4m3(w).unflatten(-1, (-1, 128)) * sw.double().repeat_interleave(128, -2)[..., :n, :, None]).flatten(-2)


def check_gemm(out, a, sa, w, sw, what):
    A, W = dequant_a(a, sa), dequant_w(w, sw)
    want, mag = A @ W.t(), A.abs() @ W.abs().t()
    k = a.shape[1]
    # products of two E4M3 values are exact; 128 terms to a block, then k / 128 folds and two scale products
    tol = 2.0**-8 * want.abs() + (128 + k // 128 + 4) * U32 * mag
    err = (out.double() - want).abs()
    bad = ~(err <= tol)
    assert not bad.any(), (what, int(bad.sum()), out[bad][:4], want[bad][:4], torch.nonzero(bad)[:4])


def run_gemm(m, n, k, seed=0):
    a, w = codes((m, k), seed), codes((n, k), seed + 1)
    sa, sw = scales((m, k // 128), seed + 2), scales((-(-n // 128), k // 128), seed + 3)
    if m > 3:
        sa[2] = 0
        a[3] = 0
    out = poisoned((m + 1, n), torch.bfloat16)
    bsq.fp8_gemm_blockscaled(a, sa, w, sw, out, m, n, k)
    check_gemm(out[:m], a, sa, w, sw, (m, n, k))
    assert out[m].isnan().all()  # nothing behind the last row


@pytest.mark.parametrize("m", [1, 2, 7, 8, 9, 16, 17, 31, 33, 64, 65, 96, 127, 128, 129, 200, 256, 257, 511, 1030])
def test_gemm_rows(m):
    run_gemm(m, 640, 1024, seed=m)


@pytest.mark.parametrize("n", [1, 2, 7, 8, 63, 100, 127, 128, 129, 130, 255, 257, 264, 576, 1000, 2112])
@pytest.mark.parametrize("m", [3, 40, 300])
def test_gemm_columns(m, n):
    run_gemm(m, n, 384, seed=n)


@pytest.mark.parametrize("m", [1, 20, 100, 260])
@pytest.mark.parametrize("k", [128, 256, 384, 640, 1408, 5120, 17408])
def test_gemm_depths(m, k):
    run_gemm(m, 264, k, seed=k)


@pytest.mark.parametrize("mnk", [(16, 5120, 5120), (128, 10240, 1024), (777, 2112, 5120), (1500, 5000, 640)])
def test_gemm_larger(mnk):
    run_gemm(*mnk, seed=9)


@pytest.mark.parametrize("m", [5, 70, 300])
def test_gemm_exact_sums(m):
    """Small integers and power-of-two scales: every sum is exact, so the
    output is the correctly rounded BF16 value, whatever the order."""
    n, k = 320, 1024
    g = gen(11)
    a = torch.randint(-4, 5, (m, k), device=DEV, generator=g).float().to(F8)
    w = torch.randint(-4, 5, (n, k), device=DEV, generator=g).float().to(F8)
    sa = 2.0 ** torch.randint(-2, 3, (m, k // 128), device=DEV, generator=g).float()
    sw = 2.0 ** torch.randint(-2, 3, (3, k // 128), device=DEV, generator=g).float()
    out = poisoned((m, n), torch.bfloat16)
    bsq.fp8_gemm_blockscaled(a.view(torch.uint8), sa, w.view(torch.uint8), sw, out, m, n, k)
    want = dequant_a(a.view(torch.uint8), sa) @ dequant_w(w.view(torch.uint8), sw).t()
    assert torch.equal(out, want.float().bfloat16())


@pytest.mark.parametrize("m", [9, 130])
def test_gemm_scales_are_per_block(m):
    """One K block and one N block at a time carry a non-zero scale."""
    n, k = 384, 512
    a, w = codes((m, k), 20), codes((n, k), 21)
    for kb in range(4):
        for nb in range(3):
            sa, sw = torch.zeros(m, 4, device=DEV), torch.zeros(3, 4, device=DEV)
            sa[:, kb] = 1 + torch.arange(m, device=DEV) / 64
            sw[nb, kb] = 0.5
            out = poisoned((m, n), torch.bfloat16)
            bsq.fp8_gemm_blockscaled(a, sa, w, sw, out, m, n, k)
            check_gemm(out, a, sa, w, sw, (kb, nb))
            other = torch.ones(n, dtype=torch.bool, device=DEV)
            other[128 * nb:128 * nb + 128] = False
            assert (out[:, other] == 0).all()


# ----------------------------------------------------------------- MoE ---

class Moe:
    def __init__(self, t, h, i, e, topk, renorm, seed=0, logits=None):
        g = gen(seed)
        self.dims = (t, h, i, e, topk, renorm)
        self.x = activations(t, h, seed + 1)
        self.logits = torch.randn(t, e, device=DEV, generator=g) if logits is None else logits
        self.w13, self.w2 = codes((e, 2 * i, h), seed + 2), codes((e, h, i), seed + 3)
        # random codes reach 448: keep gate and up near 1 so that silu is in its curved part
        self.s13 = (0.5 + torch.rand(e, 2 * i // 128, h // 128, device=DEV, generator=g)) * (2e-2 / h**0.5)
        self.s2 = (0.5 + torch.rand(e, h // 128, i // 128, device=DEV, generator=g)) * 1e-2
        self.out = poisoned((t + 1, h), torch.bfloat16)
        self.ids, self.tw = poisoned((t, topk), torch.int32), poisoned((t, topk), torch.float32)
        self.bytes = bsq.fp8_moe_workspace_bytes(t, h, i, topk)
        assert self.bytes > 0
        self.ws = poisoned((self.bytes + 64,), torch.uint8)

    def __call__(self, stream=None, ids=True):
        t, h, i, e, topk, renorm = self.dims
        bsq.fp8_moe_blockscaled(self.x, self.logits, self.w13, self.s13, self.w2, self.s2, self.out,
                                self.ids if ids else None, self.tw if ids else None, self.ws, self.bytes, t, h, i, e,
                                topk, renorm, stream)

    def check(self, what=""):
        t, h, i, e, topk, renorm = self.dims
        l = torch.where(self.logits.isnan(), -torch.inf, self.logits).double()
        ids = torch.argsort(l, dim=1, descending=True, stable=True)[:, :topk]
        assert torch.equal(self.ids.long(), ids), what
        mx = l.amax(1, keepdim=True)
        p = torch.where(l == mx, 1.0, torch.exp(l - mx))
        p = torch.where((mx == -torch.inf).expand_as(p), 0.0, p)
        pk = p.gather(1, ids)
        den = (pk if renorm else p).sum(1, keepdim=True)
        tw = torch.where(den > 0, pk / den, 0.0)
        # the difference l - max is rounded once (2^-24 of up to 100 here), exp 2 ulp, up to 512 terms to the sum
        assert ((self.tw.double() - tw).abs() <= (520 + 100) * U32 * tw + 2.0**-126).all(), what
        want = torch.zeros(t, h, dtype=torch.float64, device=DEV)
        tol = torch.zeros_like(want)
        x = self.x.double()
        for ex in ids.unique().tolist():
            tok, slot = torch.where(ids == ex)
            w13, w2 = dequant_w(self.w13[ex], self.s13[ex]), dequant_w(self.w2[ex], self.s2[ex])
            gu, mag = x[tok] @ w13.t(), x[tok].abs() @ w13.abs().t()
            gate, up = gu.split(i, 1)
            # FP32 sums of h terms (one product rounding each, the scale, the activation's FP16 grid)
            dg, du = ((h + 8) * U32 * mag).split(i, 1)
            sg = gate * torch.sigmoid(gate)
            act = sg * up
            # |d silu / dg| < 1.1; silu itself 6 roundings; act kept with 11 bits (2^-11), on a grid of 2^-38 of
            # the row's largest
            dact = (1.1 * dg + 8 * U32 * sg.abs()) * (up.abs() + du) + sg.abs() * du
            dact += 2.0**-11 * act.abs() + 2.0**-38 * act.abs().amax(1, keepdim=True)
            # a product below 2^-126 is rounded to a multiple of 2^-149 instead (half of it each for silu * up and
            # the store); the output below 2^-126 to one of 2^-133
            dact += 2.0**-149
            wt = tw[tok, slot][:, None]
            want.index_add_(0, tok, wt * (act @ w2.t()))
            m2 = act.abs() @ w2.abs().t()
            tol.index_add_(0, tok, wt * (dact @ w2.abs().t() + (i + topk + 16 + 620) * U32 * m2))
        tol += 2.0**-8 * want.abs() + 2.0**-134
        err = (self.out[:t].double() - want).abs()
        bad = ~(err <= tol)
        assert not bad.any(), (what, int(bad.sum()), torch.nonzero(bad)[:4], self.out[:t][bad][:4], want[bad][:4])
        assert self.out[t].isnan().all() and (self.ws[self.bytes:] == 0xFF).all(), what


@pytest.mark.parametrize("t,h,i,e,topk,renorm", [
    (1, 128, 128, 1, 1, 1), (1, 2048, 768, 16, 8, 1), (2, 1024, 384, 8, 2, 0), (3, 640, 128, 5, 5, 0),
    (7, 256, 256, 9, 3, 1), (8, 1408, 640, 12, 4, 0), (9, 512, 128, 33, 2, 1), (16, 1024, 1408, 24, 8, 0),
    (16, 256, 128, 4, 1, 1), (16, 384, 256, 300, 16, 0), (5, 128, 2176, 6, 2, 1), (13, 5120, 128, 8, 3, 0),
    (4, 7168, 256, 3, 2, 1), (16, 512, 256, 3, 2, 1), (16, 256, 640, 1, 1, 0), (12, 384, 1408, 2, 2, 0)])
def test_moe(t, h, i, e, topk, renorm):
    m = Moe(t, h, i, e, topk, renorm, seed=t)
    m()
    m.check()


def test_moe_routing_corners():
    t, e = 8, 40
    l = torch.randn(t, e, device=DEV, generator=gen(1))
    l[0] = -torch.inf  # nothing may be chosen
    l[1] = 0.0  # all tie: the lowest indices
    l[2, 5:] = -torch.inf  # fewer candidates than 8
    l[3, 7] = torch.nan  # counts as -inf
    l[3, 9] = torch.inf  # certain
    l[4] = -0.0
    l[4, 30] = 0.0  # equals -0
    l[5, 3] = 90.0  # others' weights underflow
    l[6] = torch.finfo(torch.float32).min  # masks of the type's lowest value
    l[6, 11] = 1.0
    l[7] = torch.nan
    for renorm in (0, 1):
        m = Moe(t, 256, 128, e, 8, renorm, seed=5, logits=l)
        m()
        m.check(renorm)
        assert (m.out[0] == 0).all() and (m.out[7] == 0).all()


def test_moe_zero_tokens_and_activations():
    m = Moe(3, 256, 256, 6, 2, 1, seed=6)
    m.x[1] = 0
    m()
    m.check()
    assert (m.out[1] == 0).all()
    before = bsq.debug_launch_count()
    bsq.fp8_moe_blockscaled(m.x, m.logits, m.w13, m.s13, m.w2, m.s2, m.out, m.ids, m.tw, m.ws, m.bytes, 0, 256, 256,
                            6, 2, 1)
    assert bsq.debug_launch_count() == before


def test_moe_wide_activation_range():
    """Elements far below their row's largest, and rows of very different size."""
    m = Moe(4, 512, 256, 4, 2, 1, seed=7)
    m.x[0] *= 2.0**60
    m.s13 *= 2.0**-60
    m.x[1] *= 2.0**-60
    m.x[2, ::2] *= 2.0**-20
    m()
    m.check()


def test_moe_weights_past_two_to_the_32_bytes():
    """The last experts of a large layer give what they give in a small one."""
    t, h, i, e, topk = 3, 2048, 2048, 512, 2
    small = Moe(t, h, i, 2, topk, 1, seed=21)
    small()
    small.check()
    w13 = torch.zeros(e, 2 * i, h, dtype=torch.uint8, device=DEV)
    w2 = torch.zeros(e, h, i, dtype=torch.uint8, device=DEV)
    assert w13.numel() > 2**32 - 1
    s13, s2 = torch.ones(e, 2 * i // 128, h // 128, device=DEV), torch.ones(e, h // 128, i // 128, device=DEV)
    logits = torch.full((t, e), -torch.inf, device=DEV)
    for to, of in ((w13, small.w13), (w2, small.w2), (s13, small.s13), (s2, small.s2)):
        to[-2:] = of
    logits[:, -2:] = small.logits
    out, ids = poisoned((t, h), torch.bfloat16), poisoned((t, topk), torch.int32)
    bsq.fp8_moe_blockscaled(small.x, logits, w13, s13, w2, s2, out, ids, None, small.ws, small.bytes, t, h, i, e, topk,
                            1)
    assert torch.equal(out, small.out[:t]) and torch.equal(ids, small.ids + e - 2)


def test_moe_ids_may_be_null():
    m = Moe(4, 256, 128, 8, 2, 0, seed=8)
    m()
    want = m.out.clone()
    m.out.view(torch.uint8).fill_(0xFF)
    m(ids=False)
    torch.cuda.synchronize()
    assert torch.equal(m.out.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("t", [1, 12])
def test_moe_same_result_every_time(t):
    m = Moe(t, 1920, 640, 16, 4, 1, seed=9)
    m()
    first = m.out.clone()
    m.check()
    for _ in range(20):
        m.ws.view(torch.uint8)[:m.bytes].random_(0, 256)
        m.out.view(torch.uint8).fill_(0xFF)
        m()
        torch.cuda.synchronize()
        assert torch.equal(m.out.view(torch.int16), first.view(torch.int16))


def test_moe_workspace_too_small():
    m = Moe(2, 256, 128, 4, 2, 1)
    m.bytes -= 1
    with pytest.raises(bsq.BsqError) as e:
        m()
    assert e.value.status == bsq.BSQ_ERR_INVALID_ARG


# ---------------------------------------------------------- together ---

class Ffn:
    """norm + residual -> gate/up product -> SiLU -> down product, and the
    same norm in front of an expert layer."""

    def __init__(self, m, h, i, seed=0):
        self.m, self.h, self.i = m, h, i
        self.x, self.res = activations(m, h, seed), activations(m, h, seed + 1)
        self.gain = (1 + 0.1 * torch.randn(h, device=DEV, generator=gen(seed + 2))).bfloat16()
        self.w = []
        for n, k in ((2 * i, h), (h, i)):
            w = (torch.randn(n, k, device=DEV, generator=gen(seed + n)) * 0.02).bfloat16()
            q, s = poisoned((n, k), torch.uint8), poisoned((n // 128, k // 128), torch.float32)
            bsq.quant_blockfp8(w, q, s, n, k)
            self.w.append((q, s))
        self.q1, self.s1 = poisoned((m, h), torch.uint8), poisoned((m, h // 128), torch.float32)
        self.q2, self.s2 = poisoned((m, i), torch.uint8), poisoned((m, i // 128), torch.float32)
        self.gu, self.out = poisoned((m, 2 * i), torch.bfloat16), poisoned((m, h), torch.bfloat16)
        self.res_out = poisoned((m, h), torch.bfloat16)

    def __call__(self, stream=None):
        m, h, i = self.m, self.h, self.i
        bsq.rmsnorm_residual_quant_fp8(self.x, self.res, self.gain, 1e-6, self.res_out, self.q1, self.s1, 128, m, h,
                                       stream)
        bsq.fp8_gemm_blockscaled(self.q1, self.s1, *self.w[0], self.gu, m, 2 * i, h, stream)
        bsq.silu_mul_quant_fp8_per128(self.gu, self.q2, self.s2, m, i, stream)
        bsq.fp8_gemm_blockscaled(self.q2, self.s2, *self.w[1], self.out, m, h, i, stream)

    def check(self):
        hid = (self.x.float() + self.res.float()).bfloat16()
        assert torch.equal(self.res_out.view(torch.int16), hid.view(torch.int16))
        check_codes(self.q1, self.s1, norm_exact(hid, self.gain, 1e-6), 128, norm_rel(self.h), "norm")
        check_gemm(self.gu, self.q1, self.s1, *self.w[0], "gate/up")
        g, u = self.gu.double().split(self.i, 1)
        check_codes(self.q2, self.s2, g * torch.sigmoid(g) * u, 128, 6 * U32, "silu")
        check_gemm(self.out, self.q2, self.s2, *self.w[1], "down")


@pytest.mark.parametrize("m", [1, 24, 200])
def test_dense_ffn_chain(m):
    f = Ffn(m, 1024, 1408)
    f()
    f.check()


def test_rowscale_chain():
    """The norm's per-row form feeds the row-scaled GEMM."""
    m, n, k = 37, 640, 1536
    x, gain = activations(m, k, 1), torch.ones(k, dtype=torch.bfloat16, device=DEV)
    q, s = poisoned((m, k), torch.uint8), poisoned((m,), torch.float32)
    w, sw = codes((n, k), 2), scales((n,), 3)
    out = poisoned((m, n), torch.bfloat16)
    bsq.rmsnorm_residual_quant_fp8(x, None, gain, 1e-6, None, q, s, 0, m, k)
    bsq.fp8_gemm_rowscale(q, s, w, sw, out, m, n, k)
    A, W = e4m3(q) * s.double()[:, None], e4m3(w) * sw.double()[:, None]
    tol = 2.0**-8 * (A @ W.t()).abs() + (k + 4) * U32 * (A.abs() @ W.abs().t())
    assert ((out.double() - A @ W.t()).abs() <= tol).all()


def test_graph_replay_and_other_streams():
    """The chain and the expert layer captured on a side stream and replayed
    with new inputs in place; back-to-back launches without a wait."""
    f, e = Ffn(24, 1024, 640), Moe(6, 1024, 256, 16, 4, 1, seed=3)
    f(), e()  # kernel attributes are set before the capture
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        for _ in range(2):
            f()
            e()
    for seed in (50, 51):
        f.x.copy_(activations(24, 1024, seed))
        e.x.copy_(activations(6, 1024, seed + 2))
        e.logits.copy_(torch.randn(6, 16, device=DEV, generator=gen(seed)))
        for t in (f.out, f.q1, f.q2, f.gu, e.out, e.ws):
            t.view(torch.uint8).fill_(0xFF)
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
        f.check()
        e.check()
    with torch.cuda.stream(side):
        f()
        e()
    side.synchronize()
    f.check()
    e.check()


def test_two_calls_at_once():
    """Two streams, each with its own buffers and workspace."""
    a, b = Moe(5, 1024, 640, 12, 3, 1, seed=1), Moe(11, 1024, 384, 12, 3, 0, seed=2)
    f, g = Ffn(40, 1024, 640, seed=1), Ffn(300, 1024, 640, seed=2)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        a(s1), b(s2), f(s1), g(s2)
    torch.cuda.synchronize()
    a.check(), b.check(), f.check(), g.check()


def test_many_streams_same_bits():
    """Every operator on a stream of its own, several launches in flight on
    each: the same bits as alone."""
    def gemm(m, n, k, seed):
        a, w = codes((m, k), seed), codes((n, k), seed + 1)
        sa, sw = scales((m, k // 128), 1), scales(((n + 127) // 128, k // 128), 2)
        out = poisoned((m, n), torch.bfloat16)
        return (lambda st: bsq.fp8_gemm_blockscaled(a, sa, w, sw, out, m, n, k, st)), out

    jobs = [gemm(700, 5120, 2048, 1), gemm(16, 5120, 5120, 3), gemm(40, 2112, 5120, 5), gemm(3, 1024, 5120, 7),
            gemm(300, 4097, 1024, 9)]
    for seed in (1, 2):
        layer = Moe(5 * seed, 1024, 768, 12, 3, 1, seed=seed)
        jobs.append((layer, layer.out))
    x = activations(500, 5120, 3)
    q, s = poisoned((500, 5120), torch.uint8), poisoned((500, 40), torch.float32)
    jobs.append((lambda st: bsq.rmsnorm_residual_quant_fp8(x, None, x[0], 1e-6, None, q, s, 128, 500, 5120, st), q))
    want = []
    for call, out in jobs:
        call(None)
        torch.cuda.synchronize()
        want.append(out.clone())
    streams = [torch.cuda.Stream() for _ in jobs]
    for _ in range(10):
        for _, out in jobs:
            out.view(torch.uint8).fill_(0xFF)
        torch.cuda.synchronize()
        for _ in range(10):
            for st, (call, _) in zip(streams, jobs):
                call(st)
        torch.cuda.synchronize()
        for (_, out), w in zip(jobs, want):
            assert torch.equal(out.view(torch.uint8), w.view(torch.uint8))
