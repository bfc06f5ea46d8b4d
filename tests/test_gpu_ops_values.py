"""Values at the ends of the number range through the operators around the grouped GEMMs, against 64-bit forms: infinities and
NaN have to stand in the same places, and finite results may not be lost on the way to them."""
import numpy as np
import pytest
import torch

import _ops_ref as ref

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
HALF = {BF16: 2.0 ** -8, F32: 2.0 ** -24}  # of a rounding, relative to the value


@pytest.fixture(scope="module")
def dg():
    import moe_grouped_gemm_03_b200 as dg

    return dg


def equal_but_for(got, want, tol, what=""):
    """NaN and infinities (with their signs) in the same places, |got - want| <= tol elsewhere."""
    got, want = (np.asarray(v.double().cpu() if torch.is_tensor(v) else v, np.float64) for v in (got, want))
    tol = np.broadcast_to(np.asarray(tol, np.float64), want.shape)
    ok = np.where(np.isnan(want), np.isnan(got), np.where(np.isinf(want), got == want, np.abs(got - want) <= tol))
    assert ok.all(), (what, int((~ok).sum()), [(got[i], want[i]) for i in map(tuple, np.argwhere(~ok)[:4])])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_swiglu_gradient_of_large_finite_values(dg, dtype):
    """d u s (1 + g (1 - s)): for a gate far below zero u (1 + g) passes the largest number and s is 0; the product is 0."""
    g = torch.tensor([-1e20, -1e20, -3e38, 3e38, 1e30, -200.0, -1e4, 0.0], dtype=F32)
    u = torch.tensor([1e20, -1e25, 3e38, 2.0, -1e8, 3e38, -3e38, 3e38], dtype=F32)
    d = torch.tensor([1.0, 1e10, -1.0, 0.5, 1e-5, 3e38, -1.0, 0.25], dtype=F32)
    gu, d = torch.cat([g, u])[None].to(dtype).cuda(), d[None].to(dtype).cuda()
    out = torch.full((1, 16), -7.5, dtype=dtype, device="cuda")
    dg.swiglu_backward(d, gu, out)
    dg.check_device_error()
    g, u = gu.double().cpu().chunk(2, 1)
    s = torch.sigmoid(g)
    want = torch.cat([d.double().cpu() * (s * (1 + g * (1 - s))) * u, d.double().cpu() * (g * s)], 1).numpy()
    assert np.isfinite(want).all() and (np.abs(want) < torch.finfo(dtype).max).all()
    # Five roundings and the functions' errors, all below 2^-20, before the last rounding.  s is held in 32 bits: one below
    # 2^-126 may count as 0, and what it is multiplied by as nothing (g = -200, u = d = 3e38: s = 1.4e-87).
    tiny = np.tile((s < 2.0 ** -126).numpy(), 2)
    equal_but_for(out, want, np.abs(want) * np.where(tiny, 1.0, HALF[dtype] + 2.0 ** -20) + 1e-37)


def test_swiglu_gradient_of_large_finite_values_to_e4m3(dg):
    gu = torch.zeros(1, 256, device="cuda")
    gu[0, :128], gu[0, 128:] = -1e20, 1e20
    gu[0, 0], gu[0, 128] = 0.0, 3.0
    d = torch.ones(1, 128, device="cuda")
    codes, sf = torch.zeros(1, 256, dtype=torch.uint8, device="cuda"), torch.zeros(2, 4, device="cuda")
    dg.swiglu_backward(d, gu, (codes, sf))
    got = codes.view(torch.float8_e4m3fn).double().cpu().numpy()
    want = np.zeros((1, 256))
    want[0, 0] = 1.5  # d u / 2
    q, s = ref.quantise(want)
    assert (got == q).all() and (sf[:, 0].cpu().double().numpy() == s[0]).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("fp8", [True, False])
def test_swiglu_of_gates_whose_sigmoid_is_not_a_normal_number(dg, dtype, fp8):
    """Between -88.7 and -87.3 sigmoid is below 2^-126 but not 0: g s u is a normal number for a u large enough."""
    g = torch.linspace(-88.625, -86.0, 128).to(dtype)
    assert float(g.min()) > -88.72  # (exp(-g) is finite in 32 bits down to there)
    gu = torch.cat([g, torch.full((128,), 2.0 ** 100, dtype=dtype)])[None].cuda()
    d = torch.ones(1, 128, dtype=dtype, device="cuda")
    forward, gradient = ref.swiglu(gu).numpy(), ref.swiglu_backward(d, gu).numpy()
    # exp's argument is rounded twice (89 2^-24 each), s below the normal numbers to 2^-150 of at least 2^-128: below 2^-16
    err = 2.0 ** -16
    for want, call, cols in ((forward, lambda o: dg.swiglu(gu, o), 128), (gradient, lambda o: dg.swiglu_backward(d, gu, o), 256)):
        if not fp8:
            out = torch.full((1, cols), -7.5, dtype=dtype, device="cuda")
            call(out)
            equal_but_for(out, want, np.abs(want) * (HALF[dtype] + err))
            continue
        codes, sf = torch.zeros(1, cols, dtype=torch.uint8, device="cuda"), torch.zeros(cols // 128, 4, device="cuda")
        call((codes, sf))
        s = sf[:, 0].cpu().double().numpy()
        top = np.abs(want).reshape(-1, 128).max(1)
        assert ((s >= ref.scale_of(top * (1 - err))) & (s <= ref.scale_of(top * (1 + err)))).all()
        wide = np.repeat(s, 128)[None]
        got = codes.view(torch.float8_e4m3fn).double().cpu().numpy() * wide
        equal_but_for(got, want, np.maximum(np.abs(want) * (1 + err) * 2.0 ** -4, wide * 2.0 ** -10) + np.abs(want) * err)
    dg.check_device_error()
