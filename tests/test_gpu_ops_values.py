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
    with np.errstate(invalid="ignore"):
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


# ------------------------------------------------------------------------- infinities, NaN and zeros into e4m3 blocks
INF, NAN = float("inf"), float("nan")


def hard_blocks():
    """Blocks of 128 (64 bits): zeros, one infinity, NaN alone and among numbers, all infinite, the largest and smallest values."""
    x = torch.zeros(8, 128, dtype=torch.float64)
    x[1, 5], x[1, 6], x[1, 7] = INF, 100.0, -3.0
    x[2, 3], x[2, 4], x[2, 100] = NAN, -INF, 0.5
    x[3, :] = NAN
    x[4, :] = -INF
    x[5] = torch.linspace(-448, 448, 128)
    x[6, 0], x[6, 1] = 1e38, -1.0
    x[7, 0], x[7, 1] = 2.0 ** -100, 2.0 ** -104
    return x


def check_e4m3(codes, sf, want, exact=True):
    """codes [rows, cols], sf [cols / 128, ld] against values: NaN codes where a value is not finite, scales of the others."""
    q, s = ref.quantise(want)
    got, sf = codes.view(torch.float8_e4m3fn).cpu().double().numpy(), sf[:, :len(want)].t().cpu().double().numpy()
    assert (np.isnan(got) == np.isnan(q)).all() and (sf == s).all()
    if exact:
        assert (got[~np.isnan(q)] == q[~np.isnan(q)]).all()
    else:  # a value next to a border between two codes may go either way: one step
        fine = ~np.isnan(q)
        assert (np.abs(got - q)[fine] <= np.maximum(np.abs(q[fine]) * 2.0 ** -3, 2.0 ** -9)).all()


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_combine_gradient_of_special_values_to_e4m3(dg, dtype, many):
    """d_rows = w d_out, where the block's largest value is |w| times that of d_out: products 0 inf, overflows, w not finite."""
    weights = [1.0, -2.0, 0.0, 2.0 ** 30, INF, NAN, 2.0 ** -140]
    x = hard_blocks().reshape(4, 256).to(dtype)
    T, k = (1200 if many else 4), len(weights)  # (from 8 tokens an SM on a warp takes a token, below a CTA)
    d = x.repeat(T // 4, 1).cuda()
    w = torch.tensor(weights).repeat(T, 1).cuda()
    row = torch.randperm(T * k, generator=torch.Generator().manual_seed(1)).to(torch.int32).view(T, k).cuda()
    rows = torch.ones(T * k, 256, dtype=dtype, device="cuda")
    codes, sf = torch.zeros(T * k, 256, dtype=torch.uint8, device="cuda"), torch.full((2, (T * k + 3) // 4 * 4), -1.0, device="cuda")
    d_w = torch.empty(T, k, device="cuda")
    dg.moe_unpermute_backward(d, rows, row, w, (codes, sf), d_w)
    dg.check_device_error()
    # each product rounded to 32 bits, as it is before it is quantised (an overflow is an infinity, which has no scale)
    with np.errstate(over="ignore", invalid="ignore"):
        products = (w.cpu().double().numpy()[:, :, None] * d.cpu().double().numpy()[:, None, :]).astype(np.float32)
    at = row.cpu().view(-1).long()
    want = np.zeros((T * k, 256), np.float32)
    want[at.numpy()] = products.reshape(T * k, 256)
    check_e4m3(codes, sf, want)
    with np.errstate(invalid="ignore"):
        sums = d.cpu().double().numpy().sum(1)
    # rows of ones: sums of at most 256 values, their chains below 2^6 additions
    size = np.where(np.isfinite(sums), np.abs(np.nan_to_num(d.cpu().double().numpy(), nan=0, posinf=0, neginf=0)).sum(1), 0)
    equal_but_for(d_w, np.repeat(sums[:, None], k, 1), np.repeat(size[:, None], k, 1) * 2.0 ** -18)


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_swiglu_of_special_values_to_e4m3(dg, dtype, backward):
    """Gates of 30 (sigmoid 1 in 32 bits): h = 30 u, d_g = d u, d_u = 30 d with infinities and NaN in u and d."""
    x = hard_blocks().reshape(8, 128).to(dtype)
    gate = torch.full_like(x, 30.0)
    d = torch.full_like(x, 1.0)
    d[0, 5], d[0, 6] = INF, NAN
    gu, d = torch.cat([gate, x], 1).cuda(), d.cuda()
    cols = 256 if backward else 128
    codes, sf = torch.zeros(8, cols, dtype=torch.uint8, device="cuda"), torch.zeros(cols // 128, 8, device="cuda")
    if backward:
        dg.swiglu_backward(d, gu, (codes, sf))
    else:
        dg.swiglu(gu, (codes, sf))
    dg.check_device_error()
    x64, d64 = x.double(), d.cpu().double()
    want = torch.cat([d64 * x64, d64 * 30], 1) if backward else x64 * 30
    if not backward:  # 30 * 1e38 is past 32 bits
        with np.errstate(over="ignore"):
            want = torch.from_numpy(want.numpy().astype(np.float32))
    check_e4m3(codes, sf, want.double().numpy(), exact=False)


@pytest.mark.parametrize("T", [8, 4000])
@pytest.mark.parametrize("X", [BF16, F32])
def test_norm_of_rows_that_are_not_finite_to_e4m3(dg, X, T):
    """An infinity makes its row's r 0 and itself NaN, a NaN the whole row; other rows are as they are without them."""
    H = 384
    g = torch.Generator(device="cuda").manual_seed(T)
    x, y, w = torch.randn(T, H, device="cuda", generator=g).to(X), torch.randn(T, H, device="cuda", generator=g).to(BF16), torch.ones(H, device="cuda")
    def call(x, y):
        codes, sf = torch.zeros(T, H, dtype=torch.uint8, device="cuda"), torch.zeros(H // 128, (T + 3) // 4 * 4, device="cuda")
        one, x_out = (codes.clone(), sf.clone()), torch.empty_like(x)
        dg.rms_norm(x, w, one)
        dg.residual_rms_norm(x, y, x_out, weight=w, out=(codes, sf), weight_post=w)
        return [one, (codes, sf)]
    clean = call(x, y)
    bad, bad_y = x.clone(), y.clone()
    bad[1, 7], bad[4, 130], bad[6, 383] = INF, NAN, -INF
    bad_y[2, 3], bad_y[5, 9] = NAN, INF
    got = call(bad, bad_y)
    dg.check_device_error()
    for n, ((c0, s0), (c1, s1)) in enumerate(zip(clean, got)):
        touched = [1, 4, 6] + ([2, 5] if n else [])
        rest = torch.tensor([t for t in range(T) if t not in touched], device="cuda")
        assert torch.equal(c0[rest], c1[rest]) and torch.equal(s0[:, :T][:, rest], s1[:, :T][:, rest])
        values = c1.view(torch.float8_e4m3fn).float()
        for t, at in ((1, 7), (6, 383)):  # x / infinity: zeros, but for infinity times 0
            want = torch.zeros(H, device="cuda")
            want[at] = NAN
            assert torch.equal(torch.isnan(values[t]), torch.isnan(want)) and float(values[t].nan_to_num().abs().max()) == 0
            assert bool((s1[:, t] == 1).all())
        assert bool(torch.isnan(values[4]).all()) and bool((s1[:, 4] == 1).all())
        if n:
            assert bool(torch.isnan(values[2]).all())
            # y's infinity: y r_y is NaN there and 0 elsewhere, so x' has one NaN and its row is NaN
            assert bool(torch.isnan(values[5]).all())


def test_swiglu_of_extreme_gates_keeps_infinities(dg):
    """Results past the largest number are infinities of the right sign; a gate of minus infinity gives NaN, as infinity times 0."""
    g = torch.tensor([0.0, -0.0, 90.0, -90.0, 1e4, -1e4, 3e38, -3e38, INF, NAN, 3e38, -INF] + [1.0] * 116, device="cuda")
    u = torch.full((128,), 2.0, device="cuda")
    u[10] = -2.0
    for dtype in (BF16, F32):
        gu = torch.cat([g, u])[None].to(dtype)
        out = torch.empty(1, 128, dtype=dtype, device="cuda")
        dg.swiglu(gu, out)
        v, uu = gu[0].double().cpu().numpy().reshape(2, 128)
        with np.errstate(over="ignore", invalid="ignore"):
            want = v / (1 + np.exp(-v)) * uu
            want[11] = NAN
            want = np.where(np.abs(want) > torch.finfo(dtype).max, np.sign(want) * np.inf, want)
        assert want[6] == np.inf and want[10] == -np.inf and want[8] == np.inf
        # (g = -90: a result of 1e-37 whose sigmoid, below 2^-126, may count as 0)
        equal_but_for(out[0], want, np.where(np.isfinite(want), np.abs(want), 0) * (HALF[dtype] + 2.0 ** -17) + 2e-37)
