"""The operators around the grouped GEMMs on the GPU against plain 64-bit forms: dispatch, combine, SwiGLU, norms.

Tolerances, in the units they come from: a rounding to bf16 is off by at most 2^-8 of the value and to fp32 by 2^-24; an
e4m3 code by 2^-4 of the value or half the smallest step, 2^-10 scales.  Sums of n fp32 terms are off by at most n
roundings of the sum of their absolute values; with the trees used here the longest chain stays below 2^6 additions in a
row's sums (2^-18), and the functions' own errors (exp, reciprocal, rsqrt: a few 2^-23) stay inside it.
"""
import numpy as np
import pytest
import torch

import _ops_ref as ref

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
STEP = {BF16: 2.0 ** -8, F32: 2.0 ** -24}
CHAIN = 2.0 ** -18  # 64 roundings of 2^-24


@pytest.fixture(scope="module")
def dg():
    import moe_grouped_gemm_03_b200 as dg

    return dg


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape, dtype=F32, scale=1.0):
    return (torch.randn(*shape, device="cuda", generator=g) * scale).to(dtype)


def near(got, want, tol, what=""):
    """|got - want| <= tol element by element (numpy or torch, 64 bits); non-finite values in the same places."""
    got, want, tol = (np.asarray(v.cpu() if torch.is_tensor(v) else v, np.float64) for v in (got, want, tol))
    assert got.shape == want.shape, (what, got.shape, want.shape)
    tol = np.broadcast_to(tol, want.shape)
    fine = np.isfinite(want)
    assert (np.isnan(got) == np.isnan(want)).all(), what
    err = np.abs(np.where(fine, got, 0) - np.where(fine, want, 0))
    bad = fine & ~(err <= tol)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} off; first at {i}: {got[i]} for {want[i]}, tolerance {tol[i]}")


class Operand:
    """An output operand filled with a sentinel: a tensor, or e4m3 codes and scales; its rows in 64 bits."""

    def __init__(self, shape, dtype, fp8):
        self.fp8, self.shape = fp8, shape
        if fp8:
            per = shape[-2]
            self.a = torch.full(shape, 0xA5, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
            self.sf = torch.full((*shape[:-2], shape[-1] // 128, (per + 3) // 4 * 4), -7.0, device="cuda")
            self.out = (self.a, self.sf)
        else:
            self.a = self.out = torch.full(shape, -7.5, dtype=dtype, device="cuda")

    def rows(self):
        return self.a.reshape(-1, self.shape[-1])

    def scales(self):
        """[rows, cols / 128] numpy."""
        sf = self.sf if self.sf.dim() == 3 else self.sf[None]
        per = self.shape[-2]
        return sf[:, :, :per].transpose(1, 2).reshape(-1, sf.shape[1]).cpu().double().numpy()

    def check(self, at, want, err):
        """Rows `at` hold `want` [n, cols] within `err` (an error before the last rounding) and that rounding; the other
        rows, and the scales' padding, hold the sentinel."""
        at, want, err = np.asarray(at), np.asarray(want, np.float64), np.broadcast_to(np.asarray(err, np.float64), np.shape(want))
        n = self.rows().shape[0]
        rest = np.setdiff1d(np.arange(n), at)
        if not self.fp8:
            got = self.rows().float().cpu().numpy().astype(np.float64)
            near(got[at], want, np.abs(want) * STEP[self.a.dtype] + err * (1 + 2.0 ** -7), "rows")
            assert (got[rest] == -7.5).all(), "rows that nothing owns were written"
            return
        codes = self.rows().view(torch.uint8).cpu()
        assert (codes[torch.from_numpy(rest)] == 0xA5).all(), "rows that nothing owns were written"
        sf = self.scales()
        assert (sf[rest] == -7.0).all(), "scales that nothing owns were written"
        if self.sf.dim() == 2:
            assert (self.sf[:, self.shape[-2]:] == -7.0).all(), "the scales' padding was written"
        got = codes.view(torch.float8_e4m3fn).double().numpy()[at]
        s = sf[at]
        blocks = want.reshape(len(at), self.shape[-1] // 128, 128)
        top = np.where(np.isfinite(blocks), np.abs(blocks), 0).max(2)
        e = np.where(np.isfinite(blocks), err.reshape(blocks.shape), 0).max(2)
        # the scale of the largest value, which may itself be off by its error
        ok = (s == ref.scale_of(top)) | (s == ref.scale_of(top + e)) | (s == ref.scale_of(np.maximum(top - e, 0)))
        assert ok.all(), f"{(~ok).sum()} scales are wrong"
        wide = np.repeat(s, 128, 1)
        near(got * wide, want, np.maximum((np.abs(want) + err) * 2.0 ** -4, wide * 2.0 ** -10) + err, "codes")
        if not err.any():
            q, _ = ref.quantise(want)
            assert ((got == q) | (np.isnan(got) & np.isnan(q))).all(), "codes"


# --------------------------------------------------------------------------------------------------------- sort
def routes(seed, T, k, G, kind):
    rng = np.random.default_rng(seed)
    if kind == "one":
        return np.full((T, k), G - 1)
    if kind == "none":
        return np.full((T, k), -1)
    if kind == "sparse":
        return rng.integers(-G, G, (T, k)).clip(-1)
    p = 1 / np.arange(1, G + 1)
    return rng.choice(G, (T, k), p=rng.permutation(p / p.sum()))


@pytest.mark.parametrize("ids_type", [torch.int32, torch.int64])
@pytest.mark.parametrize("T,k,G,kind", [
    (1, 1, 1, "zipf"), (1, 8, 256, "zipf"), (3, 5, 7, "sparse"), (0, 4, 9, "zipf"), (32, 8, 32, "zipf"), (129, 1, 33, "one"),
    (257, 32, 1024, "zipf"), (1025, 3, 64, "none"), (5000, 8, 255, "zipf"), (4099, 8, 1, "one"), (3001, 7, 1000, "sparse")])
def test_sort(dg, T, k, G, kind, ids_type):
    ids = routes(T + k, T, k, G, kind)
    t = torch.from_numpy(ids).to(ids_type).cuda().contiguous()
    new = lambda *s: torch.full(s, -99, dtype=torch.int32, device="cuda")  # noqa: E731
    for align in (128, 256):
        try:
            dg.set_m_alignment_for_contiguous_layout(align)
            M = dg.get_m_total_bound(T * k, G)
            rows, m, counts = new(T, k), new(M), new(G)
            dg.moe_sort_contiguous(t, rows, m, counts)
            dg.check_device_error()
        finally:
            dg.set_m_alignment_for_contiguous_layout(128)
        want = ref.sort(ids, "contiguous", G, align=align, m_total=M)
        for a, b in zip((rows, counts, m), want):
            assert (a.cpu().numpy() == b).all()
    rows, counts = new(T, k), new(G)
    dg.moe_sort_nopad(t, rows, counts)
    want = ref.sort(ids, "nopad", G)
    assert (rows.cpu().numpy() == want[0]).all() and (counts.cpu().numpy() == want[1]).all()
    m_max = max(1, T * k)
    if G * m_max <= 1 << 30:
        rows, counts = new(T, k), new(G)
        dg.moe_sort_masked(t, rows, counts, m_max)
        want = ref.sort(ids, "masked", G, m_max=m_max)
        assert (rows.cpu().numpy() == want[0]).all() and (counts.cpu().numpy() == want[1]).all()
    dg.check_device_error()


def test_sort_records_what_has_no_room_or_no_group(dg):
    ids = torch.tensor([[0, 1], [0, 7], [0, -2], [1, 2]], dtype=torch.int32, device="cuda")
    new = lambda *s: torch.full(s, -99, dtype=torch.int32, device="cuda")  # noqa: E731

    def status():
        with pytest.raises(dg.DGError) as e:
            dg.check_device_error()
        return e.value.status

    rows, counts = new(4, 2), new(3)
    dg.moe_sort_masked(ids, rows, counts, 2)  # expert 0 has three slots for two rows; 7 and -2 are no groups
    assert status() == -6
    assert rows.tolist() == [[0, 2], [1, -1], [-1, -1], [3, 4]] and counts.tolist() == [2, 2, 1]
    ids = torch.tensor([[0], [1], [2]], device="cuda")
    rows, counts, m = new(3, 1), new(3), new(256)
    dg.moe_sort_contiguous(ids, rows, m, counts)  # room for two groups of three
    assert status() == -6
    assert rows.tolist() == [[0], [128], [-1]] and counts.tolist() == [1, 1, 0]
    assert m.tolist() == [0] + [-1] * 127 + [1] + [-1] * 127
    dg.check_device_error()


# ------------------------------------------------------------------------------------------- dispatch and combine
def row_map(seed, T, k, rows, holes=0.2):
    """A random injective row of each slot, -1 for some."""
    rng = np.random.default_rng(seed)
    flat = rng.permutation(rows)[:T * k] if rows >= T * k else np.concatenate([rng.permutation(rows), np.full(T * k - rows, -1)])
    flat = np.where(rng.random(T * k) < holes, -1, flat)
    rng.shuffle(flat)
    return torch.from_numpy(flat.reshape(T, k).astype(np.int32)).cuda()


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,k,H,shape", [
    (1, 1, 128, (1,)), (3, 8, 256, (40,)), (33, 2, 1152, (3, 25)), (7, 32, 384, (5, 67)), (130, 17, 640, (2300,)), (64, 4, 7168, (8, 37))])
def test_permute(dg, T, k, H, shape, dtype, fp8):
    g = gen(T * H + k)
    x = randn(g, T, H, dtype=dtype) * torch.exp(2 * torch.randn(H, device="cuda", generator=g)).to(dtype)
    rows = row_map(T, T, k, int(np.prod(shape)))
    out = Operand((*shape, H), dtype, fp8)
    dg.moe_permute(x, rows, out.out)
    dg.check_device_error()
    flat = rows.cpu().numpy().reshape(-1)
    slots = np.flatnonzero(flat >= 0)
    out.check(flat[slots], x.cpu().double().numpy()[slots // k], 0.0)


@pytest.mark.parametrize("H", [8, 136, 1000, 2056])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_permute_copies_any_width(dg, H, dtype):
    x, rows = randn(gen(H), 9, H, dtype=dtype), row_map(H, 9, 3, 31)
    out = Operand((31, H), dtype, False)
    dg.moe_permute(x, rows, out.out)
    flat = rows.cpu().numpy().reshape(-1)
    slots = np.flatnonzero(flat >= 0)
    out.check(flat[slots], x.cpu().double().numpy()[slots // 3], 0.0)


def special_blocks(dtype):
    """Blocks of 128 where quantising can go wrong: zeros, borders of a scale, tiny values, infinities, NaN."""
    inf, nan = float("inf"), float("nan")
    x = torch.zeros(12, 128, dtype=torch.float64)
    x[1, 5] = 448.0
    x[2, 5] = torch.nextafter(torch.tensor(448.0, dtype=dtype), torch.tensor(1e4, dtype=dtype)).double()
    x[3] = torch.linspace(-448, 448, 128)
    x[4, 3], x[4, 4] = inf, 100.0
    x[5, 3], x[5, 4], x[5, 100] = nan, -inf, 0.5
    x[6, :] = nan
    x[7, :] = -inf
    x[8, 0], x[8, 1] = 2.0 ** -126, 2.0 ** -130  # the smallest scale, then values below its steps
    x[9, 0] = torch.finfo(dtype).max
    x[10] = torch.linspace(1.0, 2.0, 128) * 2.0 ** 20
    x[11, 127] = -(2.0 ** -100)
    return x.to(dtype).reshape(4, 384)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_permute_special_values(dg, dtype):
    x = special_blocks(dtype).cuda()
    rows = torch.tensor([[3], [0], [5], [1]], dtype=torch.int32, device="cuda")
    out = Operand((6, 384), dtype, True)
    dg.moe_permute(x, rows, out.out)
    dg.check_device_error()
    q, s = ref.quantise(x.cpu().double().numpy())
    got, sf = out.rows().cpu().double().numpy()[[3, 0, 5, 1]], out.scales()[[3, 0, 5, 1]]
    assert (sf == s).all()
    assert ((got == q) | (np.isnan(got) & np.isnan(q))).all()


def test_permute_skips_and_records_rows_out_of_range(dg):
    x = randn(gen(1), 3, 128, dtype=BF16)
    out = Operand((4, 128), BF16, False)
    dg.moe_permute(x, torch.tensor([[0], [4], [-5]], dtype=torch.int32, device="cuda"), out.out)
    with pytest.raises(dg.DGError) as e:
        dg.check_device_error()
    assert e.value.status == -6
    out.check([0], x.cpu().double().numpy()[:1], 0.0)


@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,k,H,shape", [
    (1, 1, 8, (1,)), (5, 8, 264, (50,)), (33, 3, 1000, (4, 30)), (17, 32, 2048, (600,)), (4, 9, 7168, (8, 5))])
def test_unpermute(dg, T, k, H, shape, dtype, weighted):
    g = gen(T + H)
    rows = randn(g, *shape, H, dtype=dtype)
    flat_rows = rows.view(-1, H)
    row = row_map(T, T, k, flat_rows.shape[0], 0.3)
    row[T // 2] = -1  # a token without any row
    used = torch.zeros(flat_rows.shape[0], dtype=torch.bool)
    used[row.cpu()[row.cpu() >= 0].long()] = True
    flat_rows[~used.cuda()] = float("nan")  # rows that no slot names are not read
    w = randn(g, T, k) if weighted else None
    out = torch.full((T, H), -7.5, dtype=dtype, device="cuda")
    dg.moe_unpermute(rows, row, out, w)
    dg.check_device_error()
    want = ref.combine(rows, row, w)
    size = ref.combine(rows.abs(), row, None if w is None else w.abs())
    near(out.float(), want, want.abs() * STEP[dtype] + size * (k + 1) * 2.0 ** -24 * 1.01)


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,k,H,shape", [(1, 1, 128, (1,)), (9, 8, 384, (90,)), (20, 3, 2176, (4, 20)), (5, 32, 4096, (200,)),
                                         (3, 10, 16512, (40,))])
def test_unpermute_backward(dg, T, k, H, shape, dtype, fp8):
    g = gen(T + H)
    rows, d = randn(g, *shape, H, dtype=dtype), randn(g, T, H, dtype=dtype, scale=3.0)
    row = row_map(T, T, k, int(np.prod(shape)), 0.3)
    w = randn(g, T, k)
    w[0, 0] = 0.0
    d_rows, d_w = Operand((*shape, H), dtype, fp8), torch.full((T, k), -7.5, device="cuda")
    dg.moe_unpermute_backward(d, rows, row, w, d_rows.out, d_w)
    dg.check_device_error()
    flat = row.cpu().numpy().reshape(-1)
    slots = np.flatnonzero(flat >= 0)
    value = ref.f64(w).numpy().reshape(-1)[slots, None] * ref.f64(d).numpy()[slots // k]
    d_rows.check(flat[slots], value, np.abs(value) * 2.0 ** -24 if fp8 else 0.0 + np.abs(value) * 2.0 ** -24)
    r, dd = ref.f64(rows).reshape(-1, H).numpy(), ref.f64(d).numpy()
    want, size = np.zeros(T * k), np.zeros(T * k)
    for i in slots:
        want[i], size[i] = (r[flat[i]] * dd[i // k]).sum(), np.abs(r[flat[i]] * dd[i // k]).sum()
    # a lane's chain: 8 products a vector, ceil(H / 256 / warps) <= 9 vectors, then 5 steps and at most 16 warps
    near(d_w.reshape(-1), want, size * 96 * 2.0 ** -24 + want * 0)


@pytest.mark.parametrize("T,k,H,shape,dtype,fp8", [(1201, 1, 128, (1500,), F32, True), (1190, 3, 2176, (4, 1000), BF16, True),
                                                   (1300, 8, 384, (11000,), BF16, False), (1185, 11, 640, (14000,), F32, False),
                                                   (1187, 2, 1152, (2400,), BF16, True)])
def test_unpermute_backward_of_many_tokens(dg, T, k, H, shape, dtype, fp8):
    """From 8 tokens an SM on a warp takes a token: the sums' chains are as long as those above."""
    test_unpermute_backward(dg, T, k, H, shape, dtype, fp8)


def test_unpermute_gradient_against_differences(dg):
    """<d_out, out(w + h e) - out(w - h e)> / 2h and the same for the rows: the combine is linear in each, so the
    difference is the gradient but for the fp32 roundings of the two outputs."""
    g, T, k, H, R = gen(7), 6, 4, 256, 30
    rows, d, w, row = randn(g, R, H), randn(g, T, H), randn(g, T, k), row_map(7, T, k, R, 0.2)
    d_rows, d_w = torch.zeros(R, H, device="cuda"), torch.empty(T, k, device="cuda")
    dg.moe_unpermute_backward(d, rows, row, w, d_rows, d_w)
    out = lambda r, v: (lambda o: (dg.moe_unpermute(r, row, o, v), o.double())[1])(torch.empty(T, H, device="cuda"))  # noqa: E731
    for trial in range(3):
        dw, dr = randn(g, T, k), randn(g, R, H)
        got = ((out(rows, w + dw) - out(rows, w - dw)) * d.double()).sum() / 2
        want = (d_w.double() * dw.double()).sum()
        # 2 outputs of T*H elements, each within 6 roundings of its terms (|row| |w| ~ 4): a generous 2^-20 of the sums
        size = (d.double().abs().sum() * 12)
        assert abs(got - want) <= size * 2.0 ** -20, (got, want)
        got = ((out(rows + dr, w) - out(rows - dr, w)) * d.double()).sum() / 2
        assert abs(got - (d_rows.double() * dr.double()).sum()) <= size * 2.0 ** -20


# -------------------------------------------------------------------------------------------------------- SwiGLU
def owned_rows(kind, shape, seed):
    """(keyword argument of the call, owned rows) for gate_up of `shape[:-1]` rows."""
    rng = np.random.default_rng(seed)
    R = int(np.prod(shape))
    cuda = lambda v: torch.from_numpy(np.asarray(v, np.int32)).cuda()  # noqa: E731
    if kind == "masked":
        G, M = shape
        m = rng.integers(0, M + 1, G)
        m[0], m[-1] = 0, M
        return {"masked_m": cuda(m)}, np.concatenate([g * M + np.arange(n) for g, n in enumerate(m)])
    if kind == "m_indices":
        m = np.where(rng.random(R) < 0.6, rng.integers(0, 5, R), -1)
        return {"m_indices": cuda(m)}, np.flatnonzero(m >= 0)
    if kind == "counts":
        c = rng.multinomial(R * 2 // 3, np.full(700, 1 / 700)) if R > 1 else [0]
        return {"counts": cuda(c)}, np.arange(np.sum(c))
    return {}, np.arange(R)


SWIGLU_SHAPES = [((1,), 128, "all"), ((37,), 384, "all"), ((67,), 256, "m_indices"), ((130,), 640, "counts"),
                 ((5, 33), 2048, "masked"), ((3, 7), 128, "masked"), ((256,), 4096, "m_indices"), ((1,), 8192, "counts")]


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("shape,I,kind", SWIGLU_SHAPES)
def test_swiglu(dg, shape, I, kind, dtype, fp8):
    g = gen(I + len(shape))
    gu = randn(g, *shape, 2 * I, dtype=dtype, scale=4.0)
    kw, at = owned_rows(kind, shape, I)
    flat = gu.view(-1, 2 * I)
    rest = np.setdiff1d(np.arange(flat.shape[0]), at)
    flat[torch.from_numpy(rest).cuda()] = float("nan")
    out = Operand((*shape, I), dtype, fp8)
    dg.swiglu(gu, out.out, **kw)
    dg.check_device_error()
    want = ref.swiglu(flat.cpu()[at]).numpy().reshape(len(at), I)
    # bf16 and e4m3 results: sigmoid by the fast exponential, (2 + 1.2 |g|) 2^-23 and a reciprocal of 2^-23, |g| < 30: under
    # 40 * 2^-23 < 2^-17; fp32: a few 2^-24
    out.check(at, want, np.abs(want) * (2.0 ** -17 if dtype == BF16 or fp8 else 2.0 ** -20))


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("shape,I,kind", SWIGLU_SHAPES)
def test_swiglu_backward(dg, shape, I, kind, dtype, fp8):
    g = gen(I + len(shape) + 1)
    gu, d = randn(g, *shape, 2 * I, dtype=dtype, scale=4.0), randn(g, *shape, I, dtype=dtype)
    kw, at = owned_rows(kind, shape, I)
    out = Operand((*shape, 2 * I), dtype, fp8)
    dg.swiglu_backward(d, gu, out.out, **kw)
    dg.check_device_error()
    gu64, d64 = gu.cpu().view(-1, 2 * I)[at], d.cpu().view(-1, I)[at]
    want = ref.swiglu_backward(d64, gu64).numpy().reshape(len(at), 2 * I)
    a, b = (v.numpy().reshape(len(at), I) for v in ref.f64(gu64).chunk(2, -1))
    s = 1 / (1 + np.exp(-a))
    # 1 + g (1 - s) cancels near g = -1.28: the error is of the terms' size, not of their sum's
    size = np.concatenate([np.abs(d64.double().numpy() * b * s) * (1 + np.abs(a)), np.abs(d64.double().numpy() * a * s)], 1)
    # (sigmoid as above, twice in the gradient of g)
    out.check(at, want, size * (2.0 ** -16 if dtype == BF16 or fp8 else 2.0 ** -20))


def test_swiglu_gradient_against_differences(dg):
    g, R, I, h = gen(3), 9, 128, 2.0 ** -7
    gu, d, e = randn(g, R, 2 * I), randn(g, R, I), randn(g, R, 2 * I)
    grad = torch.empty_like(gu)
    dg.swiglu_backward(d, gu, grad)

    def f(v):
        out = torch.empty(R, I, device="cuda")
        dg.swiglu(v, out)
        return (out.double() * d.double()).sum()

    got, want = (f(gu + h * e) - f(gu - h * e)) / (2 * h), (grad.double() * e.double()).sum()
    # h^2 / 6 times third derivatives (a few units an element along e) and 2^-22 roundings over 2h
    size = (d.double().abs().repeat(1, 2) * (1 + e.double().abs() ** 3) * (1 + gu.double().abs())).sum()
    assert abs(got - want) <= size * (h * h + 2.0 ** -22 / h), (got, want)


def test_swiglu_extreme_gates(dg):
    inf, nan = float("inf"), float("nan")
    g = torch.tensor([0.0, -0.0, 90.0, -90.0, 1e4, -1e4, 3e38, -3e38, inf, nan] + [1.0] * 118, device="cuda")
    for dtype in (BF16, F32):
        gu = torch.cat([g, torch.full((128,), 2.0, device="cuda")])[None].to(dtype)
        out = torch.empty(1, 128, dtype=dtype, device="cuda")
        dg.swiglu(gu, out)
        got = out[0, :10].double().cpu().numpy()
        v = gu[0, :10].double().cpu().numpy()
        with np.errstate(over="ignore", invalid="ignore"):
            want = v / (1 + np.exp(-v)) * 2
        top = torch.finfo(dtype).max
        want = np.where(np.abs(want) > top, np.inf, want)
        assert np.isnan(got[9]) and got[8] == np.inf
        near(got[:8], want[:8], np.abs(want[:8]) * 2.0 ** -7 + 1e-36)  # (results below the normal numbers may be 0)


def test_swiglu_masked_counts_out_of_range(dg):
    """Negative counts are none, counts past the rows are all: nothing outside is touched."""
    gu = randn(gen(5), 3, 10, 256, dtype=BF16)
    out = Operand((3, 10, 128), BF16, False)
    dg.swiglu(gu, out.out, masked_m=torch.tensor([-5, 1 << 30, 3], dtype=torch.int32, device="cuda"))
    at = np.concatenate([10 + np.arange(10), 20 + np.arange(3)])
    want = ref.swiglu(gu.cpu().view(30, 256)[at]).numpy()
    out.check(at, want, np.abs(want) * 2.0 ** -17)
    out = Operand((30, 128), BF16, False)
    dg.swiglu(gu.view(30, 256), out.out, counts=torch.tensor([-7, 4, 0, -1, 3], dtype=torch.int32, device="cuda"))
    want = ref.swiglu(gu.cpu().view(30, 256)[:7]).numpy()
    out.check(np.arange(7), want, np.abs(want) * 2.0 ** -17)
    out = Operand((30, 128), BF16, False)
    dg.swiglu(gu.view(30, 256), out.out, counts=torch.tensor([2 ** 31 - 1, 2 ** 31 - 1, 5], dtype=torch.int32, device="cuda"))
    want = ref.swiglu(gu.cpu().view(30, 256)).numpy()
    out.check(np.arange(30), want, np.abs(want) * 2.0 ** -17)
    out = Operand((30, 128), BF16, False)  # the sum of 1024 counts far past 32 bits
    dg.swiglu(gu.view(30, 256), out.out, counts=torch.full((1024,), 2 ** 31 - 1, dtype=torch.int32, device="cuda"))
    out.check(np.arange(30), want, np.abs(want) * 2.0 ** -17)


# --------------------------------------------------------------------------------------------------------- norms
NORMS = [(1, 8), (3, 128), (5, 1000), (37, 2048), (300, 512), (4, 4104), (7, 7168), (2, 8192), (2, 8200), (3, 16384), (1000, 256), (700, 1280)]
TYPES = [(BF16, BF16), (F32, BF16), (F32, F32)]


def norm_inputs(T, H, X, Y, P, gate, seed):
    g = gen(seed)
    t = dict(x=randn(g, T, H, dtype=X, scale=2.0), y=randn(g, T, H, dtype=Y), w=1 + 0.3 * randn(g, H), w_post=1 + 0.3 * randn(g, H))
    t["w"], t["w_post"] = t["w"].to(P), t["w_post"].to(P)
    t["gate"] = {"none": None, "row": randn(g, H).to(P), "token": randn(g, T, H, dtype=Y)}[gate]
    if T > 2:
        t["x"][1] = 0
        t["y"][1] = 0  # a row of zeros: r = 1 / sqrt(eps)
        if T > 3:
            t["x"][2] *= 100
    return t, g


@pytest.mark.parametrize("X,Y", TYPES)
@pytest.mark.parametrize("T,H", NORMS)
def test_rms_norm(dg, T, H, X, Y):
    for P, fp8 in ((BF16, False), (F32, H % 128 == 0)):
        t, _ = norm_inputs(T, H, X, Y, P, "none", T + H)
        out, rstd = Operand((T, H), Y, fp8), torch.full((T,), -1.0, device="cuda")
        dg.rms_norm(t["x"], t["w"], out.out, eps=1e-5, rstd=rstd)
        dg.check_device_error()
        _, want, r, _ = ref.norm(t["x"], w=t["w"], eps=1e-5)
        near(rstd, r, r * CHAIN)
        out.check(np.arange(T), want, want.abs() * 2 * CHAIN)


@pytest.mark.parametrize("X,Y", TYPES)
@pytest.mark.parametrize("gate", ["none", "row", "token"])
@pytest.mark.parametrize("T,H", NORMS)
def test_residual_rms_norm(dg, T, H, gate, X, Y):
    for post, pre, P, fp8 in ((True, True, F32, H % 128 == 0), (True, True, BF16, False), (False, True, F32, False),
                              (True, False, BF16, False), (False, False, F32, False)):
        t, _ = norm_inputs(T, H, X, Y, P, gate, T + H)
        out = Operand((T, H), Y, fp8)
        x_out, rstd, rp = torch.full_like(t["x"], -7.5), torch.full((T,), -1.0, device="cuda"), torch.full((T,), -1.0, device="cuda")
        w, wp = t["w"] if pre else None, t["w_post"] if post else None
        dg.residual_rms_norm(t["x"], t["y"], x_out, weight=w, out=out.out if pre else None, weight_post=wp, gate=t["gate"],
                             alpha=0.7, eps=1e-5, rstd=rstd if pre else None, rstd_post=rp if post else None)
        dg.check_device_error()
        total, want, r, r_post = ref.norm(t["x"], t["y"], w, wp, t["gate"], 0.7, 1e-5)
        size = ref.f64(t["x"]).abs() + (total - ref.f64(t["x"])).abs()
        near(x_out.float(), total, total.abs() * STEP[X] + size * 2 * CHAIN, "x_out")
        if post:
            near(rp, r_post, r_post * CHAIN)
        if pre:
            near(rstd, r, r * 4 * CHAIN)
            out.check(np.arange(T), want, size * r[:, None] * ref.f64(w).abs() * 6 * CHAIN)
        # the same call in place (a call without `out` may sum in another order, so it is not the one to compare with)
        in_place, again = t["x"].clone(), Operand((T, H), Y, fp8)
        dg.residual_rms_norm(in_place, t["y"], in_place, weight=w, out=again.out if pre else None, weight_post=wp,
                             gate=t["gate"], alpha=0.7, eps=1e-5)
        assert torch.equal(in_place, x_out) and torch.equal(again.a.view(torch.uint8), out.a.view(torch.uint8))


@pytest.mark.parametrize("X,Y", TYPES)
@pytest.mark.parametrize("gate", ["none", "row", "token"])
@pytest.mark.parametrize("T,H", NORMS)
def test_residual_rms_norm_backward(dg, T, H, gate, X, Y):
    for post, pre, skip, P in ((True, True, True, F32), (True, True, False, BF16), (False, True, True, BF16),
                               (True, False, True, F32), (False, False, True, F32)):
        t, g = norm_inputs(T, H, X, Y, P, gate, T + H + 1)
        w, wp = t["w"] if pre else None, t["w_post"] if post else None
        _, _, r, rp = ref.norm(t["x"], w=t["w"], eps=1e-5)[0:2] + (1 / torch.sqrt((ref.f64(t["x"]) ** 2).mean(1) + 1e-5),
                                                                 1 / torch.sqrt((ref.f64(t["y"]) ** 2).mean(1) + 1e-5))
        r, rp = r.float().cuda(), rp.float().cuda()
        dxo = randn(g, T, H, dtype=X) if skip else None
        do = randn(g, T, H, dtype=Y) if pre else None
        new = lambda *s, dtype=F32: torch.full(s, -7.5, dtype=dtype, device="cuda")  # noqa: E731
        d_x, d_y, d_w, d_wp = new(T, H, dtype=X), new(T, H, dtype=Y), new(H) if pre else None, new(H) if post else None
        d_gate = {"none": None, "row": new(H), "token": new(T, H, dtype=Y)}[gate]
        dg.residual_rms_norm_backward(dxo, t["y"], d_x, d_y, d_out=do, x_out=t["x"] if pre else None, weight=w,
                                      rstd=r if pre else None, weight_post=wp, rstd_post=rp if post else None, gate=t["gate"],
                                      alpha=0.7, d_weight=d_w, d_weight_post=d_wp, d_gate=d_gate)
        dg.check_device_error()
        want = ref.norm_backward(dxo, do, t["x"] if pre else None, t["y"], w, wp, t["gate"], 0.7, r, rp)
        # sizes of the terms: the errors are of theirs, not of the sums'
        x, y, r64, rp64 = ref.f64(t["x"]), ref.f64(t["y"]), ref.f64(r)[:, None], ref.f64(rp)[:, None]
        sx = torch.zeros(T, H, dtype=torch.float64) if dxo is None else ref.f64(dxo).abs()
        if pre:
            e = (ref.f64(w) * ref.f64(do)).abs()
            sx = sx + r64 * (e + x.abs() * r64 ** 2 * (e * x.abs()).mean(1, keepdim=True))
        near(d_x.float(), want["d_x"], want["d_x"].abs() * STEP[X] + sx * 4 * CHAIN, "d_x")
        gate64 = torch.ones(1, dtype=torch.float64) if t["gate"] is None else ref.f64(t["gate"]).abs()
        sn = 0.7 * gate64 * sx
        if post:
            e = ref.f64(wp).abs() * sn
            sy = rp64 * (e + y.abs() * rp64 ** 2 * (e * y.abs()).mean(1, keepdim=True))
            near(d_wp, want["d_w_post"], (sn * y.abs() * rp64).sum(0) * 8 * CHAIN, "d_weight_post")
        else:
            sy = sn
        near(d_y.float(), want["d_y"], want["d_y"].abs() * STEP[Y] + sy * 8 * CHAIN, "d_y")
        if pre:
            near(d_w, want["d_w"], (ref.f64(do).abs() * x.abs() * r64).sum(0) * 4 * CHAIN, "d_weight")
        if gate != "none":
            n = y.abs() * (rp64 * ref.f64(wp).abs() if post else 1.0)
            if gate == "row":
                near(d_gate, want["d_gate"], (0.7 * n * sx).sum(0) * 8 * CHAIN, "d_gate")
            else:
                near(d_gate.float(), want["d_gate"], want["d_gate"].abs() * STEP[Y] + n * sx * 8 * CHAIN, "d_gate")


@pytest.mark.parametrize("X,Y", TYPES)
@pytest.mark.parametrize("T,H", NORMS)
def test_rms_norm_backward(dg, T, H, X, Y):
    t, g = norm_inputs(T, H, X, Y, F32, "none", T + H + 2)
    r = (1 / torch.sqrt((ref.f64(t["x"]) ** 2).mean(1) + 1e-5)).float().cuda()
    do, skip = randn(g, T, H, dtype=Y), randn(g, T, H, dtype=X)
    for d_skip in (None, skip):
        d_x, d_w = torch.full((T, H), -7.5, dtype=X, device="cuda"), torch.full((H,), -7.5, device="cuda")
        dg.rms_norm_backward(do, t["x"], t["w"], r, d_x, d_w, d_skip=d_skip)
        dg.check_device_error()
        want = ref.norm_backward(d_skip, do, t["x"], None, t["w"], None, None, 1.0, r, None)
        x, r64, e = ref.f64(t["x"]).abs(), ref.f64(r)[:, None], (ref.f64(t["w"]) * ref.f64(do)).abs()
        size = r64 * (e + x * r64 ** 2 * (e * x).mean(1, keepdim=True)) + (0 if d_skip is None else ref.f64(skip).abs())
        near(d_x.float(), want["d_x"], want["d_x"].abs() * STEP[X] + size * 4 * CHAIN)
        near(d_w, want["d_w"], (ref.f64(do).abs() * x * r64).sum(0) * 4 * CHAIN)
    in_place = skip.clone()  # the gradient that comes in past the norm may be the buffer that goes out
    dg.rms_norm_backward(do, t["x"], t["w"], r, in_place, d_w, d_skip=in_place)
    assert torch.equal(in_place, d_x)


# more rows than the SMs take at once: a row a warp, 16 or 32 elements a thread; a gradient's CTAs take several rows each, more
# than are copied ahead, and their sums for a parameter are chains of at most 11 + 19 + 3 + 32 additions
@pytest.mark.parametrize("X,Y", TYPES)
@pytest.mark.parametrize("T,H", [(50000, 8), (4800, 256), (2500, 512), (1500, 1288), (1600, 4104)])
def test_norms_of_many_rows(dg, T, H, X, Y):
    test_rms_norm(dg, T, H, X, Y)
    test_rms_norm_backward(dg, T, H, X, Y)


@pytest.mark.parametrize("X,Y,gate,T,H", [(BF16, BF16, "token", 1600, 4104), (F32, BF16, "row", 2500, 512), (F32, F32, "none", 4800, 256),
                                          (BF16, BF16, "row", 50000, 8), (F32, F32, "token", 1500, 1288)])
def test_residual_norms_of_many_rows(dg, X, Y, gate, T, H):
    test_residual_rms_norm(dg, T, H, gate, X, Y)
    test_residual_rms_norm_backward(dg, T, H, gate, X, Y)


def test_norm_gradient_against_differences(dg):
    g, T, H, h = gen(11), 6, 256, 2.0 ** -7
    x, y, w, wp, gate = randn(g, T, H), randn(g, T, H), randn(g, H), randn(g, H), randn(g, H)
    dxo, do = randn(g, T, H), randn(g, T, H)

    def f(x, y, w, wp, gate, keep=None):
        xo, out, r, rp = torch.empty_like(x), torch.empty_like(x), torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
        dg.residual_rms_norm(x, y, xo, weight=w, out=out, weight_post=wp, gate=gate, alpha=0.7, rstd=r, rstd_post=rp)
        if keep is not None:
            keep.update(x_out=xo, rstd=r, rstd_post=rp)
        return (xo.double() * dxo.double()).sum() + (out.double() * do.double()).sum()

    keep = {}
    f(x, y, w, wp, gate, keep)
    d = [torch.empty_like(v) for v in (x, y, w, wp, gate)]
    dg.residual_rms_norm_backward(dxo, y, d[0], d[1], d_out=do, weight=w, weight_post=wp, gate=gate, alpha=0.7, d_weight=d[2],
                                  d_weight_post=d[3], d_gate=d[4], **keep)
    args = [x, y, w, wp, gate]
    for i in range(5):
        e = randn(g, *args[i].shape)
        up, down = list(args), list(args)
        up[i], down[i] = args[i] + h * e, args[i] - h * e
        got, want = (f(*up) - f(*down)) / (2 * h), (d[i].double() * e.double()).sum()
        # T*H terms of order 10, a third derivative of the same order along e, and fp32 roundings over 2h
        assert abs(got - want) <= T * H * 10 * (h * h + 2.0 ** -22 / h), (i, got, want)


def test_empty_calls_write_the_sums_of_nothing(dg):
    d_w = torch.full((256,), 3.0, device="cuda")
    e = torch.empty(0, 256, device="cuda")
    dg.rms_norm_backward(e, e, torch.ones(256, device="cuda"), torch.empty(0, device="cuda"), e, d_w)
    assert (d_w == 0).all()
    dg.rms_norm(e, torch.ones(256, device="cuda"), e)
    rows = torch.empty(0, 3, dtype=torch.int32, device="cuda")
    dg.moe_permute(e, rows, torch.empty(4, 256, device="cuda"))
    dg.moe_unpermute(torch.empty(4, 256, device="cuda"), rows, e)
    dg.moe_permute(torch.ones(2, 256, device="cuda"), torch.full((2, 1), -1, dtype=torch.int32, device="cuda"), e)
    out = torch.full((2, 256), 5.0, device="cuda")
    dg.moe_unpermute(e, torch.full((2, 1), -1, dtype=torch.int32, device="cuda"), out)  # no rows at all: zeros
    assert (out == 0).all()
    d_wt = torch.full((2, 1), 5.0, device="cuda")
    dg.moe_unpermute_backward(out, e, torch.full((2, 1), -1, dtype=torch.int32, device="cuda"), torch.ones(2, 1, device="cuda"), e, d_wt)
    assert (d_wt == 0).all()
    dg.swiglu(torch.empty(0, 512, device="cuda"), e)
    dg.check_device_error()


# ---------------------------------------------------------------------------------------- offsets, streams, devices
def test_offsets_past_32_bits(dg):
    """Operands of more than 2^31 elements: the last rows are reached, and only they."""
    H, R = 8192, 270000  # 2.2e9 codes
    x = randn(gen(1), 4, H, dtype=BF16)
    rows = torch.tensor([[R - 1, 0], [R - 2, -1], [262145, 1], [-1, R - 3]], dtype=torch.int32, device="cuda")
    a, sf = torch.zeros(R, H, dtype=torch.uint8, device="cuda"), torch.zeros(H // 128, R, device="cuda")
    dg.moe_permute(x, rows, (a, sf))
    q, s = ref.quantise(x.cpu().double().numpy())
    for t in range(4):
        for r in rows[t].tolist():
            if r >= 0:
                assert (a[r].view(torch.float8_e4m3fn).cpu().double().numpy() == q[t]).all()
                assert (sf[:, r].cpu().double().numpy() == s[t]).all()
    assert int((sf != 0).sum()) == 6 * H // 128
    del a, sf
    big = torch.zeros(R, H, dtype=BF16, device="cuda")
    dg.moe_permute(x, rows, big)
    assert torch.equal(big[R - 1], x[0]) and torch.equal(big[262145], x[2]) and torch.equal(big[R - 3], x[3])
    out = torch.empty_like(x)
    dg.moe_unpermute(big, rows, out)
    assert torch.equal(out, (x.float() * torch.tensor([2, 1, 2, 1], device="cuda")[:, None]).to(BF16))
    h = torch.zeros(R, H // 2, dtype=BF16, device="cuda")
    own = torch.full((R,), -1, dtype=torch.int32, device="cuda")
    own[R - 1] = 0
    dg.swiglu(big, h, m_indices=own)
    want = ref.swiglu(x[:1])
    near(h[R - 1:].float(), want, want.abs() * 2.0 ** -8 * 1.01)
    assert int((h[: R - 1] != 0).sum()) == 0
    dg.check_device_error()


def _calls(dg, seed=0):
    """Every operator on small inputs: (inputs to fill, outputs, the call)."""
    g = gen(seed)
    T, k, H, G, M, I = 40, 4, 512, 6, 1024, 256
    ids = torch.randint(-1, G, (T, k), device="cuda", generator=g, dtype=torch.int32)
    x, rows, d = randn(g, T, H, dtype=BF16), randn(g, M, H, dtype=BF16), randn(g, T, H, dtype=BF16)
    w, gu, dh = randn(g, T, k), randn(g, M, 2 * I, dtype=BF16), randn(g, M, I, dtype=BF16)
    pw = randn(g, H)
    z = lambda *s, dtype=F32: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
    i32 = torch.int32
    o = dict(row=z(T, k, dtype=i32), m=z(M, dtype=i32), counts=z(G, dtype=i32), a=z(M, H, dtype=torch.uint8), sf=z(H // 128, M),
             out=z(T, H, dtype=BF16), dr=z(M, H, dtype=BF16), dw=z(T, k), h=z(M, I, dtype=torch.uint8), hs=z(I // 128, M),
             dgu=z(M, 2 * I, dtype=BF16), xo=z(T, H, dtype=BF16), n=z(T, H, dtype=BF16), r=z(T), rp=z(T), dx=z(T, H, dtype=BF16),
             dy=z(T, H, dtype=BF16), gw=z(H), gp=z(H), gg=z(H))

    def run():
        dg.moe_sort_contiguous(ids, o["row"], o["m"], o["counts"])
        dg.moe_permute(x, o["row"], (o["a"], o["sf"]))
        dg.moe_unpermute(rows, o["row"], o["out"], w)
        dg.moe_unpermute_backward(d, rows, o["row"], w, o["dr"], o["dw"])
        dg.swiglu(gu, (o["h"], o["hs"]), m_indices=o["m"])
        dg.swiglu_backward(dh, gu, o["dgu"], m_indices=o["m"])
        dg.residual_rms_norm(x, o["out"], o["xo"], weight=pw, out=o["n"], weight_post=pw, gate=pw, alpha=0.5, rstd=o["r"],
                             rstd_post=o["rp"])
        dg.residual_rms_norm_backward(d, o["out"], o["dx"], o["dy"], d_out=o["n"], x_out=o["xo"], weight=pw, rstd=o["r"],
                                      weight_post=pw, rstd_post=o["rp"], gate=pw, alpha=0.5, d_weight=o["gw"],
                                      d_weight_post=o["gp"], d_gate=o["gg"])

    return dict(ids=ids, x=x, rows=rows, d=d, w=w, gu=gu, dh=dh, pw=pw), o, run


def _bits(o):
    return {k: v.clone() for k, v in o.items()}


def test_calls_repeat_bit_for_bit_and_run_on_the_current_stream(dg):
    _, o, run = _calls(dg)
    run()
    torch.cuda.synchronize()
    first = _bits(o)
    for v in o.values():
        v.zero_()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        torch.cuda._sleep(2_000_000)  # what follows on the stream has to wait for it
        run()
        late = _bits(o)
    s.synchronize()
    assert all(torch.equal(first[k], late[k]) for k in o)
    dg.check_device_error()


def test_two_captured_graphs_replay_in_turn(dg):
    """Two graphs of the same calls, each with its own inputs and outputs: replays in turn, and on two streams at once,
    give what eager calls give on the inputs' current contents."""
    sets = [_calls(dg, seed) for seed in (1, 2)]
    graphs = []
    for _, _, run in sets:
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(s):
            run()
            torch.cuda.synchronize()
            with torch.cuda.graph(graph, stream=s):
                run()
        torch.cuda.current_stream().wait_stream(s)
        graphs.append(graph)
    for trial in range(3):
        want = []
        for inputs, o, run in sets:
            inputs["x"].copy_(torch.roll(inputs["x"], 1, 0))
            inputs["ids"].copy_(torch.roll(inputs["ids"], 1, 0))
            for v in o.values():
                v.zero_()
            run()
            want.append(_bits(o))
            for v in o.values():
                v.zero_()
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in graphs]
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for (_, o, _), w in zip(sets, want):
            assert all(torch.equal(o[k], w[k]) for k in o), trial
    dg.check_device_error()


@pytest.mark.parametrize("T", [40, 200, 900])  # one CTA, clusters of 8 and of 16
def test_captured_sort_replays(dg, T):
    """Every launch shape of the sort in a graph, replayed on other ids."""
    g, G, k = gen(T), 300, 4
    ids = torch.randint(-1, G, (T, k), device="cuda", generator=g)
    M = dg.get_m_total_bound(T * k, G)
    new = lambda *s: torch.full(s, -99, dtype=torch.int32, device="cuda")  # noqa: E731
    rows, m, counts = new(T, k), new(M), new(G)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        dg.moe_sort_contiguous(ids, rows, m, counts)
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=s):
            dg.moe_sort_contiguous(ids, rows, m, counts)
    torch.cuda.current_stream().wait_stream(s)
    for trial in range(2):
        ids.copy_(torch.randint(-1, G, (T, k), device="cuda", generator=g))
        graph.replay()
        torch.cuda.synchronize()
        want = ref.sort(ids.cpu().numpy(), "contiguous", G, m_total=M)
        for a, b in zip((rows, counts, m), want):
            assert (a.cpu().numpy() == b).all()
    dg.check_device_error()


def test_calls_from_two_threads(dg):
    """Two host threads, each on its own stream with its own tensors, at once: each gets what it gets alone."""
    import threading

    sets = [_calls(dg, seed) for seed in (3, 4)]
    want = []
    for _, o, run in sets:
        run()
        torch.cuda.synchronize()
        want.append(_bits(o))
        for v in o.values():
            v.zero_()
    torch.cuda.synchronize()
    errors = []

    def work(run):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    run()
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(run,)) for _, _, run in sets]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    for (_, o, _), w in zip(sets, want):
        assert all(torch.equal(o[k], w[k]) for k in o)
    dg.check_device_error()


def test_python_refusals(dg):
    x = randn(gen(1), 4, 256, dtype=BF16)
    rows = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    out = torch.zeros(8, 256, dtype=BF16, device="cuda")
    w = torch.ones(256, device="cuda")
    f8, sf = torch.zeros(8, 256, dtype=torch.uint8, device="cuda"), torch.zeros(2, 8, device="cuda")
    bad = [
        lambda: dg.moe_permute(x.half(), rows, out), lambda: dg.moe_permute(x.t(), rows, out), lambda: dg.moe_permute(x[:, ::2], rows, out),
        lambda: dg.moe_permute(x.cpu(), rows, out), lambda: dg.moe_permute(x, rows.long(), out), lambda: dg.moe_permute(x, rows[:3], out),
        lambda: dg.moe_permute(x, rows, out.float()), lambda: dg.moe_permute(x, rows, (f8, sf[:1])),
        lambda: dg.moe_permute(x, rows, (f8, sf, sf)), lambda: dg.moe_permute(x, rows, (f8, sf.double())),
        lambda: dg.moe_permute(x[:, :100].contiguous(), rows, out[:, :100].contiguous()),
        lambda: dg.moe_unpermute(out, rows, x[:3]), lambda: dg.moe_unpermute(out, rows, x, torch.zeros(4, 3, device="cuda")),
        lambda: dg.moe_unpermute_backward(x, out, rows, torch.zeros(4, 2, device="cuda"), x, torch.zeros(4, 2, device="cuda")),
        lambda: dg.moe_sort_nopad(rows.float(), rows, rows[0]), lambda: dg.moe_sort_nopad(rows, rows, rows[0].contiguous()),
        lambda: dg.swiglu(x, out), lambda: dg.swiglu(x, x[:, :128]), lambda: dg.swiglu(out, f8[:, :128]),
        lambda: dg.swiglu(out, out[:, :128].contiguous(), masked_m=torch.zeros(2, dtype=torch.int32, device="cuda")),
        lambda: dg.swiglu(out.view(2, 4, 256), torch.zeros(2, 4, 128, dtype=BF16, device="cuda")),
        lambda: dg.rms_norm(x, w[:128], x.clone()), lambda: dg.rms_norm(x, w, x.float()), lambda: dg.rms_norm(x, w.half(), x.clone()),
        lambda: dg.residual_rms_norm(x, x, x, weight=w), lambda: dg.residual_rms_norm(x, x, x, weight=w, out=out[:4], weight_post=w.bfloat16()),
        lambda: dg.residual_rms_norm(x, x, x, gate=w[:8]), lambda: dg.residual_rms_norm(x, x, x, rstd=w[:4]),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(dg.DGError):
            call()
            raise AssertionError(f"call {i} was not refused")
