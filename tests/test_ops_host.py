"""The operators around the grouped GEMMs, on the host: refusals come back as error codes before anything is launched
(bad extents, alignments, types and combinations), empty calls are no-ops, and the 64-bit forms that the GPU tests
compare with hold on hand-written cases."""
import ctypes

import numpy as np
import pytest
import torch

import _ops_ref as ref
import moe_grouped_gemm_03_b200 as dg

L = dg.lib()
P = ctypes.c_void_p
A, B, C, D, E, F = (P(256 * i) for i in range(1, 7))  # aligned, never read: every call below is refused or empty
INVALID, ALIGNMENT, UNSUPPORTED = -1, -2, -3


def test_m_total_bound():
    assert dg.get_m_total_bound(0, 8) == 0
    assert dg.get_m_total_bound(1, 8) == 128
    assert dg.get_m_total_bound(3, 8) == 384  # three slots of three groups
    assert dg.get_m_total_bound(65536, 64) == 73600 // 128 * 128
    with pytest.raises(dg.DGError):
        dg.get_m_total_bound(-1, 8)
    with pytest.raises(dg.DGError):
        dg.get_m_total_bound(8, 0)
    try:
        dg.set_m_alignment_for_contiguous_layout(256)
        assert dg.get_m_total_bound(3, 8) == 768
    finally:
        dg.set_m_alignment_for_contiguous_layout(128)
    rng = np.random.default_rng(0)
    for _ in range(200):  # the bound holds for every split of the slots
        G, n = int(rng.integers(1, 20)), int(rng.integers(0, 600))
        counts = rng.multinomial(n, rng.dirichlet(np.full(G, 0.3)))
        assert (-(-counts // 128) * 128).sum() <= dg.get_m_total_bound(n, G)


@pytest.mark.parametrize("kw,code", [
    (dict(ids=None), INVALID), (dict(rows=None), INVALID), (dict(counts=None), INVALID), (dict(m=None), INVALID),
    (dict(id_bytes=2), INVALID), (dict(T=-1), INVALID), (dict(k=0), INVALID), (dict(k=33), INVALID), (dict(G=0), INVALID),
    (dict(G=1025), INVALID), (dict(T=1 << 26, k=32), INVALID), (dict(M=-128), INVALID), (dict(M=100), ALIGNMENT),
    (dict(rows=A), INVALID), (dict(ids=P(260), id_bytes=8), ALIGNMENT), (dict(ids=P(258)), ALIGNMENT),
    (dict(m=P(260)), ALIGNMENT), (dict(counts=P(258)), ALIGNMENT)])
def test_sort_refusals(kw, code):
    a = dict(ids=A, id_bytes=4, T=16, k=4, G=8, M=1152, rows=B, m=C, counts=D)
    a.update(kw)
    assert L.dg_moe_sort_contiguous(*a.values(), None) == code, dg.last_error()
    if not {"M", "m"} & set(kw):
        assert L.dg_moe_sort_nopad(a["ids"], a["id_bytes"], a["T"], a["k"], a["G"], a["rows"], a["counts"], None) == code
        assert L.dg_moe_sort_masked(a["ids"], a["id_bytes"], a["T"], a["k"], a["G"], 128, a["rows"], a["counts"],
                                    None) == code


def test_sort_masked_m_max():
    for m_max in (0, -1, 1 << 28):
        assert L.dg_moe_sort_masked(A, 4, 16, 4, 8, m_max, B, C, None) == INVALID


def test_sort_alignment_setting():
    try:
        dg.set_m_alignment_for_contiguous_layout(256)
        assert L.dg_moe_sort_contiguous(A, 4, 16, 4, 8, 384, B, C, D, None) == ALIGNMENT
    finally:
        dg.set_m_alignment_for_contiguous_layout(128)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), INVALID), (dict(rows=None), INVALID), (dict(out=None), INVALID), (dict(type=2), INVALID),
    (dict(type=-1), INVALID), (dict(T=-1), INVALID), (dict(k=0), INVALID), (dict(k=33), INVALID), (dict(H=0), INVALID),
    (dict(H=12), ALIGNMENT), (dict(H=264), ALIGNMENT), (dict(n=-1), INVALID), (dict(n=(1 << 30) + 1), INVALID),
    (dict(per=0), INVALID), (dict(per=48), INVALID), (dict(x=P(264)), ALIGNMENT), (dict(out=P(264)), ALIGNMENT),
    (dict(sf=P(260)), ALIGNMENT), (dict(rows=P(258)), ALIGNMENT)])
def test_permute_refusals(kw, code):
    a = dict(x=A, type=0, rows=B, T=16, k=4, H=256, n=128, per=64, out=C, sf=D)
    a.update(kw)
    assert L.dg_moe_permute(*a.values(), None) == code, dg.last_error()


def test_unpermute_refusals():
    assert L.dg_moe_unpermute(None, 0, B, C, 16, 4, 256, 128, D, None) == INVALID
    assert L.dg_moe_unpermute(A, 0, B, P(258), 16, 4, 256, 128, D, None) == ALIGNMENT
    assert L.dg_moe_unpermute(A, 0, B, C, 16, 4, 255, 128, D, None) == ALIGNMENT
    assert L.dg_moe_unpermute(A, 3, B, C, 16, 4, 256, 128, D, None) == INVALID
    args = dict(d=A, rows=B, type=0, map=C, w=D, T=16, k=4, H=256, n=128, per=128, out=E, sf=None, dw=F)
    for kw, code in ((dict(d=None), INVALID), (dict(w=None), INVALID), (dict(dw=None), INVALID), (dict(d=P(264)), ALIGNMENT),
                     (dict(H=136, sf=A), ALIGNMENT), (dict(per=100, sf=A), INVALID), (dict(w=P(258)), ALIGNMENT)):
        assert L.dg_moe_unpermute_backward(*{**args, **kw}.values(), None) == code, (kw, dg.last_error())


def test_swiglu_refusals():
    args = dict(gu=A, type=0, R=256, I=128, m=None, c=None, mm=None, G=0, out=B, sf=None)
    for kw, code in ((dict(gu=None), INVALID), (dict(out=None), INVALID), (dict(type=5), INVALID), (dict(R=-1), INVALID),
                     (dict(I=0), INVALID), (dict(I=12), ALIGNMENT), (dict(I=136, sf=C), ALIGNMENT),
                     (dict(m=C, c=D, G=4), INVALID), (dict(c=C, G=0), INVALID), (dict(mm=C, G=1025), INVALID),
                     (dict(mm=C, G=3), INVALID), (dict(gu=P(264)), ALIGNMENT), (dict(m=P(258)), ALIGNMENT),
                     (dict(sf=P(260)), ALIGNMENT)):
        a = {**args, **kw}
        assert L.dg_swiglu(*a.values(), None) == code, (kw, dg.last_error())
        assert L.dg_swiglu_backward(E, *a.values(), None) == code, (kw, dg.last_error())
    assert L.dg_swiglu_backward(None, *args.values(), None) == INVALID
    assert L.dg_swiglu_backward(P(264), *args.values(), None) == ALIGNMENT


def test_norm_refusals():
    args = dict(x=A, xt=0, w=B, pt=0, eps=1e-6, T=16, H=256, out=C, ot=0, sf=None, rstd=None)
    call = lambda kw: L.dg_rms_norm(*(ctypes.c_float(v) if k == "eps" else v for k, v in {**args, **kw}.items()), None)  # noqa: E731
    for kw, code in ((dict(x=None), INVALID), (dict(w=None), INVALID), (dict(out=None), INVALID), (dict(xt=2), INVALID),
                     (dict(pt=7), INVALID), (dict(xt=0, ot=1), UNSUPPORTED), (dict(T=-1), INVALID), (dict(H=0), INVALID),
                     (dict(H=16392), UNSUPPORTED), (dict(H=20), ALIGNMENT), (dict(H=264, sf=D), ALIGNMENT),
                     (dict(x=P(264)), ALIGNMENT), (dict(rstd=P(258)), ALIGNMENT)):
        assert call(kw) == code, (kw, dg.last_error())
    args = dict(x=A, xt=0, y=B, yt=0, w=C, wp=None, gate=None, kind=0, pt=0, alpha=1.0, eps=1e-6, T=16, H=256, xo=A, out=D,
                sf=None, rstd=None, rp=None)
    call = lambda kw: L.dg_residual_rms_norm(*(ctypes.c_float(v) if k in ("alpha", "eps") else v  # noqa: E731
                                               for k, v in {**args, **kw}.items()), None)
    for kw, code in ((dict(y=None), INVALID), (dict(xo=None), INVALID), (dict(w=None), INVALID), (dict(out=None), INVALID),
                     (dict(w=None, out=None, sf=D), INVALID), (dict(w=None, out=None, rstd=D), INVALID),
                     (dict(rp=D), INVALID), (dict(gate=E), INVALID), (dict(gate=E, kind=3), INVALID), (dict(kind=1), INVALID),
                     (dict(xt=0, yt=1), UNSUPPORTED), (dict(gate=P(264), kind=1), ALIGNMENT), (dict(y=P(264)), ALIGNMENT)):
        assert call(kw) == code, (kw, dg.last_error())


def test_norm_backward_refusals():
    args = dict(dxo=A, do=B, xo=C, xt=0, y=D, yt=0, w=E, wp=None, gate=None, kind=0, pt=0, alpha=1.0, rstd=F, rp=None, T=16,
                H=256, dx=A, dy=B, dw=C, dwp=None, dg=None)
    call = lambda kw: L.dg_residual_rms_norm_backward(*(ctypes.c_float(v) if k == "alpha" else v  # noqa: E731
                                                        for k, v in {**args, **kw}.items()), None)
    for kw in (dict(y=None), dict(dx=None), dict(dy=None), dict(do=None), dict(xo=None), dict(rstd=None), dict(dw=None),
               dict(w=None), dict(wp=F), dict(wp=F, rp=F), dict(dwp=F), dict(gate=F, kind=1), dict(dg=F),
               dict(dxo=None, do=None, xo=None, w=None, rstd=None, dw=None)):
        assert call(kw) == INVALID, (kw, dg.last_error())
    assert call(dict(H=16392)) == UNSUPPORTED
    assert call(dict(dy=P(264))) == ALIGNMENT
    assert call(dict(dw=P(258))) == ALIGNMENT
    for i in (0, 2, 5, 7, 10, 11):  # d_out, x, weight, rstd, d_x, d_weight
        a = [A, None, B, 0, 0, C, 0, D, 16, 256, E, F]
        a[{0: 0, 2: 2, 5: 5, 7: 7, 10: 10, 11: 11}[i]] = None
        assert L.dg_rms_norm_backward(*a, None) == INVALID


def test_empty_calls_are_no_ops():
    assert L.dg_moe_permute(None, 0, None, 0, 4, 256, 128, 128, C, D, None) == 0
    assert L.dg_moe_permute(A, 0, B, 16, 4, 256, 0, 0, None, None, None) == 0
    assert L.dg_moe_unpermute(A, 0, None, None, 0, 4, 256, 128, None, None) == 0
    assert L.dg_moe_unpermute_backward(None, A, 0, None, None, 0, 4, 256, 128, 128, B, None, None, None) == 0
    assert L.dg_swiglu(None, 0, 0, 128, None, None, None, 0, None, None, None) == 0
    z = ctypes.c_float(0)
    assert L.dg_rms_norm(None, 0, B, 0, z, 0, 256, None, 0, None, None, None) == 0
    assert L.dg_residual_rms_norm(None, 0, None, 0, B, None, None, 0, 0, z, z, 0, 256, None, None, None, None, None, None) == 0


def test_python_refuses_before_it_needs_a_device():
    """Types, dimensions, shapes, strides and CPU tensors, each by DGError with DG_ERR_INVALID_ARG."""
    bf16 = torch.bfloat16
    x, out = torch.zeros(4, 256, dtype=bf16), torch.zeros(8, 256, dtype=bf16)
    rows, w, wt = torch.zeros(4, 2, dtype=torch.int32), torch.ones(256), torch.ones(4, 2)
    f8, sf = torch.zeros(8, 256, dtype=torch.uint8), torch.zeros(2, 8)
    counts = torch.zeros(3, dtype=torch.int32)
    calls = {
        "topk_ids must have 2": lambda: dg.moe_sort_nopad(rows[0], rows, counts),
        "topk_ids has dtype": lambda: dg.moe_sort_masked(rows.float(), rows, counts, 8),
        "topk_ids must be a CUDA tensor": lambda: dg.moe_sort_contiguous(rows, rows, counts, counts),
        "x must be a torch.Tensor": lambda: dg.moe_permute(None, rows, out),
        "x has dtype": lambda: dg.moe_permute(x.half(), rows, out),
        "x must be contiguous": lambda: dg.moe_permute(x.t(), rows, out),
        "x must be a CUDA tensor": lambda: dg.moe_permute(x, rows, out),
        "rows must have 2 or more dims": lambda: dg.moe_unpermute(x[0], rows, out),
        "rows must be a CUDA tensor": lambda: dg.moe_unpermute_backward(x, out, rows, wt, out, wt),
        "gate_up must have 2 or more dims": lambda: dg.swiglu(torch.zeros(4, 2, 3, 2, dtype=bf16), x),
        "d_out must be a torch.Tensor": lambda: dg.swiglu_backward(None, x, x),
        "d_x must be a torch.Tensor": lambda: dg.residual_rms_norm_backward(x, x, None, x),
    }
    if torch.cuda.is_available():
        gx, gr, gw = x.cuda(), rows.cuda(), w.cuda()
        calls.update({
            "out must be a tensor or a pair": lambda: dg.moe_permute(gx, gr, (f8, sf, sf)),
            "out must be a CUDA tensor": lambda: dg.moe_permute(gx, gr, out),
            "weight and out go together": lambda: dg.residual_rms_norm(gx, gx, gx, weight=gw),
            "weight must be a torch.Tensor": lambda: dg.residual_rms_norm(gx, gx, gx, weight=3),
            "eps must be a number": lambda: dg.rms_norm(gx, gw, gx.clone(), eps="a"),
            "m_max must be an integer": lambda: dg.moe_sort_masked(gr, gr.clone(), gr[0].contiguous(), 1.5),
        })
    for message, call in calls.items():
        with pytest.raises(dg.DGError, match=message) as e:
            call()
        assert e.value.status == INVALID


# ------------------------------------------------------------------------------- the 64-bit forms on small cases
def test_reference_quantiser():
    assert ref.scale_of(448.0) == 1 and ref.scale_of(np.nextafter(448.0, 500)) == 2 and ref.scale_of(0.0) == 1
    assert ref.scale_of(1.75) == 2.0 ** -8 and ref.scale_of(1e-45) == 2.0 ** -126
    v = np.array([0.0, 2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -10, 448, 17.0, 18.0, 19.0, -1.0625, -1.1875])
    assert (ref.e4m3(v) == [0.0, 2.0 ** -9, 0.0, 2.0 ** -8, 448, 16, 18, 20, -1.0, -1.25]).all()
    t = torch.linspace(-440, 440, 4001)
    assert (ref.e4m3(t.double().numpy()) == t.to(torch.float8_e4m3fn).double().numpy()).all()


def test_reference_sort():
    ids = [[1, 0], [1, -1], [2, 1]]
    rows, counts, m = ref.sort(ids, "contiguous", 3, m_total=512)
    assert rows.tolist() == [[128, 0], [129, -1], [256, 130]] and counts.tolist() == [1, 3, 1]
    assert m[0] == 0 and m[1] == -1 and m[128:131].tolist() == [1, 1, 1] and m[131] == -1 and m[256] == 2
    assert ref.sort(ids, "nopad", 3)[0].tolist() == [[1, 0], [2, -1], [4, 3]]
    assert ref.sort(ids, "masked", 3, m_max=2)[0].tolist() == [[2, 0], [3, -1], [4, -1]]


def test_reference_gradients_against_autograd():
    g = torch.Generator().manual_seed(0)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    gu, d = r(5, 24).requires_grad_(), r(5, 12)
    a, b = gu.chunk(2, -1)
    (a * torch.sigmoid(a) * b * d).sum().backward()
    assert torch.allclose(ref.swiglu_backward(d, gu), gu.grad, rtol=1e-12)
    for gate_shape in ((16,), (6, 16)):
        x, y, w, wp, gate = (r(*s).requires_grad_() for s in ((6, 16), (6, 16), (16,), (16,), gate_shape))
        dxo, do = r(6, 16), r(6, 16)
        n = y / torch.sqrt((y * y).mean(1, keepdim=True) + 1e-6) * wp
        xo = x + 0.7 * gate * n
        h = xo / torch.sqrt((xo * xo).mean(1, keepdim=True) + 1e-6) * w
        ((xo * dxo).sum() + (h * do).sum()).backward()
        _, _, rstd, rp = ref.norm(x, y, w, wp, gate, 0.7)
        got = ref.norm_backward(dxo, do, xo, y, w, wp, gate, 0.7, rstd, rp)
        for k, t in (("d_x", x), ("d_y", y), ("d_w", w), ("d_w_post", wp), ("d_gate", gate)):
            assert torch.allclose(got[k], t.grad, rtol=1e-10, atol=1e-12), k
