"""The operators together, as an MoE layer uses them around the grouped GEMMs: norm, sort, dispatch, expert GEMM, SwiGLU,
expert GEMM, combine, residual norm, in the three grouped layouts, and the way back through the same weights.

Each step is compared with its 64-bit form on the inputs that the GPU's step before it gave it, within that step's tolerance;
the whole is then compared with the same layer in 64 bits without any quantisation.  There every e4m3 operand adds a relative
error of at most 2^-4, uniform between its neighbours: 2^-4 / sqrt(3) * (mean over a binade, about 0.72) = 2.6% in the mean
square.  Four such operands forward (two activations, two weights) add up to 5.2%, six on the way back (two more gradients)
to 6.4%; half as much again is allowed.
"""
import numpy as np
import pytest
import torch

import _ops_ref as ref
from _helpers import assert_close

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
T, K, G, H, I = 333, 3, 7, 512, 384
FORWARD, BACKWARD = 1.5 * 0.052, 1.5 * 0.064


def quantised_weight(g, n, k):
    """(fp32 weights [G, n, k], codes, scales [G, n/128, k/128]) with 128x128 blocks."""
    w = torch.randn(G, n, k, generator=g) / k ** 0.5
    blocks = w.double().reshape(G, n // 128, 128, k // 128, 128)
    s = ref.scale_of(blocks.abs().amax((2, 4)).numpy())
    q = ref.e4m3((blocks.numpy() / s[:, :, None, :, None])).reshape(G, n, k)
    return w, torch.from_numpy(q).to(torch.float8_e4m3fn).cuda(), torch.from_numpy(s).float().cuda()


def dequantise(a, sf):
    """fp64 [rows, cols] of an (e4m3, sf) operand, in any layout."""
    codes, per = a.cpu().double(), a.shape[-2]
    s = sf.cpu().double()[..., :per].transpose(-1, -2).repeat_interleave(128, -1)
    return (codes * s).reshape(-1, a.shape[-1]).numpy()


def weight64(q, s):
    return (q.cpu().double() * s.cpu().double().repeat_interleave(128, 1).repeat_interleave(128, 2)).numpy()


def relative(a, b):
    a, b = np.asarray(a, np.float64), np.asarray(b, np.float64)
    return np.linalg.norm(a - b) / np.linalg.norm(b)


def bf16_close(got, want, size):
    """Within bf16's half step of the value and 2^-14 of the size of the terms (fp32 sums and functions)."""
    got, want, size = (np.asarray(v.float().cpu() if torch.is_tensor(v) else v, np.float64) for v in (got, want, size))
    assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -14 * size).all()


class Layer:
    def __init__(self, layout, seed):
        import moe_grouped_gemm_03_b200 as dg

        self.dg, self.layout = dg, layout
        g = torch.Generator().manual_seed(seed)
        self.w1, self.q1, self.s1 = quantised_weight(g, 2 * I, H)
        self.w2, self.q2, self.s2 = quantised_weight(g, H, I)
        ids = torch.stack([torch.randperm(G, generator=g)[:K] for _ in range(T)])
        ids[torch.rand(T, K, generator=g) < 0.1] = -1  # experts of another GPU
        self.ids = ids.to(torch.int32).cuda()
        self.x = torch.randn(T, H, generator=g).to(BF16).cuda()
        self.weights = torch.softmax(torch.randn(T, K, generator=g), 1).cuda()
        self.pre, self.post, self.next, self.gate = (1 + 0.2 * torch.randn(4, H, generator=g)).cuda()
        self.row = torch.empty(T, K, dtype=torch.int32, device="cuda")
        self.counts = torch.empty(G, dtype=torch.int32, device="cuda")
        self.M = dict(contiguous=dg.get_m_total_bound(T * K, G), nopad=T * K, masked=384)[layout]
        self.m_indices = torch.empty(self.M, dtype=torch.int32, device="cuda")

    def buffer(self, cols, dtype=BF16):
        shape = (G, self.M, cols) if self.layout == "masked" else (self.M, cols)
        return torch.zeros(shape, dtype=dtype, device="cuda")

    def operand(self, cols):
        shape = (G, cols // 128, (self.M + 3) // 4 * 4) if self.layout == "masked" else (cols // 128, (self.M + 3) // 4 * 4)
        return self.buffer(cols, torch.uint8).view(torch.float8_e4m3fn), torch.ones(shape, device="cuda")

    def owned(self):
        if self.layout == "contiguous":
            return dict(m_indices=self.m_indices)
        return dict(counts=self.counts) if self.layout == "nopad" else dict(masked_m=self.counts)

    def gemm(self, lhs, b, s, out):
        dg = self.dg
        if self.layout == "contiguous":
            dg.m_grouped_fp8_gemm_nt_contiguous(lhs, (b, s), out, self.m_indices)
        elif self.layout == "nopad":
            dg.m_grouped_fp8_gemm_nt_nopad(lhs, (b, s), out, self.counts)
        else:
            dg.m_grouped_fp8_gemm_nt_masked(lhs, (b, s), out, self.counts, 128)

    def rows(self):
        """(row, expert, token) of the slots with a row."""
        row, ids = self.row.cpu().numpy().reshape(-1), self.ids.cpu().numpy().reshape(-1)
        at = np.flatnonzero(row >= 0)
        return row[at], ids[at], at // K

    def forward(self):
        dg = self.dg
        self.rstd = torch.empty(T, device="cuda")
        self.h = torch.empty(T, H, dtype=BF16, device="cuda")
        dg.rms_norm(self.x, self.pre, self.h, rstd=self.rstd)
        if self.layout == "contiguous":
            dg.moe_sort_contiguous(self.ids, self.row, self.m_indices, self.counts)
        elif self.layout == "nopad":
            dg.moe_sort_nopad(self.ids, self.row, self.counts)
        else:
            dg.moe_sort_masked(self.ids, self.row, self.counts, self.M)
        self.a = self.operand(H)
        dg.moe_permute(self.h, self.row, self.a)
        self.gu = self.buffer(2 * I)
        self.gemm(self.a, self.q1, self.s1, self.gu)
        self.act = self.operand(I)
        dg.swiglu(self.gu, self.act, **self.owned())
        self.down = self.buffer(H)
        self.gemm(self.act, self.q2, self.s2, self.down)
        self.y = torch.empty(T, H, dtype=BF16, device="cuda")
        dg.moe_unpermute(self.down, self.row, self.y, self.weights)
        self.x_out, self.out = torch.empty_like(self.x), torch.empty_like(self.x)
        self.rstd_out, self.rstd_post = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
        dg.residual_rms_norm(self.x, self.y, self.x_out, weight=self.next, out=self.out, weight_post=self.post, gate=self.gate,
                             alpha=0.8, rstd=self.rstd_out, rstd_post=self.rstd_post)

    def check_forward(self):
        rows, experts, tokens = self.rows()
        assert len(rows) == int((self.ids >= 0).sum())
        _, h, _, _ = ref.norm(self.x, w=self.pre)
        bf16_close(self.h, h, h.abs())
        q, s = ref.quantise(self.h.cpu().double().numpy())
        a = dequantise(*self.a)[rows]
        assert (a == (q * np.repeat(s, 128, 1))[tokens]).all()
        w1, w2 = weight64(self.q1, self.s1), weight64(self.q2, self.s2)
        gu = self.gu.reshape(-1, 2 * I).float().cpu().double()[rows]
        assert_close(gu.numpy(), np.stack([w1[e] @ v for e, v in zip(experts, a)]), "up")
        want, act = ref.swiglu(gu).numpy(), dequantise(*self.act)[rows]
        assert (np.abs(act - want) <= 2.0 ** -4 * np.abs(want) + 2.0 ** -9 * np.abs(want).max(1, keepdims=True) / 256).all()
        down = self.down.reshape(-1, H).float().cpu().double().numpy()[rows]
        assert_close(down, np.stack([w2[e] @ v for e, v in zip(experts, act)]), "down")
        size = ref.combine(self.down.abs(), self.row, self.weights)
        bf16_close(self.y, ref.combine(self.down, self.row, self.weights), size)
        total, out, _, _ = ref.norm(self.x, self.y, self.next, self.post, self.gate, 0.8)
        bf16_close(self.x_out, total, self.x.float().abs().cpu().double() + total.abs())
        bf16_close(self.out, out, out.abs() + 1)

    def plain(self):
        """The layer in 64 bits, without quantisation: leaves (x, weights), results (x_out, out), by autograd."""
        x, w = self.x.double().requires_grad_(), self.weights.double().requires_grad_()
        norm = lambda v, p: v / torch.sqrt((v * v).mean(1, keepdim=True) + 1e-6) * p.double()  # noqa: E731
        h = norm(x, self.pre)
        y = torch.zeros_like(x)
        for e in range(G):
            t, s = (self.ids == e).nonzero(as_tuple=True)
            g, u = (h[t] @ self.w1[e].double().cuda().T).chunk(2, 1)
            y = y.index_add(0, t, w[t, s, None] * ((g * torch.sigmoid(g) * u) @ self.w2[e].double().cuda().T))
        x_out = x + 0.8 * self.gate.double() * norm(y, self.post)
        return (x, w), (x_out, norm(x_out, self.next))


@pytest.mark.parametrize("layout", ["contiguous", "nopad", "masked"])
def test_layer_forward(layout):
    layer = Layer(layout, 11)
    layer.forward()
    layer.dg.check_device_error()
    layer.check_forward()
    _, (x_out, out) = layer.plain()
    change, want = layer.x_out.double() - layer.x.double(), x_out - layer.x.double()
    assert relative(change.cpu(), want.detach().cpu()) < FORWARD
    assert relative(layer.out.double().cpu(), out.detach().cpu()) < FORWARD


def test_layer_backward():
    """The gradient takes the same weights: B [G, N, K] of the forward GEMM is B [G, K, N] of the NN GEMM."""
    layer = Layer("contiguous", 12)
    dg = layer.dg
    layer.forward()
    g = torch.Generator().manual_seed(5)
    d_x_out, d_out = torch.randn(2, T, H, generator=g).to(BF16).cuda()
    f32 = lambda *s: torch.empty(*s, device="cuda")  # noqa: E731
    d_skip, d_y = torch.empty_like(layer.x), torch.empty_like(layer.x)
    d_next, d_post, d_gate = f32(H), f32(H), f32(H)
    dg.residual_rms_norm_backward(d_x_out, layer.y, d_skip, d_y, d_out=d_out, x_out=layer.x_out, weight=layer.next,
                                  rstd=layer.rstd_out, weight_post=layer.post, rstd_post=layer.rstd_post, gate=layer.gate,
                                  alpha=0.8, d_weight=d_next, d_weight_post=d_post, d_gate=d_gate)
    d_down, d_weights = layer.operand(H), f32(T, K)
    dg.moe_unpermute_backward(d_y, layer.down, layer.row, layer.weights, d_down, d_weights)
    d_act = layer.buffer(I)
    dg.m_grouped_fp8_gemm_nn_contiguous(d_down, (layer.q2, layer.s2), d_act, layer.m_indices)
    d_gu = layer.operand(2 * I)
    dg.swiglu_backward(d_act, layer.gu, d_gu, m_indices=layer.m_indices)
    d_a = layer.buffer(H)
    dg.m_grouped_fp8_gemm_nn_contiguous(d_gu, (layer.q1, layer.s1), d_a, layer.m_indices)
    d_h, d_x, d_pre = torch.empty_like(layer.x), torch.empty_like(layer.x), f32(H)
    dg.moe_unpermute(d_a, layer.row, d_h)
    dg.rms_norm_backward(d_h, layer.x, layer.pre, layer.rstd, d_x, d_pre, d_skip=d_skip)
    dg.check_device_error()

    rows, experts, tokens = layer.rows()
    w1, w2 = weight64(layer.q1, layer.s1), weight64(layer.q2, layer.s2)
    dd, act = dequantise(*d_down)[rows], d_act.float().cpu().double().numpy()[rows]
    assert_close(act, np.stack([v @ w2[e] for e, v in zip(experts, dd)]), "down gradient")
    want, got = ref.swiglu_backward(d_act.cpu()[rows], layer.gu.cpu()[rows]).numpy(), dequantise(*d_gu)[rows]
    # e4m3 of the value, or half the smallest step of its block, and the cancelling 1 + g (1 - s)
    top = np.abs(want).reshape(len(rows), -1, 128).max(2, keepdims=True).repeat(128, 2).reshape(want.shape)
    assert (np.abs(got - want) <= 2.0 ** -4 * np.abs(want) + top * 2.0 ** -14).all()
    assert_close(d_a.float().cpu().double().numpy()[rows], np.stack([v @ w1[e] for e, v in zip(experts, got)]), "up gradient")

    (x, w), (x_out, out) = layer.plain()
    ((x_out * d_x_out.double()).sum() + (out * d_out.double()).sum()).backward()
    assert relative(d_x.double().cpu(), x.grad.cpu()) < BACKWARD
    valid = (layer.ids >= 0).cpu()
    assert relative(d_weights.cpu()[valid], w.grad.cpu()[valid]) < BACKWARD
    assert (d_weights.cpu()[~valid] == 0).all()
