"""Plain 64-bit forms of the operators around the grouped GEMMs (CPU, float64), written from their formulas."""
import numpy as np
import torch


def scale_of(amax):
    """The smallest power of two with amax <= 448 * scale, at least 2^-126; 1 for 0 (numpy float64)."""
    amax = np.asarray(amax, np.float64)
    m, e = np.frexp(amax)  # amax = m * 2^e, m in [0.5, 1); 448 = 0.875 * 2^9
    e = np.maximum(e - 9 + (m > 0.875), -126)
    return np.where(amax == 0, 1.0, np.ldexp(1.0, e))


def e4m3(v):
    """Round to the nearest e4m3 value, ties to even; NaN stays NaN (|v| <= 448)."""
    v = np.asarray(v, np.float64)
    _, e = np.frexp(v)
    step = np.ldexp(1.0, np.maximum(np.where(np.isfinite(v), e, 0) - 1, -6) - 3)
    return np.where(np.isfinite(v), np.round(np.where(np.isfinite(v), v, 0) / step) * step, np.nan)


def quantise(x):
    """[rows, cols] -> (e4m3 values, scales [rows, cols / 128]); the scale goes by a block's finite values."""
    x = np.asarray(x, np.float64)
    b = x.reshape(x.shape[0], x.shape[1] // 128, 128)
    amax = np.where(np.isfinite(b), np.abs(b), 0).max(2)
    s = scale_of(amax)
    with np.errstate(invalid="ignore"):
        q = e4m3(np.where(np.isfinite(b), b / s[:, :, None], np.nan))
    return q.reshape(x.shape), s


def sort(ids, layout, G, align=128, m_max=0, m_total=None):
    """(row of every slot, rows of each group, m_indices): slots in order, one at a time."""
    ids = np.asarray(ids)
    flat = ids.reshape(-1)
    counts = np.array([(flat == g).sum() for g in range(G)])
    if layout == "masked":
        start = np.arange(G) * m_max
    else:
        step = counts if layout == "nopad" else -(-counts // align) * align
        start = np.concatenate([[0], np.cumsum(step)[:-1]])
    rows, seen = np.full(flat.size, -1), np.zeros(G, int)
    placed = np.zeros(G, int)
    for i, g in enumerate(flat):
        if 0 <= g < G:
            r = start[g] + seen[g]
            if not ((layout == "masked" and seen[g] >= m_max) or (m_total is not None and r >= m_total)):
                rows[i] = r
                placed[g] += 1
            seen[g] += 1
    m_indices = None
    if m_total is not None:
        m_indices = np.full(m_total, -1)
        for i, r in enumerate(rows):
            if r >= 0:
                m_indices[r] = flat[i]
    return rows.reshape(ids.shape), placed, m_indices


def f64(t):
    return t.detach().cpu().double()


def combine(rows, row_of_slot, w=None):
    rows, row = f64(rows).reshape(-1, rows.shape[-1]), row_of_slot.cpu().long()
    out = torch.zeros(row.shape[0], rows.shape[1], dtype=torch.float64)
    for t in range(row.shape[0]):
        for s in range(row.shape[1]):
            if row[t, s] >= 0:
                out[t] += (1.0 if w is None else f64(w)[t, s]) * rows[row[t, s]]
    return out


def swiglu(gu):
    g, u = f64(gu).chunk(2, -1)
    return g * torch.sigmoid(g) * u


def swiglu_backward(d, gu):
    d, (g, u) = f64(d), f64(gu).chunk(2, -1)
    s = torch.sigmoid(g)
    return torch.cat([d * u * s * (1 + g * (1 - s)), d * g * s], -1)


def norm(x, y=None, w=None, w_post=None, gate=None, alpha=1.0, eps=1e-6):
    """(x_out, out, rstd, rstd_post), any of them None."""
    total, rstd_post, out, rstd = f64(x), None, None, None
    if y is not None:
        n = f64(y)
        if w_post is not None:
            rstd_post = 1 / torch.sqrt((n * n).mean(1) + eps)
            n = n * rstd_post[:, None] * f64(w_post)
        total = total + alpha * (n if gate is None else n * f64(gate))
    if w is not None:
        rstd = 1 / torch.sqrt((total * total).mean(1) + eps)
        out = total * rstd[:, None] * f64(w)
    return total, out, rstd, rstd_post


def norm_backward(d_x_out, d_out, x_out, y, w, w_post, gate, alpha, rstd, rstd_post):
    """dict of d_x, d_y, d_w, d_w_post, d_gate."""
    res = {"d_x": torch.zeros_like(f64(x_out if x_out is not None else y)) if d_x_out is None else f64(d_x_out)}
    if w is not None:
        x, r, d = f64(x_out), f64(rstd)[:, None], f64(d_out)
        res["d_w"] = (d * x * r).sum(0)
        e = f64(w) * d
        res["d_x"] = res["d_x"] + r * (e - x * r * r * (e * x).mean(1, keepdim=True))
    if y is not None:
        n, d_n = f64(y), alpha * res["d_x"] * (1.0 if gate is None else f64(gate))
        if w_post is not None:
            r = f64(rstd_post)[:, None]
            res["d_w_post"] = (d_n * f64(y) * r).sum(0)
            e = f64(w_post) * d_n
            n = f64(y) * r * f64(w_post)
            res["d_y"] = r * (e - f64(y) * r * r * (e * f64(y)).mean(1, keepdim=True))
        else:
            res["d_y"] = d_n
        if gate is not None:
            g = alpha * n * res["d_x"]
            res["d_gate"] = g.sum(0) if gate.dim() == 1 else g
    return res
