"""The operators around the grouped GEMMs, as measured cases: dispatch (tokens sorted by expert, then gathered and
quantised), combine (expert rows weighted and summed back, and its gradient), SwiGLU between the two expert GEMMs and
its gradient, and the norms before and after a block with their gate, residual scale and gradient.

`own` False: `run` computes the operators in elementary torch operations; True: through the library's entry points.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-6
M_ALIGN = 128  # row alignment of a group in the contiguous layout
LARGEST_BYTES = 1.05e9  # no drawn case moves more than the largest listed one does


# ------------------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # decode step of 32 tokens, top 8 of 256 experts, 32 of them on this GPU: masked layout, FP8 operand
        dict(name="dispatch_decode_masked_fp8", op="dispatch", layout="masked", T=32, k=8, G=32, experts=256, H=7168,
             M_max=256, fp8=True, f32=False),
        # prompt or training micro-batch: 65536 rows over 64 experts, the contiguous layout of the FP8 GEMM
        dict(name="dispatch_contiguous_fp8", op="dispatch", layout="contiguous", T=8192, k=8, G=64, experts=64, H=7168,
             M_max=0, fp8=True, f32=False),
        # odd token count, packed rows without padding and without quantisation (a bf16 consumer)
        dict(name="dispatch_nopad_bf16", op="dispatch", layout="nopad", T=4099, k=2, G=8, experts=8, H=4096, M_max=0,
             fp8=False, f32=False),
        # the decode step's results back: weights of the routed experts, slots of other GPUs' experts skipped
        dict(name="combine_decode", op="combine", layout="masked", T=32, k=8, G=32, experts=256, H=7168, M_max=256,
             f32=False),
        # the micro-batch's results back
        dict(name="combine_contiguous", op="combine", layout="contiguous", T=8192, k=8, G=64, experts=64, H=7168,
             M_max=0, f32=False),
        # gradient of the combine: rows scaled by the weights, and the weights' own gradient
        dict(name="combine_backward", op="combine_backward", layout="contiguous", T=4099, k=8, G=64, experts=64, H=7168,
             M_max=0, fp8=False, f32=False),
        # decode: activation of the masked rows between the two expert GEMMs (N = 4096 -> K = 2048)
        dict(name="swiglu_masked_fp8", op="swiglu", layout="masked", R=8192, G=32, I=2048, fp8=True, f32=False,
             fill=0.5),
        # the micro-batch: 65536 rows in 64 skewed groups padded to 128
        dict(name="swiglu_contiguous_fp8", op="swiglu", layout="contiguous", R=69632, G=64, I=2048, fp8=True, f32=False,
             fill=0.94),
        # its gradient for the weight and data gradients
        dict(name="swiglu_backward", op="swiglu_backward", layout="contiguous", R=32768, G=8, I=2048, fp8=False,
             f32=False, fill=0.97),
        # one token between two blocks: residual add of the normed block output, next block's norm
        dict(name="norm_one_token", op="norm", T=1, H=7168, x_f32=False, y_f32=False, has_y=True, post=True, gate="row",
             pre="same", p_f32=False),
        # training forward with the residual stream in fp32; the next block's first GEMM takes e4m3
        dict(name="norm_fp8", op="norm", T=8192, H=7168, x_f32=True, y_f32=False, has_y=True, post=True, gate="row",
             pre="fp8", p_f32=True),
        # its gradient, with a gate for each token
        dict(name="norm_backward", op="norm_backward", T=8191, H=4096, x_f32=False, y_f32=False, has_y=True, post=True,
             gate="token", pre="same", p_f32=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        op = rng.choice(["dispatch", "combine", "combine_backward", "swiglu", "swiglu_backward", "norm", "norm_backward"])
        f32 = rng.random() < 0.2
        if op in ("dispatch", "combine", "combine_backward"):
            layout = rng.choice(["masked", "contiguous", "nopad"])
            G = rng.choice([1, 3, 8, 17, 32, 64, 256])
            case = dict(op=op, layout=layout, T=_log_int(rng, 1, 8192), k=rng.randint(1, 8), G=G,
                        experts=G * rng.choice([1, 1, 2, 8]), H=128 * _log_int(rng, 4, 64), M_max=0, f32=f32)
            case["k"] = min(case["k"], case["experts"])
            if op != "combine":
                case["fp8"] = rng.random() < 0.6
            if layout == "masked":
                case["T"] = min(case["T"], 512)
                case["M_max"] = 128 * -(-case["T"] // 128)
                if G * case["M_max"] * case["H"] > 2.5e8:
                    continue
        elif op in ("swiglu", "swiglu_backward"):
            layout = rng.choice(["masked", "contiguous", "nopad", "dense"])
            G = rng.choice([1, 3, 8, 17, 32, 64])
            I = 128 * _log_int(rng, 2, 64)
            if layout == "masked":
                R = G * _log_int(rng, 1, 1024)
            elif layout == "contiguous":
                R = M_ALIGN * (G + _log_int(rng, 1, 300))
            else:
                R = _log_int(rng, 1, 40000)
            case = dict(op=op, layout=layout, R=R, G=G, I=I, fp8=rng.random() < 0.6, f32=f32, fill=rng.uniform(0.2, 1.0))
        else:
            fp8 = rng.random() < 0.4
            x_f32 = rng.random() < 0.4
            has_y = rng.random() < 0.8
            case = dict(op=op, T=_log_int(rng, 1, 16384), H=(128 if fp8 else 8) * _log_int(rng, 4 if fp8 else 32, 64 if fp8 else 1024),
                        x_f32=x_f32, y_f32=x_f32 and rng.random() < 0.3, has_y=has_y, post=has_y and rng.random() < 0.7,
                        gate=rng.choice(["none", "row", "token"]) if has_y else "none", p_f32=rng.random() < 0.5)
            case["pre"] = ("same" if op == "norm_backward" or not fp8 else "fp8")
            if has_y and rng.random() < 0.15:
                case["pre"] = "none"
        if work(case)["bytes"] <= LARGEST_BYTES and _elements(case) < 6e8:
            return case


def _elements(case):
    if "k" in case:
        return case["T"] * case["k"] * case["H"]
    return case["R"] * case["I"] * 2 if "R" in case else case["T"] * case["H"] * 4


def work(case):
    op = case["op"]
    if op in ("dispatch", "combine", "combine_backward"):
        T, k, H = case["T"], case["k"], case["H"]
        e = 4 if case["f32"] else 2
        rows = T * k * min(1.0, case["G"] / case["experts"])  # rows of the experts that are here, on average
        row = (H + H // 128 * 4) if case.get("fp8") else H * e
        if op == "dispatch":  # ids and x read; the row map, the rows and their scales written
            return {"bytes": T * k * 8 + T * H * e + rows * (row + 4), "flops": 2.0 * T * H}
        if op == "combine":  # rows, weights and the row map read; out written
            return {"bytes": T * k * 8 + rows * H * e + T * H * e, "flops": 2.0 * rows * H}
        return {"bytes": T * k * 12 + T * H * e + rows * (H * e + row), "flops": 3.0 * rows * H}
    if op in ("swiglu", "swiglu_backward"):
        I, e = case["I"], 4 if case["f32"] else 2
        rows = case["R"] * (1.0 if case["layout"] == "dense" else case["fill"])
        if op == "swiglu":
            return {"bytes": rows * (2 * I * e + (I + I // 32 if case["fp8"] else I * e)), "flops": 6.0 * rows * I}
        return {"bytes": rows * (3 * I * e + (2 * I + I // 16 if case["fp8"] else 2 * I * e)), "flops": 14.0 * rows * I}
    T, H = case["T"], case["H"]
    n = T * H
    ex, ey, y, gate = 4 if case["x_f32"] else 2, 4 if case["y_f32"] else 2, case["has_y"], case["gate"] == "token"
    if op == "norm":
        h = {"none": 0, "fp8": 1 + 1 / 32, "same": ey}[case["pre"]]
        return {"bytes": n * (ex + (y * (ey + ex)) + gate * ey + h) + T * 8 + H * 8, "flops": 10.0 * n}
    h = 0 if case["pre"] == "none" else ey
    return {"bytes": n * (3 * ex + h + y * 2 * ey + gate * 2 * ey) + T * 8 + H * 16, "flops": 20.0 * n}


# ------------------------------------------------------------------------------------------------------- inputs
def _type(f32):
    return torch.float32 if f32 else torch.bfloat16


def _align(n, a):
    return -(-n // a) * a


def _activations(gen, rows, cols, dtype):
    """Normal values with channels of different size, a few of them large, as in a residual stream."""
    scale = torch.exp(0.5 * torch.randn(cols, device="cuda", generator=gen))
    scale[torch.randint(0, cols, (max(1, cols // 512),), device="cuda", generator=gen)] *= 20.0
    return torch.randn(rows, cols, device="cuda", generator=gen).mul_(scale).to(dtype)


def _routing(gen, case):
    """Expert of each slot (distinct in a token, popularity ~ 1 / rank), -1 for an expert of another GPU."""
    E = case["experts"]
    popularity = -torch.log(torch.arange(1, E + 1, device="cuda", dtype=torch.float32))
    popularity = popularity[torch.randperm(E, device="cuda", generator=gen)] * 0.7
    noise = -torch.log(-torch.log(torch.rand(case["T"], E, device="cuda", generator=gen).clamp(1e-7, 1 - 1e-7)))
    ids = torch.topk(popularity + noise, case["k"], dim=1).indices.to(torch.int32)
    return torch.where(ids < case["G"], ids, torch.full_like(ids, -1)).contiguous()


def _total_rows(case):
    slots, G = case["T"] * case["k"], case["G"]
    if case["layout"] == "masked":
        return G * case["M_max"]
    if case["layout"] == "nopad":
        return slots
    return (slots + min(G, slots) * (M_ALIGN - 1)) // M_ALIGN * M_ALIGN


def _rows_of(case, ids):
    """Row of each slot, by counting (numpy): what the sort gives, for the cases that begin behind it."""
    flat = ids.cpu().numpy().reshape(-1)
    counts = np.bincount(flat[flat >= 0], minlength=case["G"])
    if case["layout"] == "masked":
        start = np.arange(case["G"]) * case["M_max"]
    else:
        step = counts if case["layout"] == "nopad" else -(-counts // M_ALIGN) * M_ALIGN
        start = np.concatenate([[0], np.cumsum(step)[:-1]])
    order = np.argsort(flat, kind="stable")
    order = order[np.searchsorted(flat[order], 0):]
    rank = np.arange(order.size) - np.repeat(np.concatenate([[0], np.cumsum(counts)[:-1]]), counts)
    rows = np.full(flat.size, -1, np.int32)
    rows[order] = start[flat[order]] + rank
    return torch.from_numpy(rows.reshape(case["T"], case["k"])).cuda()


def _out_rows(s, key, R, cols, case, dtype):
    """Buffers of a row operand: `cols` wide rows with one spare row behind the last, e4m3 codes and scales if fp8."""
    masked = case["layout"] == "masked"
    groups = case["G"] if masked else 1
    per = R // groups
    if case["fp8"]:
        ld = _align(per, 4)
        s[key + "_full"] = torch.zeros(R + 1, cols, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
        s[key + "_sf_full"] = torch.zeros(groups * (cols // 128) * ld + 1, device="cuda")
        sf = s[key + "_sf_full"][:-1]
        s[key + "_sf"] = sf.view(groups, cols // 128, ld) if masked else sf.view(cols // 128, ld)
        s["ld"], s["per"] = ld, per
    else:
        s[key + "_full"] = torch.zeros(R + 1, cols, dtype=dtype, device="cuda")
    rows = s[key + "_full"][:R]
    s[key] = rows.view(groups, per, cols) if masked else rows
    s[key + "_out"] = (s[key], s[key + "_sf"]) if case["fp8"] else s[key]


def _groups(rs, case):
    """Rows that the groups own, for the cases that begin behind the first GEMM."""
    R, G, layout = case["R"], case["G"], case["layout"]
    want = int(R * case["fill"])
    if layout == "masked":
        M_max = R // G
        return {"masked_m": np.clip(rs.normal(case["fill"], 0.2, G) * M_max, 0, M_max).astype(np.int32)}
    share = rs.permutation(1.0 / np.arange(1, G + 1) ** 0.7)
    counts = rs.multinomial(want, share / share.sum())
    if layout == "nopad":
        return {"counts": counts.astype(np.int32)}
    m_indices, at = np.full(R, -1, np.int32), 0
    for g in range(G):
        n = min(int(counts[g]), R - at)
        m_indices[at:at + n] = g
        at = min(R, at + _align(n, M_ALIGN))
    return {"m_indices": m_indices}


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed * 7919 + 11)
    rs = np.random.RandomState((seed * 7919 + 11) % 2**32)
    s, op = {"case": case}, case["op"]
    if op in ("dispatch", "combine", "combine_backward"):
        T, k, H, dtype = case["T"], case["k"], case["H"], _type(case["f32"])
        ids = _routing(gen, case)
        R = s["R"] = _total_rows(case)
        if op == "dispatch":
            s["ids"], s["x"] = ids, _activations(gen, T, H, dtype)
            s["row_of_slot"] = torch.empty(T, k, dtype=torch.int32, device="cuda")
            s["counts"] = torch.empty(case["G"], dtype=torch.int32, device="cuda")
            s["m_indices"] = torch.empty(R, dtype=torch.int32, device="cuda") if case["layout"] == "contiguous" else None
            _out_rows(s, "a", R, H, case, dtype)
            return s
        s["row_of_slot"] = _rows_of(case, ids)
        s["rows"] = _activations(gen, R, H, dtype)
        if case["layout"] == "masked":
            s["rows"] = s["rows"].view(case["G"], case["M_max"], H)
        s["weights"] = torch.softmax(torch.randn(T, k, device="cuda", generator=gen), dim=1)
        if op == "combine":
            s["out"] = torch.empty(T, H, dtype=dtype, device="cuda")
            return s
        s["d_out"] = _activations(gen, T, H, dtype)
        s["d_weights"] = torch.empty(T, k, device="cuda")
        _out_rows(s, "d_rows", R, H, case, dtype)
        return s
    if op in ("swiglu", "swiglu_backward"):
        R, I, dtype = case["R"], case["I"], _type(case["f32"])
        s["owned"] = {} if case["layout"] == "dense" else {n: torch.from_numpy(v).cuda() for n, v in _groups(rs, case).items()}
        s["gate_up"] = _activations(gen, R, 2 * I, dtype)
        if op == "swiglu_backward":
            s["d_out"] = _activations(gen, R, I, dtype)
        if case["layout"] == "masked":
            s["gate_up"] = s["gate_up"].view(case["G"], R // case["G"], 2 * I)
            if op == "swiglu_backward":
                s["d_out"] = s["d_out"].view(case["G"], R // case["G"], I)
        _out_rows(s, "h", R, I if op == "swiglu" else 2 * I, case, dtype)
        return s
    T, H, X, Y, P = case["T"], case["H"], _type(case["x_f32"]), _type(case["y_f32"]), _type(case["p_f32"])
    weight = lambda: (1 + 0.1 * torch.randn(H, device="cuda", generator=gen)).to(P)  # noqa: E731
    s["w"] = weight() if case["pre"] != "none" else None
    s["w_post"] = weight() if case["post"] else None
    s["alpha"] = 0.7 if case["has_y"] else 1.0
    s["gate"] = {"none": None, "row": weight(), "token": (0.3 * torch.randn(T, H, device="cuda", generator=gen)).to(Y)}[case["gate"]]
    s["x"] = _activations(gen, T, H, X)  # backward: x is the sum that the forward stored
    s["y"] = _activations(gen, T, H, Y) if case["has_y"] else None
    f32 = lambda *shape: torch.empty(*shape, device="cuda")  # noqa: E731
    if op == "norm":
        s["x_out"] = torch.empty_like(s["x"]) if case["has_y"] else None
        s["rstd"], s["rstd_post"] = f32(T) if s["w"] is not None else None, f32(T) if case["post"] else None
        if case["pre"] != "none":
            _out_rows(s, "h", T, H, dict(layout="nopad", fp8=case["pre"] == "fp8"), Y)
        return s
    s["rstd"] = torch.rsqrt(s["x"].float().square().mean(1) + EPS) if s["w"] is not None else None
    s["rstd_post"] = torch.rsqrt(s["y"].float().square().mean(1) + EPS) if case["post"] else None
    s["d_x_out"] = _activations(gen, T, H, X)
    s["d_out"] = _activations(gen, T, H, Y) if s["w"] is not None else None
    s["d_x"] = torch.empty_like(s["x"])
    s["d_y"] = torch.empty_like(s["y"]) if case["has_y"] else None
    s["d_w"], s["d_w_post"] = f32(H) if s["w"] is not None else None, f32(H) if case["post"] else None
    s["d_gate"] = {"none": None, "row": f32(H), "token": torch.empty(T, H, dtype=Y, device="cuda")}[case["gate"]]
    return s


# ------------------------------------------------------------------------------------------------------- one pass
def run(s):
    op = s["case"]["op"]
    if own:
        return _OWN[op](s)
    return _PLAIN[op](s)


def _powers(sf):
    """The blocks' scales, all powers of two, in the type of powers of two: where rounding may put a block's largest
    value on either side of a power, both neighbours stand for the block equally well."""
    return sf.to(torch.float8_e8m0fnu)


def _own_dispatch(s):
    import moe_grouped_gemm_03_b200 as dg

    case = s["case"]
    if case["layout"] == "contiguous":
        dg.moe_sort_contiguous(s["ids"], s["row_of_slot"], s["m_indices"], s["counts"])
    elif case["layout"] == "nopad":
        dg.moe_sort_nopad(s["ids"], s["row_of_slot"], s["counts"])
    else:
        dg.moe_sort_masked(s["ids"], s["row_of_slot"], s["counts"], case["M_max"])
    dg.moe_permute(s["x"], s["row_of_slot"], s["a_out"])
    return [s["row_of_slot"], s["counts"], s["m_indices"], s["a_out"]]


def _own_combine(s):
    import moe_grouped_gemm_03_b200 as dg

    dg.moe_unpermute(s["rows"], s["row_of_slot"], s["out"], s["weights"])
    return s["out"]


def _own_combine_backward(s):
    import moe_grouped_gemm_03_b200 as dg

    dg.moe_unpermute_backward(s["d_out"], s["rows"], s["row_of_slot"], s["weights"], s["d_rows_out"], s["d_weights"])
    return [s["d_rows_out"], s["d_weights"]]


def _own_swiglu(s):
    import moe_grouped_gemm_03_b200 as dg

    dg.swiglu(s["gate_up"], s["h_out"], **s["owned"])
    return [s["h"], _powers(s["h_sf"])] if s["case"]["fp8"] else s["h"]


def _own_swiglu_backward(s):
    import moe_grouped_gemm_03_b200 as dg

    dg.swiglu_backward(s["d_out"], s["gate_up"], s["h_out"], **s["owned"])
    return [s["h"], _powers(s["h_sf"])] if s["case"]["fp8"] else s["h"]


def _own_norm(s):
    import moe_grouped_gemm_03_b200 as dg

    if s["y"] is None:
        dg.rms_norm(s["x"], s["w"], s["h_out"], eps=EPS, rstd=s["rstd"])
    else:
        dg.residual_rms_norm(s["x"], s["y"], s["x_out"], weight=s["w"], out=s.get("h_out"), weight_post=s["w_post"],
                             gate=s["gate"], alpha=s["alpha"], eps=EPS, rstd=s["rstd"], rstd_post=s["rstd_post"])
    return _norm_outputs(s)


def _norm_outputs(s):
    h = [s["h"], _powers(s["h_sf"])] if s["case"]["pre"] == "fp8" else s.get("h")
    return [s["x_out"], h, s["rstd"], s["rstd_post"]]


def _own_norm_backward(s):
    import moe_grouped_gemm_03_b200 as dg

    if s["y"] is None:
        dg.rms_norm_backward(s["d_out"], s["x"], s["w"], s["rstd"], s["d_x"], s["d_w"], d_skip=s["d_x_out"])
    else:
        dg.residual_rms_norm_backward(s["d_x_out"], s["y"], s["d_x"], s["d_y"], d_out=s["d_out"], x_out=s["x"],
                                      weight=s["w"], rstd=s["rstd"], weight_post=s["w_post"], rstd_post=s["rstd_post"],
                                      gate=s["gate"], alpha=s["alpha"], d_weight=s["d_w"], d_weight_post=s["d_w_post"],
                                      d_gate=s["d_gate"])
    return [s["d_x"], s["d_y"], s["d_w"], s["d_w_post"], s["d_gate"]]


_OWN = {"dispatch": _own_dispatch, "combine": _own_combine, "combine_backward": _own_combine_backward,
        "swiglu": _own_swiglu, "swiglu_backward": _own_swiglu_backward, "norm": _own_norm,
        "norm_backward": _own_norm_backward}


# ------------------------------------------------------------------------------------------------- the plain forms
def _quantise(v):
    """fp32 [rows, cols] -> e4m3 codes [rows, cols] and the power-of-two scale of each block of 128 [rows, cols / 128]."""
    blocks = v.view(v.shape[0], -1, 128)
    amax = blocks.abs().amax(2)
    mantissa, exponent = torch.frexp(amax)  # amax = mantissa * 2^exponent, 448 = 0.875 * 2^9
    exponent = (exponent - 9 + (mantissa > 0.875)).clamp_min(-126)
    exponent = torch.where(amax == 0, torch.zeros_like(exponent), exponent)
    scale = ((exponent + 127) << 23).view(torch.float32)
    return (blocks / scale[:, :, None]).view(v.shape).to(torch.float8_e4m3fn), scale


def _put(s, key, row, v, dtype):
    """Writes the rows `v` (fp32) at `row` of the operand `key`; row -1 goes to the spare row behind the last."""
    R = s[key + "_full"].shape[0] - 1
    row = torch.where(row < 0, R, row).long()
    if key + "_sf" not in s:
        s[key + "_full"][row] = v.to(dtype)
        return
    q, scale = _quantise(v)
    _put_codes(s, key, row, q, scale)


def _put_codes(s, key, row, q, scale):
    R = s[key + "_full"].shape[0] - 1
    s[key + "_full"].view(torch.uint8)[row] = q.view(torch.uint8)
    n, ld = scale.shape[1], s["ld"]
    at = (row // s["per"] * n)[:, None] * ld + torch.arange(n, device=row.device) * ld + (row % s["per"])[:, None]
    at = torch.where((row == R)[:, None], s[key + "_sf_full"].numel() - 1, at)
    s[key + "_sf_full"][at] = scale


def _plain_dispatch(s):
    case, G, R = s["case"], s["case"]["G"], s["R"]
    flat = s["ids"].view(-1).long()
    bucket = torch.where(flat < 0, G, flat)
    order = torch.argsort(bucket, stable=True)
    counts = torch.zeros(G + 1, dtype=torch.int64, device=flat.device).index_add_(0, bucket, torch.ones_like(bucket))
    first = torch.cumsum(counts, 0) - counts
    rank = torch.empty_like(flat)
    rank[order] = torch.arange(flat.numel(), device=flat.device) - first[bucket[order]]
    if case["layout"] == "masked":
        start = torch.arange(G + 1, device=flat.device) * case["M_max"]
    else:
        step = counts if case["layout"] == "nopad" else (counts + M_ALIGN - 1) // M_ALIGN * M_ALIGN
        start = torch.cumsum(step, 0) - step
    row = torch.where(flat < 0, -1, start[bucket] + rank)
    m_indices = None
    if case["layout"] == "contiguous":
        m_indices = torch.full((R + 1,), -1, dtype=torch.int32, device=flat.device)
        m_indices[torch.where(row < 0, R, row)] = flat.to(torch.int32)
        m_indices = m_indices[:R]
    token = torch.arange(flat.numel(), device=flat.device) // case["k"]
    at = torch.where(row < 0, R, row)
    if case["fp8"]:
        q, scale = _quantise(s["x"].float())
        _put_codes(s, "a", at, q[token], scale[token])
    else:
        s["a_full"][at] = s["x"][token]
    return [row.to(torch.int32).view_as(s["ids"]), counts[:G].to(torch.int32), m_indices, s["a_out"]]


def _gathered(s):
    """Rows of the slots in fp32 [T, k, H], zeros for a slot without a row."""
    H, row = s["case"]["H"], s["row_of_slot"].long()
    return torch.where((row >= 0)[:, :, None], s["rows"].view(-1, H)[row.clamp_min(0)].float(), 0.0)


def _plain_combine(s):
    return (_gathered(s) * s["weights"][:, :, None]).sum(1).to(s["rows"].dtype)


def _plain_combine_backward(s):
    d_out = s["d_out"].float()[:, None, :]
    d_weights = (_gathered(s) * d_out).sum(2)
    d_rows = (s["weights"][:, :, None] * d_out).view(-1, s["case"]["H"])
    _put(s, "d_rows", s["row_of_slot"].view(-1), d_rows, s["rows"].dtype)
    return [s["d_rows_out"], d_weights]


def _owned_rows(s):
    """Row numbers with -1 in the place of rows that no group owns."""
    R, owned = s["case"]["R"], s["owned"]
    row = torch.arange(R, device="cuda")
    if "m_indices" in owned:
        keep = owned["m_indices"] >= 0
    elif "counts" in owned:
        keep = row < owned["counts"].sum()
    elif "masked_m" in owned:
        per = R // s["case"]["G"]
        keep = row % per < owned["masked_m"][row // per]
    else:
        return row
    return torch.where(keep, row, -1)


def _plain_swiglu(s):
    I = s["case"]["I"]
    gu = s["gate_up"].view(-1, 2 * I).float()
    g, u = gu[:, :I], gu[:, I:]
    _put(s, "h", _owned_rows(s), g / (1 + torch.exp(-g)) * u, s["gate_up"].dtype)
    return [s["h"], _powers(s["h_sf"])] if s["case"]["fp8"] else s["h"]


def _plain_swiglu_backward(s):
    I = s["case"]["I"]
    gu, d = s["gate_up"].view(-1, 2 * I).float(), s["d_out"].view(-1, I).float()
    g, u = gu[:, :I], gu[:, I:]
    sig = 1 / (1 + torch.exp(-g))
    d_gu = torch.cat([d * u * sig * (1 + g * (1 - sig)), d * g * sig], 1)
    _put(s, "h", _owned_rows(s), d_gu, s["gate_up"].dtype)
    return [s["h"], _powers(s["h_sf"])] if s["case"]["fp8"] else s["h"]


def _plain_norm(s):
    total = s["x"].float()
    if s["y"] is not None:
        n = s["y"].float()
        if s["w_post"] is not None:
            s["rstd_post"] = torch.rsqrt(n.square().mean(1) + EPS)
            n = n * s["rstd_post"][:, None] * s["w_post"].float()
        if s["gate"] is not None:
            n = n * s["gate"].float()
        total = total + s["alpha"] * n
        s["x_out"] = total.to(s["x"].dtype)
    if s["w"] is not None:
        s["rstd"] = torch.rsqrt(total.square().mean(1) + EPS)
        h = total * s["rstd"][:, None] * s["w"].float()
        if s["case"]["pre"] == "fp8":
            _put(s, "h", torch.arange(h.shape[0], device=h.device), h, None)
        else:
            s["h"] = h.to(_type(s["case"]["y_f32"]))
    return _norm_outputs(s)


def _plain_norm_backward(s):
    x, d_x, H = s["x"].float(), s["d_x_out"].float(), s["case"]["H"]
    d_w = d_w_post = d_y = d_gate = None
    if s["w"] is not None:
        r, wd = s["rstd"][:, None], s["w"].float() * s["d_out"].float()
        d_w = (s["d_out"].float() * x * r).sum(0, dtype=torch.float64).float()
        d_x = d_x + r * (wd - x * r * r * ((wd * x).sum(1, keepdim=True) / H))
    if s["y"] is not None:
        y = s["y"].float()
        gate = 1.0 if s["gate"] is None else s["gate"].float()
        d_n = s["alpha"] * gate * d_x
        n = y
        if s["w_post"] is not None:
            r, w = s["rstd_post"][:, None], s["w_post"].float()
            n = y * r * w
            d_w_post = (d_n * y * r).sum(0, dtype=torch.float64).float()
            wd = w * d_n
            d_y = r * (wd - y * r * r * ((wd * y).sum(1, keepdim=True) / H))
        else:
            d_y = d_n
        if s["gate"] is not None:
            d_gate = s["alpha"] * n * d_x
            d_gate = d_gate.sum(0, dtype=torch.float64).float() if s["gate"].dim() == 1 else d_gate.to(s["gate"].dtype)
        d_y = d_y.to(s["y"].dtype)
    return [d_x.to(s["x"].dtype), d_y, d_w, d_w_post, d_gate]


_PLAIN = {"dispatch": _plain_dispatch, "combine": _plain_combine, "combine_backward": _plain_combine_backward,
          "swiglu": _plain_swiglu, "swiglu_backward": _plain_swiglu_backward, "norm": _plain_norm,
          "norm_backward": _plain_norm_backward}


# ------------------------------------------------------------------------------------- 64 bits, by the definitions
def _two_to(power):
    """2^power in 64 bits from the exponent's bits (a general power function may be off by a rounding)."""
    return ((power.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact_rows(values, rows, R, groups, fp8):
    """The operand with `values` [n, cols] (64 bits) in the rows `rows` (numpy, none below 0) and zeros elsewhere: itself,
    or e4m3 values and scales, laid out [groups, cols / 128, rows of a group to a multiple of 4]."""
    n, cols = values.shape
    at = torch.from_numpy(rows.astype(np.int64)).cuda()
    out = torch.zeros(R, cols, dtype=torch.float64, device="cuda")
    if not fp8:
        return out.index_copy_(0, at, values)
    blocks = values.view(n, cols // 128, 128)
    amax = blocks.abs().amax(2)
    power = torch.ceil(torch.log2(amax.clamp_min(2.0**-140) / 448))
    power = power + (amax > 448 * _two_to(power)).double() - (amax <= 448 * _two_to(power - 1)).double()
    scale = _two_to(torch.where(amax > 0, power.clamp_min(-126), 0.0))
    v = blocks / scale[:, :, None]
    binade = torch.floor(torch.log2(v.abs().clamp_min(2.0**-30)))
    binade = binade + (v.abs() >= _two_to(binade + 1)).double() - ((v.abs() < _two_to(binade)) & (binade > -6)).double()
    step = _two_to(binade.clamp_min(-6) - 3)
    out.index_copy_(0, at, (torch.round(v / step) * step).view(n, cols))
    per = R // groups
    sf = torch.zeros(groups, cols // 128, _align(per, 4), dtype=torch.float64, device="cuda")
    sf[at // per, :, at % per] = scale
    return [out, sf]


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    groups = case["G"] if case.get("layout") == "masked" else 1
    if op == "dispatch":
        row = _rows_of(case, s["ids"])
        flat, ids = row.cpu().numpy().reshape(-1), s["ids"].cpu().numpy().reshape(-1)
        slots = np.flatnonzero(flat >= 0)
        m_indices = None
        if case["layout"] == "contiguous":
            m_indices = np.full(s["R"], -1, np.int32)
            m_indices[flat[slots]] = ids[slots]
        x = s["x"].double()
        values = x[torch.from_numpy(slots // case["k"]).cuda()]
        counts = np.array([(ids == g).sum() for g in range(case["G"])], np.int32)
        return [row, counts, m_indices, _exact_rows(values, flat[slots], s["R"], groups, case["fp8"])]
    if op in ("combine", "combine_backward"):
        rows, row, w = s["rows"].view(-1, case["H"]), s["row_of_slot"].long(), s["weights"].double()
        valid = row >= 0
        if op == "combine":
            out = torch.zeros(case["T"], case["H"], dtype=torch.float64, device="cuda")
            for j in range(case["k"]):
                t = valid[:, j].nonzero()[:, 0]
                out[t] += w[t, j, None] * rows[row[t, j]].double()
            return out
        d, d_w = s["d_out"].double(), torch.zeros(case["T"], case["k"], dtype=torch.float64, device="cuda")
        for j in range(case["k"]):
            t = valid[:, j].nonzero()[:, 0]
            d_w[t, j] = torch.einsum("th,th->t", d[t], rows[row[t, j]].double())
        flat = row.cpu().numpy().reshape(-1)
        slots = np.flatnonzero(flat >= 0)
        pick = torch.from_numpy(slots).cuda()
        values = w.view(-1)[pick, None] * d[pick // case["k"]]
        return [_exact_rows(values, flat[slots], s["R"], groups, case["fp8"]), d_w]
    if op in ("swiglu", "swiglu_backward"):
        R, I, owned = case["R"], case["I"], {n: v.cpu().numpy() for n, v in s["owned"].items()}
        rows = np.arange(R)
        if "m_indices" in owned:
            rows = rows[owned["m_indices"] >= 0]
        elif "counts" in owned:
            rows = rows[:owned["counts"].sum()]
        elif "masked_m" in owned:
            rows = np.concatenate([g * (R // groups) + np.arange(m) for g, m in enumerate(owned["masked_m"])])
        at = torch.from_numpy(rows).cuda()
        g, u = s["gate_up"].view(R, 2, I)[at].double().unbind(1)
        if op == "swiglu":
            values = g * torch.sigmoid(g) * u
        else:
            d = s["d_out"].view(R, I)[at].double()
            e = torch.exp(-g.abs())
            sig = torch.where(g >= 0, 1 / (1 + e), e / (1 + e))
            values = torch.stack([d * u * (sig + g * sig * (1 - sig)), d * g * sig], 1).view(-1, 2 * I)
        return _exact_rows(values, rows, R, groups, case["fp8"])
    x, H = s["x"].double(), case["H"]
    d = {n: s[n].double() for n in ("y", "w", "w_post", "gate") if s[n] is not None}
    gate = d.get("gate", torch.ones(H, dtype=torch.float64, device="cuda")) * s["alpha"]
    rms = lambda v: torch.sqrt((v * v).sum(1, keepdim=True) / H + EPS)  # noqa: E731
    if op == "norm":
        total, h, rstd, rstd_post = x, None, None, None
        if "y" in d:
            n = d["y"]
            if "w_post" in d:
                rstd_post = 1 / rms(n)[:, 0]
                n = n / rms(n) * d["w_post"]
            total = x + gate * n
        if "w" in d:
            rstd = 1 / rms(total)[:, 0]
            h = _exact_rows(total / rms(total) * d["w"], np.arange(case["T"]), case["T"], 1, case["pre"] == "fp8")
        return [total if "y" in d else None, h, rstd, rstd_post]
    d_x, d_y, d_w, d_w_post, d_gate = s["d_x_out"].double(), None, None, None, None
    if "w" in d:  # x / rms(x) has the Jacobian (1 - u u^T / H) / rms for u = x / rms, with the given 1 / rms
        inv, d_h = s["rstd"].double()[:, None], s["d_out"].double()
        unit, e = x * inv, d_h * d["w"]
        d_w = (d_h * unit).sum(0)
        d_x = d_x + inv * (e - unit * (e * unit).mean(1, keepdim=True))
    if "y" in d:
        d_n, unit = gate * d_x, d["y"]
        if "w_post" in d:
            inv = s["rstd_post"].double()[:, None]
            unit = unit * inv
            d_w_post = (d_n * unit).sum(0)
            e = d_n * d["w_post"]
            d_y = inv * (e - unit * (e * unit).mean(1, keepdim=True))
            unit = unit * d["w_post"]
        else:
            d_y = d_n
        if "gate" in d:
            d_gate = d_x * unit * s["alpha"]
            d_gate = d_gate.sum(0) if d["gate"].dim() == 1 else d_gate
    return [d_x, d_y, d_w, d_w_post, d_gate]
