"""Calls of the operators around the grouped GEMMs as concurrent and captured programs make them: C callers on several host
threads, one graph of calls of several sizes."""
import os
import subprocess
import sys
import threading
import time

import numpy as np
import pytest
import torch

import _ops_ref as ref

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def dg():
    import moe_grouped_gemm_03_b200 as dg

    return dg


def at_once(*works):
    """Runs each callable on a host thread of its own and CUDA stream, all begun together; raises the first error."""
    torch.cuda.synchronize()
    errors, begin = [], threading.Barrier(len(works))

    def body(work):
        try:
            stream = torch.cuda.Stream()
            begin.wait()
            with torch.cuda.stream(stream):
                work(stream.cuda_stream)
            stream.synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=body, args=(w,)) for w in works]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    if errors:
        raise errors[0]


class NormGradient:
    """residual_rms_norm_backward with a gate [H] on T rows, by its C entry point (ctypes leaves the interpreter's lock)."""

    def __init__(self, dg, T, H, seed):
        self.dg, self.T, self.H = dg, T, H
        g = torch.Generator(device="cuda").manual_seed(seed)
        r = lambda *s, dtype=BF16: torch.randn(*s, device="cuda", generator=g).to(dtype)  # noqa: E731
        self.inputs = dict(d_x_out=r(T, H), d_out=r(T, H), x_out=r(T, H), y=r(T, H), weight=r(H), weight_post=r(H), gate=r(H),
                           rstd=torch.ones(T, device="cuda"), rstd_post=torch.ones(T, device="cuda"))
        self.d_x, self.d_y = torch.zeros_like(self.inputs["y"]), torch.zeros_like(self.inputs["y"])
        self.d_w, self.d_wp, self.d_gate = torch.zeros(3, H, device="cuda")

    def outputs(self):
        return [self.d_x, self.d_y, self.d_w, self.d_wp, self.d_gate]

    def __call__(self, stream):
        p = {k: v.data_ptr() for k, v in self.inputs.items()}
        rc = self.dg.lib().dg_residual_rms_norm_backward(
            p["d_x_out"], p["d_out"], p["x_out"], 0, p["y"], 0, p["weight"], p["weight_post"], p["gate"], 1, 0, 1.0, p["rstd"],
            p["rstd_post"], self.T, self.H, self.d_x.data_ptr(), self.d_y.data_ptr(), self.d_w.data_ptr(), self.d_wp.data_ptr(),
            self.d_gate.data_ptr(), stream)
        assert rc == 0, (self.H, rc, self.dg.last_error())


class Sort:
    """moe_sort_nopad of n tokens over G groups by its C entry point."""

    def __init__(self, dg, n, G, seed):
        self.dg, self.n, self.G = dg, n, G
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.ids = torch.randint(-1, G, (n, 4), device="cuda", generator=g, dtype=torch.int32)
        self.rows, self.counts = torch.zeros_like(self.ids), torch.zeros(G, dtype=torch.int32, device="cuda")

    def outputs(self):
        return [self.rows, self.counts]

    def __call__(self, stream):
        rc = self.dg.lib().dg_moe_sort_nopad(self.ids.data_ptr(), 4, self.n, 4, self.G, self.rows.data_ptr(),
                                             self.counts.data_ptr(), stream)
        assert rc == 0, (self.G, rc, self.dg.last_error())


def alone(calls):
    """What each call gives by itself; its outputs are zeros afterwards."""
    want = []
    for c in calls:
        c(torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        want.append([v.clone() for v in c.outputs()])
        for v in c.outputs():
            v.zero_()
    return want


def same(calls, want):
    return all(torch.equal(a, b) for c, w in zip(calls, want) for a, b in zip(c.outputs(), w))


def pairs(dg):
    """Calls of one kernel that want different amounts of shared memory."""
    return {"norm": [NormGradient(dg, 600, 7168, 1), NormGradient(dg, 600, 4096, 2)],
            "sort": [Sort(dg, 8000, 1024, 3), Sort(dg, 8000, 400, 4)]}


@pytest.mark.parametrize("kind", ["norm", "sort"])
def test_two_threads_with_different_sizes(dg, kind):
    """A kernel's shared memory is not what another thread's smaller call of it left: no valid call is refused."""
    calls = pairs(dg)[kind]
    want = alone(calls)

    def many(call):
        def work(stream):
            for _ in range(10000):
                call(stream)

        return work

    at_once(*[many(c) for c in calls])
    assert same(calls, want)
    dg.check_device_error()


@pytest.mark.parametrize("kind", ["norm", "sort"])
def test_one_graph_with_different_sizes(dg, kind):
    """The wide call first, the narrow one behind it, both in one graph."""
    calls = pairs(dg)[kind]
    want = alone(calls)
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=stream):
        for c in calls:
            c(torch.cuda.current_stream().cuda_stream)
    for _ in range(2):
        for c in calls:
            for v in c.outputs():
                v.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert same(calls, want)
    dg.check_device_error()


def test_first_calls_of_a_process_from_many_threads(dg):
    """Eight host threads make their first call of the library in a new process at once."""
    code = """
import threading, torch
import moe_grouped_gemm_03_b200 as dg
x = torch.randn(64, 512, device="cuda"); w = torch.ones(512, device="cuda")
outs = [torch.zeros_like(x) for _ in range(8)]
torch.cuda.synchronize()
begin, bad, L = threading.Barrier(8), [], dg.lib()
def work(o):
    begin.wait()
    rc = L.dg_rms_norm(x.data_ptr(), 1, w.data_ptr(), 1, 1e-6, 64, 512, o.data_ptr(), 1, None, None, None)
    if rc: bad.append(dg.last_error())
ts = [threading.Thread(target=work, args=(o,)) for o in outs]
[t.start() for t in ts]; [t.join() for t in ts]
torch.cuda.synchronize()
assert not bad, bad
assert all(torch.equal(o, outs[0]) for o in outs) and float(outs[0].abs().sum()) > 0
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    done = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0, done.stderr[-2000:]


def test_sorts_of_threads_against_the_plain_form(dg):
    """(what `alone` compares with is right)"""
    call = Sort(dg, 500, 1024, 5)
    call(torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    rows, counts, _ = ref.sort(call.ids.cpu().numpy(), "nopad", call.G)
    assert (call.rows.cpu().numpy() == rows).all() and (call.counts.cpu().numpy() == np.asarray(counts)).all()


SORT_UNDER_CAP = """
import sys, torch
import moe_grouped_gemm_03_b200 as dg
(T, k, G), kind, caps = map(int, sys.argv[1:4]), getattr(torch, sys.argv[4]), map(int, sys.argv[5:])
g = torch.Generator(device="cuda").manual_seed(T)
ids = torch.randint(-1, G, (T, k), device="cuda", generator=g).to(kind)
def run():
    rows, counts = torch.full((T, k), -9, dtype=torch.int32, device="cuda"), torch.full((G,), -9, dtype=torch.int32, device="cuda")
    dg.moe_sort_nopad(ids, rows, counts)
    m, n = torch.full((dg.get_m_total_bound(T * k, G),), -9, dtype=torch.int32, device="cuda"), torch.empty_like(counts)
    at = torch.empty_like(rows)
    dg.moe_sort_contiguous(ids, at, m, n)
    torch.cuda.synchronize()
    return rows, counts, at, m, n
want = run()
for cap in caps:
    dg.set_num_sms(cap)
    assert all(torch.equal(a, b) for a, b in zip(want, run())), cap
dg.check_device_error()
flat, (rows, counts) = ids.view(-1).long(), want[:2]
order = torch.argsort(torch.where(flat < 0, G, flat), stable=True)[: int(counts.sum())]
assert torch.equal(rows.view(-1)[order], torch.arange(len(order), device="cuda", dtype=torch.int32)) and int((rows >= 0).sum()) == len(order)
"""


@pytest.mark.parametrize("T,k,G,kind", [(20000, 8, 1024, "int64"), (1100, 1, 5, "int32")])
def test_sort_takes_no_more_sms_than_the_cap(T, k, G, kind):
    """The plan that DG_DEBUG=1 prints has a cluster that fits under set_num_sms; the rows do not depend on it."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    clusters = {16: 16, 15: 8, 8: 8, 7: 1, 1: 1, 0: 16}
    done = subprocess.run([sys.executable, "-c", SORT_UNDER_CAP, *map(str, (T, k, G, kind, *clusters))], cwd=root,
                          capture_output=True, text=True, timeout=300, env=dict(os.environ, DG_DEBUG="1"))
    assert done.returncode == 0, done.stderr[-2000:]
    plans = [int(line.rsplit("ctas=", 1)[1]) for line in done.stderr.splitlines() if line.startswith("[dg] sort")]
    assert plans == [n for n in (16, *clusters.values()) for _ in range(2)]  # (both layouts)


@pytest.mark.parametrize("cap", [1, 5])
def test_norm_gradients_under_a_cap(dg, cap):
    """Rows do not depend on set_num_sms; the parameters' gradients do by the order of their sums, over 600 rows."""
    call = NormGradient(dg, 600, 1024, 6)
    want = alone([call])[0]
    dg.set_num_sms(cap)
    try:
        call(torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
    finally:
        dg.set_num_sms(0)
    d_x, d_y, d_w, d_wp, d_gate = call.outputs()
    assert torch.equal(d_x, want[0]) and torch.equal(d_y, want[1])
    i = call.inputs
    x, y, w, wp, gate, dxo, do = (i[n].double() for n in ("x_out", "y", "weight", "weight_post", "gate", "d_x_out", "d_out"))
    got = ref.norm_backward(*(i[n] for n in ("d_x_out", "d_out", "x_out", "y", "weight", "weight_post", "gate")), 1.0, i["rstd"],
                            i["rstd_post"])
    e = (w * do).abs()
    sx = dxo.abs() + e + x.abs() * (e * x.abs()).mean(1, keepdim=True)  # size of the terms of d_x (r = 1)
    # chains of at most 600 additions for a parameter and 2^6 for a row: below 2^10 roundings of the terms' sizes
    for out, name, size in ((d_w, "d_w", do.abs() * x.abs()), (d_wp, "d_w_post", gate.abs() * sx * y.abs()),
                            (d_gate, "d_gate", wp.abs() * sx * y.abs())):
        assert bool(((out.double().cpu() - got[name]).abs() <= size.sum(0).cpu() * 2.0 ** -14).all()), name
    dg.check_device_error()


def test_swiglu_clips_counts_and_records_nothing(dg):
    """As documented: counts out of range are clipped to the rows there are, and the error word stays clear."""
    gu = torch.randn(12, 256, device="cuda").to(BF16)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    for shape, kw, owned in (((12, 256), dict(counts=i32(-3, 5, 100)), range(12)), ((12, 256), dict(counts=i32(-3, 5)), range(5)),
                             ((3, 4, 256), dict(masked_m=i32(-1, 9, 2)), [4, 5, 6, 7, 8, 9]),
                             ((12, 256), dict(m_indices=i32(*[-1, 2, 1 << 30] * 4)), [t for t in range(12) if t % 3])):
        out = torch.full((*shape[:-1], 128), -7.5, dtype=BF16, device="cuda")
        dg.swiglu(gu.view(shape), out, **kw)
        dg.check_device_error()
        assert sorted(set((out.view(12, 128) != -7.5).any(1).nonzero()[:, 0].tolist())) == list(owned)


def test_a_launch_that_waits_leaves_the_interpreter_to_other_threads(dg):
    """Behind a kernel of half a second the queue of launches fills up and a call waits in it; other Python threads go on."""
    x, w, out = torch.randn(8, 128, device="cuda"), torch.ones(128, device="cuda"), torch.empty(8, 128, device="cuda")
    dg.rms_norm(x, w, out)
    torch.cuda._sleep(1000)
    torch.cuda.synchronize()
    done, gaps, waits = threading.Event(), [0.0], [0.0]

    def tick():
        last = time.perf_counter()
        while not done.is_set():
            time.sleep(1e-3)
            now = time.perf_counter()
            gaps.append(now - last)
            last = now

    thread = threading.Thread(target=tick)
    thread.start()
    try:
        torch.cuda._sleep(1_000_000_000)  # (cycles)
        begin = time.perf_counter()
        while time.perf_counter() - begin < 0.2 and max(waits) < 0.1 and len(waits) < 50_000:
            t = time.perf_counter()
            dg.rms_norm(x, w, out)
            waits.append(time.perf_counter() - t)
    finally:
        done.set()
        thread.join()
        torch.cuda.synchronize()
    assert max(waits) > 0.1, "no launch had to wait: this shows nothing"
    assert max(gaps) < max(waits) / 2, (max(gaps), max(waits))
