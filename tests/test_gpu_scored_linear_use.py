"""The scored router and the dense product as a program uses them together: chains of
dependent launches, several streams and graphs at once, a first call under capture, another
stream than the tensors' own, buffers larger than the batch, and what the binding refuses."""
import os
import subprocess
import sys
from types import SimpleNamespace

import numpy as np
import pytest

from tests import scored_ref as ref
from tests.test_gpu_linear import check as check_linear
from tests.test_gpu_route_scored import random_case

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _ws():
    import torch
    import bit_routed_expert_fp32_b200 as moe
    ws = torch.empty(4096, dtype=torch.uint8, device="cuda")
    moe.moe_workspace_init(ws)
    return ws


@pytest.mark.parametrize("T", [1, 6, 40, 200, 700])
def test_a_chain_of_dependent_products_equals_the_same_steps_apart(T):
    """Each launch may begin before the one that writes its input has ended: forty of them in a
    row, against the same ones with the GPU waited for in between."""
    import torch
    import bit_routed_expert_fp32_b200 as moe
    ws = _ws()
    g = torch.Generator(device="cuda").manual_seed(T)
    K = 512
    w = [(torch.randn(K, K, generator=g, device="cuda") * (1.2 / K ** 0.5)).to(torch.bfloat16) for _ in range(4)]
    x = torch.randn(T, K, generator=g, device="cuda").to(torch.bfloat16)

    def steps(wait):
        a, b = x.clone(), torch.empty_like(x)
        for i in range(40):
            moe.moe_linear(a, w[i % 4], b, ws, residual=x if i % 3 else None, act=i % 5)
            if wait:
                torch.cuda.synchronize()
            a, b = b, a
        torch.cuda.synchronize()
        return a

    apart, chained = steps(True), steps(False)
    assert torch.isfinite(apart).all() and torch.equal(apart, chained)
    graph, out = torch.cuda.CUDAGraph(), {}
    with torch.cuda.graph(graph):
        a, b = x.clone(), torch.empty_like(x)
        for i in range(40):
            moe.moe_linear(a, w[i % 4], b, ws, residual=x if i % 3 else None, act=i % 5)
            a, b = b, a
        out["y"] = a
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(apart, out["y"])


def test_streams_with_every_kernel_at_once():
    """Products and routings of all sizes on four streams at once (their tensor-memory and
    cluster needs meet on the same SMs), every result as when run alone."""
    import torch
    import bit_routed_expert_fp32_b200 as moe
    g = torch.Generator(device="cuda").manual_seed(4)

    def rnd(*s):
        return (torch.randn(*s, generator=g, device="cuda") / s[-1] ** 0.5).to(torch.bfloat16)

    jobs = []
    for T, K, N, act in [(1, 1024, 512, 5), (20, 2048, 640, 2), (130, 1024, 700, 3), (600, 512, 1500, 0), (2000, 256, 900, 5)]:
        x, w = rnd(T, K) * 30, rnd(2 * N if act == 5 else N, K)
        jobs.append(lambda y, ws, x=x, w=w, act=act: moe.moe_linear(x, w, y["y"], ws["l"], act=act))
        jobs[-1].out = {"y": (T, N)}
    for T, Hd, E in [(3, 512, 64), (30, 1024, 128), (100, 1024, 72), (3000, 512, 256)]:
        cfg = SimpleNamespace(H=Hd, I=64, E=E, k=4, S=0)
        x, wr = rnd(T, Hd) * 20, torch.randn(E, Hd, generator=g, device="cuda") * 0.02
        router = moe.Router(score=moe.SCORE_SIGMOID, n_groups=4, top_groups=2, group_top=2)
        jobs.append(lambda y, ws, cfg=cfg, x=x, wr=wr, router=router, T=T:
                    moe.moe_route_scored(cfg, router, T, x, wr, None, None, y, ws["r"]))
        jobs[-1].out = None
        jobs[-1].cfg = (cfg, T)

    def buffers(job):
        ws = {"l": _ws()}
        if job.out:
            return {n: torch.zeros(s, dtype=torch.bfloat16, device="cuda") for n, s in job.out.items()}, ws
        cfg, T = job.cfg
        ws["r"] = torch.empty(moe.moe_workspace_size(cfg, T), dtype=torch.uint8, device="cuda")
        moe.moe_workspace_init(ws["r"])
        return moe.alloc_routing(cfg, T), ws

    alone = []
    for job in jobs:
        y, ws = buffers(job)
        job(y, ws)
        torch.cuda.synchronize()
        alone.append(y)
    streams = [torch.cuda.Stream() for _ in range(4)]
    mine = [[buffers(job) for job in jobs] for _ in streams]
    torch.cuda.synchronize()
    for rep in range(15):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                for j in range(len(jobs)):
                    k = (j + 3 * i + rep) % len(jobs)
                    jobs[k](*mine[i][k])
    torch.cuda.synchronize()
    for m in mine:
        for (y, ws), want in zip(m, alone):
            for n in want:
                assert torch.equal(y[n], want[n]), n
            for w in ws.values():
                assert moe.moe_get_error(w) == (0, 0)


FIRST_CALL = """
import sys, torch
sys.path.insert(0, {root!r})
from types import SimpleNamespace
import bit_routed_expert_fp32_b200 as moe
T = {T}
x = torch.randn(T, 512, device="cuda").to(torch.bfloat16)
w = torch.randn(256, 512, device="cuda").to(torch.bfloat16)
wr = torch.randn(64, 512, device="cuda") * 0.02
y = torch.zeros(T, 256, dtype=torch.bfloat16, device="cuda")
cfg = SimpleNamespace(H=512, I=64, E=64, k=4, S=0)
ws = torch.empty(moe.moe_workspace_size(cfg, T), dtype=torch.uint8, device="cuda")
moe.moe_workspace_init(ws)
rt = moe.alloc_routing(cfg, T)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    moe.moe_route_scored(cfg, moe.Router(), T, x, wr, None, None, rt, ws)
    moe.moe_linear(x, w, y, ws)
g.replay()
torch.cuda.synchronize()
y2, rt2 = torch.zeros_like(y), moe.alloc_routing(cfg, T)
moe.moe_route_scored(cfg, moe.Router(), T, x, wr, None, None, rt2, ws)
moe.moe_linear(x, w, y2, ws)
torch.cuda.synchronize()
assert torch.equal(y, y2) and all(torch.equal(rt[n], rt2[n]) for n in rt)
assert moe.moe_get_error(ws) == (0, 0)
print("first call captured")
"""


@pytest.mark.parametrize("T", [1, 20, 300, 1500])
def test_the_first_call_of_a_process_may_be_captured(T):
    r = subprocess.run([sys.executable, "-c", FIRST_CALL.format(root=ROOT, T=T)], capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "first call captured" in r.stdout, r.stderr[-2000:]


@pytest.mark.parametrize("T,most", [(1, 4), (10, 30), (64, 65), (70, 300)])
def test_buffers_larger_than_the_batch_keep_the_rest(T, most):
    import torch
    import bit_routed_expert_fp32_b200 as moe
    E, k = 32, 3
    x, wr, _, _, L = random_case(T, 256, E, 9, False, False, k, sigmoid=True)
    cfg = SimpleNamespace(H=256, I=64, E=E, k=k, S=0)
    ws = torch.empty(moe.moe_workspace_size(cfg, most), dtype=torch.uint8, device="cuda")
    moe.moe_workspace_init(ws)
    rt = moe.alloc_routing(cfg, most)
    for t in rt.values():
        t.fill_(-5)
    moe.moe_route_scored(cfg, moe.Router(score=moe.SCORE_SIGMOID), T, moe.bf16_to_device(x),
                         torch.from_numpy(wr).cuda(), None, None, rt, ws)
    torch.cuda.synchronize()
    ids, _ = ref.select(L, None, k, sigmoid=True)
    np.testing.assert_array_equal(rt["topk_ids"][:T].cpu().numpy(), ids)
    for n in ("topk_ids", "topk_w"):
        assert (rt[n][T:] == -5).all(), n
    for n in ("perm", "inv_perm"):
        assert (rt[n][T * k:] == -5).all(), n
    assert int(rt["offsets"][E]) == T * k


def test_one_workspace_serves_routings_of_changing_sizes_and_two_graphs():
    """Counters and histograms left by one call do not reach the next, whatever its size."""
    import torch
    import bit_routed_expert_fp32_b200 as moe
    E, k = 64, 4
    kw = dict(sigmoid=True)
    cfg = SimpleNamespace(H=320, I=64, E=E, k=k, S=0)
    sizes = [1, 200, 9, 1000, 64, 65, 3, 700, 8]
    cases = [random_case(T, 320, E, 40 + T, False, False, k, **kw) for T in sizes]
    ws = torch.empty(moe.moe_workspace_size(cfg, max(sizes)), dtype=torch.uint8, device="cuda")
    moe.moe_workspace_init(ws)
    router = moe.Router(score=moe.SCORE_SIGMOID)
    bufs = [(moe.bf16_to_device(c[0]), torch.from_numpy(c[1]).cuda(), moe.alloc_routing(cfg, T))
            for T, c in zip(sizes, cases)]

    def go(i):
        x, wr, rt = bufs[i]
        moe.moe_route_scored(cfg, router, sizes[i], x, wr, None, None, rt, ws)

    def right(i):
        ids, _ = ref.select(cases[i][4], None, k, **kw)
        np.testing.assert_array_equal(bufs[i][2]["topk_ids"].cpu().numpy(), ids)
        for name, want in zip(("counts", "offsets", "perm", "inv_perm"), ref.permute(ids, E)):
            np.testing.assert_array_equal(bufs[i][2][name].cpu().numpy(), want, err_msg=name)

    for i in range(len(sizes)):
        go(i)
    torch.cuda.synchronize()
    for i in range(len(sizes)):
        right(i)
    graphs = []
    for half in (range(0, len(sizes), 2), range(1, len(sizes), 2)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for i in half:
                go(i)
        graphs.append(g)
    for _ in range(3):
        for _, _, rt in bufs:
            for t in rt.values():
                t.zero_()
        for g in (graphs[1], graphs[0], graphs[1]):
            g.replay()
        torch.cuda.synchronize()
        for i in range(len(sizes)):
            right(i)
    assert moe.moe_get_error(ws) == (0, 0)


def test_the_binding_names_what_is_wrong():
    import torch
    import bit_routed_expert_fp32_b200 as moe
    ws = _ws()
    bf, dev = torch.bfloat16, "cuda"
    x = torch.zeros((4, 64), dtype=bf, device=dev)
    w = torch.zeros((32, 64), dtype=bf, device=dev)
    y = torch.full((4, 32), 3.0, dtype=bf, device=dev)
    bad = [dict(x=x.float()), dict(x=x[0]), dict(x=x.cpu()), dict(w=w.half()), dict(w=w[:, :56]), dict(y=y[:3]),
           dict(y=y.half()), dict(y=y.float()), dict(y=torch.zeros((32, 4), dtype=bf, device=dev).t()),
           dict(x=torch.zeros((64, 4), dtype=bf, device=dev).t()), dict(ws=ws.cpu()),
           dict(bias=torch.zeros(31, dtype=bf, device=dev)), dict(bias=torch.zeros(32, device=dev)),
           dict(bias=torch.zeros(64, dtype=bf, device=dev)[::2]),
           dict(residual=torch.zeros((4, 32), dtype=torch.float16, device=dev)),
           dict(residual=torch.zeros((4, 31), dtype=bf, device=dev)), dict(act=moe.ACT_SWIGLU),
           dict(w=w[:31], act=moe.ACT_SWIGLU)]
    for kw in bad:
        a = dict(x=x, w=w, y=y, ws=ws)
        a.update(kw)
        with pytest.raises(ValueError):
            moe.moe_linear(**a)
    for kw in (dict(act=9), dict(ws=ws[:1024]), dict(x=torch.zeros((4, 68), dtype=bf, device=dev)[:, :64]),
               dict(x=x[:1].expand(4, 64)), dict(y=x[:, :32])):
        a = dict(x=x, w=w, y=y, ws=ws)
        a.update(kw)
        with pytest.raises(moe.MoeError):
            moe.moe_linear(**a)
    torch.cuda.synchronize()
    assert (y == 3).all()                      # nothing was written
    moe.moe_linear(x, w, y, ws)
    assert (y == 0).all()


def test_on_a_stream_that_is_not_the_tensors_own():
    import torch
    import bit_routed_expert_fp32_b200 as moe
    ws = _ws()
    x = torch.randn(50, 256, device="cuda").to(torch.float16)
    w = torch.randn(100, 256, device="cuda").to(torch.float16) / 16
    y = torch.zeros(50, 100, dtype=torch.float16, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    moe.moe_linear(x, w, y, ws, act=moe.ACT_SILU, stream=s)
    s.synchronize()
    check_linear(y, x, w, None, None, moe.ACT_SILU)


def test_host_threads_calling_at_once():
    """Calls whose kernels ask for different amounts of shared memory, from two host threads."""
    import threading
    import torch
    import bit_routed_expert_fp32_b200 as moe
    K, N, E = 512, 384, 48
    w = (torch.randn(N, K, device="cuda") / K ** 0.5).to(torch.bfloat16)
    wr = torch.randn(E, K, device="cuda") * 0.02
    cfg = SimpleNamespace(H=K, I=64, E=E, k=4, S=0)
    torch.cuda.synchronize()
    got, failed = {}, []

    def work(me, sizes):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                jobs = []
                for T in sizes:
                    x = torch.randn(T, K, device="cuda").to(torch.bfloat16)
                    ws = torch.empty(moe.moe_workspace_size(cfg, T), dtype=torch.uint8, device="cuda")
                    moe.moe_workspace_init(ws)
                    jobs.append((T, x, torch.empty(T, N, dtype=torch.bfloat16, device="cuda"), ws, moe.alloc_routing(cfg, T)))
                for _ in range(200):
                    for T, x, y, ws, rt in jobs:
                        moe.moe_linear(x, w, y, ws)
                        moe.moe_route_scored(cfg, moe.Router(), T, x, wr, None, None, rt, ws)
                s.synchronize()
                got[me] = jobs
        except Exception as e:                                # noqa: BLE001 - shown by the assert below
            failed.append(e)

    threads = [threading.Thread(target=work, args=(i, sizes)) for i, sizes in enumerate([(12, 140, 700), (40, 90, 2000)])]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
    for jobs in got.values():
        for T, x, y, ws, rt in jobs:
            y2, rt2 = torch.empty_like(y), moe.alloc_routing(cfg, T)
            assert moe.moe_get_error(ws) == (0, 0)
            moe.moe_linear(x, w, y2, ws)
            moe.moe_route_scored(cfg, moe.Router(), T, x, wr, None, None, rt2, ws)
            torch.cuda.synchronize()
            assert torch.equal(y, y2) and all(torch.equal(rt[n], rt2[n]) for n in rt)


def test_the_router_binding_refuses_tensors_that_do_not_fit():
    import torch
    import bit_routed_expert_fp32_b200 as moe
    cfg = SimpleNamespace(H=128, I=64, E=16, k=2, S=0)
    ws = torch.empty(moe.moe_workspace_size(cfg, 8), dtype=torch.uint8, device="cuda")
    moe.moe_workspace_init(ws)
    rt = moe.alloc_routing(cfg, 8)
    x = torch.zeros((8, 128), dtype=torch.bfloat16, device="cuda")
    w, b = torch.zeros((16, 128), device="cuda"), torch.zeros(16, device="cuda")
    for kw in (dict(x=x.half()), dict(x=x.cpu()), dict(x=x[:7]), dict(x=x[:, :64]), dict(w=w.double()), dict(w=w.cpu()),
               dict(w=w[:15]), dict(w=w.t()), dict(b=b[:15]), dict(b=b.double()), dict(bal=b.cpu()),
               dict(bal=torch.zeros(32, device="cuda")[::2]), dict(ws=ws.cpu())):
        a = dict(x=x, w=w, b=b, bal=b, ws=ws)
        a.update(kw)
        with pytest.raises(ValueError):
            moe.moe_route_scored(cfg, moe.Router(), 8, a["x"], a["w"], a["b"], a["bal"], rt, a["ws"])
    moe.moe_route_scored(cfg, moe.Router(), 8, x, w, b, b, rt, ws)
    torch.cuda.synchronize()
    assert rt["topk_ids"].tolist() == [[0, 1]] * 8 and moe.moe_get_error(ws) == (0, 0)
