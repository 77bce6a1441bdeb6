"""The order of kernels that start before their predecessors have ended (programmatic dependent
launch).  The decode pass pulls its token rows into L1 before it waits, which is right only if
whatever wrote them has ended by the time it can start: a kernel of the scored router or of the
dense product releases the next one only after its own wait.  On the CPU that is read off the
sources; on the GPU layers follow one another without a wait in between, each on rows that a
product has just rewritten."""
import os
import re

import numpy as np
import pytest

import synth
from tests import harness as H

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "bit_routed_expert_fp32_b200", "csrc")


def kernels(name):
    """(name, body) of every __global__ function of a source file, comments removed."""
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
    out = []
    for m in re.finditer(r"__global__", text):
        start = text.index("{", m.end())
        depth, i = 1, start + 1
        while depth:
            depth += {"{": 1, "}": -1}.get(text[i], 0)
            i += 1
        names = [n for n in re.findall(r"(\w+)\s*\(", text[m.end():start]) if not n.startswith("__")]
        out.append((names[0], text[start:i]))
    return out


@pytest.mark.parametrize("name", ["route_scored.cu", "scored_logits.cu", "linear.cu"])
def test_a_kernel_releases_the_next_one_after_its_own_wait(name):
    found = kernels(name)
    assert found
    for kernel, body in found:
        assert body.count("griddep_wait();") == 1, kernel
        release = body.find("griddep_launch_dependents();")
        assert release > body.find("griddep_wait();"), f"{kernel} releases its dependents before it has waited"


def _layer(cfg, seed, T, width, max_tokens=None):
    import torch
    import bit_routed_expert_fp32_b200 as moe
    case = H.make_case(cfg, T=T)
    rng = np.random.default_rng(seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    shared = None
    if width:
        mk = lambda *s: (torch.randn(*s, generator=g, device="cuda") / s[1] ** 0.5).to(torch.bfloat16)   # noqa: E731
        shared = mk(2 * width, cfg.H), mk(cfg.H, width)
    router = moe.Router(score=moe.SCORE_SIGMOID, n_groups=4, top_groups=2, group_top=2, scale=1.5)
    return moe.MoeLayer(cfg, H.pack(case), case.layer.router_w, None, max_tokens or T, router=router,
                        balance=(rng.standard_normal(cfg.E) * 0.05).astype(np.float32), shared=shared)


@pytest.mark.gpu
@pytest.mark.parametrize("path", ["PATH_AUTO", "PATH_DECODE"])
@pytest.mark.parametrize("T", [1, 2, 4, 12, 40])
def test_a_layer_on_rows_that_a_product_has_just_rewritten(T, path):
    """The shared expert is a 3-bit one: it multiplies the token rows themselves, not the records
    that the router forms of them."""
    import torch
    import bit_routed_expert_fp32_b200 as moe
    cfg = synth.micro(T=T, H=256, E=16, k=4, I=128, S=1, formats="mixed", seed=61)
    lay = _layer(cfg, 3, T, None)
    g = torch.Generator(device="cuda").manual_seed(T)
    K = 8192                                             # the product takes far longer than a launch
    w = (torch.randn(cfg.H, K, generator=g, device="cuda") / K ** 0.5).to(torch.bfloat16)
    src = [torch.randn(T, K, generator=g, device="cuda").to(torch.bfloat16) for _ in range(30)]
    path = getattr(moe, path)

    def go(wait):
        x = torch.zeros(T, cfg.H, dtype=torch.bfloat16, device="cuda")
        ys = [torch.zeros_like(x) for _ in src]
        torch.cuda.synchronize()
        for a, y in zip(src, ys):
            for step in (lambda: moe.moe_linear(a, w, x, lay.ws), lambda: lay.route(x), lambda: lay.forward(x, y, path=path)):
                step()
                if wait:
                    torch.cuda.synchronize()
        torch.cuda.synchronize()
        return torch.stack(ys)

    apart, chained = go(True), go(False)
    assert moe.moe_get_error(lay.ws) == (0, 0)
    assert len({bytes(y.float().cpu().numpy().tobytes()) for y in apart}) == len(src)
    assert torch.equal(apart, chained)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 3, 6, 12, 50, 100])
def test_layers_one_after_the_other(T):
    """The first layer's last kernel is the product of its 16-bit shared expert; the next routes
    and runs on what it writes."""
    import torch
    import bit_routed_expert_fp32_b200 as moe
    cfg = synth.micro(T=T, H=256, E=16, k=4, I=128, S=1, formats="mixed", seed=63)
    one, two = _layer(cfg, 5, T, 1024), _layer(cfg, 6, T, 96)
    g = torch.Generator(device="cuda").manual_seed(T)
    xs = [torch.randn(T, cfg.H, generator=g, device="cuda").to(torch.bfloat16) for _ in range(20)]

    def go(wait):
        mid = torch.zeros_like(xs[0])
        ys = [torch.zeros_like(mid) for _ in xs]
        torch.cuda.synchronize()
        for x, y in zip(xs, ys):
            for lay, a, b in ((one, x, mid), (two, mid, y)):
                for step in (lambda: lay.route(a), lambda: lay.forward(a, b)):
                    step()
                    if wait:
                        torch.cuda.synchronize()
        torch.cuda.synchronize()
        return torch.stack(ys)

    apart, chained = go(True), go(False)
    assert moe.moe_get_error(one.ws) == (0, 0) and moe.moe_get_error(two.ws) == (0, 0)
    assert torch.isfinite(apart).all() and torch.equal(apart, chained)


@pytest.mark.parametrize("name,data", [("linear.cu", ""), ("route_scored.cu", "p.x"), ("operands.cuh", "p.x")])
def test_what_a_product_may_have_written_is_read_coherently(name, data):
    """The non-coherent loads are for data that is constant from the kernel's start on; a kernel
    started early may read rows, weights or biases that its predecessor is still writing then."""
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
    loads = [m.group(0) for m in re.finditer(r"(__ldg\s*\(|ld\.global\.nc)[^;]*;", text)]
    assert not [ld for ld in loads if data in ld]


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 3, 4, 20, 200, 700])
def test_every_input_of_a_product_written_by_the_one_before(T):
    """x, then the weights, the bias and the residual of a product are each the output of the product
    launched just before it, in buffers that earlier products of the chain have read."""
    import torch
    import bit_routed_expert_fp32_b200 as moe
    K = 256
    ws = torch.empty(4096, dtype=torch.uint8, device="cuda")
    moe.moe_workspace_init(ws)
    g = torch.Generator(device="cuda").manual_seed(T)

    def rnd(*s, std=1.0):
        return (torch.randn(*s, generator=g, device="cuda") * std).to(torch.bfloat16)

    srcs = [(rnd(T, 4096), rnd(K, 4096, std=1 / 64), rnd(K, 512, std=1 / 20), rnd(K, 512, std=1 / 20), rnd(1, 4096)) for _ in range(6)]

    def go(wait):
        x, r, y = (torch.zeros(T, K, dtype=torch.bfloat16, device="cuda") for _ in range(3))
        w, b = torch.zeros(K, K, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, K, dtype=torch.bfloat16, device="cuda")
        outs = []

        def product(a, m, out, **kw):
            moe.moe_linear(a, m, out, ws, **kw)
            if wait:
                torch.cuda.synchronize()

        def use():
            outs.append(torch.empty_like(y))
            product(x, w, outs[-1], bias=b[0], residual=r, act=moe.ACT_SILU)

        kept = [torch.empty(T, K, dtype=torch.bfloat16, device="cuda") for _ in range(30)]     # no allocation in between
        del kept
        torch.cuda.synchronize()
        for a, m, w1, w2, v in srcs:
            product(a, m, x)
            use()
            product(w1, w2, w)
            use()
            product(v, m, b)
            use()
            product(a, m, r, residual=x)
            use()
            product(a, m, r, residual=r, act=moe.ACT_RELU)                                    # in place
            use()
        torch.cuda.synchronize()
        return torch.stack(outs)

    apart, chained = go(True), go(False)
    assert moe.moe_get_error(ws) == (0, 0)
    assert torch.isfinite(apart).all() and len({o.float().cpu().numpy().tobytes() for o in apart[2:]}) == len(apart) - 2
    assert torch.equal(apart, chained)
