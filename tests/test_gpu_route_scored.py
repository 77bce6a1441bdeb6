"""moe_route_scored against the definition in 64 bits.

Most cases choose the logits exactly: token t is 1 in column t and 0 elsewhere, and column t
of the router holds the logits wanted for it, so that ties, saturated scores and switched-off
experts are decided by the definition alone.  Random tokens are drawn again while a logit
error of 8e-6 (some 2^-17, far above fp32's rounding of these sums) could change the choice."""
from types import SimpleNamespace

import numpy as np
import pytest

import synth
from tests import harness as H
from tests import scored_ref as ref

pytestmark = pytest.mark.gpu

NAMES = ("counts", "offsets", "perm", "inv_perm")


def _cfg(Hd, E, k):
    return SimpleNamespace(H=Hd, I=64, E=E, k=k, S=0)


def route(x, wr, bias, balance, k, **kw):
    """x: bf16 bits [T][H]; returns numpy routing arrays."""
    import torch
    import bit_routed_expert_fp32_b200 as moe
    T, E = x.shape[0], wr.shape[0]
    cfg = _cfg(x.shape[1], E, k)
    ws = torch.empty(moe.moe_workspace_size(cfg, T), dtype=torch.uint8, device="cuda")
    moe.moe_workspace_init(ws)
    rt = moe.alloc_routing(cfg, T)
    for t in rt.values():
        t.fill_(-77)
    dev = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a, np.float32)).cuda()   # noqa: E731
    sig = kw.pop("sigmoid", False)
    router = moe.Router(score=moe.SCORE_SIGMOID if sig else moe.SCORE_SOFTMAX, **kw)
    moe.moe_route_scored(cfg, router, T, moe.bf16_to_device(x), dev(wr), dev(bias), dev(balance), rt, ws)
    torch.cuda.synchronize()
    assert moe.moe_get_error(ws) == (0, 0)
    return {n: t.cpu().numpy() for n, t in rt.items()}


def check(rt, L, balance, k, E, rtol, **kw):
    ids, w = ref.select(L, balance, k, **kw)
    np.testing.assert_array_equal(rt["topk_ids"], ids)
    for name, want in zip(NAMES, ref.permute(ids, E)):
        np.testing.assert_array_equal(rt[name], want, err_msg=name)
    err = np.abs(rt["topk_w"] - w)
    assert (err <= rtol * np.abs(w) + 1e-45).all(), (err.max(), np.argwhere(err > rtol * np.abs(w) + 1e-45)[:4])


def exact_case(L):
    """Tokens and router whose logits are L [T][E] (fp32 values), T <= hidden."""
    T, E = L.shape
    Hd = max(64, (T + 63) // 64 * 64)
    x = np.zeros((T, Hd), np.uint16)
    x[np.arange(T), np.arange(T)] = 0x3F80                   # bf16 1.0
    wr = np.zeros((E, Hd), np.float32)
    wr[:, :T] = L.T
    return x, wr


# weights: one rounding to fp32 (2^-24) of an fp64 value that is off by far less
W_RTOL = 2.0 ** -23

GROUPS = [(8, 2, 1, 1, 1), (8, 2, 4, 2, 1), (24, 5, 3, 2, 2), (60, 12, 6, 5, 2), (72, 7, 1, 1, 2), (160, 6, 8, 3, 1),
          (250, 16, 25, 20, 2), (256, 8, 8, 4, 2), (256, 8, 32, 31, 2), (256, 16, 32, 2, 1), (256, 1, 4, 4, 2), (1, 1, 1, 1, 1),
          (256, 16, 16, 1, 2)]


@pytest.mark.parametrize("T", [1, 8, 9, 17, 33, 64, 65, 200])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("E,k,G,tg,gt", GROUPS)
def test_ties_saturation_and_groups(E, k, G, tg, gt, sigmoid, T):
    """Logits on a coarse grid (many ties), some so large that scores are 0 or 1.  Values that
    tie do so in any correct fp64: the grid has no L and -L (whose sigmoids add up to 1), and
    where a group's score is a sum of two, the balance is one value per group."""
    rng = np.random.default_rng(E * 1000 + T)
    L = (rng.integers(-8, 9, (T, E)) / 2 + 0.1484375).astype(np.float32)
    far = rng.random((T, E)) < 0.05
    L = np.where(far, rng.choice([-1e4, -60.0, 60.0, 1e4], (T, E)), L).astype(np.float32)
    L[0] = 1.25                                              # every expert ties
    balance = None
    if T % 2:
        balance = np.repeat(rng.integers(-3, 4, G), E // G) if gt == 2 else rng.integers(-3, 4, E)
        balance = balance.astype(np.float32) / 16
    kw = dict(sigmoid=sigmoid, n_groups=G, top_groups=tg, group_top=gt, renormalise=bool(T % 3), scale=2.5)
    x, wr = exact_case(L)
    check(route(x, wr, None, balance, k, **kw), L, balance, k, E, W_RTOL, **kw)


@pytest.mark.parametrize("T", [3, 100])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_switched_off_experts_and_odd_balance_values(sigmoid, T):
    """-infinity switches an expert off; where fewer than k are left the lowest ids fill up;
    whole groups off; NaN counts as -infinity; +infinity forces an expert."""
    rng = np.random.default_rng(5)
    E, k = 32, 6
    L = rng.standard_normal((T, E)).astype(np.float32)
    L = np.round(L * 1024) / 1024
    x, wr = exact_case(L)
    off = np.zeros(E, np.float32)
    off[::2] = -np.inf
    most = np.full(E, -np.inf, np.float32)
    most[[3, 17, 30]] = 0.25                                 # three experts left for six slots
    allof = np.full(E, -np.inf, np.float32)
    odd = np.zeros(E, np.float32)
    odd[4], odd[9], odd[20] = np.nan, np.inf, -np.inf
    low = np.full(E, np.finfo(np.float32).min, np.float32)   # a mask of the lowest value
    low[[1, 2, 8, 9, 10, 11, 25]] = 0
    for bal in (off, most, allof, odd, low):
        for G, tg, gt in ((1, 1, 1), (4, 2, 1), (4, 2, 2), (8, 3, 2)):
            kw = dict(sigmoid=sigmoid, n_groups=G, top_groups=tg, group_top=gt)
            check(route(x, wr, None, bal, k, **kw), L, bal, k, E, W_RTOL, **kw)


@pytest.mark.parametrize("T", [2, 70])
def test_vanishing_scores(T):
    """Sigmoid scores that are zero even in 64 bits give zero weights, not NaN."""
    L = np.full((T, 16), -2000.0, np.float32)
    L[1, 3] = 1.0
    x, wr = exact_case(L)
    kw = dict(sigmoid=True, scale=3.0)
    rt = route(x, wr, None, None, 4, **kw)
    check(rt, L, None, 4, 16, W_RTOL, **kw)
    assert (rt["topk_w"][0] == 0).all() and rt["topk_w"][1, 0] == 3.0


def random_case(T, Hd, E, seed, bias, balance, k, **kw):
    """Random tokens and router; tokens whose choice is not decided are drawn again."""
    import torch
    rng = np.random.default_rng(seed)
    wr = (rng.standard_normal((E, Hd)) * 0.02).astype(np.float32)
    b = (rng.standard_normal(E) * 0.5).astype(np.float32) if bias else None
    bal = (rng.standard_normal(E) * (0.05 if kw.get("sigmoid") else 0.3 / E)).astype(np.float32) if balance else None
    gkw = {n: v for n, v in kw.items() if n in ("sigmoid", "n_groups", "top_groups", "group_top")}
    x = synth.f32_to_bf16_bits(rng.standard_normal((T, Hd)).astype(np.float32))
    wd = torch.from_numpy(wr).double().cuda()

    def logits():
        xd = torch.from_numpy(synth.bf16_bits_to_f32(x)).double().cuda()
        L = (xd @ wd.t()).cpu().numpy()
        return L if b is None else L + b.astype(np.float64)

    for _ in range(20):
        L = logits()
        bad = np.nonzero(~ref.decided(L, bal, 8e-6, k=k, **gkw))[0]
        if bad.size == 0:
            return x, wr, b, bal, L
        x[bad] = synth.f32_to_bf16_bits(rng.standard_normal((bad.size, Hd)).astype(np.float32))
    raise RuntimeError("could not remove near-ties")


@pytest.mark.parametrize("T", [1, 3, 8, 16, 31, 64, 65, 129, 257, 700, 2500, 5000])
@pytest.mark.parametrize("Hd,E,k,G,tg,gt,sigmoid", [(64, 8, 2, 4, 2, 1, True), (192, 60, 8, 6, 3, 2, False),
                                                    (1024, 256, 8, 8, 4, 2, True), (7168, 256, 8, 8, 4, 2, True),
                                                    (2240, 130, 5, 1, 1, 1, False), (8256, 24, 4, 3, 2, 1, False)])
def test_random_tokens(Hd, E, k, G, tg, gt, sigmoid, T):
    """Weights: the logits are fp32, |L| < 16 here (one rounding: 2^-21 at most), their sums
    carry some 2^-22 of the terms' size (|x w| sums in quadrature to about |L|); a weight
    moves by the logits' errors, relative to itself (two of them when renormalised)."""
    kw = dict(sigmoid=sigmoid, n_groups=G, top_groups=tg, group_top=gt, renormalise=T % 2 == 1, scale=2.5)
    x, wr, b, bal, L = random_case(T, Hd, E, T + Hd, T % 3 == 0, T % 4 != 1, k, **kw)
    check(route(x, wr, b, bal, k, **kw), L, bal, k, E, 2.0 ** -18, **kw)


def test_softmax_without_groups_agrees_with_moe_route():
    import torch
    import bit_routed_expert_fp32_b200 as moe
    for T in (5, 90):
        x, wr, b, _, L = random_case(T, 512, 64, 3, True, False, 6)
        cfg = _cfg(512, 64, 6)
        ws = torch.empty(moe.moe_workspace_size(cfg, T), dtype=torch.uint8, device="cuda")
        moe.moe_workspace_init(ws)
        rt = moe.alloc_routing(cfg, T)
        moe.moe_route(cfg, T, moe.bf16_to_device(x), torch.from_numpy(wr).cuda(), torch.from_numpy(b).cuda(), rt, ws)
        mine = route(x, wr, b, None, 6)
        for n in ("topk_ids",) + NAMES:
            np.testing.assert_array_equal(rt[n].cpu().numpy(), mine[n], err_msg=n)
        np.testing.assert_allclose(rt["topk_w"].cpu().numpy(), mine["topk_w"], rtol=1e-5)


def scored_layer(cfg, seed, T, shared_width=None):
    """A packed layer, its tokens, the reference routing, and a MoeLayer with a scored router
    (and a 16-bit shared expert)."""
    import torch
    import bit_routed_expert_fp32_b200 as moe
    kw = dict(sigmoid=True, n_groups=4, top_groups=2, group_top=2, renormalise=True, scale=1.5)
    case = H.make_case(cfg, T=T)
    rng = np.random.default_rng(seed)
    bal = (rng.standard_normal(cfg.E) * 0.05).astype(np.float32)
    wr = case.layer.router_w
    for _ in range(20):
        L = synth.bf16_bits_to_f32(case.x).astype(np.float64) @ wr.astype(np.float64).T
        bad = np.nonzero(~ref.decided(L, bal, 8e-6, sigmoid=True, n_groups=4, top_groups=2, group_top=2, k=cfg.k))[0]
        if bad.size == 0:
            break
        case.x[bad] = synth.f32_to_bf16_bits(rng.standard_normal((bad.size, cfg.H)).astype(np.float32))
    case.ids, case.gates = ref.select(L, bal, cfg.k, **kw)
    shared = None
    if shared_width:
        g = torch.Generator(device="cuda").manual_seed(seed)
        mk = lambda *s: (torch.randn(*s, generator=g, device="cuda") / s[1] ** 0.5).to(torch.bfloat16)   # noqa: E731
        shared = mk(2 * shared_width, cfg.H), mk(cfg.H, shared_width)
    router = moe.Router(score=moe.SCORE_SIGMOID, n_groups=4, top_groups=2, group_top=2, scale=1.5)
    lay = moe.MoeLayer(cfg, H.pack(case), wr, None, T, router=router, balance=bal, shared=shared)
    return case, lay


@pytest.mark.parametrize("T", [1, 6, 12, 50, 100])
def test_routed_layer_runs_on_the_scored_routing(T):
    import torch
    import bit_routed_expert_fp32_b200 as moe
    cfg = synth.micro(T=T, H=256, E=16, k=4, I=128, S=1, seed=31)
    case, lay = scored_layer(cfg, 7, T)
    y = lay(moe.bf16_to_device(case.x))
    torch.cuda.synchronize()
    assert moe.moe_get_error(lay.ws) == (0, 0)
    np.testing.assert_array_equal(lay.rt["topk_ids"].cpu().numpy(), case.ids)
    H.check_outputs(moe.bf16_to_host(y), H.oracle_outputs(case, list(range(T))))


@pytest.mark.parametrize("T", [1, 7, 40, 150])
@pytest.mark.parametrize("width", [128, 100])
def test_layer_with_a_16_bit_shared_expert(T, width):
    """Router, packed experts and the 16-bit shared expert on the routed sum, eagerly and
    replayed from a captured graph."""
    import torch
    import bit_routed_expert_fp32_b200 as moe
    cfg = synth.micro(T=T, H=256, E=16, k=4, I=128, S=0, seed=33)
    case, lay = scored_layer(cfg, 9, T, shared_width=width)
    x = moe.bf16_to_device(case.x)
    y = lay(x)
    torch.cuda.synchronize()
    assert moe.moe_get_error(lay.ws) == (0, 0)
    w_gu, w_dn = (w.double() for w in lay.shared)
    a = x.double() @ w_gu.t()
    h = (torch.nn.functional.silu(a[:, :width]) * a[:, width:]).to(torch.bfloat16).double()
    want = H.oracle_outputs(case, list(range(T))) + (h @ w_dn.t()).cpu().numpy()
    H.check_outputs(moe.bf16_to_host(y), want)
    y2 = torch.zeros_like(y)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lay.route(x)
        lay.forward(x, y2)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, y2)


def test_layer_refusals():
    import torch
    import bit_routed_expert_fp32_b200 as moe
    cfg = synth.micro(T=4, H=128, E=8, k=2, I=64, S=0, seed=35)
    case = H.make_case(cfg)
    packed = H.pack(case)
    w = torch.zeros((128, 128), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        moe.MoeLayer(cfg, packed, case.layer.router_w, None, 4, balance=np.zeros(8))
    with pytest.raises(ValueError):
        moe.MoeLayer(cfg, packed, case.layer.router_w, None, 4, shared=(w, w))
    lay = moe.MoeLayer(cfg, packed, case.layer.router_w, None, 4, shared=(w, w[:, :64]))
    x = moe.bf16_to_device(case.x)
    lay.route(x)
    with pytest.raises(ValueError):
        lay.forward(x, torch.empty((4, 128), device="cuda"), path=moe.OUT_F32)


def test_repeats_bit_for_bit():
    x, wr, b, bal, L = random_case(100, 1024, 256, 17, False, True, 8, sigmoid=True)
    for n in (4, 100):
        a, c = (route(x[:n], wr, b, bal, 8, sigmoid=True) for _ in range(2))
        for name in a:
            np.testing.assert_array_equal(a[name], c[name])


@pytest.mark.parametrize("T,E", [(150, 64), (6000, 256)])
def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_right(T, E):
    import torch
    import bit_routed_expert_fp32_b200 as moe
    kw = dict(sigmoid=True)
    x, wr, _, _, L = random_case(T, 640, E, 3, False, False, 4, **kw)
    cfg = _cfg(640, E, 4)
    ws = torch.empty(moe.moe_workspace_size(cfg, T), dtype=torch.uint8, device="cuda")
    moe.moe_workspace_init(ws)
    rt = moe.alloc_routing(cfg, T)
    router = moe.Router(score=moe.SCORE_SIGMOID)
    xd, wd = moe.bf16_to_device(x), torch.from_numpy(wr).cuda()
    moe.moe_workspace_set_test_stall(ws, 1000)
    moe.moe_route_scored(cfg, router, T, xd, wd, None, None, rt, ws)
    st, det = moe.moe_get_error(ws)
    assert moe.STATUS[st] == "MOE_ERR_TIMEOUT" and det & 0xF00 == moe.DETAIL["TEST_STALL"], (st, hex(det))
    moe.moe_workspace_set_test_stall(ws, 0)
    moe.moe_route_scored(cfg, router, T, xd, wd, None, None, rt, ws)
    torch.cuda.synchronize()
    assert moe.moe_get_error(ws) == (0, 0)
    check({n: t.cpu().numpy() for n, t in rt.items()}, L, None, 4, E, 2.0 ** -18, **kw)
