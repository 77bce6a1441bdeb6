"""What is measured of the two operators around the packed experts: the scored router
(moe_route_scored) and the dense matrix product with its epilogue (moe_linear).

A case is a dict of plain values.  `prepare` makes a case's inputs on the GPU, `run` makes
one pass over them, as elementary torch operations or (where `own` is true) through the
package; `exact` gives the same outputs in 64 bits.  Sizes are those of the layer the
package is built around (hidden 7168, 256 experts, top-8, expert width 2048; the tiny
hidden-256 layer) and generic ones.
"""
import math
from types import SimpleNamespace

import torch

own = False

# a token is drawn again while logits off by this much could change its choice of experts:
# the choice is then the same for every way of summing a logit in fp32
LOGIT_SLACK = 8e-6


def listed():
    return [
        # ---- routing ----------------------------------------------------------------
        # one token of a generating sequence, sigmoid scores, balance bias, 4 of 8 groups
        dict(name="route_T1_sigmoid_groups", op="route", T=1, H=7168, E=256, k=8, score="sigmoid", G=8, tg=4, gt=2,
             logit_bias=False, balance=True, renorm=True, scale=2.5),
        # sixteen sequences decoding together, softmax scores kept as they are, 3 of 8 groups of 20
        dict(name="route_T16_softmax_groups", op="route", T=16, H=5120, E=160, k=6, score="softmax", G=8, tg=3, gt=1,
             logit_bias=False, balance=False, renorm=False, scale=16.0),
        # a short ragged batch just above the few-token kernels, odd expert count, no groups
        dict(name="route_T130_sigmoid_plain", op="route", T=130, H=2048, E=72, k=7, score="sigmoid", G=1, tg=1, gt=1,
             logit_bias=True, balance=True, renorm=True, scale=1.0),
        # a prompt sweep of the full-size layer
        dict(name="route_T8192_sigmoid_groups", op="route", T=8192, H=7168, E=256, k=8, score="sigmoid", G=8, tg=4,
             gt=2, logit_bias=False, balance=True, renorm=True, scale=2.5),
        # the largest sweep, softmax with a logit bias and no groups
        dict(name="route_T16384_softmax", op="route", T=16384, H=7168, E=256, k=8, score="softmax", G=1, tg=1, gt=1,
             logit_bias=True, balance=True, renorm=True, scale=1.0),
        # ---- matrix products ----------------------------------------------------------
        # the unquantised shared expert of one token: gate/up with SwiGLU, then down onto the routed sum
        dict(name="linear_T1_swiglu", op="linear", T=1, K=7168, N=2048, act="swiglu", dtype="bf16", bias=False,
             residual="", pad=0),
        dict(name="linear_T1_down_residual", op="linear", T=1, K=2048, N=7168, act="none", dtype="bf16", bias=False,
             residual="f32", pad=0),
        # sixteen sequences decoding together, a biased projection with SiLU
        dict(name="linear_T16_silu_bias", op="linear", T=16, K=7168, N=4096, act="silu", dtype="bf16", bias=True,
             residual="", pad=0),
        # a ragged batch in fp16: odd N, K that is no multiple of a tile, padded rows
        dict(name="linear_T130_gelu_odd", op="linear", T=130, K=1992, N=4999, act="gelu", dtype="fp16", bias=True,
             residual="same", pad=24),
        # a prompt chunk, tanh-GELU and residual
        dict(name="linear_T1000_gelu_tanh", op="linear", T=1000, K=4096, N=4096, act="gelu_tanh", dtype="fp16",
             bias=True, residual="same", pad=0),
        # a prompt sweep through the unquantised shared expert
        dict(name="linear_T8192_swiglu", op="linear", T=8192, K=7168, N=2048, act="swiglu", dtype="bf16", bias=False,
             residual="", pad=0),
        dict(name="linear_T8192_down_residual", op="linear", T=8192, K=2048, N=7168, act="none", dtype="bf16",
             bias=False, residual="f32", pad=0),
    ]


ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh", "swiglu")
MAX_FLOPS = 2.0 * 8192 * 7168 * 4096


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    if rng.random() < 0.5:
        E = rng.choice([8, 24, 60, 64, 72, 96, 128, 160, 192, 250, 256, 256])
        G = rng.choice([g for g in range(1, 33) if E % g == 0 and E // g >= 2])
        tg = rng.randint(1, G)
        k = rng.randint(1, min(16, tg * (E // G)))
        return dict(op="route", T=_log_int(rng, 1, 16384), H=64 * _log_int(rng, 4, 112), E=E, k=k,
                    score=rng.choice(["softmax", "sigmoid"]), G=G, tg=tg, gt=rng.choice([1, 2]),
                    logit_bias=rng.random() < 0.3, balance=rng.random() < 0.7, renorm=rng.random() < 0.7,
                    scale=rng.choice([1.0, 2.5, 16.0]))
    act = rng.choice(ACTS)
    while True:
        T, K, N = _log_int(rng, 1, 8192), _log_int(rng, 64, 8192), _log_int(rng, 64, 8192)
        if 2.0 * T * K * N * (2 if act == "swiglu" else 1) <= MAX_FLOPS:
            break
    return dict(op="linear", T=T, K=K, N=N, act=act, dtype=rng.choice(["bf16", "fp16"]), bias=rng.random() < 0.5,
                residual=rng.choice(["", "same", "f32"]), pad=rng.choice([0, 0, 8, 24]))


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float16


def _up8(n):
    return (n + 7) // 8 * 8


# ---- inputs -------------------------------------------------------------------------

def _margins_ok(case, x, wr, lb, bal):
    """Per token: no logit error up to LOGIT_SLACK changes the kept groups, the chosen
    experts or their order."""
    G, tg, gt, k = case["G"], case["tg"], case["gt"], case["k"]
    L = x.double() @ wr.double().t()
    if lb is not None:
        L = L + lb.double()
    if case["score"] == "softmax":
        s = torch.exp(L - L.max(1, keepdim=True).values)
        s = s / s.sum(1, keepdim=True)
        err = 2 * LOGIT_SLACK * s
    else:
        s = 1 / (1 + torch.exp(-L))
        err = LOGIT_SLACK * s * (1 - s) + 1e-13
    c = s if bal is None else s + bal.double()
    T, E = c.shape
    ok = torch.ones(T, dtype=torch.bool, device=c.device)
    if tg < G:
        cg, eg = c.view(T, G, E // G), err.view(T, G, E // G)
        top = cg.sort(2, descending=True).values[:, :, :gt].sum(2)
        slack = gt * eg.max(2).values
        v, i = top.sort(1, descending=True)
        sl = slack.gather(1, i)
        ok &= v[:, tg - 1] - sl[:, :tg].max(1).values > v[:, tg] + sl[:, tg:].max(1).values
        keep = torch.zeros_like(top, dtype=torch.bool).scatter_(1, i[:, :tg], True)
        c = torch.where(keep.repeat_interleave(E // G, 1), c, torch.full_like(c, -math.inf))
    v, i = c.sort(1, descending=True)
    e = err.gather(1, i)
    n = min(k, E - 1)
    ok &= (v[:, :n] - e[:, :n] > v[:, 1:n + 1] + e[:, 1:n + 1]).all(1)
    return ok


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(1000003 * (seed + 1) + len(case["op"]))

    def normal(shape, std=1.0, dtype=torch.float32):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)

    st = SimpleNamespace(case=case, own=None)
    if case["op"] == "route":
        T, H, E = case["T"], case["H"], case["E"]
        st.wr = normal((E, H), 0.02)
        st.lb = normal((E,), 0.5) if case["logit_bias"] else None
        # the size such a bias has once it balances the load: a fraction of the scores' spread
        st.bal = normal((E,), 0.05 if case["score"] == "sigmoid" else 0.3 / E) if case["balance"] else None
        st.x = normal((T, H), dtype=torch.bfloat16)
        for _ in range(50):
            bad = (~_margins_ok(case, st.x, st.wr, st.lb, st.bal)).nonzero()[:, 0]
            if bad.numel() == 0:
                break
            st.x[bad] = normal((bad.numel(), H), dtype=torch.bfloat16)
        else:
            raise RuntimeError("could not remove near-ties")
        if own:
            import bit_routed_expert_fp32_b200 as moe
            st.moe = moe
            st.cfg = SimpleNamespace(H=H, I=64, E=E, k=case["k"], S=0)
            st.router = moe.Router(score=moe.SCORE_SIGMOID if case["score"] == "sigmoid" else moe.SCORE_SOFTMAX,
                                   n_groups=case["G"], top_groups=case["tg"], group_top=case["gt"],
                                   renormalise=case["renorm"], scale=case["scale"])
            st.rt = moe.alloc_routing(st.cfg, T)
            st.ws = torch.empty(moe.moe_workspace_size(st.cfg, T), dtype=torch.uint8, device="cuda")
            moe.moe_workspace_init(st.ws)
    else:
        T, K, N, dt, pad = case["T"], case["K"], case["N"], _dtype(case), case["pad"]
        rows = 2 * N if case["act"] == "swiglu" else N
        st.x = normal((T, _up8(K) + pad), dtype=dt)[:, :K]
        st.w = normal((rows, _up8(K) + pad), 1.7 / math.sqrt(K), dtype=dt)[:, :K]
        st.b = normal((rows,), 0.5, dtype=dt) if case["bias"] else None
        st.r = None
        if case["residual"]:
            st.r = normal((T, N), dtype=torch.float32 if case["residual"] == "f32" else dt)
        if own:
            import bit_routed_expert_fp32_b200 as moe
            st.moe = moe
            st.act = {"none": moe.ACT_NONE, "relu": moe.ACT_RELU, "silu": moe.ACT_SILU, "gelu": moe.ACT_GELU,
                      "gelu_tanh": moe.ACT_GELU_TANH, "swiglu": moe.ACT_SWIGLU}[case["act"]]
            st.y = torch.empty((T, N), dtype=dt, device="cuda")
            st.ws = torch.empty(4096, dtype=torch.uint8, device="cuda")
            moe.moe_workspace_init(st.ws)
    return st


# ---- one pass -------------------------------------------------------------------------

def _arrange(ids, E):
    """Counts, offsets, permutation (experts ascending, then tokens) and its inverse."""
    flat = ids.reshape(-1)
    counts = torch.zeros(E, dtype=torch.int64, device=ids.device).scatter_add_(0, flat, torch.ones_like(flat))
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=ids.device)
    offsets[1:] = counts.cumsum(0)
    perm = flat.sort(dim=0, stable=True).indices
    inv = torch.empty_like(perm)
    inv[perm] = torch.arange(perm.numel(), device=ids.device)
    return [t.to(torch.int32) for t in (counts, offsets, perm, inv)]


def _route_plain(st):
    c_ = st.case
    T, E, G = c_["T"], c_["E"], c_["G"]
    logits = st.x.float() @ st.wr.t()
    if st.lb is not None:
        logits = logits + st.lb
    # scores in 64 bits: the sigmoid's upper end and sums of scores and biases lie close to
    # one another in 32
    L = logits.double()
    if c_["score"] == "softmax":
        s = torch.exp(L - L.max(1, keepdim=True).values)
        s = s / s.sum(1, keepdim=True)
    else:
        s = 1 / (1 + torch.exp(-L))
    c = s if st.bal is None else s + st.bal.double()
    if c_["tg"] < G:
        top = c.view(T, G, E // G).sort(2, descending=True).values[:, :, :c_["gt"]].sum(2)
        order = top.sort(dim=1, descending=True, stable=True).indices
        keep = torch.zeros((T, G), dtype=torch.bool, device=c.device).scatter_(1, order[:, :c_["tg"]], True)
        c = torch.where(keep.repeat_interleave(E // G, 1), c, torch.full_like(c, -math.inf))
    ids = c.sort(dim=1, descending=True, stable=True).indices[:, :c_["k"]]
    w = s.gather(1, ids)
    if c_["renorm"]:
        w = w / w.sum(1, keepdim=True)
    w = (w * c_["scale"]).float()
    return [ids.to(torch.int32), w] + _arrange(ids, E)


def _linear_plain(st):
    c, N = st.case, st.case["N"]
    a = st.x.float() @ st.w.float().t()
    if st.b is not None:
        a = a + st.b.float()
    act = c["act"]
    if act == "swiglu":
        gate, up = a[:, :N], a[:, N:]
        v = gate / (1 + torch.exp(-gate)) * up
    elif act == "relu":
        v = torch.where(a > 0, a, torch.zeros_like(a))
    elif act == "silu":
        v = a / (1 + torch.exp(-a))
    elif act == "gelu":
        v = 0.5 * a * (1 + torch.erf(a * math.sqrt(0.5)))
    elif act == "gelu_tanh":
        v = 0.5 * a * (1 + torch.tanh(math.sqrt(2 / math.pi) * (a + 0.044715 * a * a * a)))
    else:
        v = a
    if st.r is not None:
        v = v + st.r.float()
    return v.to(st.x.dtype)


def run(st):
    c = st.case
    if not own:
        return _route_plain(st) if c["op"] == "route" else _linear_plain(st)
    if c["op"] == "route":
        st.moe.moe_route_scored(st.cfg, st.router, c["T"], st.x, st.wr, st.lb, st.bal, st.rt, st.ws)
        return [st.rt[n] for n in ("topk_ids", "topk_w", "counts", "offsets", "perm", "inv_perm")]
    st.moe.moe_linear(st.x, st.w, st.y, st.ws, bias=st.b, residual=st.r, act=st.act)
    return st.y


def work(case):
    T = case["T"]
    if case["op"] == "route":
        H, E, k = case["H"], case["E"], case["k"]
        read = 2 * T * H + 4 * E * H + 4 * E * (int(case["logit_bias"]) + int(case["balance"]))
        write = T * k * (4 + 4 + 4 + 4) + 4 * (2 * E + 1)
        return {"bytes": read + write, "flops": 2 * T * E * H}
    K, N = case["K"], case["N"]
    rows = 2 * N if case["act"] == "swiglu" else N
    b = 2 * T * K + 2 * rows * K + 2 * T * N + (2 * rows if case["bias"] else 0)
    b += {"": 0, "same": 2, "f32": 4}[case["residual"]] * T * N
    return {"bytes": b, "flops": 2 * T * rows * K}


# ---- the definition in 64 bits ----------------------------------------------------------

def _exact_route(c, st):
    """Token by token of the definition, vectorised over tokens: repeated selection of the
    largest remaining value, the lowest index first among equals."""
    T, E, G, k = c["T"], c["E"], c["G"], c["k"]
    dev = st.x.device
    L = torch.empty((T, E), dtype=torch.float64, device=dev)
    w64 = st.wr.double()
    for t0 in range(0, T, 2048):
        L[t0:t0 + 2048] = torch.einsum("th,eh->te", st.x[t0:t0 + 2048].double(), w64)
    if st.lb is not None:
        L += st.lb.double()
    if c["score"] == "sigmoid":
        s = torch.sigmoid(L)
    else:
        s = torch.softmax(L, dim=1)
    chosen_by = s.clone()
    if st.bal is not None:
        chosen_by += st.bal.double()
    group_of = torch.arange(E, device=dev) // (E // G)
    if c["tg"] < G:
        left = chosen_by.clone()
        score = torch.zeros((T, G), dtype=torch.float64, device=dev)
        for gi in range(G):
            block = left[:, gi * (E // G):(gi + 1) * (E // G)]
            for _ in range(c["gt"]):
                m, at = block.max(1)
                score[:, gi] += m
                block.scatter_(1, at[:, None], -math.inf)
        allowed = torch.zeros((T, E), dtype=torch.bool, device=dev)
        for _ in range(c["tg"]):
            best = score.max(1, keepdim=True).values
            at = (score == best).int().argmax(1)
            allowed |= group_of[None, :] == at[:, None]
            score.scatter_(1, at[:, None], -math.inf)
        chosen_by[~allowed] = -math.inf
    ids = torch.empty((T, k), dtype=torch.int64, device=dev)
    for j in range(k):
        best = chosen_by.max(1, keepdim=True).values
        at = (chosen_by == best).int().argmax(1)
        ids[:, j] = at
        chosen_by.scatter_(1, at[:, None], -math.inf)
    w = torch.gather(s, 1, ids)
    if c["renorm"]:
        w = w / torch.sum(w, 1, keepdim=True)
    counts = torch.stack([(ids == e).sum() for e in range(E)])
    offsets = torch.cat([torch.zeros(1, dtype=counts.dtype, device=dev), torch.cumsum(counts, 0)])
    key = ids.reshape(-1) * (T * k) + torch.arange(T * k, device=dev)          # all different
    perm = torch.argsort(key)
    return [ids.int(), w * c["scale"], counts.int(), offsets.int(), perm.int(), torch.argsort(perm).int()]


def _exact_linear(c, st):
    N, w = c["N"], st.w.double()
    out = torch.empty((c["T"], N), dtype=torch.float64, device=st.x.device)
    for t0 in range(0, c["T"], 2048):
        sl = slice(t0, t0 + 2048)
        a = torch.nn.functional.linear(st.x[sl].double(), w, None if st.b is None else st.b.double())
        if c["act"] == "swiglu":
            v = torch.nn.functional.silu(a[:, :N]) * a[:, N:]
        else:
            f = {"none": lambda z: z, "relu": torch.relu, "silu": torch.nn.functional.silu,
                 "gelu": torch.nn.functional.gelu,
                 "gelu_tanh": lambda z: torch.nn.functional.gelu(z, approximate="tanh")}[c["act"]]
            v = f(a)
        out[sl] = v if st.r is None else v + st.r[sl].double()
    return out


def exact(case, seed):
    st = prepare(case, seed)
    return _exact_route(case, st) if case["op"] == "route" else _exact_linear(case, st)
