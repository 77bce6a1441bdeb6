"""moe_route_scored where values nearly meet: scores an ulp to a few apart, group scores whose two
terms cancel, balances of any size.  The choice is the fp64 one of the fp32 logits whatever the
kernel forms in fp32 on the way.  Logits are exact (see test_gpu_route_scored.exact_case); a token
whose fp64 values lie within `margin` of one another is drawn again, so that the last bits of an
fp64 exponential decide nothing (64-bit rounding of these sums stays below 65536 * 2^-52 < 2e-11)."""
import numpy as np
import pytest

from tests import scored_ref as ref
from tests.test_gpu_route_scored import W_RTOL, check, exact_case, route

pytestmark = pytest.mark.gpu

MARGIN = 2e-10


def clear(L, balance, k, margin, sigmoid, n_groups=1, top_groups=1, group_top=1):
    """Per token: the kept groups and the choice are decided by more than margin, or by values that
    are equal because their logits and balances are."""
    s = ref.scores(L, sigmoid)
    T, E = s.shape
    b = np.zeros(E) if balance is None else np.asarray(balance, np.float64)
    gs = E // n_groups
    c = s + b
    ok = np.ones(T, bool)
    keep = np.ones((T, n_groups), bool)
    if top_groups < n_groups:
        score = np.sort(c.reshape(T, n_groups, gs), axis=2)[:, :, ::-1][:, :, :group_top].sum(2)
        order = np.argsort(-score, axis=1, kind="stable")
        srt = np.take_along_axis(score, order, 1)
        ok &= srt[:, top_groups - 1] - srt[:, top_groups] > margin
        keep[:] = False
        np.put_along_axis(keep, order[:, :top_groups], True, 1)
    cand = np.where(np.repeat(keep, gs, 1), c, -np.inf)
    order = np.argsort(-cand, axis=1, kind="stable")[:, :k + 1]
    v = np.take_along_axis(cand, order, 1)
    same = (np.diff(np.take_along_axis(L, order, 1), axis=1) == 0) & (np.diff(b[order], axis=1) == 0)
    with np.errstate(invalid="ignore"):
        ok &= ((v[:, :-1] - v[:, 1:] > margin) | same).all(1)
    return ok


def settle(draw, T, balance, k, sigmoid, **g):
    """Tokens of draw(n) until T of them are clear."""
    rows = np.empty((0, draw(1).shape[1]), np.float32)
    for _ in range(50):
        new = draw(T)
        rows = np.concatenate([rows, new[clear(new, balance, k, MARGIN, sigmoid, **g)]])
        if len(rows) >= T:
            return rows[:T]
    raise RuntimeError("could not find clear tokens")


def logit(s):
    return np.log(s) - np.log1p(-s)


@pytest.mark.parametrize("T", [8, 64, 900])
@pytest.mark.parametrize("B", [0.0, 4.0, 64.0, 1000.0, 65536.0])
@pytest.mark.parametrize("E,k,G,tg", [(16, 4, 8, 4), (64, 6, 8, 3), (256, 8, 8, 4), (256, 8, 16, 5), (120, 5, 10, 4)])
@pytest.mark.parametrize("some", [False, True])
def test_group_scores_whose_terms_cancel(E, k, G, tg, some, B, T):
    """Every group's (or every other group's) two largest values are s + B and s' - B, and the group
    scores s + s' lie 1e-7 to 1e-2 apart, below and above what rounding the terms to fp32 costs."""
    rng = np.random.default_rng(int(B) + E + G + T)
    gs = E // G
    bal = np.full((G, gs), -8.0 * B - 16.0)                  # never among the two largest
    with_b = np.arange(G) % 2 == 0 if some else np.ones(G, bool)
    bal[:, 0], bal[:, 1] = np.where(with_b, B, 0.25), np.where(with_b, -B, -0.25)
    bal = bal.reshape(-1).astype(np.float32)
    g = dict(n_groups=G, top_groups=tg, group_top=2)

    def draw(n):
        spread = 10.0 ** rng.uniform(-7, -2, (n, 1))
        total = 1.0 + spread * rng.standard_normal((n, G))
        s1 = rng.uniform(0.2, 0.8, (n, G))
        L = rng.standard_normal((n, G, gs))
        L[:, :, 0], L[:, :, 1] = logit(s1), logit(total - s1)
        return L.reshape(n, E).astype(np.float32)

    kw = dict(sigmoid=True, renormalise=True, scale=2.5, **g)
    L = settle(draw, T, bal, k, True, **g)
    x, wr = exact_case(L)
    check(route(x, wr, None, bal, k, **kw), L, bal, k, E, W_RTOL, **kw)


@pytest.mark.parametrize("T", [8, 64, 900])
@pytest.mark.parametrize("B", [0.0, 3.0, 500.0])
@pytest.mark.parametrize("E,k,G,tg,gt", [(16, 4, 8, 4, 2), (256, 8, 8, 4, 2), (256, 8, 8, 4, 1), (96, 5, 1, 1, 1)])
def test_softmax_scores_with_balances_of_both_signs(E, k, G, tg, gt, B, T):
    rng = np.random.default_rng(int(B) + E + tg + T)
    gs = E // G
    bal = np.where(np.arange(E) % gs % 2 == 0, B, -B) if gs > 1 else np.zeros(E)
    bal = bal.astype(np.float32)
    g = dict(n_groups=G, top_groups=tg, group_top=gt)

    def draw(n):
        base = rng.standard_normal((n, 1, gs))
        L = base + 10.0 ** rng.uniform(-6, -2, (n, 1, 1)) * rng.standard_normal((n, G, gs))
        return L.reshape(n, E).astype(np.float32)

    kw = dict(sigmoid=False, renormalise=False, scale=1.0, **g)
    L = settle(draw, T, bal, k, False, **g)
    x, wr = exact_case(L)
    check(route(x, wr, None, bal, k, **kw), L, bal, k, E, W_RTOL, **kw)


@pytest.mark.parametrize("T", [8, 64, 900])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("balanced", [False, True])
@pytest.mark.parametrize("E,k,G,tg,gt", [(8, 3, 1, 1, 1), (64, 8, 8, 4, 1), (256, 8, 8, 4, 2), (256, 16, 1, 1, 1)])
def test_neighbours_a_few_ulp_apart(E, k, G, tg, gt, balanced, sigmoid, T):
    """Logits that are a common value plus 0 to 40 ulp (equal ones tie: lower id first); with a
    balance, scores plus balance that meet to some 1e-9 to 1e-5."""
    rng = np.random.default_rng(E + k + T)
    bal = (rng.integers(-3, 4, E) / 16).astype(np.float32) if balanced else None
    g = dict(n_groups=G, top_groups=tg, group_top=gt)

    def draw(n):
        if balanced and sigmoid:
            c = rng.uniform(0.4, 0.6, (n, 1)) + 10.0 ** rng.uniform(-9, -5, (n, 1)) * rng.standard_normal((n, E))
            return logit(c - bal).astype(np.float32)
        base = rng.choice([-6.0, -0.7, 0.3, 1.0, 2.5, 5.0], (n, 1)).astype(np.float32)
        return (base + np.spacing(base) * rng.integers(0, 41, (n, E))).astype(np.float32)

    kw = dict(sigmoid=sigmoid, renormalise=True, scale=1.0, **g)
    if gt == 2:                  # sums of two: decided by more than the margin
        L = settle(draw, T, bal, k, sigmoid, **g)
    else:
        L = draw(T)
        if balanced:
            L = settle(draw, T, bal, k, sigmoid, **g)
    x, wr = exact_case(L)
    check(route(x, wr, None, bal, k, **kw), L, bal, k, E, W_RTOL, **kw)
