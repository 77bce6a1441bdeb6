"""moe_route_scored's argument checks (host only: every call here is refused or empty)."""
import ctypes

import pytest

import bit_routed_expert_fp32_b200 as moe

WS = 1 << 30


def call(T=4, H=128, E=16, k=2, score=1, G=4, tg=2, gt=2, renorm=1, scale=1.0, x=1 << 20, wr=2 << 20, b=None, bal=None,
         rt=True, ws=4 << 20, ws_bytes=WS, router=True):
    sh = moe.Shape(H, 64, E, k, 0)
    r = moe.Router(score=score, n_groups=G, top_groups=tg, group_top=gt, scale=scale)
    r.renormalise = renorm
    out = moe.Routing(*([0x1000] * 6)) if rt else None
    return moe.lib().moe_route_scored(ctypes.byref(sh), ctypes.byref(r) if router else None, T, x, wr, b, bal,
                                      ctypes.byref(out) if rt else None, ws, ws_bytes, None)


@pytest.mark.parametrize("bad", [
    dict(router=False), dict(T=-1), dict(H=100), dict(E=257, G=1, tg=1), dict(k=17, E=32), dict(score=2), dict(score=-1),
    dict(G=0), dict(G=3), dict(E=66, G=33, k=1), dict(tg=0), dict(tg=5), dict(gt=0), dict(gt=3), dict(G=16, gt=2),
    dict(G=8, tg=1, k=3), dict(renorm=2), dict(renorm=-1), dict(scale=float("nan")), dict(scale=float("inf")),
    dict(x=None), dict(wr=None), dict(x=(1 << 20) + 8), dict(wr=(2 << 20) + 4), dict(b=(5 << 20) + 2),
    dict(bal=(5 << 20) + 1), dict(rt=False), dict(ws=None), dict(ws=(4 << 20) + 8),
])
def test_refused(bad):
    assert call(**bad) == 1


def test_workspace_and_empty_batch():
    assert call(ws_bytes=4096) == 3
    assert call(T=0) == 0
    assert call(T=0, G=3) == 1


def test_tensors_are_checked_before_their_pointers_are_used():
    """Host tensors, other types and too few rows are refused by the Python entry."""
    torch = pytest.importorskip("torch")

    class Cfg:
        H, I, E, k, S = 128, 64, 16, 2, 0
    x, w = torch.zeros((4, 128), dtype=torch.bfloat16), torch.zeros((16, 128))
    ws = torch.zeros(4096, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA device"):
        moe.moe_route_scored(Cfg, moe.Router(), 4, x, w, None, None, {}, ws)
