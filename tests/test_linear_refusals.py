"""moe_linear's argument checks (host only: every call here is refused or empty)."""
import ctypes

import pytest

import bit_routed_expert_fp32_b200 as moe


def call(T=4, K=64, N=32, dtype=0, rdtype=0, act=0, ldx=64, ldw=64, ldr=32, ldy=32, x=1 << 20, w=2 << 20, b=None,
         r=None, y=3 << 20, ws=4 << 20, ws_bytes=4096, desc=True):
    d = moe.LinearDesc(K, N, dtype, rdtype, act, ldx, ldw, ldr, ldy)
    return moe.lib().moe_linear(ctypes.byref(d) if desc else None, T, x, w, b, r, y, ws, ws_bytes, None)


@pytest.mark.parametrize("bad", [
    dict(desc=False), dict(T=-1), dict(K=0), dict(N=0), dict(dtype=2), dict(dtype=3), dict(act=-1), dict(act=6),
    dict(ldx=56), dict(ldx=65), dict(ldw=60), dict(ldw=68), dict(ldy=31), dict(ldy=1 << 40),
    dict(r=5 << 20, ldr=31), dict(r=5 << 20, rdtype=1), dict(r=5 << 20, rdtype=3), dict(x=None), dict(w=None),
    dict(y=None), dict(ws=None), dict(ws_bytes=4095), dict(x=(1 << 20) + 8), dict(w=(2 << 20) + 2),
    dict(y=(3 << 20) + 1), dict(b=(5 << 20) + 1), dict(r=(5 << 20) + 1), dict(r=(5 << 20) + 2, rdtype=2),
    dict(ws=(4 << 20) + 8),
    dict(y=1 << 20), dict(y=(1 << 20) + 64), dict(y=2 << 20), dict(b=3 << 20),       # y over x, w, the bias
    dict(r=(3 << 20) + 2), dict(r=3 << 20, ldr=40), dict(r=3 << 20, rdtype=2),       # y over another residual
    dict(act=5, y=(2 << 20) + 64 * 32 * 2),                                          # the up rows
    dict(ldx=128, ldy=128, y=(1 << 20) + 100),                                       # slices that share columns
])
def test_refused(bad):
    assert call(**bad) == 1


def test_empty_batch_and_sizes_past_the_device():
    assert call(T=0) == 0
    assert call(T=0, x=None, w=None, y=None, ws=None) == 0
    assert call(N=(1 << 31) - 8, act=5, ldy=1 << 32, w=1 << 50, y=1 << 45) == 2
