"""moe_route_scored's binding refuses routing buffers that the kernels would write past, before any
pointer reaches the library.  The tensors here are stand-ins that say they are on a GPU."""
from types import SimpleNamespace

import pytest

torch = pytest.importorskip("torch")

import bit_routed_expert_fp32_b200 as moe  # noqa: E402

CFG = SimpleNamespace(H=128, I=64, E=16, k=2, S=0)


class OnGpu:
    def __init__(self, t, dev=0):
        self.t, self.dev = t, dev

    def get_device(self):
        return self.dev

    def __getattr__(self, name):
        return getattr(self.t, name)


def routing(T, **other):
    rt = {n: OnGpu(t) for n, t in moe.alloc_routing(CFG, T, device="cpu").items()}
    rt.update({n: OnGpu(t) if isinstance(t, torch.Tensor) else t for n, t in other.items()})
    return rt


def call(monkeypatch, rt, T=8):
    seen = []
    monkeypatch.setattr(moe, "_lib", SimpleNamespace(moe_route_scored=lambda *a: seen.append(a) or moe.MOE_OK))
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    ws = OnGpu(torch.zeros(4096, dtype=torch.uint8))
    moe.moe_route_scored(CFG, moe.Router(), T, OnGpu(torch.zeros((T, 128), dtype=torch.bfloat16)),
                         OnGpu(torch.zeros((16, 128))), None, None, rt, ws, stream=SimpleNamespace(cuda_stream=0))
    return seen


def test_buffers_that_fit_reach_the_library(monkeypatch):
    assert len(call(monkeypatch, routing(8))) == 1
    assert len(call(monkeypatch, routing(40))) == 1               # room for more tokens


@pytest.mark.parametrize("other", [
    dict(topk_ids=torch.zeros((7, 2), dtype=torch.int32)), dict(topk_w=torch.zeros(15)),
    dict(topk_w=torch.zeros((8, 2), dtype=torch.float16)), dict(topk_ids=torch.zeros((8, 2), dtype=torch.int64)),
    dict(counts=torch.zeros(15, dtype=torch.int32)), dict(offsets=torch.zeros(16, dtype=torch.int32)),
    dict(perm=torch.zeros(15, dtype=torch.int32)), dict(inv_perm=torch.zeros(4, dtype=torch.int32)),
    dict(perm=torch.zeros(32, dtype=torch.int32)[::2]), dict(topk_w=torch.zeros((2, 8)).t()),
    dict(counts=OnGpu(torch.zeros(16, dtype=torch.int32), dev=1)),
    dict(counts=OnGpu(torch.zeros(16, dtype=torch.int32), dev=-1)),
])
def test_buffers_that_do_not_fit_are_refused(monkeypatch, other):
    with pytest.raises(ValueError, match=next(iter(other))):
        call(monkeypatch, routing(8, **other))


def test_buffers_of_fewer_tokens_are_refused(monkeypatch):
    with pytest.raises(ValueError, match="topk_ids"):
        call(monkeypatch, routing(7))
