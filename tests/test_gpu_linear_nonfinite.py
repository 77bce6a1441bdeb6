"""moe_linear with infinities and NaN in every input: where the definition in 64 bits is infinite or
NaN so is the output, and all else is finite; in the vector, the tile and the pair kernel."""
import pytest

from tests.test_gpu_linear import check, reference

pytestmark = pytest.mark.gpu

SIZES = [(3, 128, 64), (4, 2000, 400), (6, 128, 40), (20, 4096, 96), (40, 700, 130), (2000, 128, 4096)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("act", range(6))
@pytest.mark.parametrize("T,K,N", SIZES)
def test_where_the_definition_is_not_finite(T, K, N, act, dtype):
    import torch
    import bit_routed_expert_fp32_b200 as moe
    dt = {"bf16": torch.bfloat16, "fp16": torch.float16}[dtype]
    g = torch.Generator(device="cuda").manual_seed(T + K + act)
    rows = 2 * N if act == moe.ACT_SWIGLU else N
    inf, nan = float("inf"), float("nan")

    def rnd(*s, std=1.0):
        v = torch.randn(*s, generator=g, device="cuda") * std
        return torch.where(v.abs() < 1e-2, torch.full_like(v, 0.5), v).to(dt)     # no zero beside an infinity

    x, w, b, r = rnd(T, (K + 7) // 8 * 8)[:, :K], rnd(rows, (K + 7) // 8 * 8, std=1 / K ** 0.5)[:, :K], rnd(rows), rnd(T, N)
    x[0, K - 1] = inf                                        # one sign or the other, by the weight's
    x[1, 0], x[1, K // 2] = inf, -inf                        # opposite ones may meet
    x[2, K // 3] = nan
    w[3, 5], w[N // 2, K - 2] = inf, -inf
    b[5], b[7] = inf, -inf
    r[T - 1, 9], r[T - 1, 11], r[0, 13] = inf, nan, -inf
    y = torch.empty((T, N), dtype=dt, device="cuda")
    ws = torch.empty(4096, dtype=torch.uint8, device="cuda")
    moe.moe_workspace_init(ws)
    moe.moe_linear(x, w, y, ws, bias=b, residual=r, act=act)
    torch.cuda.synchronize()
    assert moe.moe_get_error(ws) == (0, 0)
    ref, _ = reference(x, w, b, r, act)
    assert torch.equal(torch.isnan(y), torch.isnan(ref))
    at = torch.isinf(ref)
    assert torch.equal(torch.isinf(y), at) and torch.equal(y[at].double(), ref[at])
    assert at.any() and torch.isnan(ref).any()
    # the rows and columns without any are as ever
    keep = [i for i in range(N) if i not in (3, 5, 7, 9, 11, 13, N // 2)][: N // 2]
    if act != moe.ACT_SWIGLU and T > 4:
        t = torch.arange(3, T - 1, device="cuda")
        check(y[t][:, keep], x[t], w[keep], b[keep], r[t][:, keep], act)
