"""moe_linear against the definition in 64 bits: types, activations, sizes from one value
to several tiles, strides, in-place residuals, and a layer's use of it."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


def _moe():
    import bit_routed_expert_fp32_b200 as moe
    return moe


def _ws():
    import torch
    moe = _moe()
    ws = torch.empty(4096, dtype=torch.uint8, device="cuda")
    moe.moe_workspace_init(ws)
    return ws


def reference(x, w, bias, residual, act):
    """The definition in float64; also sum_k |x w| (+ |bias|), the size of the terms of a."""
    import torch
    moe = _moe()
    a = x.double() @ w.double().t()
    mag = x.double().abs() @ w.double().abs().t()
    if bias is not None:
        a = a + bias.double()
        mag = mag + bias.double().abs()
    N = y_cols(w, act)
    if act == moe.ACT_SWIGLU:
        g, u = a[:, :N], a[:, N:]
        v = g * torch.sigmoid(g) * u
        # d silu <= 1.1, so an error of a moves the product by at most this
        mag = 1.1 * mag[:, :N] * u.abs() + mag[:, N:] * (g * torch.sigmoid(g)).abs()
    else:
        f = {moe.ACT_NONE: lambda z: z, moe.ACT_RELU: torch.relu, moe.ACT_SILU: lambda z: z * torch.sigmoid(z),
             moe.ACT_GELU: torch.nn.functional.gelu,
             moe.ACT_GELU_TANH: lambda z: torch.nn.functional.gelu(z, approximate="tanh")}[act]
        v = f(a)
        mag = 1.13 * mag                       # the largest slope of the GELUs (SiLU 1.1, ReLU 1)
    if residual is not None:
        v = v + residual.double()
    return v, mag


def y_cols(w, act):
    return w.shape[0] // 2 if act == _moe().ACT_SWIGLU else w.shape[0]


def check(y, x, w, bias, residual, act):
    """Half a step of the output's type, plus the fp32 sums.  The products are exact in
    fp32; a sum of K terms held in fp32 is off by at most about K / 16 steps of 2^-23 of
    the terms' size (16 terms enter per addition, an addition may drop up to one step), and
    in practice by far less: 4 + K / 64 steps allowed.  The activations' fast exponential,
    quotient, erf and tanh are off by at most some 2^-20 of their value's size (a value
    beside a zero of the GELUs: of the input's size)."""
    import torch
    moe = _moe()
    ref, mag = reference(x, w, bias, residual, act)
    assert torch.isfinite(y).all()
    K = x.shape[1]
    tol = torch.finfo(y.dtype).eps / 2 * ref.abs() + (4 + K / 64) * 2.0 ** -23 * mag
    tol += torch.finfo(y.dtype).smallest_normal * torch.finfo(y.dtype).eps          # fp16 subnormals
    if act != moe.ACT_NONE:
        tol += 2.0 ** -19 * (ref.abs() + mag)
    if residual is not None:
        tol += 2.0 ** -23 * residual.double().abs()
    bad = (y.double() - ref).abs() > tol
    assert not bad.any(), (f"{int(bad.sum())} of {bad.numel()} off, first {bad.nonzero()[0].tolist()}: "
                           f"{float(y[bad][0])} vs {float(ref[bad][0])} tol {float(tol[bad][0]):.3e}")


def make(T, K, N, act, dtype, bias=True, residual="same", pad=0, seed=0):
    import torch
    moe = _moe()
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    dt = {"bf16": torch.bfloat16, "fp16": torch.float16}[dtype]
    rows = 2 * N if act == moe.ACT_SWIGLU else N
    ld = (K + 7) // 8 * 8 + pad

    def rnd(*shape, std=1.0, t=dt):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(t)

    x, w = rnd(T, ld)[:, :K], rnd(rows, ld, std=1.5 / K ** 0.5)[:, :K]
    b = rnd(rows, std=0.5) if bias else None
    r = {"": None, "same": rnd(T, N + pad)[:, :N], "f32": rnd(T, N + pad, t=torch.float32)[:, :N]}[residual]
    ybuf = torch.full((T + 1, N + pad), 7.0, dtype=dt, device="cuda")
    return x, w, b, r, ybuf


def run(T, K, N, act, dtype, **kw):
    import torch
    moe = _moe()
    x, w, b, r, ybuf = make(T, K, N, act, dtype, **kw)
    ws = _ws()
    y = ybuf[:T, :N]
    moe.moe_linear(x, w, y, ws, bias=b, residual=r, act=act)
    torch.cuda.synchronize()
    assert moe.moe_get_error(ws) == (0, 0)
    check(y, x, w, b, r, act)
    # what lies behind the last row and beside the columns stays as it was
    assert (ybuf[T:] == 7).all() and (ybuf[:, N:] == 7).all()
    return y


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("act", range(6))
@pytest.mark.parametrize("T,K,N", [(1, 64, 128), (5, 200, 96), (33, 520, 257)])
def test_types_and_activations(T, K, N, act, dtype):
    run(T, K, N, act, dtype, residual="same" if dtype == "bf16" else "f32", pad=8)


@pytest.mark.parametrize("act", [0, 5])
@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300, 513, 1030])
def test_token_counts(T, act):
    run(T, 264, 200, act, "bf16", seed=T)


@pytest.mark.parametrize("act", [0, 5])
@pytest.mark.parametrize("K", [1, 7, 8, 63, 64, 65, 127, 449, 1000, 4096, 7168])
def test_inner_lengths(K, act):
    run(19, K, 130, act, "fp16", seed=K, residual="")


@pytest.mark.parametrize("act", [0, 5])
@pytest.mark.parametrize("N", [1, 2, 3, 5, 127, 128, 129, 384, 1001, 2048])
@pytest.mark.parametrize("T", [3, 400])
def test_output_widths(T, N, act):
    run(T, 96, N, act, "bf16", seed=N, residual="f32", bias=False)


@pytest.mark.parametrize("T,K,N,act", [(1, 7168, 2048, 5), (1, 2048, 7168, 0), (16, 7168, 4096, 2), (64, 4096, 1024, 3),
                                       (130, 1992, 4999, 4), (1000, 2048, 2048, 5), (2049, 1024, 1100, 0),
                                       (4096, 512, 2304, 5), (3001, 712, 4100, 1), (8000, 320, 5000, 0), (5121, 136, 2600, 5), (3878, 187, 3155, 1),
                                       (1030, 200, 4998, 3), (2050, 264, 1001, 5), (777, 900, 2561, 4)])
def test_larger(T, K, N, act):
    run(T, K, N, act, "bf16", seed=T + N, residual="same", pad=16)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("act", [0, 5])
@pytest.mark.parametrize("T", [1, 2, 3, 4, 5])
@pytest.mark.parametrize("K,N", [(1, 1), (255, 3), (256, 5), (257, 9), (2048, 33), (3001, 700), (6000, 5), (1100, 4001),
                                 (9000, 4100)])
def test_a_few_tokens(K, N, T, act, dtype):
    run(T, K, N, act, dtype, residual="f32" if N % 2 else "same", seed=K + T, pad=8 * (T % 2))


@pytest.mark.parametrize("T", [1, 40, 700])
def test_in_place_residual_and_column_slices(T):
    """The residual stream updated in place, x and y being column slices of one buffer."""
    import torch
    moe = _moe()
    ws = _ws()
    K, N = 192, 320
    buf = torch.randn(T, K + N, device="cuda").to(torch.bfloat16)
    x, y = buf[:, :K], buf[:, K:]
    w = (torch.randn(N, K, device="cuda") / K ** 0.5).to(torch.bfloat16)
    x0, r0 = x.clone(), y.clone()
    moe.moe_linear(x, w, y, ws, residual=y)
    torch.cuda.synchronize()
    check(y, x0, w, None, r0, moe.ACT_NONE)
    assert torch.equal(x, x0)


def test_repeats_bit_for_bit():
    import torch
    moe = _moe()
    ws = _ws()
    x, w, b, r, ybuf = make(200, 1000, 300, 5, "bf16", pad=8)
    outs = []
    for _ in range(3):
        y = torch.empty((200, 300), dtype=torch.bfloat16, device="cuda")
        moe.moe_linear(x, w, y, ws, bias=b, residual=r, act=5)
        outs.append(y)
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


def test_infinities_and_nan_stay_in_their_row():
    import torch
    moe = _moe()
    ws = _ws()
    x = torch.randn(6, 128, device="cuda").to(torch.float16)
    w = torch.randn(40, 128, device="cuda").to(torch.float16)
    x[1, 5] = float("nan")
    x[4, 7] = float("inf")
    y = torch.empty((6, 40), dtype=torch.float16, device="cuda")
    for act in range(6):
        n = 20 if act == moe.ACT_SWIGLU else 40
        moe.moe_linear(x, w, y[:, :n], ws, act=act)
        assert torch.isnan(y[1, :n]).all()
        rows = torch.tensor([0, 2, 3, 5], device="cuda")
        assert torch.isfinite(y[rows][:, :n]).all()
        check(y[rows][:, :n], x[rows], w, None, None, act)
        # a sum past the type's range becomes an infinity
    big = torch.full((2, 64), 200.0, dtype=torch.float16, device="cuda")
    y2 = torch.empty((2, 2), dtype=torch.float16, device="cuda")
    moe.moe_linear(big, torch.stack([big[0], -big[0]]), y2, ws)
    assert torch.equal(y2, torch.tensor([[float("inf"), float("-inf")]] * 2, dtype=torch.float16, device="cuda"))


def test_two_streams_share_a_workspace_and_a_graph_replays():
    import torch
    moe = _moe()
    ws = _ws()
    cases = [make(7, 640, 500, 2, "bf16", seed=s) for s in range(2)]
    ys = [torch.empty((7, 500), dtype=torch.bfloat16, device="cuda") for _ in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(20):
        for (x, w, b, r, _), y, s in zip(cases, ys, streams):
            moe.moe_linear(x, w, y, ws, bias=b, residual=r, act=2, stream=s)
    torch.cuda.synchronize()
    for (x, w, b, r, _), y in zip(cases, ys):
        check(y, x, w, b, r, 2)
    x, w, b, r, _ = cases[0]
    want = ys[0].clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.moe_linear(x, w, ys[0], ws, bias=b, residual=r, act=2)
    ys[0].zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(ys[0], want)


def test_empty_batch_is_a_no_op():
    import torch
    moe = _moe()
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.ones((8, 64), dtype=torch.bfloat16, device="cuda")
    moe.moe_linear(x, w, torch.empty((0, 8), dtype=torch.bfloat16, device="cuda"), _ws())


@pytest.mark.parametrize("T", [20, 300, 2000])              # up to four tokens nothing waits
def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_right(T):
    import torch
    moe = _moe()
    ws = _ws()
    x, w, b, r, ybuf = make(T, 512, 256, 0, "bf16")
    y = torch.empty((T, 256), dtype=torch.bfloat16, device="cuda")
    moe.moe_workspace_set_test_stall(ws, 1000)
    moe.moe_linear(x, w, y, ws, bias=b, residual=r)
    st, det = moe.moe_get_error(ws)
    assert moe.STATUS[st] == "MOE_ERR_TIMEOUT" and det & 0xF00 == moe.DETAIL["TEST_STALL"], (st, hex(det))
    moe.moe_workspace_set_test_stall(ws, 0)
    moe.moe_linear(x, w, y, ws, bias=b, residual=r)
    assert moe.moe_get_error(ws) == (0, 0)
    check(y, x, w, b, r, 0)
