"""moe_linear's activations value by value, against their definitions in 64 bits: x is 1 and w the
argument itself (K = 1), so that the fp32 sum is exact and only the activation and the one rounding
of its result are off.

Tolerance: half a step of the type, and what the fp32 formulas may lose, in steps of 2^-23 of the
value, z being the argument of the exponential:
  SiLU       2^(-z log2 e - 15): the argument's rounding, half a step of 1.45 z + 15, 5.2 + 0.5 z,
             log2 e itself 0.25 z, ex2.approx 2; the sum 0.5, rcp.approx 1, the product 0.5
                                                                                     10 + 0.8 z
  tanh GELU  the same; z itself (seven roundings of half a step, times z): 4 z       10 + 4.8 z
  GELU       erfc's fit 5.4, its seven terms with alternating signs (the largest is 0.4, their sum
             down to 0.06) and the quotient 8, z = a a / 2: z, the exponential 2 + 1.17 z
                                                                                     16 + 2.5 z
and half of the smallest subnormal, which in fp32 loses bits too below 2^-126: 2^-149 (1 + |a|)."""
import pytest

pytestmark = pytest.mark.gpu


def _moe():
    import bit_routed_expert_fp32_b200 as moe
    return moe


def values(dtype):
    """All of the type's values of some sizes, and a fine walk through the activations' range."""
    import torch
    dt = {"bf16": torch.bfloat16, "fp16": torch.float16}[dtype]
    v = torch.cat([torch.linspace(-14, 14, 6001), torch.linspace(-110, 110, 1501),
                   torch.tensor([0.0, 1e-7, 1e-4, 1e-3, 500.0, 6e4])]).to(dt)
    v = torch.cat([v, -v]).unique()
    return v[: v.numel() // 8 * 8].cuda()


def definition(act, a):
    """act(a) in float64, and the argument of its exponential."""
    import torch
    moe = _moe()
    a = a.double()
    if act in (moe.ACT_SILU, moe.ACT_SWIGLU):
        return a * torch.exp(torch.nn.functional.logsigmoid(a)), a.abs()
    if act == moe.ACT_GELU:
        return 0.5 * a * torch.special.erfc(-a * 0.5 ** 0.5), a * a / 2
    z = 2 * (2 / torch.pi) ** 0.5 * (a + 0.044715 * a ** 3)
    return a * torch.exp(torch.nn.functional.logsigmoid(z)), z.abs()


# (T, copies of the values side by side): the vector, the tile and the pair kernel
KERNELS = [(3, 1), (40, 1), (2048, 4)]


def one(act, dtype, T, copies):
    import torch
    moe = _moe()
    v = values(dtype)
    a = v.repeat(copies)
    N, dt = a.numel(), a.dtype
    glu = act == moe.ACT_SWIGLU
    w = torch.zeros((2 * N if glu else N, 8), dtype=dt, device="cuda")
    w[:N, 0] = a
    if glu:
        w[N:, 0] = 1
    x = torch.zeros((T, 8), dtype=dt, device="cuda")
    x[:, 0] = 1
    y = torch.empty((T, N), dtype=dt, device="cuda")
    ws = torch.empty(4096, dtype=torch.uint8, device="cuda")
    moe.moe_workspace_init(ws)
    moe.moe_linear(x[:, :1], w[:, :1], y, ws, act=act)
    torch.cuda.synchronize()
    assert moe.moe_get_error(ws) == (0, 0)
    assert torch.equal(y, y[:1].expand(T, N))
    ref, z = definition(act, a)
    c0, c1 = {moe.ACT_SILU: (10, 0.8), moe.ACT_SWIGLU: (10, 0.8), moe.ACT_GELU_TANH: (10, 4.8), moe.ACT_GELU: (16, 2.5)}[act]
    fi = torch.finfo(dt)
    tol = (fi.eps / 2 + (c0 + c1 * z.clamp_max(120)) * 2.0 ** -23) * ref.abs()
    tol = tol + fi.smallest_normal * fi.eps / 2 + 2.0 ** -149 * (1 + a.double().abs())
    bad = (y[0].double() - ref).abs() > tol
    i = int(bad.nonzero()[0]) if bad.any() else 0
    assert not bad.any(), (f"{int(bad.sum())} of {N} off, first {float(a[i])}: {float(y[0, i])} against {float(ref[i])}, "
                           f"tolerance {float(tol[i]):.3e}")


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("T,copies", KERNELS)
def test_gelu(T, copies, dtype):
    one(_moe().ACT_GELU, dtype, T, copies)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("T,copies", KERNELS)
@pytest.mark.parametrize("act", ["SILU", "SWIGLU", "GELU_TANH"])
def test_sigmoid_forms(act, T, copies, dtype):
    """Down to where fp32 ends: bf16 holds SiLU's values far past -87, where 1 + e^-a leaves the
    range of the fast quotient's divisor."""
    one(getattr(_moe(), "ACT_" + act), dtype, T, copies)
