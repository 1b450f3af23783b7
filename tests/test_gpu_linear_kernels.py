"""Every kernel that sv_linear may take (tests/linear_kernels.py), with
operands and outputs of every type, each activation, with and without bias
and residual, against float64.

Elements are multiples of 2^-3 of magnitude below 1 and scales powers of two
from 1/2 to 2, so that the scaled sums with their bias are multiples of 2^-8
below 2^14 and exact in float32.  What is off then is the activation, the
addition of the residual and the one rounding of the output: relative errors
of exp (a few units in the last place, its argument's rounding magnified by
|z|) and erfc (its argument's by 2 z^2 + 1)."""
import math

import numpy as np
import pytest

from oracle import last_layer as ref
from tests.harness import log
from tests.linear_kernels import KERNELS

pytestmark = pytest.mark.gpu

ULP = 2.0 ** -23
ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]


def _t(name):
    import torch

    return {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}[name]


def tanh_argument(v):
    return 2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)


def activate(v, act):
    """float64 tensors."""
    import torch

    if act == "relu":
        return v.clamp_min(0)
    if act == "silu":
        return v * torch.sigmoid(v)
    if act == "gelu":
        return 0.5 * v * torch.special.erfc(-v / math.sqrt(2))
    if act == "gelu_tanh":
        return v * torch.sigmoid(tanh_argument(v))
    return v


def relative(v, act):
    """The activation's relative error."""
    if act == "gelu":
        return (v * v + 1) * 2 * ULP + 20 * ULP  # 2 z^2 with z = v / sqrt 2
    if act == "gelu_tanh":
        return (8 + 4 * tanh_argument(v).abs()) * ULP
    if act == "silu":
        return (8 + 4 * v.abs()) * ULP
    return 0 * v


def grid(g, shape, dtype):
    import torch

    return (torch.randint(-7, 8, shape, device="cuda", generator=g).float() / 8).to(_t(dtype))


def close(got, want, v, y, act, odt):
    tol = relative(v, act) * y.abs() + 2.0 ** -120 + ULP * want.abs() + (2.0 ** -8 * want.abs() if odt == "bf16" else 0.0)
    bad = (~((got.double() - want).abs() <= tol)).nonzero()  # NaN is bad
    assert bad.numel() == 0, (act, len(bad), bad[:3].tolist(), got[tuple(bad[0])].item(), want[tuple(bad[0])].item())


def test_the_reference_is_the_oracle_s():
    import torch

    v = np.linspace(-12, 12, 301)
    for act in ACTS:
        assert np.allclose(activate(torch.from_numpy(v).cuda(), act).cpu().numpy(), ref.activate(v, act), rtol=1e-12, atol=1e-30), act


@pytest.mark.parametrize("odt", ["f32", "bf16"])
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("kernel,M,N,K", KERNELS)
def test_every_kernel_with_every_epilogue(kernel, M, N, K, dtype, odt):
    import torch

    from rejection_sampling_verify_09_amd import linear

    log(f"[linear kernel {kernel}] M={M} N={N} K={K} {dtype} -> {odt}")
    g = torch.Generator(device="cuda")
    g.manual_seed(M + N + K)
    x, w = grid(g, (M, K), dtype), grid(g, (N, K), dtype)
    sc = {}
    s = (x.float().cpu() @ w.float().cpu().T).cuda().double()  # exact
    if dtype == "e4m3":
        sc = dict(x_scale=torch.exp2(torch.randint(-1, 2, (M,), device="cuda", generator=g).float()),
                  weight_scale=torch.exp2(torch.randint(-1, 2, (N,), device="cuda", generator=g).float()))
        s = s * sc["x_scale"].double()[:, None] * sc["weight_scale"].double()
    bias = grid(g, (N,), odt)
    part = next(p for p in (3, 5, 7) if N % p == 0)
    shared, whole = grid(g, (M, N // part), odt), grid(g, (M, N), odt)
    o = _t(odt)
    for act in ACTS:
        y = activate(s, act)
        close(linear(x, w, activation=act, out_dtype=o, **sc), y, s, y, act, odt)
        v = s + bias.double()
        y = activate(v, act)
        close(linear(x, w, bias=bias, activation=act, out_dtype=o, **sc), y, v, y, act, odt)
        want = y + shared.double().repeat(1, part)
        close(linear(x, w, bias=bias, residual=shared, activation=act, out_dtype=o, **sc), want, v, y, act, odt)
        mine = whole.clone()
        linear(x, w, bias=bias, residual=mine, activation=act, out_dtype=o, out=mine, **sc)
        close(mine, y + whole.double(), v, y, act, odt)
        y = activate(s, act)
        close(linear(x, w, residual=whole, activation=act, out_dtype=o, **sc), y + whole.double(), s, y, act, odt)


EXTREME = [0.0, -0.0, 1e-45, -1e-45, 1.2e-38, -1.2e-38, 1e-20, -1e-20, 1e4, -1e4, 1e10, -1e10, 1e20, -1e20, 3e38, -3e38]
EXTREME += [s * k for k in (0.5, 1.0, 5.0, 9.0, 13.0, 14.5, 20.0, 86.0, 87.5, 88.5, 100.0, 103.5, 127.0, 128.0, 129.0)
            for s in (1.0, -1.0)]


@pytest.mark.parametrize("odt", ["f32", "bf16"])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("kernel,M,N,K", KERNELS)
def test_every_kernel_on_extreme_values(kernel, M, N, K, act, odt):
    """Brought in by the bias of a product of zeros; NaN and the infinities too, each in columns of its own."""
    import torch

    from rejection_sampling_verify_09_amd import linear

    log(f"[linear kernel {kernel}] extremes, {act} -> {odt}")
    v = torch.tensor(EXTREME + [float("inf"), float("nan")]).to(_t(odt))
    b = v.double().numpy()
    with np.errstate(all="ignore"):
        y = torch.from_numpy(ref.activate(b, act))
        z = np.minimum(np.abs(tanh_argument(b)) if act == "gelu_tanh" else np.abs(b), 200.0)
        rel = (z * z + 1) * 2 * ULP + 20 * ULP if act == "gelu" else (8 + 4 * z) * ULP if act != "none" else 0 * z
        tol = torch.from_numpy(rel) * y.abs() + 2.0 ** -120 + (2.0 ** -8 * y.abs() if odt == "bf16" else 0.0)
    bias = v.repeat(N // len(v) + 1)[:N].cuda()
    got = linear(torch.zeros((M, K), device="cuda", dtype=torch.bfloat16), torch.zeros((N, K), device="cuda", dtype=torch.bfloat16),
                 bias=bias, activation=act, out_dtype=_t(odt)).cpu().double()
    wide = lambda t: t.repeat(N // len(v) + 1)[:N].expand(M, N)  # noqa: E731
    y, tol = wide(y), wide(tol)
    nan, inf = torch.isnan(y), torch.isinf(y)
    assert torch.equal(torch.isnan(got), nan) and torch.equal(got[inf], y[inf])
    ok = ~nan & ~inf
    assert ((got[ok] - y[ok]).abs() <= tol[ok]).all()
