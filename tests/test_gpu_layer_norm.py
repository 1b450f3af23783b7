"""GPU parity of layer_norm with the float64 oracle.

Bound of the float32 steps, u = 2^-24 each.  A sum over a row is at most 64 +
6 + 16 rounded terms a thread, a wave and a workgroup deep, below 90 u of the
sum of magnitudes.  With c = h - mean h and s = sqrt(mean c^2):
- the mean the kernel takes off first is wrong by at most D = 90 u mean|h|; the
  mean of what is left is taken off again, so of D only roundings remain: c is
  off by e_c = 3 u (|c| + D) + 92 u (mean|c| + D), and by u |h| + u mean|h| where h
  is a rounded sum with the residual;
- the variance: 95 u (s^2 + D^2) from its sums, 2 s u rms(h) from the rounded h,
  and half of its relative error, plus 4 u, is the reciprocal root's;
- two products, the bias' addition: 3 u |c r w| + 2 u |y|.
An output type adds its half step: 2^-8 for bfloat16, and for e4m3 2^-4 (2^-10
of the scale below its normal range)."""
import numpy as np
import pytest

from oracle import fine_tune as ref
from oracle import last_layer
from tests.harness import log

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {"f32": U, "bf16": 2.0 ** -8, "e4m3": 2.0 ** -4}


def _t(name):
    import torch

    return {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}[name]


def np64(t):
    return None if t is None else t.detach().float().cpu().numpy().astype(np.float64)


def bound(h, w, b, eps, residual):
    """(y, the bound of its float32 error)."""
    y, _ = ref.layer_norm(h, w, b, eps=eps)
    mean = lambda v: np.mean(v, axis=-1, keepdims=True)  # noqa: E731
    c = h - mean(h)
    var = mean(c * c)
    ah = mean(np.abs(h))
    D = 90 * U * ah
    ec = 3 * U * (np.abs(c) + D) + 92 * U * (mean(np.abs(c)) + D)
    ev = 95 * U * (var + D * D)
    if residual:
        ec = ec + U * (np.abs(h) + ah)
        ev = ev + 2 * U * np.sqrt(var * mean(h * h))
    r = 1 / np.sqrt(var + eps)
    rel = 0.5 * ev / (var + eps) + 4 * U
    aw = 1.0 if w is None else np.abs(w)
    return y, aw * r * ec + np.abs(c) * r * aw * (rel + 3 * U) + 2 * U * np.abs(y)


def check(x, w, b, r, eps, out, scale, hres, dtype, odt):
    h = np64(x) + (0.0 if r is None else np64(r))
    want, e = bound(h, np64(w), np64(b), eps, r is not None)
    got = np64(out)
    if odt == "e4m3":
        s, es = np64(scale), last_layer.e4m3_scale(want)
        assert np.all(np.abs(s - es) <= np.max(e, axis=1) / 448 + 2 * U * es)
        got = got * s[:, None]
        tol = e + HALF[odt] * (np.abs(want) + e) + 2.0 ** -10 * es[:, None] * (1 + 2.0 ** -16) + np.abs(want) * 4 * U
        assert np.all(np.max(np.abs(np64(out)), axis=1)[es > last_layer.FLT_MIN] == 448.0)
    else:
        tol = e + HALF[odt] * (np.abs(want) + e) + 2.0 ** -130
    err = np.abs(got - want)
    assert np.all(err <= tol), (np.max(err / (tol + 1e-300)), np.argwhere(err > tol)[:3])
    if r is not None:
        assert np.all(np.abs(np64(hres) - h) <= (HALF[dtype] + U) * np.abs(h) + 2.0 ** -140)
    return float(np.max(err / (tol + 1e-300)))


@pytest.mark.parametrize("odt", ["bf16", "f32", "e4m3"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,d", [(1, 1), (1, 64), (3, 100), (1, 4096), (5, 4097), (7, 2048), (448, 512), (70, 1000),
                                    (33, 8192), (2, 16384), (3, 20001), (1, 65536), (2, 40000), (1500, 72), (9, 513)])
def test_matches_the_oracle(rows, d, dtype, odt):
    import torch

    from rejection_sampling_verify_09_amd import layer_norm

    g = torch.Generator(device="cuda")
    g.manual_seed(rows * 1000003 + d)
    for residual, affine in ((False, 3), (True, 3), (True, 0), (False, 1), (False, 2)):
        log(f"[layer] rows={rows} d={d} {dtype} -> {odt} residual={residual} affine={affine}")
        x = (torch.randn((rows, d), device="cuda", generator=g) * 3 + 1).to(_t(dtype))
        w = torch.randn((d,), device="cuda", generator=g).to(_t(dtype)) if affine & 1 else None
        b = torch.randn((d,), device="cuda", generator=g).to(_t(dtype)) if affine & 2 else None
        r = torch.randn((rows, d), device="cuda", generator=g).to(_t(dtype)) if residual else None
        out, scale, hres = layer_norm(x, w, b, residual=r, eps=1e-5, out_dtype=_t(odt))
        assert out.dtype == _t(odt) and (scale is not None) == (odt == "e4m3") and (hres is not None) == residual
        log(f"   worst err / bound {check(x, w, b, r, 1e-5, out, scale, hres, dtype, odt):.3g}")


@pytest.mark.parametrize("odt", ["bf16", "f32", "e4m3"])
def test_rows_of_one_value_of_close_values_and_of_non_finite_ones(odt):
    import torch

    from rejection_sampling_verify_09_amd import layer_norm

    log(f"[layer] edge rows -> {odt}")
    d = 520
    x = torch.randn((10, d), device="cuda", dtype=torch.float32)
    x[0] = 0
    x[1] = 12345.678             # nothing but the mean
    x[2] = x[2] * 0.01 + 1000    # differences far below the mean
    x[3] *= 1e-30                # far below eps
    x[4] *= 1e15                 # squares near 1e30
    x[5, 0] = 3e4                # one value that outweighs the others
    x[6, 17] = float("nan")
    x[7, 5] = float("inf")
    x[8, 511] = -float("inf")
    w = torch.rand((d,), device="cuda") + 0.5
    b = torch.rand((d,), device="cuda") + 0.5
    out, scale, _ = layer_norm(x, w, b, eps=1e-6, out_dtype=_t(odt))
    fin = [0, 1, 2, 3, 4, 5, 9]
    check(x[fin], w, b, None, 1e-6, out[fin], None if scale is None else scale[fin], None, "f32", odt)
    assert torch.isnan(out[6:9].float()).all()
    if odt == "e4m3":
        assert torch.isnan(scale[6:9]).all()
    out, scale, _ = layer_norm(x[:1], w, out_dtype=_t(odt))
    assert (out.float() == 0).all()
    if odt == "e4m3":
        assert scale.item() == 2.0 ** -126


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 100, 4096])
def test_in_place_and_misaligned_rows(d, dtype):
    """out = x, out_residual = residual; then bases one element past 16-byte
    alignment, inside a larger buffer whose margins stay as they were."""
    import torch

    from rejection_sampling_verify_09_amd import layer_norm

    log(f"[layer] in place and misaligned d={d} {dtype}")
    t = _t(dtype)
    x, r = torch.randn((9, d), device="cuda").to(t), torch.randn((9, d), device="cuda").to(t)
    w, b = torch.randn((d,), device="cuda").to(t), torch.randn((d,), device="cuda").to(t)
    y, _, h = layer_norm(x, w, b, residual=r)
    x2, r2 = x.clone(), r.clone()
    out, _, hr = layer_norm(x2, w, b, residual=r2, out=x2, out_residual=r2)
    assert out.data_ptr() == x2.data_ptr() and torch.equal(x2, y) and torch.equal(r2, h)
    x3, r3 = x.clone(), r.clone()
    layer_norm(x3, w, b, residual=r3, out=r3, out_residual=x3)
    assert torch.equal(r3, y) and torch.equal(x3, h)

    def off(v):
        buf = torch.full((v.numel() + 9,), 7.0, device="cuda", dtype=t)
        buf[1:1 + v.numel()] = v.reshape(-1)
        return buf, buf[1:1 + v.numel()].view(v.shape)

    bufs = [off(v) for v in (x, w, b, r, torch.zeros_like(x), torch.zeros_like(x))]
    xo, wo, bo, ro, oo, ho = (v for _, v in bufs)
    layer_norm(xo, wo, bo, residual=ro, out=oo, out_residual=ho)
    assert torch.equal(oo, y) and torch.equal(ho, h)
    for buf, v in bufs:
        assert buf[0].item() == 7.0 and (buf[1 + v.numel():] == 7.0).all()


def test_empty_batches_and_leading_dimensions():
    import torch

    from rejection_sampling_verify_09_amd import layer_norm

    out, scale, h = layer_norm(torch.empty((0, 64), device="cuda"))
    assert out.shape == (0, 64) and scale is None and h is None
    x = torch.randn((2, 3, 64), device="cuda")
    y, scale, _ = layer_norm(x, out_dtype=torch.float8_e4m3fn)
    assert y.shape == x.shape and scale.shape == (2, 3)
    a, s, _ = layer_norm(x.view(6, 64), out_dtype=torch.float8_e4m3fn)
    assert torch.equal(a.view(torch.uint8), y.view(6, 64).view(torch.uint8)) and torch.equal(s, scale.view(6))
