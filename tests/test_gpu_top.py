"""GPU parity of top_logits with the float64 oracle: values and tokens equal,
the log-sum-exp within the bound of its float32 sum.

u = 2^-24.  An exponential's argument is rounded once (a fused product and
sum) and carries the rounding of log2(e) / T over its distance from the
reference, which lies 8 powers of two below the maximum at most: 2.5 u (|x - m| /
T + 8 ln 2) of its value, within 4 u |x - m| / T + 14 u, and 2 u from exp2 itself.
The sum of a thread's V / threads terms, of a wave and of a workgroup is less
than D = V / threads + 8 + 22 deep (a thread's terms are summed in runs of 8,
two at a time, so that its depth is V / (8 threads) + 5: the 14 u are within D), so
the sum is off by (4 E + D + 4) u, E being the mean of |x - m| / T under the
distribution; log turns that into an absolute error, and the result is rounded
once."""
import math

import numpy as np
import pytest

from oracle import fine_tune as ref
from tests.harness import log

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _t(name):
    import torch

    return {"f32": torch.float32, "bf16": torch.bfloat16}[name]


def threads(V, dtype):
    run = 4 if dtype == "f32" else 8
    return min(1024, max(64, -(-V // run) // 64 * 64))


def sum_bound(x, T, V, dtype):
    """Relative bound of a float32 sum of exponentials over x (finite or -inf)."""
    z = (x[x > -np.inf] - np.max(x)) / T
    p = np.exp(z)
    return (4 * float(np.sum(p * -z) / np.sum(p)) + V / threads(V, dtype) + 8 + 22 + 4) * U


def check(x, k, T=1.0, rows=None):
    import torch

    from rejection_sampling_verify_09_amd import top_logits

    dtype = "f32" if x.dtype == torch.float32 else "bf16"
    V = x.shape[-1]
    values, index, lse = top_logits(x, k, temperature=T)
    assert values.dtype == torch.float32 and index.dtype == torch.int32 and lse.dtype == torch.float32
    xs = x.float().cpu().numpy()
    v, i, s = values.cpu().numpy(), index.cpu().numpy(), lse.cpu().numpy()
    for r in range(x.shape[0]) if rows is None else rows:
        wv, wi, ws = ref.top_logits(xs[r], k, T)
        assert np.array_equal(i[r], wi), (r, i[r][:8], wi[:8])
        assert np.array_equal(v[r], wv.astype(np.float32), equal_nan=True)
        if math.isnan(ws) or math.isinf(ws):
            assert np.array_equal(s[r], np.float32(ws), equal_nan=True), (s[r], ws)
        else:
            tol = sum_bound(xs[r].astype(np.float64), T, V, dtype) + U * abs(ws)
            assert abs(float(s[r]) - ws) <= tol, (s[r], ws, tol)
    again = top_logits(x, k, with_lse=False)
    assert again[2] is None and torch.equal(again[1], index) and torch.equal(again[0].nan_to_num(), values.nan_to_num())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,V,k", [
    (1, 1, 1), (3, 5, 5), (2, 63, 10), (4, 64, 64), (3, 100, 100), (5, 513, 1), (2, 520, 64), (3, 1000, 256), (2, 1500, 1024),
    (4, 4104, 64), (2, 8193, 20), (3, 8192, 1024), (300, 2049, 7), (3, 24979, 33), (2, 32000, 8), (6, 128256, 64),
    (2, 128256, 1024), (3, 152064, 256), (1, 262144, 1), (2, 262145, 100), (1, 300001, 17), (1, 2097152, 50)])
def test_matches_the_oracle(rows, V, k, dtype):
    import torch

    g = torch.Generator(device="cuda")
    g.manual_seed(V * 1009 + k)
    for T, spread in ((1.0, 2.0), (0.6, 8.0), (3.0, 0.05)):
        log(f"[top] rows={rows} V={V} k={k} {dtype} T={T} spread={spread}")
        check((torch.randn((rows, V), device="cuda", generator=g) * spread).to(_t(dtype)), k, T)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V,k", [(70, 70), (3000, 64), (24979, 300), (128256, 64), (200000, 1000)])
def test_rows_in_order_of_many_equal_values_and_masked(V, k, dtype):
    import torch

    log(f"[top] orders and ties V={V} k={k} {dtype}")
    g = torch.Generator(device="cuda")
    g.manual_seed(V)
    x = torch.randn((14, V), device="cuda", generator=g) * 3
    inf = float("inf")
    x[0] = x[0].sort(descending=True).values          # all of the list next to each other
    x[1] = x[1].sort().values
    x[2] = 1.5                                         # one value
    x[3] = -inf                                        # nothing left
    x[4] = torch.where(torch.rand(V, device="cuda", generator=g) < 20 / V, x[4], -inf)  # fewer left than k
    x[5] = x[5].round()                                # a few values, each many times
    x[6] = torch.where(torch.arange(V, device="cuda") % 2 == 0, 0.0, -0.0)
    x[7, 3:] = -inf
    x[8] = torch.finfo(torch.float32 if dtype == "f32" else torch.bfloat16).min  # masked by the lowest value
    x[8, V // 2:V // 2 + 9] = torch.arange(9, device="cuda").float()
    x[9, V - 1] = inf
    x[9, 5] = inf
    x[10, ::7] = -inf
    x[11] = torch.arange(V, device="cuda") // 100 % 2  # runs of ones
    x[12] = x[12].abs() * 1e-40                        # below the normal numbers
    x[13] = (torch.arange(V, device="cuda") >= V - k // 2).float()  # fewer large ones than k, at the end
    check(x.to(_t(dtype)), k)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_nan(dtype):
    import torch

    x = torch.randn((4, 5000), device="cuda")
    nan, inf = float("nan"), float("inf")
    x[0, 4321] = nan
    x[1, 17], x[1, 3], x[1, 4000] = nan, inf, -inf
    x[2] = nan
    x[3, 11] = -torch.tensor(nan)
    check(x.to(_t(dtype)), 40)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V,k", [(5000, 300), (128256, 1000), (200000, 1024)])
def test_many_nan_and_infinities_and_long_lists(V, k, dtype):
    """More reach the bound than the list holds, and threads with NaN or
    infinities, few to all of them, have no maximum to go by."""
    import torch

    log(f"[top] many NaN V={V} k={k} {dtype}")
    g = torch.Generator(device="cuda")
    g.manual_seed(V)
    nan, inf = float("nan"), float("inf")
    x = torch.randn((8, V), device="cuda", generator=g)
    at = [torch.randperm(V, device="cuda", generator=g) for _ in range(8)]
    x[0, at[0][:100]], x[0, at[0][100:300]] = nan, inf
    x[1, at[1][:k + 50]] = nan
    x[2, at[2][:k - 7]] = inf
    x[3, :V // 2] = nan
    x[4, 3::8] = inf
    x[5] = torch.where(torch.rand(V, device="cuda", generator=g) < 0.9, x[5].round(), inf)
    x[6, at[6][:5]], x[6, at[6][5:V - 40]] = nan, -inf
    x[7, at[7][:30]] = torch.finfo(torch.bfloat16).max
    check(x.to(_t(dtype)), k)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [1000, 24979, 128256])
def test_misaligned_rows_and_margins(V, dtype):
    """Logits and outputs one element past alignment, inside larger buffers that
    stay as they were; the same result as aligned."""
    import torch

    from rejection_sampling_verify_09_amd import top_logits

    log(f"[top] misaligned V={V} {dtype}")
    t, rows, k = _t(dtype), 5, 48
    x = torch.randn((rows, V), device="cuda").to(t)
    # what lies around the rows would win if it were read as theirs
    buf = torch.full((rows * V + 32,), 1e30, device="cuda", dtype=t)
    buf[1:1 + rows * V] = x.view(-1)
    ov = torch.full((rows * k + 9,), 7.0, device="cuda")
    oi = torch.full((rows * k + 9,), 7, device="cuda", dtype=torch.int32)
    os = torch.full((rows + 9,), 7.0, device="cuda")
    view = lambda b, n, *s: b[1:1 + n].view(*s)  # noqa: E731
    got = top_logits(view(buf, rows * V, rows, V), k, out_values=view(ov, rows * k, rows, k),
                     out_index=view(oi, rows * k, rows, k), out_lse=view(os, rows, rows))
    for a, b in zip(got, top_logits(x, k)):
        assert torch.equal(a, b)
    for b, n in ((ov, rows * k), (oi, rows * k), (os, rows)):
        assert b[0].item() == 7 and (b[1 + n:] == 7).all()
    check(x, k)


def test_empty_batches_and_leading_dimensions():
    import torch

    from rejection_sampling_verify_09_amd import SpecVerifyError, top_logits

    v, i, s = top_logits(torch.empty((0, 50), device="cuda"), 3)
    assert v.shape == (0, 3) and i.shape == (0, 3) and s.shape == (0,)
    x = torch.randn((2, 3, 50), device="cuda")
    v, i, s = top_logits(x, 3)
    assert v.shape == (2, 3, 3) and s.shape == (2, 3)
    w = top_logits(x.view(6, 50), 3)
    assert torch.equal(v.view(6, 3), w[0]) and torch.equal(i.view(6, 3), w[1]) and torch.equal(s.view(6), w[2])
    with pytest.raises(SpecVerifyError):
        top_logits(x, 51)


def test_more_rows_than_compute_units_hold():
    import torch

    x = torch.randn((20000, 300), device="cuda").bfloat16()
    log("[top] 20000 rows of 300")
    check(x, 12, rows=list(range(0, 20000, 997)) + [19999])


def test_element_offsets_past_32_bits():
    """2^31 + 2^20 logits: the last rows' addresses do not fit 32 bits."""
    import torch

    from rejection_sampling_verify_09_amd import top_logits

    V = 2097152
    rows = 1025
    log(f"[top] {rows} rows of {V}")
    x = torch.zeros((rows, V), device="cuda", dtype=torch.bfloat16)
    at = (torch.arange(rows, device="cuda") * 2039) % V
    x[torch.arange(rows, device="cuda"), at] = 3.0
    v, i, s = top_logits(x, 2)
    assert torch.equal(i[:, 0].long(), at) and (v[:, 0] == 3).all() and (v[:, 1] == 0).all()
    assert torch.equal(i[:, 1], (at == 0).int())
    assert (s - math.log(V - 1 + math.exp(3))).abs().max().item() < 1e-4
