"""The e4m3 output of rms_norm is its float32 row over its scale, rounded once:
rows whose elements lie on, next to and between the ties of e4m3 times an
uneven scale, where one rounding more on the way gives the neighbouring value.

The rows are made so that every float32 step before the division is exact: all
elements of x are 1 and eps is below half a step of 1, so that the mean of the
squares plus eps and its root are 1 and the output is the weight."""
import numpy as np
import pytest

from oracle import last_layer as ref
from tests.harness import log

pytestmark = pytest.mark.gpu


def nearest_e4m3(v):
    """float64 values of magnitude at most 448 rounded to e4m3, ties to the even pattern."""
    pos = ref.e4m3_values()[:0x7F]  # 0 .. 448, by bit pattern
    a = np.abs(v)
    hi = np.clip(np.searchsorted(pos, a), 0, len(pos) - 1)
    lo = np.maximum(hi - 1, 0)
    dh, dl = pos[hi] - a, a - pos[lo]
    pick = np.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, lo)
    return np.copysign(pos[pick], v)


def tie_row(largest, d):
    """A float32 row [d] whose largest magnitude is `largest`: the floats around every tie of e4m3 times its scale."""
    scale = np.float32(largest) / np.float32(448.0)
    pos = ref.e4m3_values()[:0x7F]
    ties = (pos[1:] + pos[:-1]) / 2
    near = np.float32(ties * np.float64(scale))
    bits = (near.view(np.int32)[:, None] + np.arange(-6, 7)).astype(np.int32).reshape(-1)
    row = bits.view(np.float32)
    row = row[row < largest]
    out = np.full(d, np.float32(largest))
    n = min(d - 1, row.size)
    out[1:1 + n] = row[:n] * np.where(np.arange(n) % 2, -1, 1)
    return out, scale


@pytest.mark.parametrize("d", [1700, 4096, 4099])
@pytest.mark.parametrize("largest", [448.0 * 1.1, 3.0, 0.7, 448.0 * 1.9999, 123.456])
def test_e4m3_rounds_the_row_over_its_scale_once(largest, d):
    import torch

    from rejection_sampling_verify_09_amd import rms_norm

    log(f"[norm] ties of e4m3, largest {largest}, d={d}")
    w, scale = tie_row(np.float32(largest), d)
    x = torch.ones((3, d), device="cuda")
    wt = torch.from_numpy(w).cuda()
    y, _, _ = rms_norm(x, wt, eps=1e-9)
    assert torch.equal(y, wt.expand(3, d))  # the steps before the scale are exact
    out, s, _ = rms_norm(x, wt, eps=1e-9, out_dtype=torch.float8_e4m3fn)
    assert (s.cpu().numpy() == scale).all()
    want = nearest_e4m3((w / scale).astype(np.float64))
    got = out.float().cpu().numpy().astype(np.float64)
    assert np.array_equal(got, np.tile(want, (3, 1)))
    # the test's own sharpness: a product with the rounded reciprocal differs somewhere
    inv = np.float32(1.0) / scale
    other = nearest_e4m3(np.clip((w * inv).astype(np.float64), -448, 448))
    assert (other != want).any()


def test_e4m3_of_a_row_whose_output_overflows():
    """An infinite element makes the scale infinite: it comes out NaN, the finite ones as zeros."""
    import torch

    from rejection_sampling_verify_09_amd import rms_norm

    log("[norm] e4m3 of an infinite element")
    w = torch.ones((256,), device="cuda")
    w[7] = float("inf")
    out, s, _ = rms_norm(torch.ones((2, 256), device="cuda"), w, out_dtype=torch.float8_e4m3fn)
    o = out.float()
    assert torch.isinf(s).all() and torch.isnan(o[:, 7]).all()
    o[:, 7] = 0
    assert (o == 0).all()
