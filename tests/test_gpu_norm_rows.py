"""Rows of rms_norm alone, beside others, and beside rows of NaN: bit for bit
the same.  Up to 512 columns four rows share a workgroup."""
import pytest

from tests.harness import log

pytestmark = pytest.mark.gpu


def _bytes(t):
    import torch

    return t.contiguous().view(torch.uint8)


@pytest.mark.parametrize("odt", ["bf16", "f32", "e4m3"])
@pytest.mark.parametrize("rows", [5, 63])
@pytest.mark.parametrize("d", [64, 100, 512, 513, 4096, 20000])
def test_a_row_depends_on_itself_alone(d, rows, odt):
    import torch

    from rejection_sampling_verify_09_amd import rms_norm

    log(f"[norm rows] {rows} x {d} -> {odt}")
    t = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}[odt]
    g = torch.Generator(device="cuda")
    g.manual_seed(d + rows)
    rnd = lambda *s: torch.randn(s, device="cuda", generator=g).bfloat16()  # noqa: E731
    x, r, w = rnd(rows, d), rnd(rows, d), rnd(d)
    size = torch.exp2(torch.randint(-20, 20, (rows, 1), device="cuda", generator=g).float()).bfloat16()
    x, r = x * size, r * size
    out = rms_norm(x, w, residual=r, out_dtype=t)
    assert (out[1] is not None) == (odt == "e4m3")
    pick = sorted({0, 1, 2, 3, 4, rows // 2, rows - 2, rows - 1})
    for i in pick:
        one = rms_norm(x[i:i + 1], w, residual=r[i:i + 1], out_dtype=t)
        for a, b in zip(out, one):
            assert a is None or torch.equal(_bytes(a[i:i + 1]), _bytes(b)), i
    for i in pick:
        x2, r2 = rnd(rows, d) * 3, rnd(rows, d)
        x2[::2] = float("nan")
        r2[1::3] = float("inf")
        x2[i], r2[i] = x[i], r[i]
        among = rms_norm(x2, w, residual=r2, out_dtype=t)
        for a, b in zip(out, among):
            assert a is None or torch.equal(_bytes(a[i:i + 1]), _bytes(b[i:i + 1])), i
