"""The norms' gradients over millions of rows: sums over rows are formed of
parts of at most 1024 rows, so that a row, and a rounding, of the first million
counts as one of the last.

u = 2^-24.  A column's sum over rows is a sum of blocks of up to 1024 rows, one
after another (1024 u of the magnitudes' sum), folded one after another (a u for
each block of a workgroup), joined over up to 8 rows side by side and 256
workgroups (8 + 4 + 16 + 2 u)."""
import pytest

from tests.harness import log
from tests.test_gpu_top import U, _t

pytestmark = pytest.mark.gpu


def _both():
    import rejection_sampling_verify_09_amd as sv

    def rms(*a, **kw):
        return (*sv.rms_norm_backward(*a, **kw), None)

    return ("layer", sv.layer_norm_backward), ("rms", rms)


@pytest.mark.parametrize("rows,d,dtype", [
    ((1 << 20) + 3000, 2048, "bf16"), (3000001, 24, "f32"), (5000003, 200, "bf16"), (2100001, 64, "bf16"),
    (270001, 16384, "bf16"), (264001, 10000, "f32"), (600001, 4, "f32"), (530001, 6, "bf16"), (266001, 16400, "bf16")])
def test_every_row_counts_once(rows, d, dtype):
    """h of +-1 (mean 0, mean square 1, exactly so for these d, whose product with their rounded reciprocal rounds to 1)
    and gradients of -1, 0 and 1, eps below a rounding of 1: every product is -1, 0 or 1, and every sum of them a whole
    number below 2^24, with no rounding at all."""
    import torch

    log(f"[norm sums] rows={rows} d={d} {dtype}")
    g = torch.Generator(device="cuda")
    g.manual_seed(d)
    t = _t(dtype)
    h, dy = torch.empty((rows, d), device="cuda", dtype=t), torch.empty((rows, d), device="cuda", dtype=t)
    dw, db = torch.zeros(d, device="cuda", dtype=torch.float64), torch.zeros(d, device="cuda", dtype=torch.float64)
    pattern = torch.where(torch.arange(d, device="cuda") % 2 == 0, 1.0, -1.0)[torch.randperm(d, device="cuda", generator=g)]
    at = max(1, (1 << 26) // d)
    for r in range(0, rows, at):
        n = min(at, rows - r)
        sign = torch.randint(0, 2, (n, 1), device="cuda", generator=g).mul_(2).sub_(1)
        h[r:r + n] = pattern * sign
        dy[r:r + n] = torch.randint(-1, 2, (n, d), device="cuda", generator=g, dtype=torch.int8)
        db += dy[r:r + n].sum(0, dtype=torch.float64)
        dw += (dy[r:r + n].float() * h[r:r + n].float()).sum(0, dtype=torch.float64)
    assert rows < 2 ** 24
    for name, back in _both():
        _, gw, gb = back(dy, h, eps=2.0 ** -40)
        assert torch.equal(gw.double(), dw), (name, (gw - dw).abs().max())
        if gb is not None:
            assert torch.equal(gb.double(), db), (gb - db).abs().max()


@pytest.mark.parametrize("rows,d", [(1 << 26, 8), (1 << 24, 4), ((1 << 24) + 77, 6)])
def test_roundings_do_not_add_up(rows, d):
    """One row many times, whose gradient a long float32 sum rounds the same way each time."""
    import torch

    log(f"[norm sums] one row {rows} times, d={d}")
    dy = torch.full((rows, d), 1 + 2.0 ** -11, device="cuda")
    row = torch.where(torch.arange(d, device="cuda") % 2 == 0, 1.0, -1.0)
    h = row.expand(rows, d).contiguous()
    turns = -(-rows // (8 if d == 8 else 1) // 256)
    # the sums' own, and 4 u of a term's value: 1 / sqrt of 1 + eps, and two products
    tol = (1024 + turns / 1024 + 30 + 4) * U
    for name, back in _both():
        out, gw, gb = back(dy, h, eps=2.0 ** -40)
        want = rows * (1 + 2.0 ** -11)
        assert ((gw.double() - want * row.double()).abs() <= tol * want).all(), (name, gw / want)
        if gb is not None:
            assert ((gb.double() - want).abs() <= tol * want).all(), (name, gb / want)
        del out


@pytest.mark.parametrize("rows,d,dtype", [(2200001, 24, "bf16"), (600001, 4, "f32"), (266001, 16400, "bf16"), (264001, 10000, "bf16")])
def test_one_sum_alone_in_place_and_in_a_graph(rows, d, dtype):
    """Folded sums: one of the two alone, grad_h over its inputs, and captured and replayed, give the same bits."""
    import torch

    import rejection_sampling_verify_09_amd as sv

    log(f"[norm sums] forms rows={rows} d={d} {dtype}")
    t = _t(dtype)
    h, dy = torch.empty((rows, d), device="cuda", dtype=t).normal_(), torch.empty((rows, d), device="cuda", dtype=t).normal_()
    dres = torch.empty((rows, d), device="cuda", dtype=t).normal_()
    want = sv.layer_norm_backward(dy, h, grad_residual=dres)
    dh = want[0]
    for kw in (dict(with_bias=False), dict(with_weight=False)):
        _, dw, db = sv.layer_norm_backward(dy, h, grad_residual=dres, out=dh, **kw)
        assert (dw is None or torch.equal(dw, want[1])) and (db is None or torch.equal(db, want[2]))
    keep = dh.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = sv.layer_norm_backward(dy, h, grad_residual=dres, out=dh)
    for _ in range(3):
        dh.zero_(), got[1].zero_(), got[2].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(dh, keep) and torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])
    del graph, dh
    got = sv.layer_norm_backward(dy, h, grad_residual=dres, out=dres)
    assert torch.equal(got[0], keep) and torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])
