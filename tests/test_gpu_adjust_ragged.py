"""Ragged batches of few sequences, whose rows are split among many workgroups
by the longest one: sequences from none of max_k drafts to all of them."""
import numpy as np
import pytest

from tests.harness import log
from tests.test_gpu_adjust import _bits, call, check, make

pytestmark = pytest.mark.gpu

LENGTHS = {"all or none": (64, 0), "none at first": (0, 0, 64, 1), "one each": (1, 1, 1), "steps of a group": (3, 4, 5, 8, 0, 64)}


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("bonus", [0, 1])
@pytest.mark.parametrize("name", list(LENGTHS))
def test_draft_lengths_far_below_the_longest(name, bonus, dtype):
    import torch

    log(f"[adjust ragged] {name}, bonus {bonus}, {dtype}")
    ks = LENGTHS[name]
    c = make(len(name), B=len(ks), R=0, K=64, V=1500, cap=300, dtype=dtype, ks=ks, bonus=bonus, nbias=30, mask="index")
    got = call(c)
    check(c, got)
    mine = c["logits"].clone()
    call(c, out=mine, logits=mine)
    assert torch.equal(mine.view(_bits(c)), got.view(_bits(c)))


def test_batches_whose_rows_all_belong_to_one_sequence():
    """No row of the others is touched, in front of it or behind."""
    import torch

    log("[adjust ragged] one sequence has every row")
    for ks in ((0, 20, 0), (20, 0, 0), (0, 0, 20)):
        c = make(9, B=3, R=0, K=64, V=900, cap=50, dtype="f32", ks=ks, bonus=0, nbias=12, mask="rows")
        n = c["logits"].numel()
        buf = torch.full((n + 16,), 7.0, device="cuda")
        out = buf[8:8 + n].view(c["logits"].shape)
        check(c, call(c, out=out))
        assert (buf[:8] == 7).all() and (buf[8 + n:] == 7).all()
    assert np.array_equal(out.cpu().numpy(), call(c).cpu().numpy())
