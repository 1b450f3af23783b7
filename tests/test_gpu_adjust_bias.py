"""The biases of adjust_logits where their order and number matter: added to
each other in the order they are listed, in float32, and then to the logit."""
import numpy as np
import pytest

from tests.harness import log

pytestmark = pytest.mark.gpu


def cuda(a):
    import torch

    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def summed(tok, val, V):
    """float32 sums of each token's biases in their order, and which tokens have any."""
    out, has = np.zeros(V, dtype=np.float32), np.zeros(V, dtype=bool)
    for t in np.unique(tok):
        out[t] = np.add.accumulate(val[tok == t], dtype=np.float32)[-1]
        has[t] = True
    return out, has


@pytest.mark.parametrize("n", [2, 16, 17, 40, 900, 1500])
def test_biases_are_added_to_each_other_before_the_logit(n):
    """1e8, whose neighbours are 8 away, and n biases of 3: one by one they would not move it."""
    import torch

    from rejection_sampling_verify_09_amd import adjust_logits

    log(f"[adjust] {n} small biases of a large logit")
    V = 700
    tok, val = np.full(n, 123, dtype=np.int32), np.full(n, 3.0, dtype=np.float32)
    total = np.float32(3 * n)
    lg = torch.full((2, V), 1e8, device="cuda")
    bias = (cuda(np.array([0, n, n], dtype=np.int32)), cuda(tok), cuda(val))
    for out in (None, lg):
        got = adjust_logits(lg, bias=bias, out=out).cpu().numpy()
        want = np.full((2, V), 1e8, dtype=np.float32)
        want[0, 123] = np.float32(1e8) + total
        assert want[0, 123] >= np.float32(1e8) + 8 and np.array_equal(got, want)


def test_biases_at_the_end_of_the_longest_list():
    """Offsets next to 2^31, where positions a few past the last bias do not fit a signed number; all but the last
    60 entries of the list are in no sequence."""
    import torch

    from rejection_sampling_verify_09_amd import adjust_logits

    n, V, m = (1 << 31) - 1, 3000, 60
    log(f"[adjust] the last {m} of {n} biases")
    tok = torch.empty((n,), device="cuda", dtype=torch.int32)
    val = torch.empty((n,), device="cuda", dtype=torch.float32)
    g = np.random.default_rng(3)
    t, v = g.integers(-1, 40, m).astype(np.int32) * 71, g.standard_normal(m).astype(np.float32)
    tok[-m:], val[-m:] = cuda(t), cuda(v)
    cu = torch.tensor([n - m, n - m + 20, n], device="cuda", dtype=torch.int32)
    lg = torch.zeros((2, V), device="cuda")
    for out in (None, lg):
        got = adjust_logits(lg, bias=(cu, tok, val), out=out).cpu().numpy()
        for b, s in enumerate((slice(0, 20), slice(20, m))):
            ok = t[s] >= 0
            assert np.array_equal(got[b], summed(t[s][ok], v[s][ok], V)[0]), b
