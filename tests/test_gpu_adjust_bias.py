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
