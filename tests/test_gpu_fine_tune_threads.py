"""Calls of several host threads at once, each on a stream of its own, of one
kernel with unlike amounts of LDS: every call's result is what it is alone."""
import threading

import pytest

from tests.harness import log

pytestmark = pytest.mark.gpu


def test_calls_of_two_threads_with_unlike_rows():
    import torch

    import rejection_sampling_verify_09_amd as sv

    log("[fine-tune] two threads")
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    b = torch.bfloat16

    def top(V, k):
        x = torch.randn((8, V), device="cuda", generator=g).to(b)
        return lambda: sv.top_logits(x, k)

    def distill(V, k):
        x = torch.randn((4, V), device="cuda", generator=g).to(b)
        index = torch.randint(0, V, (4, k), device="cuda", generator=g, dtype=torch.int32)
        values = torch.randn((4, k), device="cuda", generator=g)
        return lambda: sv.distill_loss(x, index, values, with_grad=True)

    for one, other in ((top(2000000, 1024), top(128256, 600)), (distill(1048576, 1024), distill(400000, 1000)),
                       (top(200000, 1000), distill(1048576, 64))):
        want = [one(), other()]
        torch.cuda.synchronize()
        bad = []

        def work(call, expect):
            try:
                s = torch.cuda.Stream()
                with torch.cuda.stream(s):
                    for _ in range(100):
                        got = call()
                        s.synchronize()
                        if not all(torch.equal(a, w) for a, w in zip(got, expect)):
                            bad.append("result")
                            return
            except Exception as e:
                bad.append(repr(e))

        threads = [threading.Thread(target=work, args=a) for a in ((one, want[0]), (other, want[1]))]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        assert not bad
