"""The workspace of the norms' gradients, without a GPU: rows whose sums are
folded in it have room for that, and a call with less is refused."""
import ctypes

import pytest

from rejection_sampling_verify_09_amd import _lib as L


def P(i):
    return ctypes.c_void_p((i + 1) << 44)


@pytest.mark.parametrize("d,stride", [(1, 4), (4, 4), (6, 8), (7, 8), (16385, 16388), (65536, 65536)])
def test_wide_and_narrow_rows_fold_in_the_workspace(d, stride):
    f = L.lib().sv_norm_backward_workspace
    assert f(256 * 1024, d) == 256 * stride * 8
    rows = 256 * 1024 + 1  # 1025 turns on 256 workgroups, the last of which have none
    groups = -(-rows // 1025)
    assert f(rows, d) == 2 * groups * stride * 8
    assert f(2 ** 30, d) == 2 * 256 * stride * 8


@pytest.mark.parametrize("d", [8, 64, 4096, 16384])
def test_other_rows_fold_in_lds(d):
    f = L.lib().sv_norm_backward_workspace
    for rows in (8 * 256 * 1024 + 1, 2 ** 30):
        assert f(rows, d) <= 256 * d * 8


@pytest.mark.parametrize("rows,d", [(256 * 1024 + 1, 4), (2 ** 30, 7), (300001, 16400)])
def test_a_smaller_workspace_is_refused(rows, d):
    n = L.lib().sv_norm_backward_workspace(rows, d)
    call = lambda nbytes, dw=P(5), db=P(6): L.lib().sv_layer_norm_backward(  # noqa: E731
        P(0), P(1), None, None, 1e-5, P(4), dw, db, P(7), nbytes, rows, d, L.SV_BF16, None)
    assert call(n - 16) == L.SV_ERR_WORKSPACE
    assert call(n // 2) == L.SV_ERR_WORKSPACE
    assert call(n // 2 - 16, db=None) == L.SV_ERR_WORKSPACE
    assert call(n // 2 - 16, dw=None) == L.SV_ERR_WORKSPACE
    assert L.lib().sv_rms_norm_backward(P(0), P(1), None, None, 1e-5, P(4), P(5), P(7), n // 2 - 16, rows, d, L.SV_BF16,
                                        None) == L.SV_ERR_WORKSPACE
