"""Ends of the ranges that sv_rms_norm, sv_linear and sv_adjust_logits accept,
without a GPU: refusals only, which are answered before any HIP call."""
import ctypes

import pytest

from rejection_sampling_verify_09_amd import _lib as L


def P(i):
    """Addresses a terabyte apart, never dereferenced."""
    return ctypes.c_void_p((i + 1) << 40)


@pytest.mark.parametrize("d", [1, 64, 511, 512])
@pytest.mark.parametrize("rows", [(1 << 26) - 3, (1 << 26) - 2, (1 << 26) - 1, 1 << 26])
def test_rms_norm_counts_the_rows_that_fill_up_the_last_workgroup(rows, d):
    """Rows of one wave go four to a workgroup, so that 2^26 - 3 rows take the 2^32 threads of 2^26."""
    assert L.lib().sv_rms_norm(P(0), None, P(2), 1e-6, P(30), None, None, rows, d, L.SV_BF16, L.SV_BF16, None) == L.SV_ERR_SHAPE


@pytest.mark.parametrize("d,rows", [(513, 1 << 25), (1024, 1 << 25), (8192, 1 << 22), (65536, 1 << 22)])
def test_rms_norm_refuses_rows_past_one_launch(rows, d):
    assert L.lib().sv_rms_norm(P(0), None, P(2), 1e-6, P(30), None, None, rows, d, L.SV_BF16, L.SV_BF16, None) == L.SV_ERR_SHAPE
