"""How many compilers the build starts, whatever MAX_JOBS holds."""
import os

import pytest

from rejection_sampling_verify_09_amd import build


@pytest.mark.parametrize("value,jobs", [
    ("1", 1), ("3", 3), (" 2 ", 2), ("16", 8), ("0", None), ("-4", None), ("", None), ("all", None), ("2.5", None), (None, None)])
def test_max_jobs(monkeypatch, value, jobs):
    if value is None:
        monkeypatch.delenv("MAX_JOBS", raising=False)
    else:
        monkeypatch.setenv("MAX_JOBS", value)
    assert build._jobs() == (jobs or max(1, min(8, len(build.SOURCES), os.cpu_count() or 1)))
