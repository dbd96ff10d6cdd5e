"""The expert layer's unit lookup on the host (no GPU): whatever unwritten entries of the list
of active experts hold, nothing of them becomes an index, also where no slot names an expert."""
import os

import pytest

from test_sanitizers import CSRC, ENV, HERE, HIPCC, _run


def test_units_without_rows_index_nothing(tmp_path):
    if not os.path.exists(HIPCC):
        pytest.skip("no hipcc")
    exe = str(tmp_path / "moe_units")
    rc, out = _run([HIPCC, "-x", "hip", "--offload-host-only", "-std=c++17", "-O1", "-g",
                    "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
                    "-Xarch_host", "-fno-sanitize-recover=all", "-I", CSRC,
                    os.path.join(HERE, "moe_units_driver.cpp"), "-o", exe])
    assert rc == 0, out
    rc, out = _run([exe], env=ENV, timeout=120)
    assert rc == 0 and "moe units run: ok" in out, out
