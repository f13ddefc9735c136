"""The debug build's switches do nothing in the ordinary library."""
import os

import pytest


def test_wait_limit(zs):
    if os.environ.get("ZS_CHECKED") == "1":
        pytest.skip("the debug build is loaded")
    L = zs.lib()
    assert L.zero_debug_wait_limit(5) == 0
    assert L.zero_debug_wait_limit(-1) == zs.ZS_ERR_ARG and L.zero_debug_wait_limit((1 << 20) + 1) == zs.ZS_ERR_ARG
