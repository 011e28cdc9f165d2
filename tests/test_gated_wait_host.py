"""Refusals of the test hook for the gated recurrence's bounded wait, before any launch."""
import ctypes

import pytest

from selective_state_space_54_b200 import _lib
from selective_state_space_54_b200.build import build


@pytest.mark.parametrize("ws,n,us,code", [
    (None, 512, 100, _lib.SSM_ERR_WORKSPACE), (256, 128, 100, _lib.SSM_ERR_WORKSPACE),
    (264, 512, 100, _lib.SSM_ERR_WORKSPACE), (256, 512, 0, _lib.SSM_ERR_INVALID_ARG),
    (256, 512, -5, _lib.SSM_ERR_INVALID_ARG), (256, 512, 1000001, _lib.SSM_ERR_INVALID_ARG)])
def test_bad_arguments(ws, n, us, code):
    build()
    assert _lib.load().ssm_gated_scan_test_wait_timeout(None if ws is None else ctypes.c_void_p(ws), n, us, None) == code
