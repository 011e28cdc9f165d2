"""The shape structs that the gated recurrence's binding hands out are the caller's own:
editing one (a path or flags for a second workspace query) changes no other call."""
import ctypes

import pytest

import selective_state_space_54_b200 as ssm


def _u(*size, dtype="bfloat16"):
    import torch
    return torch.zeros(size, dtype=getattr(torch, dtype))


FIELDS = [name for name, _ in ssm.ssm_shape._fields_]


@pytest.mark.parametrize("kw", [{}, dict(tied=False), dict(save_states=True), dict(token_major=True),
                                dict(path=ssm.SSM_PATH_LOOKBACK)])
def test_an_edited_shape_changes_no_later_one(kw):
    u = _u(2, 16, 64)
    mine = ssm.gated_scan_shape(u, **kw)
    before = [getattr(mine, n) for n in FIELDS]
    for n in FIELDS:
        setattr(mine, n, 77)
    again = ssm.gated_scan_shape(u, **kw)
    assert again is not mine and [getattr(again, n) for n in FIELDS] == before


def test_an_edited_shape_changes_no_call():
    # the struct that calls on such tensors pass to the library
    u = _u(3, 5, 70)
    mine = ssm.gated_scan_shape(u, save_states=True)
    mine.batch = 64
    key = ssm._gated_key(u, True, True, False, ssm.SSM_PATH_AUTO)
    assert ssm._gated_shape(*key).batch == 3
    mine = ssm.gated_scan_shape(_u(4, 9, 1))
    mine.dim = 1 << 20
    ref = ssm._gated_step_ref(4, 9, ssm.SSM_BF16, 0)
    assert ctypes.cast(ref, ctypes.POINTER(ssm.ssm_shape)).contents.dim == 9
