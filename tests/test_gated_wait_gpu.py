"""The bounded wait of the gated recurrence's tiles: real calls of many tiles leave the
error word clear, the giving-up branch reports within its limit, and calls that share the
workspace afterwards run as ever."""
import ctypes
import time

import pytest

import synth
from test_gated_gpu import Case, _path

pytestmark = pytest.mark.gpu

# sequences of many tiles: tiles that are groups of their own, and groups of several
SHAPES = {False: [(2, 30, 30000), (1, 3, 70000)], True: [(24, 200, 3000), (1, 70, 9000)]}


@pytest.mark.parametrize("tok", [False, True])
@pytest.mark.parametrize("which", [0, 1])
@pytest.mark.parametrize("dtype", [synth.BF16, synth.F32])
def test_calls_of_many_tiles_report_no_timeout(cuda_device, tok, which, dtype):
    batch, dim, L = SHAPES[tok][which]
    c = Case(cuda_device, batch, dim, L, dtype, 5, tok=tok, starts=0.0005)
    y, last = c.fwd("lookback", check_status=True)
    saved = c.bwd("lookback", save=True, check_status=True)
    again = c.bwd("lookback", save=False, check_status=True)  # the forward's tiles once more
    import torch
    assert torch.isfinite(y.float()).all() and torch.isfinite(last).all()
    assert all(torch.equal(saved[k], again[k]) for k in saved)


def _probe(ws, us):
    import torch
    from selective_state_space_54_b200 import _lib
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    return _lib.load().ssm_gated_scan_test_wait_timeout(ctypes.c_void_p(ws.data_ptr()), ws.nbytes, us, stream)


def test_a_wait_for_nothing_gives_up_and_reports(cuda_device):
    import torch
    import selective_state_space_54_b200 as ssm
    c = Case(cuda_device, 1, 70, 2500, synth.BF16, 6, tok=True)
    shape = ssm.gated_scan_shape(c.t["u"], token_major=True, path=_path("lookback"))
    ws = torch.empty(ssm.gated_scan_fwd_workspace_bytes(shape), dtype=torch.uint8, device=cuda_device)
    want, _ = c.fwd("lookback", workspace=ws, check_status=True)
    torch.cuda.synchronize()
    for us in (1, 20000):
        t = time.perf_counter()
        assert _probe(ws, us) == 0
        with pytest.raises(ssm.ScanError) as e:
            ssm.check(ws)
        assert e.value.code == ssm._lib.SSM_ERR_DEVICE_TIMEOUT
        assert us / 1e6 <= time.perf_counter() - t < us / 1e6 + 1.0
        ssm.check(ws)  # read and cleared
    got, _ = c.fwd("lookback", workspace=ws, check_status=True)
    assert torch.equal(got, want)
