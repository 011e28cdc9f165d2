"""The gated recurrence's and layer norm's C entry points without a GPU: bad
arguments get the documented status before any launch."""
import ctypes

import pytest

from selective_state_space_54_b200 import _lib
from selective_state_space_54_b200.build import build

INV, UNS, WS = _lib.SSM_ERR_INVALID_ARG, _lib.SSM_ERR_UNSUPPORTED, _lib.SSM_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    build()
    return _lib.load()


def v(x):
    return None if x is None else ctypes.c_void_p(x)


def _shape(**kw):
    d = dict(batch=2, dim=16, seqlen=64, dstate=1, io_dtype=_lib.SSM_BF16)
    d.update(kw)
    return _lib.ssm_shape(**d)


BAD_SHAPES = [(dict(batch=-1), INV), (dict(dim=-1), INV), (dict(seqlen=-2), INV), (dict(dstate=2), INV),
              (dict(dstate=0), INV), (dict(io_dtype=3), UNS), (dict(path=_lib.SSM_PATH_SPLIT_L), UNS),
              (dict(path=_lib.SSM_PATH_LOOKBACK_WS), UNS), (dict(path=17), UNS), (dict(lanes=2), UNS),
              (dict(flags=_lib.SSM_FLAG_ZOH_EXACT), INV), (dict(flags=16), INV),
              (dict(flags=_lib.SSM_FLAG_TOKEN_MAJOR, path=_lib.SSM_PATH_PER_GROUP), UNS),
              (dict(batch=1 << 20, dim=1 << 20, seqlen=1), UNS)]


def _fwd(lib, shape, **over):
    p = dict(u=32, f=64, z=None, bias=None, starts=None, h0=None, y=96, last=None, ws=None, n=0)
    p.update(over)
    return lib.ssm_gated_scan_fwd(None if shape is None else ctypes.byref(shape),
                                  *[v(p[k]) for k in ("u", "f", "z", "bias", "starts", "h0", "y", "last", "ws")],
                                  p["n"], None)


def _bwd(lib, shape, **over):
    p = dict(u=32, f=64, z=None, bias=None, starts=None, h0=None, dout=128, dlast=None, fws=None, du=160, df=192,
             dz=None, dbias=None, dh0=None, ws=None, n=0)
    p.update(over)
    return lib.ssm_gated_scan_bwd(
        None if shape is None else ctypes.byref(shape),
        *[v(p[k]) for k in ("u", "f", "z", "bias", "starts", "h0", "dout", "dlast", "fws", "du", "df", "dz", "dbias",
                            "dh0", "ws")], p["n"], None)


def _step(lib, shape, **over):
    p = dict(u=32, f=64, z=None, bias=None, state=96, y=128)
    p.update(over)
    return lib.ssm_gated_scan_step(None if shape is None else ctypes.byref(shape),
                                   *[v(p[k]) for k in ("u", "f", "z", "bias", "state", "y")], None)


@pytest.mark.parametrize("kw,code", BAD_SHAPES)
def test_gated_bad_shapes(lib, kw, code):
    sh = _shape(**kw)
    assert _fwd(lib, sh) == code and _bwd(lib, sh) == code
    assert lib.ssm_gated_scan_fwd_workspace_bytes(ctypes.byref(sh)) == 0
    assert lib.ssm_gated_scan_bwd_workspace_bytes(ctypes.byref(sh)) == 0
    assert lib.ssm_gated_scan_path(ctypes.byref(sh)) == _lib.SSM_PATH_AUTO
    if "seqlen" not in kw:
        assert _step(lib, _shape(**dict(kw, seqlen=1))) == code


def test_gated_null_shape(lib):
    assert _fwd(lib, None) == INV and _bwd(lib, None) == INV and _step(lib, None) == INV
    assert lib.ssm_gated_scan_fwd_workspace_bytes(None) == 0


@pytest.mark.parametrize("over", [dict(u=None), dict(f=None), dict(y=None), dict(u=33), dict(f=65), dict(z=1),
                                  dict(y=97), dict(bias=6), dict(h0=2), dict(last=5), dict(y=32), dict(y=64),
                                  dict(z=96)])
def test_gated_forward_bad_pointers(lib, over):
    assert _fwd(lib, _shape(), **over) == INV


@pytest.mark.parametrize("over", [dict(u=None), dict(f=None), dict(dout=None), dict(du=None), dict(df=None),
                                  dict(z=320), dict(dz=320), dict(bias=320), dict(dbias=320), dict(du=161),
                                  dict(dbias=2, bias=4), dict(dlast=2), dict(dh0=3), dict(fws=256), dict(du=32),
                                  dict(df=160), dict(dz=128, z=320), dict(dz=160, z=320)])
def test_gated_backward_bad_pointers(lib, over):
    assert _bwd(lib, _shape(), **over) == INV


def test_gated_workspaces(lib):
    save = _lib.SSM_FLAG_SAVE_STATES
    sh = _shape(flags=save)
    need = lib.ssm_gated_scan_fwd_workspace_bytes(ctypes.byref(sh))
    # the state entering every 64-step chunk, and the header
    assert need == 0 or need >= 256 + 4 * 2 * 16
    assert _fwd(lib, sh) in (WS, _lib.SSM_ERR_CUDA)
    assert _fwd(lib, sh, ws=256, n=16) in (WS, _lib.SSM_ERR_CUDA)
    assert _fwd(lib, sh, ws=264, n=1 << 20) in (WS, _lib.SSM_ERR_CUDA)
    assert _bwd(lib, _shape()) in (WS, _lib.SSM_ERR_CUDA)
    assert _bwd(lib, sh, fws=272) == INV


def test_gated_empty_problems(lib):
    none = dict(u=None, f=None, y=None)
    assert _fwd(lib, _shape(batch=0), **none) == 0 and _fwd(lib, _shape(dim=0), **none) == 0
    assert _fwd(lib, _shape(seqlen=0), **none) == 0
    assert _step(lib, _shape(batch=0, seqlen=1), u=None, f=None, state=None, y=None) == 0


@pytest.mark.parametrize("over,code", [(dict(u=None), INV), (dict(state=None), INV), (dict(y=None), INV),
                                       (dict(state=98), INV), (dict(y=32), INV), (dict(y=96), INV),
                                       (dict(state=64), INV)])
def test_step_bad_pointers(lib, over, code):
    assert _step(lib, _shape(seqlen=1), **over) == code


def test_step_is_one_token(lib):
    for L in (0, 2, 64):
        assert _step(lib, _shape(seqlen=L)) == INV
    assert _step(lib, _shape(seqlen=1, flags=_lib.SSM_FLAG_SAVE_STATES)) == UNS
    assert _step(lib, _shape(seqlen=1, path=_lib.SSM_PATH_LOOKBACK)) == UNS


def _norm(lib, rows=4, dim=32, io=_lib.SSM_BF16, rd=_lib.SSM_BF16, x=32, res=None, w=64, b=None, eps=1e-5, y=96,
          ro=None):
    return lib.ssm_layer_norm(rows, dim, io, rd, v(x), v(res), v(w), v(b), eps, v(y), v(ro), None)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), INV), (dict(dim=-1), INV), (dict(io=5), UNS), (dict(rd=7), UNS),
    (dict(io=_lib.SSM_F32, rd=_lib.SSM_BF16), UNS), (dict(eps=-1e-3), INV), (dict(eps=float("nan")), INV),
    (dict(eps=float("inf")), INV), (dict(x=None), INV), (dict(w=None), INV), (dict(y=None), INV), (dict(x=33), INV),
    (dict(w=66), INV), (dict(b=3), INV), (dict(res=128), INV), (dict(ro=128), INV), (dict(y=32), INV),
    (dict(res=128, ro=32), INV), (dict(res=128, ro=96), INV), (dict(res=130, ro=160, rd=_lib.SSM_F32), INV)])
def test_norm_bad_arguments(lib, kw, code):
    assert _norm(lib, **kw) == code


def test_norm_empty(lib):
    assert _norm(lib, rows=0, x=None, y=None) == 0 and _norm(lib, dim=0, x=None, w=None, y=None) == 0


def _norm_bwd(lib, rows=4, dim=32, io=_lib.SSM_BF16, rd=_lib.SSM_BF16, s=32, w=64, eps=1e-5, dy=96, dro=None, dx=128,
              dres=None, dw=160, db=None, ws=None, n=0):
    return lib.ssm_layer_norm_bwd(rows, dim, io, rd, v(s), v(w), eps, v(dy), v(dro), v(dx), v(dres), v(dw), v(db),
                                  v(ws), n, None)


@pytest.mark.parametrize("kw", [
    dict(rows=-1), dict(s=None), dict(w=None), dict(dy=None), dict(dx=None), dict(dw=None), dict(dres=256),
    dict(rd=_lib.SSM_F32), dict(dx=32), dict(dx=96), dict(dro=128), dict(dw=6), dict(db=2), dict(eps=-1.0),
    dict(rd=_lib.SSM_F32, dres=32), dict(rd=_lib.SSM_F32, s=34, dres=256)])
def test_norm_backward_bad_arguments(lib, kw):
    assert _norm_bwd(lib, **kw) == INV


def test_norm_backward_workspace(lib):
    assert _norm_bwd(lib) in (WS, _lib.SSM_ERR_CUDA)
    assert lib.ssm_layer_norm_bwd_workspace_bytes(-1, 8) == 0


def test_injected_failures_reach_the_layer_operators(lib, capfd):
    lib.ssm_scan_test_fail_next(3)
    assert _norm(lib, rows=-1) == INV  # checks first: nothing consumed
    assert _norm(lib) == _lib.SSM_ERR_CUDA
    assert _step(lib, _shape(seqlen=1)) == _lib.SSM_ERR_CUDA
    assert _norm(lib, res=256, ro=256) == _lib.SSM_ERR_CUDA  # in place
    assert capfd.readouterr().err.count("launch failure") == 3
    lib.ssm_scan_test_fail_next(0)


def test_python_refuses_what_is_not_on_a_gpu():
    import torch
    import selective_state_space_54_b200 as ssm
    x = torch.zeros((2, 4, 8))
    with pytest.raises(ValueError):
        ssm.gated_scan_fwd(x, x)
    with pytest.raises(ValueError):
        ssm.gated_scan_bwd(x, x, None, None, x)
    with pytest.raises(ValueError):
        ssm.gated_scan_step(x[0], x[0], state=x[0])
    with pytest.raises(ValueError):
        ssm.layer_norm(x, x[0, 0])
    with pytest.raises(ValueError):
        ssm.layer_norm_bwd(x, x[0, 0], None, x)
    with pytest.raises(ValueError):
        ssm.gated_scan_shape(x[0])
    with pytest.raises(TypeError):
        ssm.gated_scan_shape(x.half())
