"""Values that the gated recurrence's runs have to carry whatever lies between: what is
not a number, under packed sequences and gates that close; and the factors of gates that
are nearly closed, digit by digit."""
import numpy as np
import pytest

import synth
from gpu_util import to_f64
from test_gated_gpu import PATHS, Case

pytestmark = pytest.mark.gpu

# (batch, dim, seqlen) whose tiles are groups of their own, and whose tiles share groups
SHAPES = {False: [(2, 30, 9000), (1, 3, 9000)], True: [(24, 200, 700), (1, 70, 2500)]}


@pytest.mark.parametrize("path,tok", PATHS)
@pytest.mark.parametrize("which", [0, 1])
@pytest.mark.parametrize("f_mean", [-8.0, 1.0])
@pytest.mark.parametrize("packed", ["absent", "none", "before", "between"])
def test_not_a_number_lasts_until_a_start(cuda_device, path, tok, which, f_mean, packed):
    # A NaN in u reaches every later state of its sequence, one in dy every earlier gradient,
    # one in f both, however small the product of the gates between has become (at a mean of
    # -8 it is 0 in fp32 after 11 steps) and whether or not a starts tensor is given: the
    # reference's pattern, element by element
    batch, dim, L = SHAPES[tok][which]
    at = {"u": L // 3, "f": L // 2 + 5, "dy": L - L // 4}

    def edit(raw, case):
        case.starts = None if packed == "absent" else np.zeros((batch, L), bool)
        if packed in ("before", "between"):
            case.starts[:, [0, 7, L // 3 - 20]] = True
        if packed == "between":
            case.starts[:, [L // 3 + 130, L // 2 + 70, L // 2 + 71]] = True
        for i, (k, t) in enumerate(at.items()):
            raw[k][0, i, t] = np.nan
    c = Case(cuda_device, batch, dim, L, synth.F32, 60, tok=tok, f_mean=f_mean, edit=edit, bias=False)
    y, last = c.fwd(path)
    g = c.bwd(path)
    with np.errstate(invalid="ignore"):
        ref, rb = c.ref(), c.ref_bwd()
    pairs = [("y", c.rows(y), ref["y"]), ("last_state", to_f64(last), ref["last_state"])]
    pairs += [(k, c.rows(g[k]), rb[k]) for k in ("du", "df", "dz")]
    pairs += [("dinitial_state", to_f64(g["dinitial_state"]), rb["dinitial_state"])]
    for k, got, want in pairs:
        bad = np.isnan(got) != np.isnan(want)
        assert not bad.any(), (k, int(bad.sum()), np.argwhere(bad)[:3].tolist())
        assert np.isnan(want).any() or k in ("dinitial_state", "last_state")
        assert np.isfinite(got[~np.isnan(want)]).all(), k


# The factor a = 1 / (1 + e^-x) of one step, x the logit with |x| <= 18, |f_bias| <= 2, relative.
# Nearly closed gates (e^x < 1/32) as e^x g:
#   exponent   x log2(e) in fp32: its own rounding and f_bias log2(e)'s, 2^-24 each of 26 and 3,
#              and the constant's 2^-25 of 26, times ln 2:               1.8e-6
#   functions  2^v to 2^-22, the reciprocal to 2^-23, 1 + e^x to 2^-24:   4.2e-7
# the others as 1 - g, where a >= 1/33 and |x| counts up to 3.5:
#   g          to 2^-24 + 2^-23, of 1/33:                                5.9e-6
#   exponent   as above, 2^-24 of 5.1 and 3 and 2^-25 of 5.1, times ln 2:  4.4e-7
# and in both the step itself, its product, its sum and a run's join, 2^-24 each: 1.8e-7.
# So less than DELTA a step in all, relative to the state that the same gates make of the
# absolute values (no cancellation), plus what is flushed below 2^-126.
DELTA = 6.6e-6
TINY = 1e-37


def _absolute(c):
    """States and gradients of the absolute values, and the number of steps behind (up) and
    ahead (down) of each that are not exactly open (a = 1)."""
    from oracle.layer import sigmoid
    x = c.n["f"] + (0 if c.n["b"] is None else c.n["b"][None, :, None].astype(np.float64))
    a, g = sigmoid(x), sigmoid(-x)
    u, dy = np.abs(c.n["u"]), np.abs(c.n["dy"])
    add = g * u if c.tied else u
    H, G = np.zeros_like(u), np.zeros_like(u)
    h, P = np.abs(c.n["h0"]).astype(np.float64), np.abs(c.n["dlast"]).astype(np.float64)
    prev = np.zeros_like(u)
    for t in range(c.L):
        prev[:, :, t] = h
        h = H[:, :, t] = a[:, :, t] * h + add[:, :, t]
    for t in range(c.L - 1, -1, -1):
        G[:, :, t] = dy[:, :, t] + P
        P = a[:, :, t] * G[:, :, t]
    step = (a < 1).astype(np.float64)
    up = np.cumsum(step, 2)
    down = np.cumsum(step[:, :, ::-1], 2)[:, :, ::-1]
    return {"H": H, "prev": prev, "G": G, "P": P, "a": a, "g": g, "up": up, "down": down}


def _digits(c, path):
    """Every output against the reference, element by element."""
    assert c.t["z"] is None and c.starts is None
    m = _absolute(c)
    worst = {}

    def near(name, got, want, scale, steps):
        excess = np.abs(got - want) - (DELTA * (steps + 1) * scale + TINY)
        worst[name] = float(np.max(np.abs(got - want) / (DELTA * (steps + 1) * scale + TINY)))
        assert (excess <= 0).all(), (name, worst[name], np.unravel_index(np.argmax(excess), excess.shape))
    y, last = c.fwd(path)
    g = c.bwd(path)
    ref, rb = c.ref(), c.ref_bwd()
    near("last_state", to_f64(last), ref["last_state"], m["H"][:, :, -1], m["up"][:, :, -1])
    near("dinitial_state", to_f64(g["dinitial_state"]), rb["dinitial_state"], m["P"], m["down"][:, :, 0])
    if c.dtype == synth.F32:
        near("y", c.rows(y), ref["y"], m["H"], m["up"])
        near("du", c.rows(g["du"]), rb["du"], m["G"] * (m["g"] if c.tied else 1), m["down"])
        near("df", c.rows(g["df"]), rb["df"], m["G"] * m["a"] * m["g"] * (m["prev"] + np.abs(c.n["u"]) * c.tied),
             m["up"] + m["down"])
    return worst


@pytest.mark.parametrize("path,tok", PATHS)
@pytest.mark.parametrize("dtype", [synth.BF16, synth.F32])
@pytest.mark.parametrize("tied", [True, False])
@pytest.mark.parametrize("logit", [-1.0, -3.0, -5.0, -8.0, -12.0])
def test_nearly_closed_gates_keep_their_digits(cuda_device, path, tok, dtype, tied, logit):
    # pieces of a few steps, whose gradients of the initial state (and states, where the input
    # is small or 0) are products of such factors
    for L in (1, 2, 5):
        for u in ("normal", "none"):
            def edit(raw, case):
                raw["f"][:] = np.clip(0.7 * (raw["f"] - 1.0), -3, 3) + logit
                if u == "none":
                    raw["u"][:] = 0
            c = Case(cuda_device, 2, 70, L, dtype, 70 + L, z=False, tied=tied, tok=tok, edit=edit)
            c.n["b"] = np.clip(c.n["b"], -2, 2)
            c.t["b"].clamp_(-2, 2)
            _digits(c, path)


@pytest.mark.parametrize("path,tok", PATHS)
@pytest.mark.parametrize("dtype", [synth.BF16, synth.F32])
@pytest.mark.parametrize("tied", [True, False])
@pytest.mark.parametrize("which", [0, 1])
def test_closed_gates_far_apart(cuda_device, path, tok, dtype, tied, which):
    # gates that hold the state exactly (f = inf) but for four over the whole sequence, at other
    # steps in every channel, so that the factors pass through lanes', warps' and tiles' runs
    batch, dim, L = SHAPES[tok][which]

    def edit(raw, case):
        g = np.random.default_rng(5)
        raw["f"][:] = np.inf
        raw["u"][:, :, 1:] = 0
        raw["dy"][:, :, :-1] = 0
        for _ in range(4):
            at = g.integers(0, L, (batch, dim, 1))
            np.put_along_axis(raw["f"], at, np.clip(g.normal(-7, 2, at.shape), -14, -1), 2)
        if not tied:
            raw["u"][:, :, ::5] = 0
    c = Case(cuda_device, batch, dim, L, dtype, 80, z=False, bias=False, tied=tied, tok=tok, edit=edit)
    _digits(c, path)


@pytest.mark.parametrize("dtype", [synth.BF16, synth.F32])
@pytest.mark.parametrize("tied", [True, False])
@pytest.mark.parametrize("dim", [77, 264])
def test_nearly_closed_gates_of_single_steps(cuda_device, dtype, tied, dim):
    import torch
    import selective_state_space_54_b200 as ssm
    for logit in (-1.0, -3.0, -5.0, -8.0, -12.0):
        def edit(raw, case):
            raw["f"][:] = np.clip(0.7 * (raw["f"] - 1.0), -3, 3) + logit
            raw["u"][:] = 0
        c = Case(cuda_device, 3, dim, 4, dtype, 90, z=False, bias=False, tied=tied, edit=edit)
        state, ref, m = c.t["h0"].clone(), c.ref(), _absolute(c)
        for t in range(4):
            one = lambda k: c.t[k][:, :, t].contiguous()
            ssm.gated_scan_step(one("u"), one("f"), state=state, tied=tied)
            err = np.abs(to_f64(state) - ref["h"][:, :, t])
            assert (err <= DELTA * (t + 2) * m["H"][:, :, t] + TINY).all(), (logit, t)
        assert torch.isfinite(state).all()
