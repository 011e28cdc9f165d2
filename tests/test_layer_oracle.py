"""CPU pins of the fp64 references of the gated recurrence and layer norm:
gradients against central differences, the gated recurrence against the
selective scan's oracle (the gating reduction N = 1, A = -1, B = C = 1 with
exact zero-order hold), and closed forms."""
import numpy as np
import pytest

import oracle
import synth
from oracle import layer


def _case(batch, dim, L, seed):
    g = np.random.default_rng(seed)
    r = lambda *s: g.standard_normal(s)
    return dict(u=r(batch, dim, L), f=r(batch, dim, L) + 1, z=r(batch, dim, L), b=r(dim), h0=r(batch, dim),
                dy=r(batch, dim, L), dlast=r(batch, dim), starts=g.random((batch, L)) < 0.2)


def _loss(c, **kw):
    o = layer.gated_scan(c["u"], c["f"], c["z"], c["b"], h0=c["h0"], **kw)
    return (o["y"] * c["dy"]).sum() + (o["last_state"] * c["dlast"]).sum()


@pytest.mark.parametrize("tied", [True, False])
@pytest.mark.parametrize("packed", [True, False])
def test_gated_gradients_against_differences(tied, packed):
    c = _case(2, 3, 12, 1)
    starts = c["starts"] if packed else None
    g = layer.gated_scan_bwd(c["u"], c["f"], c["z"], c["b"], c["dy"], tied=tied, starts=starts, h0=c["h0"],
                             dlast=c["dlast"])
    h = 1e-6
    for key, name in (("u", "du"), ("f", "df"), ("z", "dz"), ("b", "df_bias"), ("h0", "dinitial_state")):
        num = np.zeros_like(c[key])
        for i in np.ndindex(*c[key].shape):
            d = dict(c)
            d[key] = c[key].copy()
            d[key][i] += h
            up = _loss(d, tied=tied, starts=starts)
            d[key][i] -= 2 * h
            num[i] = (up - _loss(d, tied=tied, starts=starts)) / (2 * h)
        # central differences: truncation h^2, rounding 1e-16 |loss| / h
        np.testing.assert_allclose(g[name], num, atol=1e-7)


def test_gated_recurrence_is_the_scan_s_gating_reduction():
    # S6 with one state, A = -1, B = C = 1, exact zero-order hold and Delta =
    # softplus(s): exp(-Delta) = sigmoid(-s) is the forget gate, 1 - exp(-Delta)
    # = sigmoid(s) the input gate, so f = -s (fp32 inputs, exact in fp64)
    case = synth.make_case(2, 5, 70, 1, synth.F32, seed=3, with_D=False, with_bias=False)
    case["A"] = -np.ones((5, 1), np.float32)
    case["B"] = np.ones_like(case["B"])
    case["C"] = np.ones_like(case["C"])
    ref = oracle.fwd(case, zoh_exact=True)
    got = layer.gated_scan(case["u"], -case["delta"], case["z"])
    np.testing.assert_allclose(got["y"], ref["y"], rtol=1e-10, atol=1e-12)


def test_a_start_separates_the_packed_sequences():
    c = _case(1, 4, 20, 5)
    starts = np.zeros((1, 20), bool)
    starts[0, 7] = True
    both = layer.gated_scan(c["u"], c["f"], c["z"], c["b"], starts=starts, h0=c["h0"])
    cut = lambda k, s: c[k][:, :, s]
    first = layer.gated_scan(cut("u", slice(0, 7)), cut("f", slice(0, 7)), cut("z", slice(0, 7)), c["b"], h0=c["h0"])
    second = layer.gated_scan(cut("u", slice(7, 20)), cut("f", slice(7, 20)), cut("z", slice(7, 20)), c["b"])
    assert np.array_equal(both["y"], np.concatenate([first["y"], second["y"]], -1))
    assert np.array_equal(both["last_state"], second["last_state"])


def test_norm_gradients_against_differences():
    g = np.random.default_rng(2)
    s, w, b, dy = g.standard_normal((3, 9)), g.standard_normal(9), g.standard_normal(9), g.standard_normal((3, 9))
    loss = lambda s, w, b: (layer.layer_norm(s, w, b) * dy).sum()
    ref = layer.layer_norm_bwd(s, w, dy)
    h = 1e-6
    for x, name, call in ((s, "ds", lambda v: loss(v, w, b)), (w, "dweight", lambda v: loss(s, v, b)),
                          (b, "dbias", lambda v: loss(s, w, v))):
        num = np.zeros_like(x)
        for i in np.ndindex(*x.shape):
            up, dn = x.copy(), x.copy()
            up[i] += h
            dn[i] -= h
            num[i] = (call(up) - call(dn)) / (2 * h)
        np.testing.assert_allclose(ref[name], num, atol=1e-7)


def test_norm_rows_have_mean_zero_and_variance_one():
    s = np.random.default_rng(3).standard_normal((4, 50)) * 3 + 7
    y = layer.layer_norm(s, np.ones(50), eps=0.0)
    assert np.allclose(y.mean(-1), 0, atol=1e-13) and np.allclose((y * y).mean(-1), 1, atol=1e-12)
