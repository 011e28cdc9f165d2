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
