"""Seeded random sweep of the gated recurrence and layer norm: sizes, options,
paths, layouts, dtypes and buffers off their alignment by one to seven values,
each against the fp64 reference with the library's tolerances."""
import numpy as np
import pytest

import synth
from test_gated_gpu import Case as GatedCase
from test_norm_gpu import TYPES, Case as NormCase

pytestmark = pytest.mark.gpu


def _spread(g, lo, hi):
    return int(round(np.exp(g.uniform(np.log(lo), np.log(hi)))))


def _off(t, k):
    """t's values k elements into an allocation of their own."""
    import torch
    if t is None:
        return None
    flat = torch.empty(t.numel() + 16, dtype=t.dtype, device=t.device)
    v = flat[k:k + t.numel()].view(t.shape)
    v.copy_(t)
    return v


@pytest.mark.parametrize("seed", range(40))
def test_gated_sweep(cuda_device, seed):
    g = np.random.default_rng([7, seed])
    path, tok = [("auto", False), ("auto", True), ("per_group", False), ("lookback", False), ("lookback", True)][seed % 5]
    L = _spread(g, 1, 12000)
    dim = _spread(g, 1, max(1, min(300, 400000 // L)))
    batch = _spread(g, 1, max(1, min(12, 400000 // (L * dim))))
    flag = lambda p: bool(g.random() < p)
    c = GatedCase(cuda_device, batch, dim, L, synth.BF16 if flag(0.6) else synth.F32, 1000 + seed, z=flag(0.7),
                  bias=flag(0.7), tied=flag(0.6), starts=float(g.choice([0.0, 0.0, 0.003, 0.2])), h0=flag(0.6), tok=tok,
                  f_mean=float(g.uniform(-2, 7)))
    if flag(0.4):
        k = int(g.integers(1, 8))
        for name in ("u", "f", "z", "dy"):
            c.t[name] = _off(c.t[name], k if flag(0.8) else int(g.integers(0, 8)))
    c.check_fwd(*c.fwd(path))
    dlast = flag(0.7)
    c.check_bwd(c.bwd(path, save=flag(0.5), dlast=dlast), dlast)


@pytest.mark.parametrize("seed", range(30))
def test_norm_sweep(cuda_device, seed):
    g = np.random.default_rng([8, seed])
    dim = _spread(g, 3, 24000)
    rows = _spread(g, 1, max(1, min(3000, 400000 // dim)))
    dtype, residual = TYPES[seed % len(TYPES)]
    c = NormCase(cuda_device, rows, dim, dtype, residual, 2000 + seed, bias=bool(g.random() < 0.7))
    if g.random() < 0.5:
        k = int(g.integers(1, 8))
        for name in ("x", "res", "dy", "dro"):
            setattr(c, name, _off(getattr(c, name), k))
    c.check()
