"""Layer norm on the GPU, forward (with the residual's addition) and backward,
against the fp64 reference.

Tolerances: gpu_util.assert_close (one rounding to the output's type plus 2e-5
of the largest value; fp32 rel-L2 1e-5).  The reference takes s as the kernel
stored it, whose own values are checked to be the exactly rounded sums."""
import numpy as np
import pytest

import synth
from gpu_util import assert_close, to_f64
from oracle import layer

pytestmark = pytest.mark.gpu

TYPES = [(synth.BF16, "none"), (synth.BF16, "same"), (synth.BF16, "f32"), (synth.F32, "none"), (synth.F32, "same")]


class Case:
    def __init__(self, device, rows, dim, dtype, residual, seed, bias=True, offset=0.3, scale=1.0):
        import torch
        td = torch.bfloat16 if dtype == synth.BF16 else torch.float32
        g = np.random.default_rng(seed)
        r = lambda *s, m=0.0, sd=1.0: torch.from_numpy((g.standard_normal(s) * sd + m).astype(np.float32))
        self.dtype, self.rows, self.dim = dtype, rows, dim
        self.rdtype = synth.F32 if residual == "f32" else dtype
        rt = torch.float32 if residual == "f32" else td
        self.x = r(rows, dim, m=offset * scale, sd=scale).to(td).to(device)
        self.res = None if residual == "none" else r(rows, dim, m=offset, sd=3.0).to(rt).to(device)
        self.w, self.b = r(dim, m=1.0, sd=0.3).to(device), r(dim).to(device) if bias else None
        self.dy = r(rows, dim).to(td).to(device)
        self.dro = None if residual == "none" else r(rows, dim).to(rt).to(device)

    def check(self, eps=1e-5, **more):
        import torch
        import selective_state_space_54_b200 as ssm
        out = ssm.layer_norm(self.x, self.w, self.b, residual=self.res, eps=eps, **more)
        y, s = out if self.res is not None else (out, self.x)
        if self.res is not None:
            want = (self.x.double() + self.res.double()).to(self.res.dtype)
            assert torch.equal(s, want)
        g = ssm.layer_norm_bwd(s, self.w, self.b, self.dy, eps=eps, dresidual_out=self.dro)
        torch.cuda.synchronize()
        n = lambda t: None if t is None else to_f64(t)
        assert_close(n(y), layer.layer_norm(n(s), n(self.w), n(self.b), eps), self.dtype, "y")
        ref = layer.layer_norm_bwd(n(s), n(self.w), n(self.dy), eps, n(self.dro))
        assert_close(n(g["dx"]), ref["ds"], self.dtype, "dx")
        if self.dtype == self.rdtype:
            assert g["dresidual"] is g["dx"]
        else:
            assert_close(n(g["dresidual"]), ref["ds"], self.rdtype, "dresidual")
        assert_close(n(g["dweight"]), ref["dweight"], synth.F32, "dweight")
        if self.b is not None:
            assert_close(n(g["dbias"]), ref["dbias"], synth.F32, "dbias")
        else:
            assert g["dbias"] is None
        return y, s, g


@pytest.mark.parametrize("dtype,residual", TYPES)
@pytest.mark.parametrize("dim", [2, 3, 8, 31, 64, 100, 255, 256, 257, 1000, 1024, 1537, 2048, 2560, 4096, 5120, 8192,
                                 8193, 10007, 16384, 20000, 33000])
def test_widths(cuda_device, dtype, residual, dim):
    # (two columns normalise to +-1 and leave no gradient but what eps leaves: a wide eps there)
    Case(cuda_device, 13, dim, dtype, residual, dim).check(eps=0.5 if dim == 2 else 1e-5)


@pytest.mark.parametrize("dtype,residual", TYPES)
@pytest.mark.parametrize("rows", [1, 2, 3, 7, 8, 9, 147, 149, 600, 1201])
def test_row_counts(cuda_device, dtype, residual, rows):
    Case(cuda_device, rows, 192, dtype, residual, rows).check()
    Case(cuda_device, rows, 77, dtype, residual, rows, bias=False).check()


def test_many_rows(cuda_device):
    Case(cuda_device, 20011, 264, synth.BF16, "f32", 3).check()


@pytest.mark.parametrize("dtype,residual", TYPES)
def test_one_column(cuda_device, dtype, residual):
    # s - mean is 0: y is the bias, and nothing reaches s through the norm
    Case(cuda_device, 5, 1, dtype, residual, 9).check()


@pytest.mark.parametrize("dim", [24, 1000, 8192, 20000])
def test_a_mean_far_from_zero(cuda_device, dim):
    # values near 1000 with deviation 1: the variance is formed from the centred
    # values.  The mean's own error, at most 2^-24 * 1000 * a few roundings = 2e-4 of the
    # deviation, shifts y by as much; a shift drops out of the centred squares to first order.
    import torch
    import selective_state_space_54_b200 as ssm
    c = Case(cuda_device, 6, dim, synth.F32, "none", 4, offset=1000.0)
    y = ssm.layer_norm(c.x, c.w, c.b)
    ref = layer.layer_norm(to_f64(c.x), to_f64(c.w), to_f64(c.b))
    assert np.abs(to_f64(y) - ref).max() <= 2e-4 * np.abs(to_f64(c.w)).max()


@pytest.mark.parametrize("dtype", [synth.BF16, synth.F32])
def test_rows_of_one_value(cuda_device, dtype):
    # no variance: eps alone divides; y is the bias
    import torch
    import selective_state_space_54_b200 as ssm
    td = torch.bfloat16 if dtype == synth.BF16 else torch.float32
    x = torch.full((3, 520), 1.5, dtype=td, device=cuda_device)
    w, b = torch.randn(520, device=cuda_device), torch.randn(520, device=cuda_device)
    assert torch.equal(ssm.layer_norm(x, w, b), b.to(td).expand(3, 520))


@pytest.mark.parametrize("scale", [1e-4, 1e4, 1e15])
def test_scales(cuda_device, scale):
    c = Case(cuda_device, 4, 700, synth.F32, "none", 6, scale=scale, offset=0.0)
    c.check(eps=1e-5 if scale < 1e10 else 0.0)


def test_bad_rows_stay_their_own(cuda_device):
    import torch
    import selective_state_space_54_b200 as ssm
    for dim in (40, 3000, 20000):
        c = Case(cuda_device, 9, dim, synth.BF16, "f32", 7)
        want = ssm.layer_norm(c.x, c.w, c.b, residual=c.res)[0].clone()
        c.x[4, 3] = float("nan")
        c.res[6, 1] = float("inf")
        y = ssm.layer_norm(c.x, c.w, c.b, residual=c.res)[0]
        ok = [i for i in range(9) if i not in (4, 6)]
        assert torch.equal(y[ok], want[ok]) and torch.isnan(y[4]).all() and not torch.isfinite(y[6]).any()


def test_leading_axes_and_in_place_residual(cuda_device):
    import torch
    import selective_state_space_54_b200 as ssm
    for dim in (96, 9000, 20000):
        c = Case(cuda_device, 12, dim, synth.BF16, "f32", 8)
        y, s = ssm.layer_norm(c.x, c.w, c.b, residual=c.res)
        x3, r3 = c.x.view(3, 4, dim), c.res.clone().view(3, 4, dim)
        y3, s3 = ssm.layer_norm(x3, c.w, c.b, residual=r3, residual_out=r3)
        assert y3.shape == x3.shape and s3 is r3
        assert torch.equal(y3.view_as(y), y) and torch.equal(r3.view_as(s), s)
        g = ssm.layer_norm_bwd(s, c.w, c.b, c.dy, dresidual_out=c.dro)
        dro = c.dro.clone()
        g2 = ssm.layer_norm_bwd(s, c.w, c.b, c.dy, dresidual_out=dro, out={"dresidual": dro})
        assert g2["dresidual"] is dro
        assert all(torch.equal(g[k], g2[k]) for k in g)


@pytest.mark.parametrize("dtype,residual", TYPES)
def test_offset_buffers_and_guards(cuda_device, dtype, residual):
    import torch
    import selective_state_space_54_b200 as ssm
    for dim in (64, 1021, 4096, 17000):
        c = Case(cuda_device, 7, dim, dtype, residual, 10)

        def off(t):
            if t is None:
                return None, None
            flat = torch.full((t.numel() + 129,), 7.0, dtype=t.dtype, device=cuda_device)
            v = flat[65:65 + t.numel()].view(t.shape)
            v.copy_(t)
            return v, flat
        for k in ("x", "res", "dy", "dro", "w", "b"):
            setattr(c, k, off(getattr(c, k))[0])
        y, yf = off(torch.zeros_like(c.x))
        dx, dxf = off(torch.zeros_like(c.x))
        dw, dwf = off(torch.zeros_like(c.w))
        out = ssm.layer_norm(c.x, c.w, c.b, residual=c.res, y=y)
        s = c.x if c.res is None else out[1]
        g = ssm.layer_norm_bwd(s, c.w, c.b, c.dy, dresidual_out=c.dro, out={"dx": dx, "dweight": dw})
        # against the reference, not against the aligned call: two correctly rounded results
        # may stand on either side of a rounding boundary, a whole step apart
        n = lambda t: None if t is None else to_f64(t)
        assert_close(n(y), layer.layer_norm(n(s), n(c.w), n(c.b)), dtype, "y")
        ref = layer.layer_norm_bwd(n(s), n(c.w), n(c.dy), dresidual=n(c.dro))
        assert_close(n(g["dx"]), ref["ds"], dtype, "dx")
        assert_close(n(dw), ref["dweight"], synth.F32, "dweight")
        for v, flat in ((y, yf), (dx, dxf), (dw, dwf)):
            assert (flat[:65] == 7).all() and (flat[65 + v.numel():] == 7).all()


def test_repeated_two_streams_and_captured(cuda_device):
    import torch
    import selective_state_space_54_b200 as ssm
    for rows, dim in ((5000, 1024), (40, 12000)):
        c = Case(cuda_device, rows, dim, synth.BF16, "f32", 12)

        def both(stream=None):
            y, s = ssm.layer_norm(c.x, c.w, c.b, residual=c.res, stream=stream)
            g = ssm.layer_norm_bwd(s, c.w, c.b, c.dy, dresidual_out=c.dro, stream=stream)
            return [y, s, g["dx"], g["dresidual"], g["dweight"], g["dbias"]]
        want = both()
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in range(2)]
        got = [both(s) for s in streams for _ in range(2)]
        torch.cuda.synchronize()
        for o in got:
            assert all(torch.equal(a, b) for a, b in zip(want, o))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            kept = both()
        for t in kept:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, kept))


def test_no_rows_and_no_columns(cuda_device):
    import torch
    import selective_state_space_54_b200 as ssm
    w = torch.ones(8, device=cuda_device)
    e = torch.zeros((0, 8), device=cuda_device)
    assert ssm.layer_norm(e, w, w).shape == (0, 8)
    g = ssm.layer_norm_bwd(e, w, w, e)
    assert not g["dweight"].any() and not g["dbias"].any() and g["dx"].shape == (0, 8)
    e, w = torch.zeros((4, 0), device=cuda_device), torch.ones(0, device=cuda_device)
    assert ssm.layer_norm(e, w).shape == (4, 0)


def test_offsets_past_32_bits(cuda_device):
    import torch
    import selective_state_space_54_b200 as ssm
    rows, dim = 600_011, 4096
    gen = torch.Generator(device=cuda_device).manual_seed(3)
    x, dy = (torch.randn((rows, dim), generator=gen, device=cuda_device, dtype=torch.bfloat16) for _ in range(2))
    w = torch.rand(dim, generator=gen, device=cuda_device) + 0.5
    y = ssm.layer_norm(x, w)
    g = ssm.layer_norm_bwd(x, w, w, dy)
    at = [0, 1, 299_999, 524_288, rows - 1]
    n = lambda t: to_f64(t[at])
    assert_close(n(y), layer.layer_norm(n(x), to_f64(w)), synth.BF16, "y")
    assert_close(n(g["dx"]), layer.layer_norm_bwd(n(x), to_f64(w), n(dy))["ds"], synth.BF16, "dx")
    ref = torch.zeros(dim, dtype=torch.float64, device=cuda_device)
    for i in range(0, rows, 50_000):
        ref += dy[i:i + 50_000].double().sum(0)
    assert_close(to_f64(g["dbias"]), to_f64(ref), synth.F32, "dbias")


def test_refusals(cuda_device):
    import torch
    import selective_state_space_54_b200 as ssm
    x = torch.zeros((4, 8), dtype=torch.bfloat16, device=cuda_device)
    w = torch.ones(8, device=cuda_device)
    with pytest.raises(TypeError):
        ssm.layer_norm(x, w.bfloat16())
    with pytest.raises(TypeError):
        ssm.layer_norm(x.float(), w, residual=x)  # a residual narrower than x
    with pytest.raises(ValueError):
        ssm.layer_norm(x, w[:4])
    with pytest.raises(ValueError):
        ssm.layer_norm(x, w, residual=x[:2])
    with pytest.raises(ValueError):
        ssm.layer_norm(x.t(), torch.ones(4, device=cuda_device))
    with pytest.raises(ValueError):
        ssm.layer_norm(x, w, residual_out=x)
    with pytest.raises(ssm.ScanError):
        ssm.layer_norm(x, w, eps=-1.0)
    with pytest.raises(ssm.ScanError):
        ssm.layer_norm(x, w, y=x)
    with pytest.raises(TypeError):
        ssm.layer_norm_bwd(x, w, None, x.float())
    with pytest.raises(ssm.ScanError):
        ssm.layer_norm_bwd(x, w, None, x, out={"dx": x})


def test_gradients_that_are_not_formed_are_refused(cuda_device):
    import torch
    import selective_state_space_54_b200 as ssm
    x, w = torch.ones((4, 16), device=cuda_device), torch.ones(16, device=cuda_device)
    with pytest.raises(ValueError):  # the residual's gradient is dx itself
        ssm.layer_norm_bwd(x, w, w, x, out={"dresidual": torch.empty_like(x)})
    with pytest.raises(ValueError):
        ssm.layer_norm_bwd(x, w, None, x, out={"dbias": torch.empty_like(w)})
