"""The gated linear recurrence on the GPU against its fp64 reference: forward,
backward and single step, every path, layout and dtype, at the sizes and masks
where they can go wrong.

Tolerances are the library's own (gpu_util.assert_close), which count one
rounding to the output's type (half a step: bf16 2^-9 of the binade's upper
end) plus 2e-5 of the largest value for the fp32 arithmetic; fp32 outputs and
the fp32 sums df_bias hold rel-L2 1e-5 (a sum of n terms rounds n times by
2^-24 of a partial sum that grows like sqrt(n): 2^-24 sqrt(n/2) < 1e-5 of the
result up to n = 56000 terms)."""
import numpy as np
import pytest

import synth
from gpu_util import assert_close, to_f64
from oracle import layer

pytestmark = pytest.mark.gpu

PATHS = [("per_group", False), ("lookback", False), ("lookback", True)]  # path, token-major


def _path(name):
    import selective_state_space_54_b200 as ssm
    return {"auto": ssm.SSM_PATH_AUTO, "per_group": ssm.SSM_PATH_PER_GROUP, "lookback": ssm.SSM_PATH_LOOKBACK}[name]


def _torch_dtype(dtype):
    import torch
    return torch.bfloat16 if dtype == synth.BF16 else torch.float32


class Case:
    """Inputs on the GPU and the same values in fp64 (batch, dim, seqlen)."""

    def __init__(self, device, batch, dim, L, dtype, seed, *, z=True, bias=True, tied=True, starts=0.0, h0=True,
                 tok=False, f_mean=1.0, edit=None):
        import torch
        self.tied, self.tok, self.dtype, self.device = tied, tok, dtype, device
        self.batch, self.dim, self.L = batch, dim, L
        g = np.random.default_rng(seed)
        td = _torch_dtype(dtype)
        raw = {"u": g.standard_normal((batch, dim, L)), "f": g.standard_normal((batch, dim, L)) + f_mean,
               "z": g.standard_normal((batch, dim, L)) if z else None, "dy": g.standard_normal((batch, dim, L))}
        self.starts = None
        if starts:
            self.starts = g.random((batch, L)) < starts
        if edit is not None:
            edit(raw, self)
        self.t, self.n = {}, {}
        for k, v in raw.items():
            if v is None:
                self.t[k] = self.n[k] = None
                continue
            x = torch.from_numpy(v.astype(np.float32)).to(td)
            self.n[k] = x.double().numpy()
            self.t[k] = (x.transpose(1, 2) if tok else x).contiguous().to(device)
        f32 = lambda *s: g.standard_normal(s).astype(np.float32)
        self.n["b"] = f32(dim) if bias else None
        self.n["h0"] = f32(batch, dim) if h0 else None
        self.n["dlast"] = f32(batch, dim)
        for k in ("b", "h0", "dlast"):
            self.t[k] = None if self.n[k] is None else torch.from_numpy(self.n[k]).to(device)
        self.t["starts"] = None if self.starts is None else torch.from_numpy(self.starts).to(device)

    def kw(self, path):
        return dict(tied=self.tied, starts=self.t["starts"], initial_state=self.t["h0"], token_major=self.tok,
                    path=_path(path))

    def rows(self, t):
        """An activation-shaped GPU tensor as fp64 (batch, dim, seqlen)."""
        v = to_f64(t)
        return v.transpose(0, 2, 1) if self.tok else v

    def fwd(self, path="auto", **more):
        import selective_state_space_54_b200 as ssm
        return ssm.gated_scan_fwd(self.t["u"], self.t["f"], self.t["z"], self.t["b"], return_last_state=True,
                                  **self.kw(path), **more)

    def bwd(self, path="auto", save=True, dlast=True, **more):
        import torch
        import selective_state_space_54_b200 as ssm
        ws = None
        if save:
            shape = ssm.gated_scan_shape(self.t["u"], tied=self.tied, save_states=True, token_major=self.tok,
                                         path=_path(path))
            ws = torch.empty(ssm.gated_scan_fwd_workspace_bytes(shape), dtype=torch.uint8, device=self.device)
            ws.fill_(255)
            self.fwd(path, workspace=ws, save_states=True)
        return ssm.gated_scan_bwd(self.t["u"], self.t["f"], self.t["z"], self.t["b"], self.t["dy"],
                                  dlast_state=self.t["dlast"] if dlast else None, want_dinitial_state=True,
                                  fwd_workspace=ws, **self.kw(path), **more)

    def ref(self):
        n = self.n
        return layer.gated_scan(n["u"], n["f"], n["z"], n["b"], tied=self.tied, starts=self.starts, h0=n["h0"])

    def ref_bwd(self, dlast=True):
        n = self.n
        return layer.gated_scan_bwd(n["u"], n["f"], n["z"], n["b"], n["dy"], tied=self.tied, starts=self.starts,
                                    h0=n["h0"], dlast=n["dlast"] if dlast else None)

    def check_fwd(self, y, last):
        ref = self.ref()
        assert_close(self.rows(y), ref["y"], self.dtype, "y")
        assert_close(to_f64(last), ref["last_state"], synth.F32, "last_state")

    def check_bwd(self, g, dlast=True):
        ref = self.ref_bwd(dlast)
        for k in ("du", "df", "dz"):
            assert (g[k] is None) == (ref[k] is None), k
            if g[k] is not None:
                assert_close(self.rows(g[k]), ref[k], self.dtype, k)
        assert (g["df_bias"] is None) == (ref["df_bias"] is None)
        if g["df_bias"] is not None:
            assert_close(to_f64(g["df_bias"]), ref["df_bias"], synth.F32, "df_bias")
        assert_close(to_f64(g["dinitial_state"]), ref["dinitial_state"], synth.F32, "dinitial_state")


LENGTHS = [1, 2, 7, 15, 16, 17, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 511, 512, 513, 1000, 1024, 2049]


@pytest.mark.parametrize("path,tok", PATHS)
@pytest.mark.parametrize("L", LENGTHS)
def test_lengths(cuda_device, path, tok, L):
    c = Case(cuda_device, 2, 37, L, synth.BF16, L, tok=tok)
    c.check_fwd(*c.fwd(path))
    c.check_bwd(c.bwd(path, save=L % 2 == 0))


@pytest.mark.parametrize("path,tok", PATHS)
@pytest.mark.parametrize("L", [1, 16, 31, 257, 1030, 4096, 8200])
def test_lengths_fp32(cuda_device, path, tok, L):
    c = Case(cuda_device, 1, 9, L, synth.F32, L + 1, tok=tok)
    c.check_fwd(*c.fwd(path))
    c.check_bwd(c.bwd(path, save=L % 2 == 0))


@pytest.mark.parametrize("path,tok", PATHS)
@pytest.mark.parametrize("dim", [1, 2, 7, 8, 31, 32, 33, 63, 64, 65, 130, 256])
def test_channel_counts(cuda_device, path, tok, dim):
    for dtype in (synth.BF16, synth.F32):
        c = Case(cuda_device, 3, dim, 150, dtype, dim, tok=tok, starts=0.02)
        c.check_fwd(*c.fwd(path))
        c.check_bwd(c.bwd(path))


@pytest.mark.parametrize("path,tok", PATHS)
@pytest.mark.parametrize("dtype", [synth.BF16, synth.F32])
@pytest.mark.parametrize("opt", ["all", "no_z", "no_bias", "no_state", "untied", "packed", "untied_packed_no_z",
                                 "bare"])
def test_options(cuda_device, path, tok, dtype, opt):
    kw = {"all": {}, "no_z": dict(z=False), "no_bias": dict(bias=False), "no_state": dict(h0=False),
          "untied": dict(tied=False), "packed": dict(starts=0.01),
          "untied_packed_no_z": dict(tied=False, starts=0.05, z=False),
          "bare": dict(z=False, bias=False, h0=False)}[opt]
    c = Case(cuda_device, 2, 48, 1200, dtype, 11, tok=tok, **kw)
    c.check_fwd(*c.fwd(path))
    c.check_bwd(c.bwd(path, dlast=opt != "bare"), dlast=opt != "bare")
    c.check_bwd(c.bwd(path, save=False))


@pytest.mark.parametrize("path,tok", PATHS)
def test_long_sequences_cross_many_tiles(cuda_device, path, tok):
    # the chain of tiles is long, and the memory (a = sigmoid(5 +- 1), hundreds of
    # steps) carries across them
    for dtype, tied in ((synth.BF16, True), (synth.F32, True), (synth.F32, False)):
        c = Case(cuda_device, 1, 3, 40000, dtype, 21, tok=tok, f_mean=5.0, tied=tied, starts=0.0001)
        c.check_fwd(*c.fwd(path))
        c.check_bwd(c.bwd(path))


@pytest.mark.parametrize("path,tok", PATHS)
@pytest.mark.parametrize("dim", [3, 200])
def test_outer_states_reach_across_tiles(cuda_device, path, tok, dim):
    # an initial state and a gradient of the last state far above everything else, under
    # a long memory (a = 1 - 1e-4): every tile's outputs depend on them
    def edit(raw, case):
        raw["f"][:] = 9.0
    c = Case(cuda_device, 1, dim, 9000, synth.F32, 33, tok=tok, bias=False, edit=edit)
    for k in ("h0", "dlast"):
        c.n[k] = c.n[k] * 1000
        c.t[k].mul_(1000)
    c.check_fwd(*c.fwd(path))
    c.check_bwd(c.bwd(path))


@pytest.mark.parametrize("path,tok", PATHS)
def test_many_batches(cuda_device, path, tok):
    c = Case(cuda_device, 70, 11, 90, synth.BF16, 22, tok=tok, starts=0.03)
    c.check_fwd(*c.fwd(path))
    c.check_bwd(c.bwd(path, save=False))


@pytest.mark.parametrize("path,tok", PATHS)
def test_memory_of_a_hundred_thousand_steps(cuda_device, path, tok):
    # a = sigmoid(11.5) = 1 - 1e-5 everywhere: the state is a sum over the whole
    # sequence.  The state moves by g (u - h), so its rounding is one half step
    # (2^-24 of the state) a step, random in sign: 2^-24 sqrt(1 / (2 g)) = 1.3e-5 of
    # the state's scale at worst; the last state and y are held to 5e-5 of it.
    def edit(raw, case):
        raw["f"][:] = 11.5
        raw["u"][:] = np.abs(raw["u"]) + 1
    c = Case(cuda_device, 1, 4, 100000, synth.F32, 23, tok=tok, bias=False, z=False, edit=edit)
    y, last = c.fwd(path)
    ref = c.ref()
    scale = np.abs(ref["y"]).max()
    assert np.abs(c.rows(y) - ref["y"]).max() <= 5e-5 * scale
    assert np.abs(to_f64(last) - ref["last_state"]).max() <= 5e-5 * scale


@pytest.mark.parametrize("path,tok", PATHS)
@pytest.mark.parametrize("dtype", [synth.BF16, synth.F32])
def test_extreme_gates(cuda_device, path, tok, dtype):
    # logits over [-200, 200] and the infinities: a closed gate takes the input, an
    # open one holds the state; gradients stay finite
    def edit(raw, case):
        f = raw["f"]
        f[:] = np.random.default_rng(1).uniform(-200, 200, f.shape)
        f[:, :, 5::40] = np.inf
        f[:, :, 7::40] = -np.inf
        raw["z"][:, :, ::3] *= 100
    c = Case(cuda_device, 2, 33, 700, dtype, 24, tok=tok, edit=edit)
    c.check_fwd(*c.fwd(path))
    c.check_bwd(c.bwd(path))


@pytest.mark.parametrize("path,tok", PATHS)
@pytest.mark.parametrize("bad", [np.nan, np.inf])
def test_a_start_stops_what_is_not_finite(cuda_device, path, tok, bad):
    # one packed sequence of garbage between good ones, in u, f, z, dy and the initial
    # state: the neighbours' outputs and gradients are as if it were not there
    L, lo, hi = 900, 300, 650

    def edit(raw, case):
        for k in ("u", "f", "z", "dy"):
            raw[k][:, :, lo + 3:hi] = bad
        case.starts = np.zeros((2, L), bool)
        case.starts[:, [0, lo, hi, 700]] = True
    c = Case(cuda_device, 2, 20, L, synth.F32, 25, tok=tok, edit=edit)
    c.t["h0"].fill_(bad)
    y, last = c.fwd(path)
    c.t["dlast"].zero_()
    g = c.bwd(path)
    keep = np.ones(L, bool)
    keep[lo:hi] = False
    # the reference on the same inputs with the garbage replaced by ones
    for k in ("u", "f", "z", "dy"):
        c.n[k] = np.where(np.isfinite(c.n[k]), c.n[k], 1.0)
    c.n["h0"] = np.zeros_like(c.n["h0"])
    c.n["dlast"] = np.zeros_like(c.n["dlast"])
    ref, rb = c.ref(), c.ref_bwd()
    assert_close(c.rows(y)[:, :, keep], ref["y"][:, :, keep], synth.F32, "y")
    assert_close(to_f64(last), ref["last_state"], synth.F32, "last_state")
    for k in ("du", "df", "dz"):
        assert_close(c.rows(g[k])[:, :, keep], rb[k][:, :, keep], synth.F32, k)
    assert not to_f64(g["dinitial_state"]).any()  # every sequence starts at 0


@pytest.mark.parametrize("path,tok", PATHS)
def test_not_a_number_reaches_every_later_output(cuda_device, path, tok):
    def edit(raw, case):
        raw["f"][0, 2, 100] = np.nan
    c = Case(cuda_device, 1, 5, 900, synth.F32, 26, tok=tok, edit=edit)
    y, last = c.fwd(path)
    v = c.rows(y)
    assert np.isnan(v[0, 2, 100:]).all() and np.isnan(to_f64(last)[0, 2])
    assert np.isfinite(v[0, 2, :100]).all() and np.isfinite(np.delete(v, 2, 1)).all()


@pytest.mark.parametrize("path,tok", PATHS)
def test_pieces_continue_one_another(cuda_device, path, tok):
    # two calls chained through the state give the whole sequence's results, and two
    # backward calls chained through dlast_state its gradients
    import torch
    import selective_state_space_54_b200 as ssm
    c = Case(cuda_device, 2, 24, 1000, synth.F32, 27, tok=tok, starts=0.01)
    cut = 417
    ax = 1 if tok else 2
    part = lambda t, a, b: t.narrow(ax, a, b - a).contiguous()
    kw = dict(tied=True, token_major=tok, path=_path(path))
    outs, h = [], c.t["h0"]
    spans = [(0, cut), (cut, 1000)]
    h_in = []
    for a, b in spans:
        h_in.append(h)
        y, h = ssm.gated_scan_fwd(part(c.t["u"], a, b), part(c.t["f"], a, b), part(c.t["z"], a, b), c.t["b"],
                                  starts=c.t["starts"][:, a:b].contiguous(), initial_state=h, return_last_state=True,
                                  **kw)
        outs.append(y)
    c.check_fwd(torch.cat(outs, ax), h)
    dl, gs = c.t["dlast"], []
    for (a, b), h0 in zip(spans[::-1], h_in[::-1]):
        g = ssm.gated_scan_bwd(part(c.t["u"], a, b), part(c.t["f"], a, b), part(c.t["z"], a, b), c.t["b"],
                               part(c.t["dy"], a, b), starts=c.t["starts"][:, a:b].contiguous(), initial_state=h0,
                               dlast_state=dl, want_dinitial_state=True, **kw)
        dl = g["dinitial_state"]
        gs.insert(0, g)
    whole = {k: torch.cat([g[k] for g in gs], ax) for k in ("du", "df", "dz")}
    whole["df_bias"] = gs[0]["df_bias"] + gs[1]["df_bias"]
    whole["dinitial_state"] = dl
    c.check_bwd(whole)


@pytest.mark.parametrize("tied", [True, False])
@pytest.mark.parametrize("dtype", [synth.BF16, synth.F32])
def test_steps_are_the_scan(cuda_device, dtype, tied):
    import torch
    import selective_state_space_54_b200 as ssm
    for batch, dim in ((1, 1), (3, 77), (5, 264)):
        c = Case(cuda_device, batch, dim, 9, dtype, 28, tied=tied)
        state, ys = c.t["h0"].clone(), []
        for t in range(9):
            one = lambda k: c.t[k][:, :, t].contiguous()
            ys.append(ssm.gated_scan_step(one("u"), one("f"), one("z"), c.t["b"], state=state, tied=tied))
        c.check_fwd(torch.stack(ys, -1), state)


def test_step_options(cuda_device):
    import selective_state_space_54_b200 as ssm
    for z, bias in ((False, True), (True, False), (False, False)):
        c = Case(cuda_device, 4, 130, 1, synth.BF16, 29, z=z, bias=bias)
        state = c.t["h0"].clone()
        y = ssm.gated_scan_step(c.t["u"][:, :, 0], c.t["f"][:, :, 0], c.t["z"][:, :, 0] if z else None, c.t["b"],
                                state=state)
        c.check_fwd(y[:, :, None], state)


@pytest.mark.parametrize("path,tok", PATHS)
def test_offset_buffers_and_guards(cuda_device, path, tok):
    # every buffer one element into its allocation (no 16-byte access possible), with a
    # guard behind and before each output
    import torch
    import selective_state_space_54_b200 as ssm
    for dtype, L in ((synth.BF16, 528), (synth.F32, 300), (synth.BF16, 77)):
        c = Case(cuda_device, 2, 40, L, dtype, 30, tok=tok)

        def off(t, guard=64):
            if t is None:
                return None, None
            flat = torch.full((t.numel() + 2 * guard + 1,), 7.0, dtype=t.dtype, device=cuda_device)
            v = flat[guard + 1:guard + 1 + t.numel()].view(t.shape)
            v.copy_(t)
            return v, flat
        for k in ("u", "f", "z", "dy"):
            c.t[k], _ = off(c.t[k])
        outs = {k: off(torch.zeros_like(c.t["u"])) for k in ("y", "du", "df", "dz")}
        last, lflat = off(torch.zeros_like(c.t["h0"]))
        y, _ = c.fwd(path, y=outs["y"][0], last_state=last)
        g = c.bwd(path, out={k: outs[k][0] for k in ("du", "df", "dz")})
        c.check_fwd(y, last)
        c.check_bwd(g)
        for v, flat in list(outs.values()) + [(last, lflat)]:
            n = v.numel()
            assert (flat[:65] == 7).all() and (flat[65 + n:] == 7).all()


@pytest.mark.parametrize("path,tok", PATHS)
def test_repeated_calls_give_equal_bits(cuda_device, path, tok):
    import torch
    c = Case(cuda_device, 3, 200, 3000, synth.BF16, 31, tok=tok, starts=0.001)
    first, g1 = c.fwd(path), c.bwd(path)
    for save in (True, False, True):
        again, g2 = c.fwd(path), c.bwd(path, save=save)
        assert all(torch.equal(a, b) for a, b in zip(first, again))
        assert all(torch.equal(g1[k], g2[k]) for k in g1)


@pytest.mark.parametrize("path,tok", PATHS)
def test_two_streams_at_once(cuda_device, path, tok):
    import torch
    cases = [Case(cuda_device, 2, 64, 6000, synth.BF16, 40 + i, tok=tok) for i in range(2)]
    want = [(c.fwd(path), c.bwd(path)) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(4):
        got = []
        for c, s in zip(cases, streams):
            got.append((c.fwd(path, stream=s), c.bwd(path, save=False, stream=s)))
        torch.cuda.synchronize()
        for (f1, g1), (f2, g2) in zip(want, got):
            assert all(torch.equal(a, b) for a, b in zip(f1, f2))
            assert all(torch.equal(g1[k], g2[k]) for k in g1)


@pytest.mark.parametrize("path,tok", PATHS)
def test_captured_and_replayed(cuda_device, path, tok):
    # forward and backward in one graph, replayed on new inputs
    import torch
    c = Case(cuda_device, 2, 100, 1500, synth.BF16, 50, tok=tok)
    other = Case(cuda_device, 2, 100, 1500, synth.BF16, 51, tok=tok)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        c.fwd(path), c.bwd(path)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f, g = c.fwd(path), c.bwd(path)
    for src in (c, other, c):
        keep = {k: src.t[k].clone() for k in ("u", "f", "z", "dy", "b", "h0", "dlast")}
        want_f, want_g = src.fwd(path), src.bwd(path)
        saved = {k: c.t[k].clone() for k in keep}
        for k in keep:
            c.t[k].copy_(keep[k])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want_f, f))
        assert all(torch.equal(want_g[k], g[k]) for k in g)
        for k in keep:
            c.t[k].copy_(saved[k])


def test_zero_lengths_pass_the_state_through(cuda_device):
    import torch
    import selective_state_space_54_b200 as ssm
    u = torch.zeros((2, 6, 0), dtype=torch.bfloat16, device=cuda_device)
    h0, dl = torch.randn((2, 6), device=cuda_device), torch.randn((2, 6), device=cuda_device)
    y, last = ssm.gated_scan_fwd(u, u, initial_state=h0, return_last_state=True)
    _, zero = ssm.gated_scan_fwd(u, u, return_last_state=True)
    g = ssm.gated_scan_bwd(u, u, None, torch.zeros(6, device=cuda_device), u, dlast_state=dl, want_dinitial_state=True)
    assert y.numel() == 0 and torch.equal(last, h0) and not zero.any()
    assert torch.equal(g["dinitial_state"], dl) and not g["df_bias"].any()
    e = torch.zeros((0, 6, 5), device=cuda_device)
    g = ssm.gated_scan_bwd(e, e, None, torch.ones(6, device=cuda_device), e)
    assert not g["df_bias"].any()  # no batch: the bias's gradient is 0, not left as it was


@pytest.mark.parametrize("path,tok", PATHS)
def test_offsets_past_32_bits(cuda_device, path, tok):
    # more than 2^31 values a tensor: the last channels of the last batch element
    # against the reference
    import torch
    import selective_state_space_54_b200 as ssm
    batch, dim, L = 3, 720, 1_000_003
    g = torch.Generator(device=cuda_device).manual_seed(5)
    shape = (batch, L, dim) if tok else (batch, dim, L)
    u, f, dy = (torch.randn(shape, generator=g, device=cuda_device, dtype=torch.bfloat16) for _ in range(3))
    y, last = ssm.gated_scan_fwd(u, f, return_last_state=True, token_major=tok, path=_path(path))
    gr = ssm.gated_scan_bwd(u, f, None, None, dy, token_major=tok, path=_path(path), want_dinitial_state=True)
    torch.cuda.synchronize()
    rows = [(2, 719), (2, 0), (1, 300)]
    pick = lambda t: np.stack([to_f64(t[b, :, d] if tok else t[b, d]) for b, d in rows])[None]
    un, fn, dn = pick(u), pick(f), pick(dy)
    ref = layer.gated_scan(un, fn)
    rb = layer.gated_scan_bwd(un, fn, None, None, dn)
    assert_close(pick(y), ref["y"], synth.BF16, "y")
    assert_close(np.array([to_f64(last)[b, d] for b, d in rows]), ref["last_state"][0], synth.F32, "last")
    assert_close(pick(gr["du"]), rb["du"], synth.BF16, "du")
    assert_close(pick(gr["df"]), rb["df"], synth.BF16, "df")


@pytest.mark.parametrize("path,tok", PATHS)
@pytest.mark.parametrize("L", [1, 700, 9000])
def test_states_in_place(cuda_device, path, tok, L):
    # last_state over initial_state and dinitial_state over dlast_state, the way a state
    # is carried along: the same bits as with buffers of their own
    import torch
    c = Case(cuda_device, 2, 21, L, synth.BF16, 34, tok=tok, f_mean=8.0)
    y, last = c.fwd(path)
    g = c.bwd(path)
    state, grad = c.t["h0"].clone(), c.t["dlast"].clone()
    keep = c.t["h0"], c.t["dlast"]
    c.t["h0"] = state
    y2, _ = c.fwd(path, last_state=state)
    c.t["h0"], c.t["dlast"] = keep[0], grad
    g2 = c.bwd(path, out={"dinitial_state": grad})
    assert torch.equal(y, y2) and torch.equal(state, last)
    assert all(torch.equal(g[k], g2[k]) for k in g)


@pytest.mark.parametrize("path,tok", PATHS)
def test_a_closed_gate_forgets_any_state(cuda_device, path, tok):
    # f = -inf (g = 1 exactly): h = u whatever the state before it was, here 2^40 times u
    import torch
    import selective_state_space_54_b200 as ssm

    def edit(raw, case):
        raw["f"][:, :, 0::10] = -np.inf
        raw["u"][:, :, 5::10] *= 2.0 ** 40
    c = Case(cuda_device, 1, 12, 600, synth.F32, 35, tok=tok, z=False, bias=False, edit=edit)
    c.t["h0"].fill_(2.0 ** 60)
    y, _ = c.fwd(path)
    assert np.array_equal(c.rows(y)[:, :, 0::10], c.n["u"][:, :, 0::10])
    state = torch.full((1, 12), 2.0 ** 60, device=cuda_device)
    one = torch.randn((1, 12), device=cuda_device)
    assert torch.equal(ssm.gated_scan_step(one, torch.full_like(one, -np.inf), state=state), one)


def test_device_and_argument_refusals(cuda_device):
    import torch
    import selective_state_space_54_b200 as ssm
    u = torch.zeros((2, 8, 16), dtype=torch.bfloat16, device=cuda_device)
    with pytest.raises(ValueError):
        ssm.gated_scan_fwd(u, u.cpu())
    with pytest.raises(ValueError):
        ssm.gated_scan_fwd(u, u.transpose(1, 2).contiguous())
    with pytest.raises(TypeError):
        ssm.gated_scan_fwd(u, u.float())
    with pytest.raises(TypeError):
        ssm.gated_scan_fwd(u.half(), u.half())
    with pytest.raises(TypeError):
        ssm.gated_scan_fwd(u, u, starts=torch.zeros((2, 16), dtype=torch.int32, device=cuda_device))
    with pytest.raises(ValueError):
        ssm.gated_scan_fwd(u, u, starts=torch.zeros((16, 2), dtype=torch.bool, device=cuda_device).t())
    with pytest.raises(ValueError):
        ssm.gated_scan_fwd(u, u, save_states=True)
    with pytest.raises(ssm.ScanError):
        ssm.gated_scan_fwd(u, u, token_major=True, path=ssm.SSM_PATH_PER_GROUP)
    with pytest.raises(ssm.ScanError):
        ssm.gated_scan_fwd(u, u, path=ssm.SSM_PATH_SPLIT_L)
    with pytest.raises(ssm.ScanError):
        ssm.gated_scan_fwd(u, u, y=u)  # y may not be an input
    with pytest.raises(ValueError):
        ssm.gated_scan_bwd(u, u, None, None, u, fwd_workspace=torch.empty(16, dtype=torch.uint8, device=cuda_device))
    with pytest.raises(ValueError):
        ssm.gated_scan_step(u[:, :, 0], u[:, :, 0], state=torch.zeros((2, 8), device=cuda_device))  # strided


@pytest.mark.parametrize("shape", [(0, 8, 16), (2, 0, 16), (2, 8, 0), (0, 0, 0)])
@pytest.mark.parametrize("token_major", [False, True])
def test_queries_of_empty_shapes(cuda_device, shape, token_major):
    import torch
    import selective_state_space_54_b200 as ssm
    u = torch.zeros(shape, device=cuda_device)
    for path in (ssm.SSM_PATH_AUTO, ssm.SSM_PATH_LOOKBACK):
        sh = ssm.gated_scan_shape(u, token_major=token_major, path=path)
        assert ssm.gated_scan_fwd_workspace_bytes(sh) == 0 and ssm.gated_scan_bwd_workspace_bytes(sh) == 0
        assert ssm.gated_scan_path(sh) in ssm.PATH_NAMES.values()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("path", ["per_group", "lookback"])
@pytest.mark.parametrize("seqlen", [1, 17, 513, 2051, 4099])
def test_saved_states_serve_differently_aligned_gradients(cuda_device, dtype, path, seqlen):
    """Where rows are cut depends on the shape alone: states saved beside aligned tensors serve
    a backward whose dout starts off every boundary, with the same bits; nothing outside the
    gradients is written."""
    import torch
    import selective_state_space_54_b200 as ssm
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    path = ssm.SSM_PATH_PER_GROUP if path == "per_group" else ssm.SSM_PATH_LOOKBACK
    shape = (2, 5, seqlen)
    gen = torch.Generator(device=cuda_device).manual_seed(seqlen)
    u, f, z, dy = (torch.randn(shape, device=cuda_device, generator=gen).to(dt) for _ in range(4))
    bias = torch.linspace(-1, 3, 5, device=cuda_device)
    h0 = torch.randn(2, 5, device=cuda_device, generator=gen)
    sh = ssm.gated_scan_shape(u, save_states=True, path=path)
    ws = torch.empty(max(ssm.gated_scan_fwd_workspace_bytes(sh), 256), dtype=torch.uint8, device=cuda_device)
    ssm.gated_scan_fwd(u, f, z, bias, initial_state=h0, workspace=ws, save_states=True, path=path)
    want = ssm.gated_scan_bwd(u, f, z, bias, dy, initial_state=h0, path=path, want_dinitial_state=True)

    def off(fill):  # one element past a 16-byte boundary, with a guard on either side
        whole = torch.full((u.numel() + 64,), 7.0, dtype=dt, device=cuda_device)
        part = whole[33:33 + u.numel()].view(shape)
        if fill is not None:
            part.copy_(fill)
        return whole, part

    outs = {k: off(None) for k in ("du", "df", "dz")}
    got = ssm.gated_scan_bwd(u, f, z, bias, off(dy)[1], initial_state=h0, path=path, want_dinitial_state=True,
                             fwd_workspace=ws, out={k: v[1] for k, v in outs.items()})
    for k, v in want.items():
        assert torch.equal(got[k], v), k
    for k, (whole, _) in outs.items():
        assert bool((whole[:33] == 7).all()) and bool((whole[33 + u.numel():] == 7).all()), k
