"""The layer operators together, as a model uses them: residual add + norm,
projections, causal conv1d + SiLU, gated recurrence with its output gate,
projection, residual add + norm; forward and every gradient against autograd in
fp64, prefill continued by decode steps, and the training step in one CUDA graph."""
import numpy as np
import pytest

from gpu_util import rel_l2, to_f64

pytestmark = pytest.mark.gpu

B, L, D, DI, K = 2, 330, 96, 160, 4


def _params(seed):
    import torch
    g = torch.Generator().manual_seed(seed)
    r = lambda *s, sd=1.0: torch.randn(s, generator=g) * sd
    p = {"x": r(B, L, D), "res": r(B, L, D, sd=2.0), "w1": 1 + r(D, sd=0.2), "b1": r(D, sd=0.2),
         "win": r(3 * DI, D, sd=D ** -0.5), "cw": r(DI, K, sd=0.5), "cb": r(DI, sd=0.2), "fb": r(DI).abs() * 3,
         "wout": r(D, DI, sd=DI ** -0.5), "w2": 1 + r(D, sd=0.2), "b2": r(D, sd=0.2)}
    starts = torch.rand((B, L), generator=g) < 0.02
    return p, starts, r(B, L, D), r(B, L, D)


def _reference(p, starts, g1, g2):
    import torch
    q = {k: v.double().requires_grad_(True) for k, v in p.items()}
    norm = lambda s, w, b: torch.nn.functional.layer_norm(s, (D,), w, b, 1e-5)
    r1 = q["x"] + q["res"]
    proj = norm(r1, q["w1"], q["b1"]) @ q["win"].t()
    xc, f, z = (t.transpose(1, 2) for t in proj.split(DI, -1))
    c = torch.nn.functional.conv1d(torch.nn.functional.pad(xc, (K - 1, 0)), q["cw"][:, None], q["cb"], groups=DI)
    c = torch.nn.functional.silu(c)
    a = torch.sigmoid(f + q["fb"][:, None])
    h, hs = torch.zeros(B, DI, dtype=torch.float64), []
    for t in range(L):
        h = a[:, :, t] * torch.where(starts[:, t, None], 0.0, h) + (1 - a[:, :, t]) * c[:, :, t]
        hs.append(h)
    y = torch.stack(hs, -1) * torch.nn.functional.silu(z)
    r2 = r1 + y.transpose(1, 2) @ q["wout"].t()
    y2 = norm(r2, q["w2"], q["b2"])
    ((y2 * g1.double()).sum() + (r2 * g2.double()).sum()).backward()
    return {"y2": y2.detach().numpy(), "r2": r2.detach().numpy(), "last": h.detach().numpy(),
            **{"d" + k: v.grad.numpy() for k, v in q.items()}}


def _step(p, starts, g1, g2, token_major, ws):
    """One training step with the framework's calls; matrix products by torch."""
    import torch
    import selective_state_space_54_b200 as ssm
    rows = lambda t: t.reshape(-1, t.shape[-1])
    y1, r1 = ssm.layer_norm(p["x"], p["w1"], p["b1"], residual=p["res"])
    proj = y1 @ p["win"].t()
    xc = proj[..., :DI].transpose(1, 2).contiguous()
    c = ssm.causal_conv1d(xc, p["cw"], p["cb"])
    flip = lambda t: t.transpose(1, 2).contiguous()
    u = flip(c) if token_major else c
    f, z = (proj[..., i * DI:(i + 1) * DI].contiguous() for i in (1, 2))
    if not token_major:
        f, z = flip(f), flip(z)
    y, last = ssm.gated_scan_fwd(u, f, z, p["fb"], starts=starts, return_last_state=True, workspace=ws,
                                 save_states=True, token_major=token_major)
    yt = y if token_major else flip(y)
    y2, r2 = ssm.layer_norm(yt @ p["wout"].t(), p["w2"], p["b2"], residual=r1)
    n2 = ssm.layer_norm_bwd(r2, p["w2"], p["b2"], g1, dresidual_out=g2)
    do = n2["dx"]
    dyt = do @ p["wout"]
    gs = ssm.gated_scan_bwd(u, f, z, p["fb"], dyt if token_major else flip(dyt), starts=starts, fwd_workspace=ws,
                            token_major=token_major)
    du, df, dz = (gs[k] if not token_major else flip(gs[k]) for k in ("du", "df", "dz"))
    gc = ssm.causal_conv1d_bwd(xc, p["cw"], p["cb"], du)
    dproj = torch.cat([gc["dx"], df, dz], 1).transpose(1, 2).contiguous()
    n1 = ssm.layer_norm_bwd(r1, p["w1"], p["b1"], dproj @ p["win"], dresidual_out=do)
    return {"y2": y2, "r2": r2, "last": last, "dx": n1["dx"], "dres": n1["dresidual"], "dw1": n1["dweight"],
            "db1": n1["dbias"], "dwin": rows(dproj).t() @ rows(y1), "dcw": gc["dweight"], "dcb": gc["dbias"],
            "dfb": gs["df_bias"], "dwout": rows(do).t() @ rows(yt), "dw2": n2["dweight"], "db2": n2["dbias"]}


def _workspace(device, token_major):
    import torch
    import selective_state_space_54_b200 as ssm
    u = torch.empty((B, L, DI) if token_major else (B, DI, L), device=device)
    shape = ssm.gated_scan_shape(u, save_states=True, token_major=token_major)
    return torch.empty(ssm.gated_scan_fwd_workspace_bytes(shape), dtype=torch.uint8, device=device)


def _compare(got, ref):
    # ten fp32 stages, each within the library's 1e-5 rel-L2 of its own inputs, every one
    # of condition about 1: 1e-4 in all
    for k, v in ref.items():
        assert rel_l2(to_f64(got[k]), v) <= 1e-4, (k, rel_l2(to_f64(got[k]), v))


@pytest.mark.parametrize("token_major", [False, True])
def test_training_step(cuda_device, token_major):
    p, starts, g1, g2 = _params(1)
    ref = _reference(p, starts, g1, g2)
    dev = lambda t: t.to(cuda_device)
    got = _step({k: dev(v) for k, v in p.items()}, dev(starts), dev(g1), dev(g2), token_major,
                _workspace(cuda_device, token_major))
    _compare(got, ref)


@pytest.mark.parametrize("token_major", [False, True])
def test_training_step_in_a_graph(cuda_device, token_major):
    import torch
    import selective_state_space_54_b200 as ssm  # noqa: F401
    ws = _workspace(cuda_device, token_major)
    cases = [_params(s) for s in (2, 3)]
    put = lambda c: ({k: v.to(cuda_device) for k, v in c[0].items()}, *(t.to(cuda_device) for t in c[1:]))
    p, starts, g1, g2 = put(cases[0])
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        _step(p, starts, g1, g2, token_major, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = _step(p, starts, g1, g2, token_major, ws)
    for c in cases[::-1]:
        q = put(c)
        for k in p:
            p[k].copy_(q[0][k])
        for a, b in zip((starts, g1, g2), q[1:]):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        _compare(got, _reference(*c))


def test_prefill_then_decode(cuda_device):
    # a prompt through conv1d and the recurrence, then token by token with the states they
    # left: the same outputs as the whole sequence at once
    import torch
    import selective_state_space_54_b200 as ssm
    g = torch.Generator(device=cuda_device).manual_seed(4)
    r = lambda *s: torch.randn(s, generator=g, device=cuda_device)
    n, m = 45, 12
    x, f, z = r(3, DI, n + m), r(3, DI, n + m), r(3, DI, n + m)
    cw, cb, fb = r(DI, K), r(DI), r(DI).abs() * 3
    whole = ssm.gated_scan_fwd(ssm.causal_conv1d(x, cw, cb), f, z, fb)
    cut = lambda t, a, b: t[:, :, a:b].contiguous()
    c, tail = ssm.causal_conv1d(cut(x, 0, n), cw, cb, return_final_state=True)
    y, state = ssm.gated_scan_fwd(c, cut(f, 0, n), cut(z, 0, n), fb, return_last_state=True)
    out = [y]
    for t in range(n, n + m):
        c, tail = ssm.causal_conv1d(cut(x, t, t + 1), cw, cb, initial_state=tail, return_final_state=True)
        one = lambda v: v[:, :, t].contiguous()
        out.append(ssm.gated_scan_step(c[:, :, 0].contiguous(), one(f), one(z), fb, state=state)[:, :, None])
    got, want = to_f64(torch.cat(out, -1)), to_f64(whole)
    assert rel_l2(got, want) <= 1e-5


def test_residual_stream_in_fp32_under_bf16_activations(cuda_device):
    # the stream's own rounding never touches it: after many layers s is the exact fp32 sum
    import torch
    import selective_state_space_54_b200 as ssm
    w = torch.ones(D, device=cuda_device)
    s = torch.randn(7, D, device=cuda_device)
    want = s.clone()
    for _ in range(20):
        x = torch.randn(7, D, device=cuda_device).bfloat16()
        y, s = ssm.layer_norm(x, w, residual=s, residual_out=s)
        want = want + x.float()
        assert torch.equal(s, want) and y.dtype == torch.bfloat16
