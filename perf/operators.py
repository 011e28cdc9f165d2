"""Cases of the gated linear recurrence and of layer norm: their inputs, plain forms and exact values.

A case names an operator and a size:

* ``step``        one token of the gated recurrence for every (batch, channel), the state updated in place;
* ``scan``        the gated recurrence over whole sequences (a prompt's prefill), with the last state;
* ``scan_train``  a training step of it: the forward and the gradients of every input;
* ``norm``        layer norm, alone or with the residual stream's addition before it;
* ``norm_train``  a training step of that: the forward and the gradients of x, residual, weight and bias.

The recurrence, per batch element, channel d and step t, with g_t = sigmoid(-(f_t + f_bias_d)), a_t = 1 - g_t and
h_{t-1} taken as 0 where a packed sequence starts:

    h_t = a_t h_{t-1} + g_t u_t      (tied)      or      h_t = a_t h_{t-1} + u_t      (untied)
    y_t = h_t SiLU(z_t)

Layer norm, per row of dim values: s = x + residual, rounded to the residual's type (s = x without one), and
y = (s - mean(s)) / sqrt(var(s) + eps) * weight + bias.
"""
import math

import torch

own = False

EPS = 1e-5
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}


def _step(name, batch, dim, dtype, z=True, tied=True):
    return {"name": name, "op": "step", "batch": batch, "dim": dim, "dtype": dtype, "z": z, "tied": tied}


def _scan(name, op, batch, dim, length, dtype, tokens, z=True, tied=True, state=True, starts=False):
    return {"name": name, "op": op, "batch": batch, "dim": dim, "len": length, "dtype": dtype, "tokens": tokens,
            "z": z, "tied": tied, "state": state, "starts": starts}


def _norm(name, op, rows, dim, dtype, residual, bias=True):
    return {"name": name, "op": op, "rows": rows, "dim": dim, "dtype": dtype, "residual": residual, "bias": bias}


def listed():
    return [
        # one user's next token in a small layer: nothing but latency
        _step("step-1x1536", 1, 1536, "bf16"),
        # the next token of a full serving batch
        _step("step-128x5120", 128, 5120, "bf16"),
        # a short prompt of one user, an odd length
        _scan("scan-1x1536x77", "scan", 1, 1536, 77, "bf16", tokens=False),
        # a ragged fp32 batch as a projection leaves it, continued from a state, inputs gated by the caller
        _scan("scan-3x1001x1999-f32", "scan", 3, 1001, 1999, "f32", tokens=True, z=False, tied=False),
        # a large layer's prefill, channel rows as the causal convolution leaves them
        _scan("scan-4x5120x8192", "scan", 4, 5120, 8192, "bf16", tokens=False, state=False),
        # one very long sequence: few rows, each to be split over the machine
        _scan("scan-1x1024x1M", "scan", 1, 1024, 1 << 20, "bf16", tokens=False, state=False),
        # a training step on packed sequences, token rows as a projection leaves them
        _scan("train-8x4096x2048-packed", "scan_train", 8, 4096, 2048, "bf16", tokens=True, state=False, starts=True),
        # a small fp32 training step of odd length, carried over from the sequence's previous piece
        _scan("train-2x1536x3001-f32", "scan_train", 2, 1536, 3001, "f32", tokens=False, tied=False),
        # the norm before a layer of a serving batch's next token, on an fp32 residual stream
        _norm("norm-128x5120", "norm", 128, 5120, "bf16", "f32"),
        # the final norm over a long prompt
        _norm("norm-32768x4096", "norm", 32768, 4096, "bf16", "none"),
        # a training step of the norm before a layer, on an fp32 residual stream
        _norm("norm-train-16384x4096", "norm_train", 16384, 4096, "bf16", "f32"),
        # the same in fp32 with odd rows
        _norm("norm-train-4099x1537-f32", "norm_train", 4099, 1537, "f32", "f32"),
    ]


def draw(rng):
    def spread(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    op = rng.choice(["step", "scan", "scan", "scan_train", "scan_train", "norm", "norm_train"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    case = {"op": op}
    if op == "step":
        case.update(batch=spread(1, 512), dim=spread(64, 8192), dtype=dtype, z=rng.random() < 0.7, tied=rng.random() < 0.6)
    elif op in ("scan", "scan_train"):
        # up to 2^27 values a tensor, from wide batches of one token to single long sequences
        length = spread(1, 1 << 18)
        dim = spread(16, max(16, min(8192, (1 << 27) // length)))
        batch = spread(1, max(1, min(64, (1 << 27) // (length * dim))))
        case.update(batch=batch, dim=dim, len=length, dtype=dtype, tokens=rng.random() < 0.5, z=rng.random() < 0.7,
                    tied=rng.random() < 0.6, state=rng.random() < 0.5, starts=rng.random() < 0.5)
    else:
        dim = spread(8, 20000)
        case.update(rows=spread(1, max(1, min(100000, (1 << 27) // dim))), dim=dim, dtype=dtype,
                    residual=rng.choice(["none", "same", "f32"]), bias=rng.random() < 0.7)
    return case


def _residual_type(case):
    return torch.float32 if case["residual"] == "f32" else TYPES[case["dtype"]]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(shape, dtype=torch.float32, mean=0.0, std=1.0):
        return torch.randn(shape, generator=gen, device="cuda", dtype=dtype).mul_(std).add_(mean)

    s = dict(case)
    if case["op"] in ("norm", "norm_train"):
        shape, dt, rt = (case["rows"], case["dim"]), TYPES[case["dtype"]], _residual_type(case)
        s["x"] = normal(shape, dt)
        # a residual stream is wider than what a layer adds to it, and off centre
        s["residual"] = normal(shape, rt, 0.3, 3.0) if case["residual"] != "none" else None
        s["weight"] = normal((case["dim"],), mean=1.0, std=0.2)
        s["bias"] = normal((case["dim"],), std=0.2) if case["bias"] else None
        if case["op"] == "norm_train":
            s["dy"] = normal(shape, dt)
            s["dresidual"] = normal(shape, rt) if case["residual"] != "none" else None
        return s
    batch, dim, dt = case["batch"], case["dim"], TYPES[case["dtype"]]
    one = case["op"] == "step"
    tokens = (not one) and case["tokens"]
    shape = (batch, dim) if one else (batch, case["len"], dim) if tokens else (batch, dim, case["len"])
    s["u"] = normal(shape, dt)
    s["f"] = normal(shape, dt)
    s["z"] = normal(shape, dt) if case["z"] else None
    # from a memory of a few steps to one of some hundreds, channel by channel
    s["f_bias"] = torch.rand((dim,), generator=gen, device="cuda") * 6.0
    if one:
        s["state"] = normal((batch, dim))
        return s
    s["state0"] = normal((batch, dim)) if case["state"] else None
    s["starts"] = None
    if case["starts"]:  # packed sequences of some 400 steps on average, single tokens among them
        s["starts"] = torch.rand((batch, case["len"]), generator=gen, device="cuda") < 0.0025
    if case["op"] == "scan_train":
        s["dy"] = normal(shape, dt)
    return s


# ---- the plain forms -------------------------------------------------------------
def _recur(a, b):
    """h_t = a_t h_{t-1} + b_t from h = 0 along the last axis: pairs of steps are joined, the half-length
    recurrence gives every second state, and one step more the others."""
    n = a.shape[-1]
    if n == 1:
        return b
    even = n - n % 2
    a0, a1, b0, b1 = a[..., 0:even:2], a[..., 1:even:2], b[..., 0:even:2], b[..., 1:even:2]
    odd = _recur(a0 * a1, a1 * b0 + b1)
    h = torch.empty_like(b)
    h[..., 1:even:2] = odd
    h[..., 0] = b[..., 0]
    h[..., 2::2] = a[..., 2::2] * odd[..., : (n - 1) // 2] + b[..., 2::2]
    return h


def _gates(s):
    """u, a, g and z with the steps on the last axis, in 32 bits; a is 0 where a sequence starts."""
    def rows(t):
        return None if t is None else (t.transpose(1, 2) if s["tokens"] else t).float().contiguous()

    f = rows(s["f"]) + s["f_bias"][:, None]
    a, g = torch.sigmoid(f), torch.sigmoid(-f)
    keep = None if s["starts"] is None else (~s["starts"]).float()[:, None, :]
    return rows(s["u"]), a, g, rows(s["z"]), keep


def _plain_scan(s):
    u, a, g, z, keep = _gates(s)
    ak = a if keep is None else a * keep
    b = g * u if s["tied"] else u.clone()
    if s["state0"] is not None:
        b[..., 0] += ak[..., 0] * s["state0"]
    h = _recur(ak, b)
    y = h if z is None else h * z * torch.sigmoid(z)
    back = (lambda t: t.transpose(1, 2)) if s["tokens"] else (lambda t: t)
    out = {"y": back(y).to(s["u"].dtype).contiguous(), "last_state": h[..., -1].contiguous()}
    if s["op"] == "scan":
        return out
    dy = back(s["dy"]).float()
    dh = dy
    if z is not None:
        sz = torch.sigmoid(z)
        dh = dy * z * sz
        out["dz"] = back(dy * h * sz * (1 + z * (1 - sz))).to(s["u"].dtype).contiguous()
    # G_t = dh_t + a_{t+1} G_{t+1}: the same recurrence, backwards
    later = torch.zeros_like(ak)
    later[..., :-1] = ak[..., 1:]
    G = _recur(later.flip(-1), dh.flip(-1)).flip(-1)
    before = torch.empty_like(h)
    before[..., 1:] = h[..., :-1]
    before[..., 0] = 0 if s["state0"] is None else s["state0"]
    if keep is not None:
        before = before * keep
    df = G * (before - u if s["tied"] else before) * a * g
    out["du"] = back(G * g if s["tied"] else G).to(s["u"].dtype).contiguous()
    out["df"] = back(df).to(s["u"].dtype).contiguous()
    out["df_bias"] = df.double().sum((0, 2)).float()
    if s["state0"] is not None:
        out["dinitial_state"] = (ak[..., 0] * G[..., 0]).contiguous()
    return out


def _plain_step(s):
    f = s["f"].float() + s["f_bias"]
    a, g, u = torch.sigmoid(f), torch.sigmoid(-f), s["u"].float()
    h = a * s["state"] + (g * u if s["tied"] else u)
    s["state"].copy_(h)
    y = h
    if s["z"] is not None:
        z = s["z"].float()
        y = h * z * torch.sigmoid(z)
    return {"y": y.to(s["u"].dtype), "state": s["state"]}


def _plain_norm(s):
    dt = s["x"].dtype
    total = s["x"] if s["residual"] is None else (s["x"].float() + s["residual"].float()).to(s["residual"].dtype)
    r = total.float()
    c = r - r.mean(-1, keepdim=True)
    rstd = torch.rsqrt((c * c).mean(-1, keepdim=True) + EPS)
    xhat = c * rstd
    y = xhat * s["weight"]
    out = {"y": (y if s["bias"] is None else y + s["bias"]).to(dt)}
    if s["residual"] is not None:
        out["residual_out"] = total
    if s["op"] == "norm":
        return out
    dy = s["dy"].float()
    wdy = dy * s["weight"]
    dr = (wdy - wdy.mean(-1, keepdim=True) - xhat * (wdy * xhat).mean(-1, keepdim=True)) * rstd
    if s["dresidual"] is not None:
        dr = dr + s["dresidual"].float()
        out["dresidual"] = dr.to(s["residual"].dtype)
    out["dx"] = dr.to(dt)
    out["dweight"] = (dy * xhat).sum(0)
    if s["bias"] is not None:
        out["dbias"] = dy.sum(0)
    return out


# ---- the framework's calls -------------------------------------------------------
def _own(s):
    import selective_state_space_54_b200 as ssm
    if s["op"] == "step":
        y = ssm.gated_scan_step(s["u"], s["f"], s["z"], s["f_bias"], state=s["state"], tied=s["tied"])
        return {"y": y, "state": s["state"]}
    if s["op"] in ("scan", "scan_train"):
        kw = {"tied": s["tied"], "starts": s["starts"], "initial_state": s["state0"], "token_major": s["tokens"]}
        if s["op"] == "scan":
            y, last = ssm.gated_scan_fwd(s["u"], s["f"], s["z"], s["f_bias"], return_last_state=True, **kw)
            return {"y": y, "last_state": last}
        shape = ssm.gated_scan_shape(s["u"], token_major=s["tokens"], save_states=True)
        ws = torch.empty(ssm.gated_scan_fwd_workspace_bytes(shape), dtype=torch.uint8, device=s["u"].device)
        y, last = ssm.gated_scan_fwd(s["u"], s["f"], s["z"], s["f_bias"], return_last_state=True, save_states=True,
                                     workspace=ws, **kw)
        g = ssm.gated_scan_bwd(s["u"], s["f"], s["z"], s["f_bias"], s["dy"], fwd_workspace=ws,
                               want_dinitial_state=s["state0"] is not None, **kw)
        out = {"y": y, "last_state": last, "du": g["du"], "df": g["df"], "df_bias": g["df_bias"]}
        if s["z"] is not None:
            out["dz"] = g["dz"]
        if s["state0"] is not None:
            out["dinitial_state"] = g["dinitial_state"]
        return out
    if s["residual"] is None:
        y, total = ssm.layer_norm(s["x"], s["weight"], s["bias"], eps=EPS), s["x"]
        out = {"y": y}
    else:
        y, total = ssm.layer_norm(s["x"], s["weight"], s["bias"], residual=s["residual"], eps=EPS)
        out = {"y": y, "residual_out": total}
    if s["op"] == "norm":
        return out
    g = ssm.layer_norm_bwd(total, s["weight"], s["bias"], s["dy"], eps=EPS, dresidual_out=s["dresidual"])
    out.update(dx=g["dx"], dweight=g["dweight"])
    if s["residual"] is not None:
        out["dresidual"] = g["dresidual"]
    if s["bias"] is not None:
        out["dbias"] = g["dbias"]
    return out


def run(state):
    if own:
        return _own(state)
    if state["op"] == "step":
        return _plain_step(state)
    if state["op"] in ("scan", "scan_train"):
        return _plain_scan(state)
    return _plain_norm(state)


def work(case):
    e = BYTES[case["dtype"]]
    if case["op"] in ("norm", "norm_train"):
        n, r = case["rows"] * case["dim"], 4 if case["residual"] == "f32" else e
        stream = case["residual"] != "none"
        b = n * (2 * e + (2 * r if stream else 0)) + 4 * case["dim"] * (1 + case["bias"])
        if case["op"] == "norm":
            return {"bytes": b, "flops": 8 * n}
        # the gradients of x and of a residual of x's type are the same values: written once
        more = 0 if not stream else 2 * r if case["residual"] == "f32" else r
        return {"bytes": b + n * (2 * e + more) + 4 * case["dim"] * (1 + case["bias"]), "flops": 24 * n}
    n = case["batch"] * case["dim"]
    if case["op"] == "step":
        return {"bytes": n * (e * (3 + case["z"]) + 8) + 4 * case["dim"], "flops": 14 * n}
    full = n * case["len"]
    b = full * e * (3 + case["z"]) + 4 * n * (1 + case["state"]) + 4 * case["dim"] + case["starts"] * case["batch"] * case["len"]
    if case["op"] == "scan":
        return {"bytes": b, "flops": 14 * full}
    return {"bytes": b + full * e * (3 + case["z"]) + 4 * n * case["state"] + 4 * case["dim"], "flops": 45 * full}


# ---- exact values, in 64 bits and step by step -------------------------------------
def exact(case, seed):
    if case["op"] in ("scan", "scan_train") and case["len"] > 1 << 17:
        return None
    s = prepare(case, seed)
    wide = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v for k, v in s.items()}
    if case["op"] in ("norm", "norm_train"):
        return _exact_norm(case, wide, s)
    if case["op"] == "step":
        forget = 1 / (1 + torch.exp(-(wide["f"] + wide["f_bias"])))
        take = 1 / (1 + torch.exp(wide["f"] + wide["f_bias"]))
        h = forget * wide["state"] + (take * wide["u"] if case["tied"] else wide["u"])
        return {"y": h if wide["z"] is None else h * wide["z"] / (1 + torch.exp(-wide["z"])), "state": h}
    return _exact_scan(case, wide)


def _exact_scan(case, w):
    L, tied = case["len"], case["tied"]
    # [step][batch][dim] throughout
    first = lambda t: None if t is None else t.movedim(1 if case["tokens"] else 2, 0).contiguous()  # noqa: E731
    u, z, logit = first(w["u"]), first(w["z"]), first(w["f"]) + w["f_bias"]
    forget, take = 1 / (1 + torch.exp(-logit)), 1 / (1 + torch.exp(logit))
    carry = forget.clone()
    if w["starts"] is not None:
        carry[w["starts"].t()] = 0
    h0 = w["state0"] if w["state0"] is not None else torch.zeros_like(u[0])
    added = take * u if tied else u
    H = torch.empty_like(u)
    h = h0
    for t, (c, v, out) in enumerate(zip(carry.unbind(0), added.unbind(0), H.unbind(0))):
        h = torch.addcmul(v, c, h, out=out)
    place = lambda t: t.movedim(0, 1 if case["tokens"] else 2)  # noqa: E731
    silu = None if z is None else z / (1 + torch.exp(-z))
    out = {"y": place(H if z is None else H * silu), "last_state": H[L - 1]}
    if case["op"] == "scan":
        return out
    dy = first(w["dy"])
    G = dy.clone() if z is None else dy * silu
    for t in range(L - 2, -1, -1):
        G[t].addcmul_(carry[t + 1], G[t + 1])
    previous = torch.cat([h0[None], H[:-1]])
    if w["starts"] is not None:
        previous[w["starts"].t()] = 0
    df = G * forget * take * ((previous - u) if tied else previous)
    out.update(du=place(G * take if tied else G), df=place(df), df_bias=df.sum((0, 1)))
    if z is not None:
        p = 1 / (1 + torch.exp(-z))
        out["dz"] = place(dy * H * (p + z * p * (1 - p)))
    if w["state0"] is not None:
        out["dinitial_state"] = carry[0] * G[0]
    return out


def _exact_norm(case, w, s):
    x, dim = w["x"], case["dim"]
    r = x if w["residual"] is None else (x + w["residual"]).to(s["residual"].dtype).double()
    mean = r.sum(1, keepdim=True) / dim
    dev = (((r - mean) ** 2).sum(1, keepdim=True) / dim + EPS).sqrt()
    n = (r - mean) / dev
    out = {"y": n * w["weight"] + (0 if w["bias"] is None else w["bias"])}
    if w["residual"] is not None:
        out["residual_out"] = r
    if case["op"] == "norm":
        return out
    q = w["dy"] * w["weight"]
    d = (q - q.sum(1, keepdim=True) / dim - n * ((q * n).sum(1, keepdim=True) / dim)) / dev
    if w["dresidual"] is not None:
        d = d + w["dresidual"]
        out["dresidual"] = d
    out.update(dx=d, dweight=(w["dy"] * n).sum(0))
    if w["bias"] is not None:
        out["dbias"] = w["dy"].sum(0)
    return out
