"""fp64 references of the layer operators beside the selective scan, in numpy:
the gated linear recurrence (step by step) and layer norm, with their
gradients.  Written from the formulas; shares no code with the CUDA path.

Shapes are token-last: u, f, z, dy (batch, dim, seqlen); states (batch, dim);
starts (batch, seqlen) truth values.
"""
from __future__ import annotations

import numpy as np


def sigmoid(x):
    """1 / (1 + e^-x) without overflow, exact at the infinities."""
    x = np.asarray(x, np.float64)
    with np.errstate(over="ignore"):
        return np.where(x >= 0, 1.0 / (1.0 + np.exp(-np.abs(x))), np.exp(-np.abs(x)) / (1.0 + np.exp(-np.abs(x))))


def gated_scan(u, f, z=None, f_bias=None, *, tied=True, starts=None, h0=None):
    """{"y", "last_state", "h"}: h (batch, dim, seqlen) holds every state."""
    u, f = np.asarray(u, np.float64), np.asarray(f, np.float64)
    logit = f if f_bias is None else f + np.asarray(f_bias, np.float64)[None, :, None]
    a, g = sigmoid(logit), sigmoid(-logit)
    batch, dim, L = u.shape
    h = np.zeros((batch, dim)) if h0 is None else np.array(h0, np.float64)
    H = np.zeros_like(u)
    for t in range(L):
        prev = h if starts is None else np.where(np.asarray(starts)[:, t, None], 0.0, h)
        h = a[:, :, t] * prev + (g[:, :, t] * u[:, :, t] if tied else u[:, :, t])
        H[:, :, t] = h
    y = H
    if z is not None:
        z = np.asarray(z, np.float64)
        y = H * z * sigmoid(z)
    return {"y": y, "last_state": h, "h": H}


def gated_scan_bwd(u, f, z, f_bias, dy, *, tied=True, starts=None, h0=None, dlast=None):
    """Gradients of sum(dy * y) + sum(dlast * last_state)."""
    u, f, dy = (np.asarray(x, np.float64) for x in (u, f, dy))
    logit = f if f_bias is None else f + np.asarray(f_bias, np.float64)[None, :, None]
    a, g = sigmoid(logit), sigmoid(-logit)
    H = gated_scan(u, f, z, f_bias, tied=tied, starts=starts, h0=h0)["h"]
    batch, dim, L = u.shape
    out = {"du": np.zeros_like(u), "df": np.zeros_like(u), "dz": None}
    dh = dy
    if z is not None:
        z = np.asarray(z, np.float64)
        s = sigmoid(z)
        dh = dy * z * s
        out["dz"] = dy * H * (s + z * s * (1 - s))
    P = np.zeros((batch, dim)) if dlast is None else np.array(dlast, np.float64)
    for t in range(L - 1, -1, -1):
        prev = H[:, :, t - 1] if t else (np.zeros((batch, dim)) if h0 is None else np.asarray(h0, np.float64))
        cut = np.zeros((batch, 1), bool) if starts is None else np.asarray(starts)[:, t, None].astype(bool)
        prev = np.where(cut, 0.0, prev)
        G = dh[:, :, t] + P
        out["du"][:, :, t] = G * g[:, :, t] if tied else G
        out["df"][:, :, t] = G * (prev - u[:, :, t] if tied else prev) * a[:, :, t] * g[:, :, t]
        P = np.where(cut, 0.0, a[:, :, t] * G)
    out["dinitial_state"] = P
    out["df_bias"] = out["df"].sum((0, 2)) if f_bias is not None else None
    return out


def layer_norm(s, weight, bias=None, eps=1e-5):
    """y of rows s (rows, dim)."""
    s = np.asarray(s, np.float64)
    c = s - s.mean(-1, keepdims=True)
    y = c / np.sqrt((c * c).mean(-1, keepdims=True) + eps) * np.asarray(weight, np.float64)
    return y if bias is None else y + np.asarray(bias, np.float64)


def layer_norm_bwd(s, weight, dy, eps=1e-5, dresidual=None):
    """{"ds", "dweight", "dbias"} of sum(dy * y) (+ dresidual reaching s past the norm)."""
    s, dy, weight = (np.asarray(x, np.float64) for x in (s, dy, weight))
    c = s - s.mean(-1, keepdims=True)
    r = 1.0 / np.sqrt((c * c).mean(-1, keepdims=True) + eps)
    q, wd = c * r, dy * weight
    ds = r * (wd - wd.mean(-1, keepdims=True) - q * (wd * q).mean(-1, keepdims=True))
    if dresidual is not None:
        ds = ds + np.asarray(dresidual, np.float64)
    return {"ds": ds, "dweight": (dy * q).sum(0), "dbias": dy.sum(0)}
