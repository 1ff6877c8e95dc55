"""CPU oracle of the operators behind the MoE layer -- test infrastructure only.

Plain NumPy: the norm of a block's output with its gate, the residual's addition and the next norm, low-rank
adapters of many requests, and their gradients. float64, except where a rounding is
part of an operator's definition.
"""
from __future__ import annotations

import numpy as np

from .block import round_bf16


def inverse_rms(v, eps) -> np.ndarray:
    """[T, 1] float64."""
    v = np.asarray(v, dtype=np.float64)
    with np.errstate(all="ignore"):
        return 1.0 / np.sqrt((v * v).sum(1, keepdims=True) / v.shape[1] + eps)


def gate_act(z, act) -> np.ndarray:
    z = np.asarray(z, dtype=np.float64)
    if act == "sigmoid":
        e = np.exp(-np.abs(z))
        return np.where(z >= 0, 1.0, e) / (1.0 + e)
    return np.tanh(z) if act == "tanh" else z


def gate_slope(z, act) -> np.ndarray:
    z = np.asarray(z, dtype=np.float64)
    e = np.exp(-np.abs(z))
    if act == "sigmoid":
        return e / (1.0 + e) ** 2
    return 4.0 * e * e / (1.0 + e * e) ** 2 if act == "tanh" else np.ones_like(z)


def sandwich(x, res, wp, gate, act, res_scale, branch_scale, post_eps):
    """(s, post_rstd, p) in float64 of bf16 inputs, s not yet rounded."""
    x = np.asarray(x, dtype=np.float64)
    r1 = None if wp is None else inverse_rms(x, post_eps)
    p = x if wp is None else x * r1 * wp
    f = branch_scale if gate is None else gate_act(gate, act) * branch_scale
    return p * f + (0.0 if res is None else np.asarray(res, dtype=np.float64) * res_scale), r1, p


def sandwich_bits(x, res, wp, gate, res_scale, branch_scale, post_eps):
    """(s, post_rstd) as stored, step by step in float32, for a gate without an activation (or none)."""
    f32 = np.float32
    p, r1 = f32(x), None
    if wp is not None:
        r1 = inverse_rms(x, post_eps).astype(f32)
        p = (p * r1) * f32(wp)
    p = p * (f32(branch_scale) if gate is None else f32(gate) * f32(branch_scale))
    return round_bf16(p if res is None else f32(res) * f32(res_scale) + p), r1


def sandwich_norm(s, w, eps):
    """(rstd, y) as stored, of the stream as it is stored."""
    r = inverse_rms(s, eps).astype(np.float32)
    return r, round_bf16((np.float32(s) * r) * np.float32(w))


def sandwich_backward(dy, d_s, x, s, wp, w, gate, act, res_scale, branch_scale, r1, r2):
    """float64 gradients {dx, d_res, d_gate (of every value), dw, dwp} of float64 inputs; d_gate before any sum."""
    H = x.shape[1]
    ds = np.zeros_like(x) if d_s is None else d_s
    out = {}
    if w is not None:
        xs, g = s * r2, dy * w
        ds = ds + r2 * (g - xs * (g * xs).sum(1, keepdims=True) / H)
        out["dw"] = (dy * xs).sum(0)
    out["d_res"] = res_scale * ds
    f = branch_scale * (1.0 if gate is None else gate_act(gate, act))
    xh = x if wp is None else x * r1
    p = xh if wp is None else xh * wp
    dp = f * ds
    if gate is not None:
        out["d_gate"] = branch_scale * gate_slope(gate, act) * ds * p
    if wp is not None:
        g = dp * wp
        out["dwp"] = (dp * xh).sum(0)
        dp = r1 * (g - xh * (g * xh).sum(1, keepdims=True) / H)
    out["dx"] = dp * np.ones_like(x)
    return out


def adapter(x, ids, a, b, scale=None, ranks=None, base=None):
    """(out, v) in float64: out[t] = base[t] + scale B A x[t] of the row's adapter; v = A x (0 past its rank)."""
    T, n, R = x.shape[0], a.shape[0], a.shape[1]
    out = np.zeros((T, b.shape[1])) if base is None else np.array(base, dtype=np.float64)
    v = np.zeros((T, R))
    for i in range(n):
        t = np.nonzero(ids == i)[0]
        k = R if ranks is None else min(max(int(ranks[i]), 0), R)
        v[t, :k] = x[t] @ a[i, :k].T
        out[t] += (1.0 if scale is None else float(scale[i])) * (v[t, :k] @ b[i, :, :k].T)
    return out, v


def adapter_backward(dout, x, v, ids, a, b, scale=None, ranks=None, dx_base=None):
    """float64 (dx, da, db)."""
    n, R = a.shape[0], a.shape[1]
    dx = np.zeros(x.shape) if dx_base is None else np.array(dx_base, dtype=np.float64)
    da, db = np.zeros(a.shape), np.zeros(b.shape)
    for i in range(n):
        t = np.nonzero(ids == i)[0]
        k = R if ranks is None else min(max(int(ranks[i]), 0), R)
        f = 1.0 if scale is None else float(scale[i])
        dv = f * (dout[t] @ b[i, :, :k])
        dx[t] += dv @ a[i, :k]
        da[i, :k] = dv.T @ x[t]
        db[i, :, :k] = f * (dout[t].T @ v[t, :k])
    return dx, da, db
