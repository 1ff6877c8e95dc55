"""CPU oracle of the operators around the MoE layer -- test infrastructure only.

Plain NumPy in float64, row by row where that is plainest: the RMS norm with the residual's
addition and its gradients, the router's choice with its gradient, and the expert FFN of a
few tokens through MXFP4 experts. Roundings that are part of an operator's definition (the
bf16 stream, the fp32 products of the norm, MXFP8 of x and h) are written out.
"""
from __future__ import annotations

import numpy as np

from .moe_oracle import quantize_groups, silu
from .mx import dequantize_mx_e4m3, dequantize_mx_fp4, quantize_mx_e4m3

FLT_MAX = float(np.finfo(np.float32).max)


def round_bf16(v) -> np.ndarray:
    """float32 -> the float32 value of its bf16 (round to nearest, ties to even)."""
    v = np.ascontiguousarray(v, dtype=np.float32)
    b = v.view(np.uint32).astype(np.uint64)
    r = ((b + 0x7FFF + ((b >> 16) & 1)) >> 16).astype(np.uint32) << np.uint32(16)
    return np.where(np.isnan(v), np.float32(np.nan), r.view(np.float32)).astype(np.float32)


def rmsnorm(x, res, w, eps):
    """(s, rstd, y) of float32 inputs (bf16 values; w bf16 or fp32), each in float32 as stored."""
    with np.errstate(all="ignore"):
        s = round_bf16(np.float32(x) + np.float32(res)) if res is not None else np.float32(x)
        s64 = s.astype(np.float64)
        rstd = (1.0 / np.sqrt((s64 * s64).sum(1) / s.shape[1] + eps)).astype(np.float32)
        y = round_bf16((s * rstd[:, None]) * np.float32(w))
    return s, rstd, y


def quantize_rows(y, dtype):
    """(codes, scales) of finite bf16 rows in the layer's format: fp32 scales per 128 (fp8), E8M0
    bytes per 32 padded to whole words (mxfp4)."""
    if dtype == "fp8":
        return quantize_groups(y)
    codes, b = quantize_mx_e4m3(y)
    words = (y.shape[1] + 127) // 128
    return codes, np.pad(b, ((0, 0), (0, 4 * words - b.shape[1])))


def rmsnorm_backward(dy, s, w, rstd, d_res=None):
    """float64 (dx, dweight) of float64 inputs."""
    xhat = s * rstd[:, None]
    g = dy * w
    dx = rstd[:, None] * (g - xhat * (g * xhat).mean(1, keepdims=True))
    return (dx if d_res is None else dx + d_res), (dy * xhat).sum(0)


def router_topk(logits, K, *, score="softmax", normalize=True, groups=1, topk_groups=1, group_top=1, scale=1.0,
                bias=None):
    """(idx int [T, K], weights float64 [T, K]), one token after another."""
    l = np.asarray(logits, dtype=np.float64)
    T, E = l.shape
    size = E // groups
    idx = np.full((T, K), -1, dtype=np.int64)
    weights = np.zeros((T, K))
    for t in range(T):
        on = [e for e in range(E) if l[t, e] > -np.inf and (bias is None or bias[e] > -np.inf)]
        sc = scores(l[t], score)
        key = {e: min(l[t, e], FLT_MAX) for e in on}
        if bias is not None or (groups > 1 and group_top == 2):
            key = {e: sc[e] + (0.0 if bias is None else float(bias[e])) for e in on}
        rank = {}
        for g in range(groups):
            members = sorted((key[e] for e in on if e // size == g), reverse=True)[:group_top]
            if members:
                rank[g] = sum(members)
        kept = set(sorted(rank, key=lambda g: (-rank[g], g))[:topk_groups])
        pick = sorted((e for e in on if e // size in kept), key=lambda e: (-key[e], e))[:K]
        idx[t, :len(pick)] = pick
        if pick:
            weights[t, :len(pick)] = chosen_weights(l[t], pick, score, normalize) * scale
    return idx, weights


def scores(row, score) -> np.ndarray:
    """A token's scores; 0 for an expert that is switched off."""
    out = np.zeros(row.shape)
    on = row > -np.inf
    z = np.minimum(row, FLT_MAX)
    with np.errstate(over="ignore", under="ignore"):
        if score == "sigmoid":
            out[on] = 1.0 / (1.0 + np.exp(-z[on]))
        elif on.any():
            out[on] = np.exp(z[on] - z[on].max())
            out /= out.sum()
    return out


def chosen_weights(row, pick, score, normalize) -> np.ndarray:
    z = np.minimum(row, FLT_MAX)
    if score == "softmax" and normalize:
        with np.errstate(over="ignore", under="ignore"):
            e = np.exp(z[pick] - z[pick].max())
        return e / e.sum()
    s = scores(row, score)[pick]
    return s / s.sum() if normalize and s.sum() > 0 else (s * 0.0 if normalize else s)


def router_topk_backward(d_weights, logits, idx, *, score="softmax", normalize=True, scale=1.0, **_):
    """float64 d_logits [T, E] by the derivative of chosen_weights, entry by entry."""
    l = np.asarray(logits, dtype=np.float64)
    T, E = l.shape
    out = np.zeros((T, E))
    for t in range(T):
        at = [k for k in range(idx.shape[1]) if 0 <= idx[t, k] < E and l[t, idx[t, k]] > -np.inf]
        if not at:
            continue
        pick = [int(idx[t, k]) for k in at]
        d = np.asarray(d_weights[t], dtype=np.float64)[at] * scale
        w = chosen_weights(l[t], pick, score, normalize)
        s = scores(l[t], score)
        if score == "softmax" and normalize:
            for i, e in enumerate(pick):
                out[t, e] += w[i] * (d[i] - (w * d).sum())
        elif score == "softmax":
            out[t] -= s * (s[pick] * d).sum()
            for i, e in enumerate(pick):
                out[t, e] += s[e] * d[i]
        else:
            total = s[pick].sum() if normalize else 1.0
            mean = (w * d).sum() if normalize else 0.0
            for i, e in enumerate(pick):
                if total > 0:
                    out[t, e] += (d[i] - mean) / total * s[e] * (1.0 - s[e])
    return out


def expert_ffn_decode(x, x_s, idx, weights, w1, w1_s, w2, w2_s, expert_begin=0):
    """float64 out [T, H]. x: MXFP8 codes with E8M0 bytes (row-major, padded words), or float32
    rows with x_s None (quantised here); weights in row-major MXFP4 (codes, E8M0 bytes)."""
    if x_s is None:
        x, x_s = quantize_mx_e4m3(x)
    xv = dequantize_mx_e4m3(x, x_s[:, :x.shape[1] // 32])
    T, H = xv.shape
    I = w1.shape[1] // 2
    out = np.zeros((T, H))
    for t in range(T):
        for k in range(idx.shape[1]):
            e = int(idx[t, k]) - expert_begin
            if not 0 <= e < w1.shape[0]:
                continue
            g = dequantize_mx_fp4(w1[e], w1_s[e]) @ xv[t]
            h = silu(g[:I]) * g[I:]
            h = dequantize_mx_e4m3(*quantize_mx_e4m3(h.astype(np.float32)[None]))[0]
            out[t] += float(weights[t, k]) * (dequantize_mx_fp4(w2[e], w2_s[e]) @ h)
    return out
