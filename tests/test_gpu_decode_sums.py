"""The few-token expert FFN's two products by themselves, through the workspace that lies between them.

h's codes are compared one by one. The inputs make W1 x a sum of whole multiples of one unit, less than 2^24 of them in all
magnitudes together, so that fp32 sums are exact in any order; large products that cancel stand next to small ones.
What is left is SwiGLU in fp32: exp(-g) is off by |g| 2^-24 (the argument's
rounding) and a few units, the sum, the quotient and the product by half a unit each: relative (|g| + 8) 2^-24. A code has to be
that of a value of float64's h within it.

out is compared with the float64 product of W2 and the very codes that the call left in the workspace: bf16's half step 2^-8,
and fp32 sums of exact products, I of them a pair in some order, K pairs, 16 partial sums and a product with the weight:
(I + K + 20) 2^-24 of the sum of magnitudes."""
import numpy as np
import pytest
import torch

import combine_moe_dispatch_02_amd as moe
import oracle
from oracle.mx import dequantize_mx_e4m3, dequantize_mx_fp4, quantize_mx_e4m3

from _gpu import say

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def call(x, idx, weights, w1, w1_s, w2, w2_s):
    """(out, codes of h [T * K, I], its scale bytes) of one call; x: bf16 rows, or codes and scales."""
    T, K = idx.shape
    I = w1.shape[1] // 2
    n = moe.expert_ffn_decode_workspace_bytes(T, K, I)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    x, x_s = x if isinstance(x, tuple) else (x, None)
    out = torch.empty(T, 2 * w1.shape[2], dtype=torch.bfloat16, device="cuda")
    moe.moe_expert_ffn_decode(x.cuda(), None if x_s is None else x_s.cuda(), idx.cuda(), weights.cuda(),
                              moe.moe_pack_weights(w1.cuda(), "mxfp4"), moe.moe_pack_mx_scales(w1_s.cuda()),
                              moe.moe_pack_weights(w2.cuda(), "mxfp4"), moe.moe_pack_mx_scales(w2_s.cuda()), ws, out)
    torch.cuda.synchronize()
    ws = ws.cpu().numpy()
    at = (T * K * I + 255) // 256 * 256
    return out, ws[:T * K * I].reshape(T * K, I), ws[at:at + T * K * (I // 32)].reshape(T * K, I // 32)


def e4m3(v):
    """v rounded to e4m3's values (float64, saturating)."""
    step = np.exp2(np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -6))) - 3)
    return np.clip(np.rint(v / step) * step, -448.0, 448.0)


def whole_case(T, H, I, E, seed):
    """x codes and scales, W1: products are whole multiples of 2^-9, up to 180 of them, but for two blocks of 32
    with a pair of values that are up to 2^14 times as large and whose products cancel."""
    rng = np.random.default_rng(seed)
    ints = oracle.e4m3_encode(np.arange(16, dtype=np.float32) * np.float32(2.0 ** -9)).astype(np.uint8)
    x = ints[rng.integers(0, 16, (T, H))] | (rng.integers(0, 2, (T, H)).astype(np.uint8) << 7)
    w = rng.integers(0, 16, (E, 2 * I, H), dtype=np.uint8)
    for block in rng.permutation(H // 32)[:2]:
        i, j = block * 32 + rng.permutation(32)[:2]
        x[:, i] = x[:, j] = oracle.e4m3_encode(np.float32(448.0))
        w[:, :, j] = w[:, :, i] ^ 8
    w1 = (w[:, :, ::2] | (w[:, :, 1::2] << 4)).astype(np.uint8)
    return x, np.full((T, H // 32), 127, np.uint8), w1, np.full((E, 2 * I, H // 32), 128, np.uint8)


# one wave's K blocks and several, the kernel for few pairs (8 waves), for many, and for many on few experts
@pytest.mark.parametrize("T,H,I,E", [(1, 128, 1024, 1), (8, 512, 256, 3), (9, 512, 256, 8), (40, 1152, 128, 4), (64, 2048, 128, 30)])
def test_every_code_of_h(T, H, I, E):
    say("decode every code of h", T, H, I, E)
    x, x_s, w1, w1_s = whole_case(T, H, I, E, T + H)
    idx = torch.from_numpy(np.random.default_rng(T).integers(0, E, (T, 1)).astype(np.int32))
    t = torch.from_numpy
    w2, w2_s = torch.zeros(E, H, I // 2, dtype=torch.uint8), torch.full((E, H, I // 32), 127, dtype=torch.uint8)
    _, codes, scales = call((t(x), t(x_s)), idx, torch.ones(T, 1), t(w1), t(w1_s), w2, w2_s)
    xv = dequantize_mx_e4m3(x, x_s)
    differs = 0
    for i in range(T):
        w = dequantize_mx_fp4(w1[idx[i, 0]], w1_s[idx[i, 0]])
        assert (np.abs(w) @ np.abs(xv[i])).max() < 2.0 ** 24 * 2.0 ** -9
        g = w @ xv[i]
        g, up = g[:I], g[I:]
        h = g / (1.0 + np.exp(-g)) * up
        bound = (np.abs(g) + 8) * U
        amax = np.abs(h).reshape(-1, 32).max(1)
        e = np.floor(np.log2(amax)) - 8
        wide = bound.reshape(-1, 32).max(1)
        sure = np.floor(np.log2(amax * (1 - wide))) == np.floor(np.log2(amax * (1 + wide)))   # else the scale may differ
        assert sure.mean() > 0.99 and np.array_equal(scales[i][sure], (e + 127).astype(np.uint8)[sure])
        v = h.reshape(-1, 32) * np.exp2(-e)[:, None]
        b = bound.reshape(-1, 32)
        low, high = e4m3(v * (1 - b)), e4m3(v * (1 + b))
        got = dequantize_mx_e4m3(codes[i:i + 1], np.full((1, I // 32), 127, np.uint8)).reshape(-1, 32)
        assert (((got == low) | (got == high))[sure]).all()
        differs += (low != high).sum()
    assert differs <= 2e-4 * T * I + 2                          # the comparison leaves hardly any code open


# W1's rows differ by up to 2^9, so that h's codes are of all sizes; then ordinary rows and more of everything, the last two by
# workgroups of 16 waves
@pytest.mark.parametrize("T,H,I,E,K,spread", [(1, 256, 128, 2, 1, 9), (5, 512, 128, 3, 1, 9), (16, 256, 256, 4, 2, 9), (33, 384, 128, 2, 2, 9),
                                              (64, 256, 128, 6, 1, 9), (64, 2048, 384, 5, 3, 9), (64, 4096, 640, 8, 4, 5),
                                              (3, 128, 1536, 6, 4, 0), (24, 512, 512, 40, 8, 0),
                                              (16, 128, 1536, 30, 8, 0), (64, 256, 1536, 16, 4, 0)])
def test_out_is_summed_in_fp32(T, H, I, E, K, spread):
    say("decode out's sums", T, H, I, E, K, spread)
    g = torch.Generator().manual_seed(T + H + I)
    r = lambda *s: torch.randint(0, 256, s, generator=g, dtype=torch.uint8)  # noqa: E731
    w1, w2 = r(E, 2 * I, H // 2), r(E, H, I // 2)
    w1_s = 127 - int(np.log2(H) / 2 + 2) - torch.randint(0, spread + 1, (E, 2 * I, 1), generator=g)
    w1_s = w1_s.expand(E, 2 * I, H // 32).contiguous().to(torch.uint8)
    w2_s = torch.randint(118, 123, (E, H, I // 32), generator=g, dtype=torch.uint8)
    x = torch.randn(T, H, generator=g).to(torch.bfloat16)
    idx = torch.randn(T, E, generator=g).topk(K, dim=1)[1].to(torch.int32)
    weights = torch.softmax(torch.randn(T, K, generator=g), 1)
    out, codes, scales = call(x, idx, weights, w1, w1_s, w2, w2_s)
    hv = dequantize_mx_e4m3(codes, scales).reshape(T, K, I)
    ref, mag = np.zeros((T, H)), np.zeros((T, H))
    for e in range(E):
        v = dequantize_mx_fp4(w2[e].numpy(), w2_s[e].numpy())
        for t, k in np.argwhere(idx.numpy() == e):
            p = float(weights[t, k])
            ref[t] += p * (v @ hv[t, k])
            mag[t] += p * (np.abs(v) @ np.abs(hv[t, k]))
    err = np.abs(oracle.bf16_to_f64(out.cpu()) - ref)
    assert (err <= 2.0 ** -8 * np.abs(ref) * (1 + 2.0 ** -7) + (I + K + 20) * U * mag).all()


def test_codes_of_h_far_below_zero():
    """silu of gates near -80: exp has to be right to its last bits there too, not off by |g| 2^-24. Each gate is a sum of four
    products, exact in fp32; exp is off by two units, 1 + exp, the quotient and the product by half a unit each: 6 * 2^-24 in all."""
    say("decode codes of h far below zero")
    T, H, I = 8, 128, 16384
    rng = np.random.default_rng(0)
    x = np.zeros((T, H), np.uint8)
    x[:, ::32] = oracle.e4m3_encode(np.float32(1.0))
    x[:, 96] = oracle.e4m3_encode((1 + np.arange(T) / 8).astype(np.float32))
    w = np.zeros((1, 2 * I, H), np.uint8)
    w[0, :I, 0], w[0, :I, 32] = 14, 14                                  # -4 * 16 - 4 * 4
    w[0, :I, 64], w[0, :I, 96] = rng.integers(0, 16, I), rng.integers(0, 16, I)
    w[0, I:, 64], w[0, I:, 96] = rng.integers(4, 8, I), rng.integers(0, 16, I)
    w1 = (w[:, :, ::2] | (w[:, :, 1::2] << 4)).astype(np.uint8)
    w1_s = np.broadcast_to(np.array([131, 129, 126, 121], np.uint8), (1, 2 * I, 4)).copy()
    t = torch.from_numpy
    w2, w2_s = torch.zeros(1, H, I // 2, dtype=torch.uint8), torch.full((1, H, I // 32), 127, dtype=torch.uint8)
    x_s = np.full((T, 4), 127, np.uint8)
    _, codes, scales = call((t(x), t(x_s)), torch.zeros(T, 1, dtype=torch.int32), torch.ones(T, 1), t(w1), t(w1_s), w2, w2_s)
    g = dequantize_mx_e4m3(x, x_s) @ dequantize_mx_fp4(w1[0], w1_s[0]).T
    assert (g[:, :I] < -75).all()
    h = (g[:, :I] / (1.0 + np.exp(-g[:, :I])) * g[:, I:]).reshape(-1, 32)
    e = np.floor(np.log2(np.abs(h).max(1))) - 8
    sure = np.floor(np.log2(np.abs(h).max(1) * (1 - 6 * U))) == np.floor(np.log2(np.abs(h).max(1) * (1 + 6 * U)))
    v = h * np.exp2(-e)[:, None]
    low, high = e4m3(v * (1 - 6 * U)), e4m3(v * (1 + 6 * U))
    got = dequantize_mx_e4m3(codes, np.full((T, I // 32), 127, np.uint8)).reshape(-1, 32)
    assert np.array_equal(scales.reshape(-1)[sure], (e + 127).astype(np.uint8)[sure])
    assert (((got == low) | (got == high))[sure]).all() and (low != high).mean() < 1e-4


@pytest.mark.parametrize("w_byte,x_byte", [(0, 240), (1, 240), (10, 246), (127, 127), (240, 3), (252, 8)])
def test_scales_at_the_ends(w_byte, x_byte):
    """The largest and smallest scales that are taken, each against one that brings the products back: h's codes are float64's."""
    say("decode scales at the ends", w_byte, x_byte)
    T, H, I = 4, 128, 256
    x, x_s, w1, w1_s = whole_case(T, H, I, 1, w_byte)
    if w_byte == 252:                                           # and the products stay in fp32
        x = np.where(x & 0x7F == 0x7E, x ^ 0x7E, x).astype(np.uint8)
    x_s[:], w1_s[:] = x_byte, w_byte
    t = torch.from_numpy
    w2, w2_s = torch.zeros(1, H, I // 2, dtype=torch.uint8), torch.full((1, H, I // 32), 127, dtype=torch.uint8)
    _, codes, scales = call((t(x), t(x_s)), torch.zeros(T, 1, dtype=torch.int32), torch.ones(T, 1), t(w1), t(w1_s), w2, w2_s)
    g = dequantize_mx_e4m3(x, x_s) @ dequantize_mx_fp4(w1[0], w1_s[0]).T
    h = g[:, :I] / (1.0 + np.exp(-g[:, :I])) * g[:, I:]
    ref, ref_s = quantize_mx_e4m3(h.astype(np.float32))
    assert (codes == ref).mean() > 0.999 and (scales == ref_s).all()
