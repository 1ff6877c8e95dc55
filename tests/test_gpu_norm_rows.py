"""The norm's backward pass where a workgroup has several rows, and a wave of the narrow layout a few or none, against
float64.

dx: bf16's half step 2^-8 and, in fp32, the roundings of three products and of the row's sum of H terms (at most 32 a lane,
then 64 lanes and 16 waves in a tree: at most 72 in a chain with those of a term): 2^-24 (8 |g| + 72 |xhat| mean|g xhat|) rstd. dweight:
a sum of T fp32 terms of two roundings, in some order, partial sums joined: (T + 24) 2^-24 of the sum of magnitudes."""
import pytest
import torch

import combine_moe_dispatch_02_amd as moe

from _gpu import say

pytestmark = pytest.mark.gpu

U = 2.0 ** -24

CASES = [(H, T) for H in (8, 24, 256, 472, 512) for T in (1025, 2049, 3500, 4333)]
CASES += [(H, T) for H in (520, 1024, 2048) for T in (2500, 3001)]
CASES += [(H, T) for H in (2056, 4096, 8192) for T in (1025, 1601)] + [(8200, 601), (16392, 600), (32768, 601)]


@pytest.mark.parametrize("H,T", CASES)
@pytest.mark.parametrize("wdt,with_res", [(torch.bfloat16, True), (torch.float32, False)])
def test_backward_of_many_rows(H, T, wdt, with_res):
    say("norm backward of many rows", H, T, wdt, with_res)
    g = torch.Generator(device="cuda").manual_seed(H + T)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    # rows and columns of their own sizes, so that none can stand for another
    s = (r(T, H) * (1 + torch.arange(T, device="cuda") % 7)[:, None]).to(torch.bfloat16)
    dy = (r(T, H) * (1 + torch.arange(H, device="cuda") % 5)).to(torch.bfloat16)
    w, d_res = r(H).to(wdt), r(T, H).to(torch.bfloat16) if with_res else None
    y, rstd = torch.empty_like(s), torch.empty(T, device="cuda")
    moe.moe_rmsnorm(s, w, 1e-6, y, rstd=rstd)
    dx, dw = torch.full_like(s, 7.0), torch.full((H + 8,), 7.0, device="cuda")
    ws = torch.full((moe.rmsnorm_backward_workspace_bytes(T, H),), 255, dtype=torch.uint8, device="cuda")
    moe.moe_rmsnorm_backward(dy, s, w, rstd, dx, dw[:H], ws, d_res=d_res)
    torch.cuda.synchronize()
    assert bool((dw[H:] == 7.0).all())
    R = rstd.double()[:, None]
    xhat = s.double() * R
    gd = dy.double() * w.double()
    t = gd * xhat
    ref = R * (gd - xhat * t.mean(1, keepdim=True))
    tol = 1.01 * U * R * (8 * gd.abs() + 72 * xhat.abs() * t.abs().mean(1, keepdim=True))
    if with_res:
        ref += d_res.double()
        tol += 2 * 1.01 * U * d_res.double().abs()
    assert bool(((dx.double() - ref).abs() <= tol + 2.0 ** -8 * ref.abs()).all())
    t = dy.double() * xhat
    assert bool(((dw[:H].double() - t.sum(0)).abs() <= (T + 24) * U * t.abs().sum(0)).all())
