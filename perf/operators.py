"""What stands around the expert FFN in a transformer's MoE block, as it is measured.

Four operators, each in a plain form (elementary torch operations, ``own`` false) and as the
framework's own calls (``own`` true):

* ``norm``: the residual's addition, the root-mean-square norm and an 8-bit copy with scales
  (the two quantised activation formats of the layer), and the backward pass;
* ``router``: the K experts of each token and their weights from the router's logits, and the
  backward pass;
* ``dispatch``: rows that already are 8-bit codes with scales into the expert-major pool;
* ``decode``: the expert FFN of a few tokens as matrix-vector products with MXFP4 weights,
  straight from the routing (no pool).

Sizes are those of this repository's workloads (H 4096 / I 1536 / 128 experts / top-8, and the
expert-parallel share H 7168 / I 2048 / 32 of 256 experts) and what serves them: one token,
small batches, ragged ones.
"""
import math

import numpy as np
import torch

own = False

BF16, F32, F64, E4M3, E8M0 = torch.bfloat16, torch.float32, torch.float64, torch.float8_e4m3fn, torch.float8_e8m0fnu
FLT_MAX = 3.4028234663852886e38
EPS = 1e-6


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------
def listed():
    return [
        # one generated token: the residual stream, the normed row for the router and its MXFP8 copy for the experts
        {"name": "norm_token_mx", "op": "norm", "T": 1, "H": 4096, "q": "mxfp4", "w": "bf16", "res": True, "train": False},
        # a prefill batch in front of the fp8 experts
        {"name": "norm_prefill_fp8", "op": "norm", "T": 8192, "H": 4096, "q": "fp8", "w": "bf16", "res": True, "train": False},
        # a training step of the skew workload: forward and backward, bf16
        {"name": "norm_train", "op": "norm", "T": 16384, "H": 4096, "q": "bf16", "w": "bf16", "res": True, "train": True},
        # a ragged training micro-batch at the expert-parallel width, fp32 master weight
        {"name": "norm_train_ragged", "op": "norm", "T": 1021, "H": 7168, "q": "bf16", "w": "f32", "res": True, "train": True},
        # one generated token's routing
        {"name": "router_token", "op": "router", "T": 1, "E": 128, "K": 8, "score": "softmax", "normalize": True,
         "groups": 1, "topk_groups": 1, "group_top": 1, "bias": False, "logits": "f32", "masked": 0.0, "train": False},
        # the skew workload's routing in training: softmax over the chosen experts
        {"name": "router_train", "op": "router", "T": 16384, "E": 128, "K": 8, "score": "softmax", "normalize": True,
         "groups": 1, "topk_groups": 1, "group_top": 1, "bias": False, "logits": "f32", "masked": 0.0, "train": True},
        # sigmoid scores, a selection bias that balances the experts, groups of experts; some experts switched off
        {"name": "router_groups", "op": "router", "T": 8192, "E": 256, "K": 8, "score": "sigmoid", "normalize": True,
         "groups": 8, "topk_groups": 4, "group_top": 2, "bias": True, "logits": "f32", "masked": 0.02, "train": True},
        # the fp8 workload's rows, quantised by the norm, into the pool
        {"name": "dispatch_fp8", "op": "dispatch", "T": 8192, "H": 4096, "E": 128, "E_local": 128, "begin": 0, "K": 8, "q": "fp8"},
        # a ragged MXFP8 batch on one expert-parallel rank: most pairs belong to other ranks
        {"name": "dispatch_mx_share", "op": "dispatch", "T": 1021, "H": 7168, "E": 256, "E_local": 32, "begin": 32, "K": 8, "q": "mxfp4"},
        # one generated token
        {"name": "decode_1", "op": "decode", "T": 1, "H": 4096, "I": 1536, "E": 128, "E_local": 128, "begin": 0, "K": 8, "x": "mxfp8"},
        # a small batch on one expert-parallel rank, unquantised rows
        {"name": "decode_13_share", "op": "decode", "T": 13, "H": 7168, "I": 2048, "E": 256, "E_local": 32, "begin": 32, "K": 8, "x": "bf16"},
        # a serving batch that reaches nearly every expert
        {"name": "decode_64", "op": "decode", "T": 64, "H": 4096, "I": 1536, "E": 128, "E_local": 128, "begin": 0, "K": 8, "x": "mxfp8"},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def _ranks(rng, pairs, most):
    """How many ranks the experts are spread over: so few that this one has some of the pairs."""
    return rng.choice([1] + [n for n in (2, 4, 8) if n <= most and pairs >= 8 * n])


def draw(rng):
    op = rng.choice(["norm", "router", "dispatch", "decode"])
    if op == "norm":
        q = rng.choice(["bf16", "fp8", "mxfp4"])
        step = {"bf16": 8, "fp8": 128, "mxfp4": 32}[q]
        return {"op": op, "T": _log(rng, 1, 8192), "H": step * _log(rng, max(1, 64 // step), 8192 // step), "q": q,
                "w": rng.choice(["bf16", "f32"]), "res": rng.random() < 0.7, "train": q == "bf16" and rng.random() < 0.7}
    if op == "router":
        groups = rng.choice([1, 1, 4, 8])
        E = groups * _log(rng, max(2, 8 // groups), 512 // groups)
        keep = 1 if groups == 1 else rng.randint(2, groups)
        K = rng.randint(1, min(16, keep * (E // groups)))
        # one chosen expert's normalised weight is 1 whatever the logits: its gradient is rounding alone
        return {"op": op, "T": _log(rng, 1, 16384), "E": E, "K": K,
                "score": rng.choice(["softmax", "sigmoid"]), "normalize": K > 1 and rng.random() < 0.6, "groups": groups,
                "topk_groups": keep, "group_top": rng.choice([1, 2]), "bias": rng.random() < 0.4,
                "logits": rng.choice(["f32", "bf16"]), "masked": rng.choice([0.0, 0.05]), "train": rng.random() < 0.6}
    if op == "dispatch":
        E_local = rng.choice([8, 32, 61, 128])
        T, K = _log(rng, 1, 8192), rng.randint(1, 8)
        ranks = _ranks(rng, T * K, 4)
        q = rng.choice(["fp8", "mxfp4"])
        step = {"fp8": 128, "mxfp4": 32}[q]
        return {"op": op, "T": T, "H": step * _log(rng, max(1, 128 // step), 4096 // step), "E": E_local * ranks,
                "E_local": E_local, "begin": E_local * rng.randrange(ranks), "K": K, "q": q}
    E_local = rng.choice([8, 16, 30, 64])
    T, K = _log(rng, 1, 64), rng.randint(1, 8)
    ranks = _ranks(rng, T * K, 8)
    return {"op": op, "T": T, "H": 128 * rng.randint(2, 40), "I": 128 * rng.randint(1, 16), "E": E_local * ranks,
            "E_local": E_local, "begin": E_local * rng.randrange(ranks), "K": K, "x": rng.choice(["bf16", "mxfp8"])}


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------
def _blocks(q):
    return {"fp8": 128, "mxfp4": 32}[q]


def _words(H):
    return (H + 127) // 128


def _quantise(y, q):
    """The layer's activation formats of fp32 rows: e4m3 codes, and scales per 128 values (fp32, amax / 448) or per 32
    values (the E8M0 byte of 2^(floor(log2 amax) - 8))."""
    g = y.unflatten(-1, (-1, _blocks(q)))
    amax = g.abs().amax(-1, keepdim=True)
    if q == "fp8":
        s = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
        codes = (g / s).clamp(-448.0, 448.0).to(E4M3)
        return codes.view(torch.uint8).flatten(-2), s.squeeze(-1)
    e = torch.where(amax > 0, torch.frexp(amax)[1] - 9, torch.full_like(amax, -127, dtype=torch.int32)).clamp(-127, 127)
    codes = (g * ((127 - e) << 23).view(F32)).clamp(-448.0, 448.0).to(E4M3)
    return codes.view(torch.uint8).flatten(-2), (e + 127).to(torch.uint8).squeeze(-1)


def _scale_values(byte):
    """E8M0 bytes as the powers of two that they stand for."""
    return torch.where(byte > 0, byte.int() << 23, torch.full_like(byte, 1, dtype=torch.int32) << 22).view(F32)


def _as_values(codes):
    return codes.view(E4M3)


def _routing(g, T, E, K):
    logits = torch.randn(T, E, generator=g, device="cuda")
    top, idx = torch.topk(logits, K, dim=1)
    return idx.to(torch.int32), torch.softmax(top, dim=1)


def _prep_norm(c, g):
    T, H = c["T"], c["H"]
    s = {"x": torch.randn(T, H, generator=g, device="cuda").to(BF16),
         "weight": (1.0 + 0.1 * torch.randn(H, generator=g, device="cuda")).to(BF16 if c["w"] == "bf16" else F32)}
    s["res"] = (3.0 * torch.randn(T, H, generator=g, device="cuda")).to(BF16) if c["res"] else None
    # what a program allocates once and hands to every call
    s["y"] = torch.empty(T, H, dtype=BF16, device="cuda")
    s["res_out"] = torch.empty(T, H, dtype=BF16, device="cuda") if c["res"] else None
    s["rstd"] = torch.empty(T, dtype=F32, device="cuda") if c["train"] else None
    s["q"] = s["q_s"] = None
    if c["q"] != "bf16":
        s["q"] = torch.empty(T, H, dtype=torch.uint8, device="cuda")
        s["q_s"] = (torch.empty(T, _words(H), dtype=F32, device="cuda") if c["q"] == "fp8"
                    else torch.empty(T, 4 * _words(H), dtype=torch.uint8, device="cuda"))
    if c["train"]:
        s["dy"] = torch.randn(T, H, generator=g, device="cuda").to(BF16)
        s["d_res"] = torch.randn(T, H, generator=g, device="cuda").to(BF16) if c["res"] else None
        s["dx"] = torch.empty(T, H, dtype=BF16, device="cuda")
        s["dweight"] = torch.empty(H, dtype=F32, device="cuda")
        if own:
            import combine_moe_dispatch_02_amd as moe
            s["ws"] = torch.empty(moe.rmsnorm_backward_workspace_bytes(T, H), dtype=torch.uint8, device="cuda")
    return s


def _prep_router(c, g):
    T, E, K = c["T"], c["E"], c["K"]
    l = torch.randn(T, E, generator=g, device="cuda") - 1.2 * torch.log(torch.arange(1, E + 1, device="cuda"))
    if c["masked"]:
        l = torch.where(torch.rand(T, E, generator=g, device="cuda") < c["masked"], -math.inf, l)
    dt = F32 if c["logits"] == "f32" else BF16
    s = {"logits": l.to(dt), "idx": torch.empty(T, K, dtype=torch.int32, device="cuda"),
         "weights": torch.empty(T, K, dtype=F32, device="cuda"),
         "bias": 0.1 * torch.randn(E, generator=g, device="cuda") if c["bias"] else None}
    if c["train"]:
        s["d_weights"] = torch.randn(T, K, generator=g, device="cuda")
        s["d_logits"] = torch.empty(T, E, dtype=dt, device="cuda")
    if own:
        import combine_moe_dispatch_02_amd as moe
        s["cfg"] = moe.RouterConfig(score=c["score"], normalize=c["normalize"], groups=c["groups"],
                                    topk_groups=c["topk_groups"], group_top=c["group_top"], scale=_route_scale(c))
    return s


def _route_scale(c):
    return 2.5 if c["score"] == "sigmoid" else 1.0


TILE = 128


def _prep_dispatch(c, g):
    T, H = c["T"], c["H"]
    codes, scales = _quantise(torch.randn(T, H, generator=g, device="cuda").to(BF16).float(), c["q"])
    if c["q"] == "mxfp4":
        scales = torch.nn.functional.pad(scales, (0, 4 * _words(H) - scales.shape[1]))
    idx, _ = _routing(g, T, c["E"], c["K"])
    rows = (T * c["K"] + c["E_local"] * (TILE - 1)) // TILE * TILE
    s = {"q": codes, "q_s": scales, "idx": idx, "rows": rows, "pool": torch.zeros(rows, H, dtype=torch.uint8, device="cuda")}
    s["pool_s"] = torch.zeros(rows, scales.shape[1], dtype=scales.dtype, device="cuda")
    if own:
        import combine_moe_dispatch_02_amd as moe
        s["plan"] = moe.Plan.allocate(T, c["K"], c["begin"], c["E_local"], TILE)
        s["ws"] = moe.Workspace(T, c["K"], c["E_local"], TILE)
    return s


def _prep_decode(c, g):
    T, H, I, E = c["T"], c["H"], c["I"], c["E_local"]

    def matrix(rows, K):
        # codes of every value alike (their spread is that of a quantised normal), scaled to 1 / sqrt(K)
        w = torch.randint(0, 256, (E, rows, K // 2), generator=g, device="cuda", dtype=torch.uint8)
        b = 127 + round(math.log2(K ** -0.5 / 2.9))
        return w, torch.randint(b, b + 2, (E, rows, K // 32), generator=g, device="cuda", dtype=torch.uint8)

    w1, w1_s = matrix(2 * I, H)
    w2, w2_s = matrix(H, I)
    # the same weights in the layer's load-time layout: 16 x 128 tiles, lane l of a tile holds 32 codes (one scale)
    # of row l % 16 from column 32 * (l / 16)
    pack = lambda w: w.view(E, w.shape[1] // 16, 16, -1, 4, 16).permute(0, 1, 3, 4, 2, 5).contiguous().view_as(w)  # noqa: E731
    pack_s = lambda s: s.view(E, s.shape[1] // 16, 16, -1, 4).permute(0, 1, 3, 4, 2).contiguous().view_as(s)  # noqa: E731
    idx, wt = _routing(g, T, c["E"], c["K"])
    x = torch.randn(T, H, generator=g, device="cuda").to(BF16)
    s = {"w1": w1, "w1_s": w1_s, "w2": w2, "w2_s": w2_s, "idx": idx, "weights": wt, "x": x, "x_s": None,
         "w1p": pack(w1), "w1p_s": pack_s(w1_s), "w2p": pack(w2), "w2p_s": pack_s(w2_s),
         "out": torch.empty(T, H, dtype=BF16, device="cuda")}
    if c["x"] == "mxfp8":
        s["x"], s["x_s"] = _quantise(x.float(), "mxfp4")
    if own:
        import combine_moe_dispatch_02_amd as moe
        s["ws"] = torch.empty(moe.expert_ffn_decode_workspace_bytes(T, c["K"], I), dtype=torch.uint8, device="cuda")
    return s


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"norm": _prep_norm, "router": _prep_router, "dispatch": _prep_dispatch, "decode": _prep_decode}[case["op"]](case, g)
    s["case"] = case
    return s


# ---------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------
def _norm_outputs(c, s):
    H = c["H"]
    out = {"y": s["y"]}
    if c["res"]:
        out["res_out"] = s["res_out"]
    if c["q"] == "fp8":
        out["codes"], out["scales"] = _as_values(s["q"]), s["q_s"]
    elif c["q"] == "mxfp4":
        out["codes"], out["scales"] = _as_values(s["q"]), s["q_s"][:, :H // 32].view(E8M0)
    if c["train"]:
        out["rstd"], out["dx"], out["dweight"] = s["rstd"], s["dx"], s["dweight"]
    return out


def _norm_plain(c, s):
    x, w = s["x"].float(), s["weight"].float()
    r = {"case": c, **s}
    if c["res"]:
        r["res_out"] = (x + s["res"].float()).to(BF16)   # the stream as it is stored is what is normed
        x = r["res_out"].float()
    # the statistic in 64 bits: codes and scales next to a rounding border hang on its last bit
    rstd = torch.rsqrt(x.double().square().mean(1, keepdim=True) + EPS).float()
    r["y"] = (x * rstd * w).to(BF16)
    if c["q"] != "bf16":
        r["q"], r["q_s"] = _quantise(r["y"].float(), c["q"])   # of the row as it is stored, as dispatch does it
    if c["train"]:
        g, xhat = s["dy"].float() * w, x * rstd
        dx = rstd * (g - xhat * (g * xhat).mean(1, keepdim=True))
        r["dx"] = (dx + s["d_res"].float() if c["res"] else dx).to(BF16)
        r["dweight"] = (s["dy"].float() * xhat).double().sum(0).float()
        r["rstd"] = rstd[:, 0]
    return _norm_outputs(c, r)


def _norm_own(c, s):
    import combine_moe_dispatch_02_amd as moe
    moe.moe_rmsnorm(s["x"], s["weight"], EPS, s["y"], res=s["res"], res_out=s["res_out"], rstd=s["rstd"], q=s["q"], q_s=s["q_s"],
                    dtype=c["q"])
    if c["train"]:
        moe.moe_rmsnorm_backward(s["dy"], s["res_out"] if c["res"] else s["x"], s["weight"], s["rstd"], s["dx"], s["dweight"],
                                 s["ws"], d_res=s["d_res"])
    return _norm_outputs(c, s)


def _keys(c, l, bias, score):
    """What experts are chosen by: the logits where their order is the scores', else the scores with the bias. In 64 bits:
    a sum next to another must not change places with it."""
    on = l > -math.inf
    l = l.double().clamp(max=FLT_MAX)
    if bias is None and (c["groups"] == 1 or c["group_top"] == 1):
        return torch.where(on, l, -math.inf)
    l = torch.where(on, l, -math.inf)
    if score == "sigmoid":
        key = torch.sigmoid(l)
    else:
        m = l.amax(1, keepdim=True)
        p = torch.where(on, torch.exp(l - m), 0.0)
        key = p / p.sum(1, keepdim=True)
    return torch.where(on, key if bias is None else key + bias.double(), -math.inf)


def _choose(c, key):
    """The K largest keys of each row, ties to the lowest index, out of the groups that are kept; -1 where there are none."""
    G = c["groups"]
    if G > 1:
        top = key.unflatten(1, (G, -1)).sort(dim=2, descending=True)[0][:, :, :c["group_top"]]
        on = top[:, :, :1].amax(2) > -math.inf
        of = torch.where(on, torch.where(top > -math.inf, top, 0.0).sum(2), -math.inf)
        at = of.sort(dim=1, descending=True, stable=True)[1]
        rank = torch.empty_like(at).scatter_(1, at, torch.arange(G, device=at.device).expand_as(at))
        kept = (rank < c["topk_groups"]) & on
        key = torch.where(kept.unsqueeze(2), key.unflatten(1, (G, -1)), -math.inf).flatten(1)
    v, at = key.sort(dim=1, descending=True, stable=True)
    K = c["K"]
    return torch.where(v[:, :K] > -math.inf, at[:, :K], -1)


def _route(c, l, bias, d_weights, dt):
    """idx, weights and, with d_weights, the gradient of the logits; l and the arithmetic of the weights in type dt."""
    idx = _choose(c, _keys(c, l, bias, c["score"]))
    on, scale = l > -math.inf, _route_scale(c)
    l = torch.where(on, l.to(dt).clamp(max=FLT_MAX), -FLT_MAX)
    got = idx >= 0
    at = idx.clamp(min=0)
    chosen = l.gather(1, at)
    if c["score"] == "softmax":
        m = (torch.where(got, chosen, -FLT_MAX) if c["normalize"] else l).amax(1, keepdim=True)
        e = torch.where(got, torch.exp(chosen - m), 0.0)
        total = e.sum(1, keepdim=True) if c["normalize"] else torch.where(on, torch.exp(l - m), 0.0).sum(1, keepdim=True)
    else:
        e = torch.where(got, torch.sigmoid(chosen), 0.0)
        total = e.sum(1, keepdim=True) if c["normalize"] else torch.ones_like(e[:, :1])
    total = torch.where(total > 0, total, 1.0)
    w = e / total
    if d_weights is None:
        return idx, w * scale, None
    d = torch.where(got, d_weights.to(dt), 0.0) * scale
    mean = (w * d).sum(1, keepdim=True)
    dl = torch.zeros_like(l)
    if c["score"] == "softmax" and not c["normalize"]:
        dl = -torch.where(on, torch.exp(l - m), 0.0) / total * mean
        part = w * d
    elif c["score"] == "softmax":
        part = w * (d - mean)
    else:
        part = (d - mean if c["normalize"] else d) / total * e * torch.sigmoid(-chosen)
    dl = dl.scatter_add(1, at, torch.where(got, part, 0.0))
    return idx, w * scale, dl


def _router_outputs(c, s):
    out = {"idx": s["idx"], "weights": s["weights"]}
    if c["train"]:
        out["d_logits"] = s["d_logits"]
    return out


def _router_plain(c, s):
    idx, w, dl = _route(c, s["logits"], s["bias"], s["d_weights"] if c["train"] else None, F32)
    return _router_outputs(c, {"idx": idx.to(torch.int32), "weights": w,
                               "d_logits": dl.to(s["logits"].dtype) if c["train"] else None})


def _router_own(c, s):
    import combine_moe_dispatch_02_amd as moe
    moe.moe_router_topk(s["logits"], s["idx"], s["weights"], s["cfg"], bias=s["bias"])
    if c["train"]:
        moe.moe_router_topk_backward(s["d_weights"], s["logits"], s["idx"], s["d_logits"], s["cfg"])
    return _router_outputs(c, s)


def _dispatch_outputs(c, pos, pool, pool_s):
    return {"pos": pos, "pool": _as_values(pool), "scales": pool_s if c["q"] == "fp8" else pool_s.view(E8M0)}


def _dispatch_plain(c, s):
    T, K, E, rows = c["T"], c["K"], c["E_local"], s["rows"]
    e = (s["idx"].long() - c["begin"]).flatten()
    e = torch.where((e >= 0) & (e < E), e, E)                     # E: another rank's
    counts = torch.zeros(E + 1, dtype=torch.int64, device=e.device).scatter_add_(0, e, torch.ones_like(e))
    whole = (counts + TILE - 1) // TILE * TILE
    start, first = whole.cumsum(0) - whole, counts.cumsum(0) - counts
    order = e.argsort(stable=True)                                # an expert's pairs in the order of the tokens
    es = e[order]
    row = torch.where(es < E, start[es] + torch.arange(T * K, device=e.device) - first[es], rows)
    pos = torch.empty_like(row).scatter_(0, order, torch.where(es < E, row, -1)).to(torch.int32)
    src = torch.full((rows + 1,), -1, dtype=torch.int64, device=e.device).scatter_(0, row, order)[:rows]
    real, t = (src >= 0).unsqueeze(1), (src // K).clamp(min=0)
    pool = torch.where(real, s["q"][t], s["pool"])
    # scales: one 4-byte word for 128 columns, the words of a tile's rows next to each other
    word = s["q_s"].view(F32)
    tiles = torch.where(real, word[t], s["pool_s"].view(F32).view(rows // TILE, -1, TILE).transpose(1, 2).reshape(rows, -1))
    tiles = tiles.view(rows // TILE, TILE, -1).transpose(1, 2).contiguous().view(rows, -1)
    return _dispatch_outputs(c, pos, pool, tiles.view(s["q_s"].dtype))


def _dispatch_own(c, s):
    import combine_moe_dispatch_02_amd as moe
    moe.moe_plan(s["idx"], s["plan"], s["ws"])
    moe.moe_dispatch_quantized(s["q"], s["q_s"], s["plan"], s["pool"], s["pool_s"], 1, s["ws"], dtype=c["q"])
    return _dispatch_outputs(c, s["plan"].pos, s["pool"], s["pool_s"])


FP4 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def _weights(codes, scales, dt):
    """[n, rows, K] values of MXFP4 weights."""
    pair = torch.tensor([(FP4[b & 15], FP4[b >> 4]) for b in range(256)], dtype=dt, device=codes.device)
    v = pair[codes.int()].flatten(-2).unflatten(-1, (-1, 32))
    return (v * _scale_values(scales).to(dt).unsqueeze(-1)).flatten(-2)


def _values(codes, scales, dt):
    v = _as_values(codes).to(dt).unflatten(-1, (-1, 32))
    return (v * _scale_values(scales).to(dt).unsqueeze(-1)).flatten(-2)


def _hidden(g, I):
    return torch.nn.functional.silu(g[..., :I]) * g[..., I:]


def _decode_plain(c, s):
    T, K, E, I = c["T"], c["K"], c["E_local"], c["I"]
    x, xs = (s["x"], s["x_s"]) if c["x"] == "mxfp8" else _quantise(s["x"].float(), "mxfp4")
    x = _values(x, xs, F32)
    e = s["idx"].long() - c["begin"]
    local = (e >= 0) & (e < E)
    wt = torch.where(local, s["weights"], 0.0)
    if T * K <= E:       # the experts of the pairs
        e = e.clamp(0, E - 1).flatten()
        w1, w2 = _weights(s["w1"][e], s["w1_s"][e], F32), _weights(s["w2"][e], s["w2_s"][e], F32)
        rows, wt = x.repeat_interleave(K, 0).unsqueeze(2), wt.flatten().unsqueeze(1)
        h = _hidden(torch.bmm(w1, rows).squeeze(2), I)
        h = _values(*_quantise(h, "mxfp4"), F32)
        y = torch.bmm(w2, h.unsqueeze(2)).squeeze(2) * wt
        return {"out": y.view(T, K, -1).sum(1).to(BF16)}
    # every expert here, each with all the tokens
    w1 = _weights(s["w1"], s["w1_s"], F32)
    h = _hidden(torch.matmul(x, w1.transpose(1, 2).contiguous()), I)
    h = _values(*_quantise(h, "mxfp4"), F32)
    w2 = _weights(s["w2"], s["w2_s"], F32)
    y = torch.matmul(h, w2.transpose(1, 2).contiguous())
    share = torch.zeros(T, E + 1, device=x.device).scatter_add_(1, torch.where(local, e, E), wt)[:, :E]
    return {"out": (y * share.t().unsqueeze(2)).sum(0).to(BF16)}


def _decode_own(c, s):
    import combine_moe_dispatch_02_amd as moe
    moe.moe_expert_ffn_decode(s["x"], s["x_s"], s["idx"], s["weights"], s["w1p"], s["w1p_s"], s["w2p"], s["w2p_s"], s["ws"],
                              s["out"], expert_begin=c["begin"])
    return {"out": s["out"]}


def run(state):
    c = state["case"]
    if own:
        return {"norm": _norm_own, "router": _router_own, "dispatch": _dispatch_own, "decode": _decode_own}[c["op"]](c, state)
    return {"norm": _norm_plain, "router": _router_plain, "dispatch": _dispatch_plain, "decode": _decode_plain}[c["op"]](c, state)


# ---------------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------------
def work(case):
    c = case
    if c["op"] == "norm":
        n, wb = c["T"] * c["H"], 2 if c["w"] == "bf16" else 4
        b = 2 * n + 2 * n + wb * c["H"] + (4 * n if c["res"] else 0)
        b += n + 4 * c["T"] * _words(c["H"]) if c["q"] != "bf16" else 0
        f = 4 * n + (n if c["res"] else 0) + (3 * n if c["q"] != "bf16" else 0)
        if c["train"]:   # the stored stream and dy again, the stream's gradient, dx
            b += 2 * n + 2 * n + 2 * n + (2 * n if c["res"] else 0) + (wb + 4) * c["H"] + 8 * c["T"]
            f += 10 * n
        return {"bytes": b, "flops": f}
    if c["op"] == "router":
        n, k, lb = c["T"] * c["E"], c["T"] * c["K"], 4 if c["logits"] == "f32" else 2
        b = lb * n + 8 * k + (4 * c["E"] if c["bias"] else 0)
        b += 2 * lb * n + 8 * k if c["train"] else 0
        return {"bytes": b, "flops": n * (4 if c["train"] else 2)}
    if c["op"] == "dispatch":
        pairs = c["T"] * c["K"]
        mine = pairs * c["E_local"] / c["E"]
        row = c["H"] + 4 * _words(c["H"])
        reach = 1.0 - (1.0 - c["E_local"] / c["E"]) ** c["K"]    # tokens with a pair here
        return {"bytes": 8 * pairs + row * (c["T"] * reach + mine), "flops": 0}
    experts = c["E_local"] * (1.0 - (1.0 - c["K"] / c["E"]) ** c["T"])
    one = 3 * c["H"] * c["I"]
    pairs = c["T"] * c["K"] * c["E_local"] / c["E"]
    return {"bytes": experts * one * (0.5 + 1 / 32) + c["T"] * c["H"] * (4 if c["x"] == "bf16" else 3 + 1 / 32), "flops": 2 * pairs * one}


# ---------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------------
def _exact_norm(c, s):
    x, w = s["x"].double(), s["weight"].double()
    out = {}
    if c["res"]:
        out["res_out"] = x + s["res"].double()
        x = out["res_out"].to(BF16).double()
    rstd = 1.0 / torch.sqrt((x * x).sum(1, keepdim=True) / c["H"] + EPS)
    out["y"] = x * rstd * w
    if c["q"] != "bf16":
        # the copy is of the row as it is stored: its roundings are part of the definition
        row = (x.float() * rstd.float() * w.float()).to(BF16)
        g = row.double().unflatten(1, (-1, _blocks(c["q"])))
        amax = g.abs().amax(2, keepdim=True)
        scale = amax / 448.0 if c["q"] == "fp8" else torch.exp2(torch.floor(torch.log2(amax)) - 8.0)
        scale = torch.where(amax > 0, scale, 1.0 if c["q"] == "fp8" else 2.0 ** -127)
        out["codes"] = (g / scale).clamp(-448.0, 448.0).flatten(1)
        out["scales"] = scale.squeeze(2)
    if c["train"]:
        dy = s["dy"].double()
        g = dy * w
        dot = (g * x).sum(1, keepdim=True) / c["H"]
        out["dx"] = g * rstd - x * dot * rstd ** 3 + (s["d_res"].double() if c["res"] else 0.0)
        out["dweight"] = (dy * x * rstd).sum(0)
        out["rstd"] = rstd[:, 0]
    return out


def _exact_router(c, s):
    """Row by row in numpy, from the definition."""
    l = s["logits"].double().cpu().numpy()
    bias = np.zeros(c["E"]) if s["bias"] is None else s["bias"].double().cpu().numpy()
    T, E, K, G = c["T"], c["E"], c["K"], c["groups"]
    scale, of = _route_scale(c), E // G
    idx, w = np.full((T, K), -1, np.int64), np.zeros((T, K))
    dl = np.zeros((T, E))
    dw = s["d_weights"].double().cpu().numpy() * scale if c["train"] else np.zeros((T, K))
    with np.errstate(over="ignore"):
        for t in range(T):
            on = np.nonzero(l[t] > -np.inf)[0]
            if not on.size:
                continue
            z = np.minimum(l[t], FLT_MAX)
            score = np.zeros(E)
            if c["score"] == "sigmoid":
                score[on] = 1.0 / (1.0 + np.exp(-z[on]))
            else:
                score[on] = np.exp(z[on] - z[on].max())
                score[on] /= score[on].sum()
            # scores without a bias are ordered as their logits are
            key = z if s["bias"] is None else score + bias
            pool = on
            if G > 1:
                by = {}
                for a in range(G):
                    m = on[on // of == a]
                    if m.size:
                        v = key[m] if c["group_top"] == 1 else (score + bias)[m]
                        by[a] = np.sort(v)[::-1][:c["group_top"]].sum()
                kept = sorted(by, key=lambda a: (-by[a], a))[:c["topk_groups"]]
                pool = on[np.isin(on // of, kept)]
            pick = pool[np.lexsort((pool, -key[pool]))][:K]
            n = pick.size
            idx[t, :n] = pick
            v = score[pick]
            total = v.sum() if c["normalize"] and v.sum() > 0 else 1.0
            w[t, :n] = scale * v / total
            d = dw[t, :n]
            if c["normalize"]:
                d = (d - (v * d).sum() / total) / total
            if c["score"] == "sigmoid":
                dl[t, pick] = d * v * (1.0 - v)
            else:
                dl[t, on] = -score[on] * (v * d).sum()
                dl[t, pick] += v * d
    out = {"idx": torch.from_numpy(idx), "weights": torch.from_numpy(w)}
    if c["train"]:
        out["d_logits"] = torch.from_numpy(dl)
    return out


def _exact_decode(c, s):
    I, E = c["I"], c["E_local"]
    if c["x"] == "mxfp8":
        x = _values(s["x"], s["x_s"], F64)
    else:
        x = _round_mx(s["x"].double())
    out = torch.zeros(c["T"], c["H"], dtype=F64, device="cuda")
    e = s["idx"].cpu().numpy() - c["begin"]
    for a in range(E):
        t, k = np.nonzero(e == a)
        if not t.size:
            continue
        t, k = torch.from_numpy(t).cuda(), torch.from_numpy(k).cuda()
        g = x[t] @ _weights(s["w1"][a], s["w1_s"][a], F64).t()
        h = g[:, :I] / (1.0 + torch.exp(-g[:, :I])) * g[:, I:]
        y = _round_mx(h) @ _weights(s["w2"][a], s["w2_s"][a], F64).t()
        out.index_add_(0, t, y * s["weights"][t, k].double().unsqueeze(1))
    return {"out": out}


def _round_mx(v):
    """The values that MXFP8 holds in place of v."""
    g = v.unflatten(1, (-1, 32))
    amax = g.abs().amax(2, keepdim=True)
    scale = torch.where(amax > 0, torch.exp2(torch.floor(torch.log2(amax)) - 8.0), 1.0)
    u = (g / scale).clamp(-448.0, 448.0)
    step = torch.exp2(torch.floor(torch.log2(u.abs().clamp(min=2.0 ** -6))) - 3.0)   # of e4m3 at that size
    return (torch.round(u / step) * step * scale).flatten(1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(case, s)
    if case["op"] == "router":
        return _exact_router(case, s) if case["T"] * case["E"] <= 4 << 20 else None
    if case["op"] == "dispatch":
        return None   # rows are moved: equal bit for bit, which the plain form says already
    return _exact_decode(case, s)
