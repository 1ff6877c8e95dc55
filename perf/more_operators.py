"""What stands behind the MoE layer in a fine-tuned transformer block, as it is measured.

Two operators with their backward passes, each in a plain form (elementary torch operations,
``own`` false) and as the framework's own calls (``own`` true):

* ``sandwich``: the norm behind a block, the block's gate, both branches' scales, the residual's
  addition, the next block's norm and its 8-bit copy in the layer's activation formats;
* ``adapter``: low-rank adapters of many requests at once beside a shared projection: each row
  through its own request's pair of factors, added to what the projection gave.

Sizes are those of this repository's workloads (H 4096 and 7168; 1 to 16384 rows; the ragged
1021 rows) and what serves and trains them: one token, small batches of many requests, prompts
of several requests, one fine-tune of a whole batch.
"""
import math

import torch

own = False

BF16, F32, F64, E4M3, E8M0 = torch.bfloat16, torch.float32, torch.float64, torch.float8_e4m3fn, torch.float8_e8m0fnu
EPS, POST_EPS = 1e-6, 1e-5


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------
def _sandwich(name, **kw):
    c = {"op": "sandwich", "q": "bf16", "w": "bf16", "post": True, "pre": True, "gate": "none", "act": "none", "gate_t": "bf16",
         "res_scale": 1.0, "branch_scale": 1.0, "train": False, **kw}
    return {"name": name, **c}


def _adapter(name, **kw):
    c = {"op": "adapter", "n": 1, "ids": "mixed", "none": 0.0, "ranks": "full", "base": True, "plan": False, "train": False, **kw}
    return {"name": name, **c}


def listed():
    return [
        # one generated token behind the experts: post-norm, a learned gate of the token, and the MXFP8 copy the next layer takes
        _sandwich("sandwich_token_mx", T=1, H=4096, q="mxfp4", gate="row", act="sigmoid"),
        # a prefill batch between two layers with fp8 experts
        _sandwich("sandwich_prefill_fp8", T=8192, H=4096, q="fp8"),
        # a training step: forward and backward with a learned scale for each channel
        _sandwich("sandwich_train", T=16384, H=4096, gate="channel", train=True),
        # a ragged training micro-batch at the expert-parallel width: a gate for every value, fp32 master weights, scaled residual
        _sandwich("sandwich_train_ragged", T=1021, H=7168, w="f32", gate="full", act="sigmoid", res_scale=0.5, branch_scale=1.5, train=True),
        # a serving batch of a model without post-norms: a shared branch's token gate and a residual multiplier
        _sandwich("sandwich_scaled", T=333, H=5120, post=False, gate="row", act="sigmoid", gate_t="f32", branch_scale=0.22),
        # one generated token of one request
        _adapter("adapter_token", T=1, K=4096, N=4096, R=16, n=64),
        # a serving batch: nearly every row another request's adapter, of different ranks, some rows with none
        _adapter("adapter_decode_64", T=64, K=4096, N=4096, R=64, n=64, ranks="mixed", none=0.1),
        # prompts of several requests, the batch's first projection (its rows are grouped here)
        _adapter("adapter_prompt", T=8192, K=4096, N=4096, R=64, n=16, ids="runs", plan=True),
        # a ragged prompt batch into a narrow projection, some requests without an adapter
        _adapter("adapter_prompt_ragged", T=1021, K=7168, N=2048, R=24, n=32, ids="runs", ranks="mixed", none=0.2),
        # one adapter fine-tuned on a whole batch
        _adapter("adapter_train", T=8192, K=4096, N=4096, R=64, n=1, ids="runs", train=True),
        # several fine-tunes in one batch
        _adapter("adapter_train_many", T=4333, K=4096, N=7168, R=16, n=8, ids="runs", none=0.05, train=True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    if rng.random() < 0.5:
        q = rng.choice(["bf16", "bf16", "fp8", "mxfp4"])
        step = {"bf16": 8, "fp8": 128, "mxfp4": 32}[q]
        c = _sandwich("", T=_log(rng, 1, 8192), H=step * _log(rng, max(1, 64 // step), 8192 // step), q=q, w=rng.choice(["bf16", "f32"]),
                      post=rng.random() < 0.7, pre=q != "bf16" or rng.random() < 0.8, gate=rng.choice(["none", "row", "channel", "full"]),
                      act=rng.choice(["none", "sigmoid", "tanh"]), gate_t=rng.choice(["bf16", "f32"]), res_scale=rng.choice([1.0, 1.0, 0.5, 3.0]),
                      branch_scale=rng.choice([1.0, 0.22, 1.5]), train=q == "bf16" and rng.random() < 0.6)
    else:
        T = _log(rng, 1, 8192)
        c = _adapter("", T=T, K=8 * _log(rng, 8, 512), N=8 * _log(rng, 8, 512), R=8 * rng.randint(1, 8), n=_log(rng, 1, 64),
                     ids=rng.choice(["runs", "mixed"]), none=rng.choice([0.0, 0.1]), ranks=rng.choice(["full", "mixed"]),
                     base=rng.random() < 0.8, plan=T > 64 and rng.random() < 0.4, train=rng.random() < 0.4)
    del c["name"]
    return c


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------
def _blocks(q):
    return {"fp8": 128, "mxfp4": 32}[q]


def _words(H):
    return (H + 127) // 128


def _type(t):
    return BF16 if t == "bf16" else F32


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _prep_sandwich(c, g):
    T, H = c["T"], c["H"]
    s = {"x": (0.7 * _normal(g, T, H)).to(BF16), "res": (3.0 * _normal(g, T, H)).to(BF16),
         "w": (1.0 + 0.1 * _normal(g, H)).to(_type(c["w"])) if c["pre"] else None,
         "wp": (0.8 + 0.1 * _normal(g, H)).to(_type(c["w"])) if c["post"] else None}
    shape = {"none": None, "row": (T, 1), "channel": (H,), "full": (T, H)}[c["gate"]]
    # a gate without an activation is a learned factor around one, the others are logits
    s["gate"] = None if shape is None else ((1.0 + 0.3 * _normal(g, *shape)) if c["act"] == "none" else _normal(g, *shape)).to(_type(c["gate_t"]))
    # what a program allocates once and hands to every call
    s["s"] = torch.empty(T, H, dtype=BF16, device="cuda")
    s["y"] = torch.empty(T, H, dtype=BF16, device="cuda") if c["pre"] else None
    s["rstd"] = torch.empty(T, dtype=F32, device="cuda") if c["train"] and c["pre"] else None
    s["post_rstd"] = torch.empty(T, dtype=F32, device="cuda") if c["train"] and c["post"] else None
    s["q"] = s["q_s"] = None
    if c["q"] != "bf16":
        s["q"] = torch.empty(T, H, dtype=torch.uint8, device="cuda")
        s["q_s"] = (torch.empty(T, _words(H), dtype=F32, device="cuda") if c["q"] == "fp8"
                    else torch.empty(T, 4 * _words(H), dtype=torch.uint8, device="cuda"))
    if c["train"]:
        s["dy"] = _normal(g, T, H).to(BF16) if c["pre"] else None
        s["d_s"] = _normal(g, T, H).to(BF16)
        s["dx"], s["d_res"] = torch.empty_like(s["x"]), torch.empty_like(s["x"])
        s["dw"] = torch.empty(H, dtype=F32, device="cuda") if c["pre"] else None
        s["dwp"] = torch.empty(H, dtype=F32, device="cuda") if c["post"] else None
        s["d_gate"] = None if shape is None else torch.empty(shape, dtype=F32 if c["gate"] == "channel" else s["gate"].dtype, device="cuda")
        if own:
            import combine_moe_dispatch_02_amd as moe
            s["ws"] = torch.empty(moe.sandwich_norm_backward_workspace_bytes(T, H), dtype=torch.uint8, device="cuda")
    return s


def _prep_adapter(c, g):
    T, K, N, R, n = c["T"], c["K"], c["N"], c["R"], c["n"]
    if c["ids"] == "runs":     # requests one behind another, of uneven lengths
        q = min(T, 2 * n)
        cuts = torch.rand(T, generator=g, device="cuda").argsort()[:q]
        of = torch.zeros(T, dtype=torch.int64, device="cuda").scatter_(0, cuts, 1).cumsum(0).clamp(max=q - 1)
        which = torch.randint(0, n, (q,), generator=g, device="cuda")
        which = torch.where(torch.rand(q, generator=g, device="cuda") < c["none"], -1, which)
        ids = which[of]
    else:
        ids = torch.randint(0, n, (T,), generator=g, device="cuda")
        ids = torch.where(torch.rand(T, generator=g, device="cuda") < c["none"], -1, ids)
    s = {"x": _normal(g, T, K).to(BF16), "ids": ids.to(torch.int32),
         "a": (_normal(g, n, R, K) / math.sqrt(K)).to(BF16), "b": (_normal(g, n, N, R) / math.sqrt(R)).to(BF16),
         "scale": 0.5 + 1.5 * torch.rand(n, generator=g, device="cuda"),
         "base": _normal(g, T, N).to(BF16) if c["base"] else None, "out": torch.empty(T, N, dtype=BF16, device="cuda")}
    # an adapter of lower rank has its first rows of a, its first columns of b; the others hold anything
    s["ranks"] = None
    if c["ranks"] == "mixed":
        s["ranks"] = torch.randint(0, 4, (n,), generator=g, device="cuda").add(1).mul(R).div(4, rounding_mode="floor").to(torch.int32)
    if c["train"]:
        s["dout"], s["dx_base"] = _normal(g, T, N).to(BF16), _normal(g, T, K).to(BF16)
        s["v"] = torch.empty(T, R, dtype=F32, device="cuda")
        s["dx"] = torch.empty(T, K, dtype=BF16, device="cuda")
        s["da"], s["db"] = torch.empty(n, R, K, dtype=F32, device="cuda"), torch.empty(n, N, R, dtype=F32, device="cuda")
    if own:
        import combine_moe_dispatch_02_amd as moe
        s["ws"] = torch.empty(moe.adapter_workspace_bytes(T, K, R), dtype=torch.uint8, device="cuda")
        s["plan"] = None
        if T > 64 or c["train"]:
            # the rows' grouping, which all projections of a batch share
            tile = moe.adapter_tile(T, n)
            s["plan"], s["plan_ws"] = moe.Plan.allocate(T, 1, 0, n, tile), moe.Workspace(T, 1, n, tile)
            moe.moe_plan(s["ids"].view(T, 1), s["plan"], s["plan_ws"])
        if c["train"]:
            s["bws"] = torch.empty(moe.adapter_backward_workspace_bytes(T, n, K, N, R), dtype=torch.uint8, device="cuda")
    return s


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"sandwich": _prep_sandwich, "adapter": _prep_adapter}[case["op"]](case, g)
    s["case"] = case
    return s


# ---------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------
def _quantise(y, q):
    """The layer's activation formats of fp32 rows: e4m3 codes, and scales per 128 values (fp32, amax / 448) or per 32
    values (the E8M0 byte of 2^(floor(log2 amax) - 8))."""
    g = y.unflatten(-1, (-1, _blocks(q)))
    amax = g.abs().amax(-1, keepdim=True)
    if q == "fp8":
        s = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
        return (g / s).clamp(-448.0, 448.0).to(E4M3).flatten(-2), s.squeeze(-1)
    e = torch.where(amax > 0, torch.frexp(amax)[1] - 9, torch.full_like(amax, -127, dtype=torch.int32)).clamp(-127, 127)
    codes = (g * ((127 - e) << 23).view(F32)).clamp(-448.0, 448.0).to(E4M3)
    return codes.flatten(-2), (e + 127).to(torch.uint8).squeeze(-1).view(E8M0)


def _sandwich_outputs(c, s):
    out = {"s": s["s"]}
    if c["pre"]:
        out["y"] = s["y"]
    if c["q"] == "fp8":
        out["codes"], out["scales"] = s["q"].view(E4M3), s["q_s"]
    elif c["q"] == "mxfp4":
        out["codes"], out["scales"] = s["q"].view(E4M3), s["q_s"][:, :c["H"] // 32].view(E8M0)
    if c["train"]:
        for k in ("rstd", "post_rstd", "dx", "d_res", "dw", "dwp", "d_gate"):
            if s[k] is not None:
                out[k] = s[k]
    return out


def _inverse_rms(v, eps):
    # in 64 bits: what is rounded to codes afterwards hangs on the last bit
    return torch.rsqrt(v.double().square().mean(1, keepdim=True) + eps).float()


def _sandwich_plain(c, s):
    x, res = s["x"].float(), s["res"].float()
    r = dict.fromkeys(("rstd", "post_rstd", "dw", "dwp", "d_gate"))
    p = x
    if c["post"]:
        r1 = _inverse_rms(x, POST_EPS)
        wp = s["wp"].float()
        p = x * r1 * wp
        r["post_rstd"] = r1[:, 0]
    f = c["branch_scale"]
    if s["gate"] is not None:
        gate = s["gate"].float()
        act = {"none": gate, "sigmoid": torch.sigmoid(gate), "tanh": torch.tanh(gate)}[c["act"]]
        f = act * f
    st = (res * c["res_scale"] + p * f).to(BF16)
    r["s"] = st
    xs = st.float()      # the stream as it is stored is what is normed
    if c["pre"]:
        r2 = _inverse_rms(xs, EPS)
        w = s["w"].float()
        xs = xs * r2
        y = (xs * w).to(BF16)
        r["y"], r["rstd"] = y, r2[:, 0]
        if c["q"] != "bf16":
            codes, scales = _quantise(y.float(), c["q"])
            return {"s": st, "y": y, "codes": codes, "scales": scales}
    if c["train"]:
        ds = s["d_s"].float()
        if c["pre"]:
            dy = s["dy"].float()
            g = dy * w
            ds = ds + r2 * (g - xs * (g * xs).mean(1, keepdim=True))
            r["dw"] = (dy * xs).double().sum(0).float()
        r["d_res"] = (ds * c["res_scale"]).to(BF16)
        dp = ds * f
        if s["gate"] is not None:
            dg = ds * p * c["branch_scale"]
            dg = {"none": dg, "sigmoid": dg * (act * (1.0 - act)), "tanh": dg * (1.0 - act * act)}[c["act"]]
            if c["gate"] == "row":
                dg = dg.double().sum(1, keepdim=True).to(s["gate"].dtype)
            elif c["gate"] == "channel":
                dg = dg.double().sum(0).float()
            r["d_gate"] = dg.to(s["d_gate"].dtype)
        if c["post"]:
            xh, g = x * r1, dp * wp
            r["dwp"] = (dp * xh).double().sum(0).float()
            dp = r1 * (g - xh * (g * xh).mean(1, keepdim=True))
        r["dx"] = dp.to(BF16)
    return _sandwich_outputs(c, r)


def _sandwich_own(c, s):
    import combine_moe_dispatch_02_amd as moe
    gate = dict(gate=s["gate"], gate_act=c["act"], res_scale=c["res_scale"], branch_scale=c["branch_scale"])
    moe.moe_sandwich_norm(s["x"], s["res"], s["w"], EPS, s["s"], s["y"], post_weight=s["wp"], post_eps=POST_EPS, **gate,
                          rstd=s["rstd"], post_rstd=s["post_rstd"], q=s["q"], q_s=s["q_s"], dtype=c["q"])
    if c["train"]:
        moe.moe_sandwich_norm_backward(s["dy"], s["d_s"], s["x"], s["s"], s["w"], s["rstd"], s["dx"], s["d_res"], s["dw"], s["ws"],
                                       post_weight=s["wp"], post_rstd=s["post_rstd"], **gate, d_post_weight=s["dwp"], d_gate=s["d_gate"])
    return _sandwich_outputs(c, s)


def _mine(c, s):
    """[T, n * R]: whether a place of the adapters' ranks, side by side, is one of the row's own adapter."""
    of = s["ids"].unsqueeze(1) == torch.arange(c["n"], device="cuda")
    on = of.unsqueeze(2).expand(-1, -1, c["R"])
    if s["ranks"] is not None:
        on = on & (torch.arange(c["R"], device="cuda") < s["ranks"].unsqueeze(1))
    return on.flatten(1)


def _adapter_plain(c, s):
    T, K, N, R, n = c["T"], c["K"], c["N"], c["R"], c["n"]
    base = 0.0 if s["base"] is None else s["base"].float()
    if T * R * (K + N) <= 1 << 26 and not c["train"]:
        # few rows: each row's own factors
        at = s["ids"].clamp(min=0).long()
        on = (s["ids"] >= 0).unsqueeze(1)
        if s["ranks"] is not None:
            on = on & (torch.arange(R, device="cuda") < s["ranks"][at].unsqueeze(1))
        v = torch.where(on, torch.bmm(s["a"][at].float(), s["x"].float().unsqueeze(2)).squeeze(2), 0.0)
        d = torch.bmm(s["b"][at].float(), (v * s["scale"][at].unsqueeze(1)).unsqueeze(2)).squeeze(2)
        return {"out": (base + d).to(BF16)}
    # all adapters side by side, a row's own places kept
    on, scale = _mine(c, s), s["scale"].repeat_interleave(R)
    a = s["a"].float().view(n * R, K)
    b = s["b"].float().transpose(0, 1).reshape(N, n * R) * scale
    x = s["x"].float()
    v = torch.where(on, x @ a.t(), 0.0)
    out = {"out": (base + v @ b.t()).to(BF16)}
    if c["train"]:
        dout = s["dout"].float()
        dv = torch.where(on, dout @ b, 0.0)
        out["dx"] = (s["dx_base"].float() + dv @ a).to(BF16)
        out["da"] = (dv.t() @ x).view(n, R, K)
        out["db"] = ((dout.t() @ v) * scale).view(N, n, R).transpose(0, 1).contiguous()
    return out


def _adapter_own(c, s):
    import combine_moe_dispatch_02_amd as moe
    if c["plan"]:
        moe.moe_plan(s["ids"].view(-1, 1), s["plan"], s["plan_ws"])
    by = {"plan": s["plan"]} if s["plan"] is not None else {"ids": s["ids"]}
    moe.moe_adapter(s["x"], s["a"], s["b"], s["out"], s["ws"], base=s["base"], scale=s["scale"], ranks=s["ranks"], v=s.get("v"), **by)
    out = {"out": s["out"]}
    if c["train"]:
        moe.moe_adapter_backward(s["dout"], s["x"], s["v"], s["a"], s["b"], s["plan"], s["bws"], s["da"], s["db"], s["dx"],
                                 dx_base=s["dx_base"], scale=s["scale"], ranks=s["ranks"])
        out.update(dx=s["dx"], da=s["da"], db=s["db"])
    return out


def run(state):
    c = state["case"]
    if own:
        return {"sandwich": _sandwich_own, "adapter": _adapter_own}[c["op"]](c, state)
    return {"sandwich": _sandwich_plain, "adapter": _adapter_plain}[c["op"]](c, state)


# ---------------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------------
def work(case):
    c = case
    T = c["T"]
    if c["op"] == "sandwich":
        n, wb = T * c["H"], 2 if c["w"] == "bf16" else 4
        weights = wb * c["H"] * (c["pre"] + c["post"])
        gate = {"none": 0, "row": T, "channel": c["H"], "full": n}[c["gate"]] * (2 if c["gate_t"] == "bf16" else 4)
        b = 4 * n + 2 * n + (2 * n if c["pre"] else 0) + weights + gate
        b += n + 4 * T * _words(c["H"]) if c["q"] != "bf16" else 0
        f = n * (3 + (4 if c["post"] else 0) + (4 if c["pre"] else 0) + (3 if c["q"] != "bf16" else 0))
        if c["train"]:     # d_s, dy, x and the stream again; dx and d_res
            b += 2 * n + (4 * n if c["pre"] else 0) + (2 * n if c["post"] or gate else 0) + 4 * n + weights + 2 * gate
            b += 4 * c["H"] * (c["pre"] + c["post"]) + 8 * T * (c["pre"] + c["post"])
            f += n * (3 + (8 if c["pre"] else 0) + (8 if c["post"] else 0) + (3 if gate else 0))
        return {"bytes": b, "flops": f}
    K, N, n = c["K"], c["N"], c["n"]
    rows = T * (1.0 - c["none"])
    share = 1.0 if c["ranks"] == "full" else 0.625
    reached = n * (1.0 - (1.0 - 1.0 / n) ** (rows if c["ids"] == "mixed" else min(rows, 2 * n * (1.0 - c["none"])))) if n > 1 else 1.0
    factors = reached * c["R"] * share * (K + N)
    b = 2 * rows * K + 2 * T * N * (2 if c["base"] else 1) + 2 * factors + 4 * T
    f = 2 * rows * c["R"] * share * (K + N)
    if c["train"]:     # v; dout and x again, dx on top of the projection's own; the factors' gradients
        b += 8 * rows * c["R"] + 2 * rows * N + 2 * rows * K + 4 * T * K + 2 * factors + 4 * n * c["R"] * (K + N)
        f += 2 * f
    return {"bytes": b, "flops": f}


# ---------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------------
def _exact_sandwich(c, s):
    H = c["H"]
    x, res = s["x"].double(), s["res"].double()
    out = {}
    branch, r1 = x, None
    if c["post"]:
        r1 = 1.0 / torch.sqrt((x * x).sum(1) / H + POST_EPS)
        branch = x * r1[:, None] * s["wp"].double()
    z, slope = torch.ones(1, 1, dtype=F64, device="cuda"), None
    if s["gate"] is not None:
        z = s["gate"].double()
        if c["act"] == "sigmoid":
            z = 1.0 / (1.0 + torch.exp(-z))
            slope = z - z * z
        elif c["act"] == "tanh":
            u = torch.exp(-2.0 * z.abs())
            z, slope = torch.sign(z) * (1.0 - u) / (1.0 + u), 4.0 * u / (1.0 + u) ** 2
        else:
            slope = torch.ones_like(z)
    out["s"] = c["res_scale"] * res + c["branch_scale"] * z * branch
    # norm, codes and gradients are of the stream as it is stored: in 32 bits up to its rounding, as it is defined
    st = s["res"].float() * c["res_scale"] + _branch_f32(c, s) * _factor_f32(c, s)
    st = st.to(BF16).double()
    if c["pre"]:
        w = s["w"].double()
        r2 = 1.0 / torch.sqrt((st * st).sum(1) / H + EPS)
        out["y"] = st * r2[:, None] * w
        if c["q"] != "bf16":
            row = (st.float() * r2[:, None].float() * s["w"].float()).to(BF16).double().unflatten(1, (-1, _blocks(c["q"])))
            amax = row.abs().amax(2, keepdim=True)
            scale = amax / 448.0 if c["q"] == "fp8" else torch.exp2(torch.floor(torch.log2(amax)) - 8.0)
            scale = torch.where(amax > 0, scale, 1.0 if c["q"] == "fp8" else 2.0 ** -127)
            out["codes"], out["scales"] = (row / scale).clamp(-448.0, 448.0).flatten(1), scale.squeeze(2)
    if not c["train"]:
        return out
    if c["pre"]:
        out["rstd"] = r2
    if c["post"]:
        out["post_rstd"] = r1
    ds = s["d_s"].double()
    if c["pre"]:
        dy = s["dy"].double()
        ds = ds + dy * w * r2[:, None] - st * ((dy * w * st).sum(1) * r2 ** 3 / H)[:, None]
        out["dw"] = (dy * st * r2[:, None]).sum(0)
    out["d_res"] = c["res_scale"] * ds
    dbranch = c["branch_scale"] * z * ds
    out["dx"] = dbranch
    if c["post"]:
        g = dbranch * s["wp"].double()
        out["dx"] = g * r1[:, None] - x * ((g * x).sum(1) * r1 ** 3 / H)[:, None]
        out["dwp"] = (dbranch * x * r1[:, None]).sum(0)
    if s["gate"] is not None:
        dz = c["branch_scale"] * ds * branch * slope
        out["d_gate"] = dz.sum(1, keepdim=True) if c["gate"] == "row" else dz.sum(0) if c["gate"] == "channel" else dz
    return out


def _branch_f32(c, s):
    """The branch in 32 bits, its statistic in 64."""
    x = s["x"].float()
    if not c["post"]:
        return x
    rms = torch.sqrt((s["x"].double() ** 2).sum(1, keepdim=True) / c["H"] + POST_EPS)
    return x * (1.0 / rms).float() * s["wp"].float()


def _factor_f32(c, s):
    if s["gate"] is None:
        return c["branch_scale"]
    z = s["gate"].float()
    return (torch.sigmoid(z) if c["act"] == "sigmoid" else torch.tanh(z) if c["act"] == "tanh" else z) * c["branch_scale"]


def _exact_adapter(c, s):
    T, R = c["T"], c["R"]
    out = torch.zeros(T, c["N"], dtype=F64, device="cuda") if s["base"] is None else s["base"].double()
    ids = s["ids"].cpu()
    ranks = [R] * c["n"] if s["ranks"] is None else s["ranks"].tolist()
    if c["train"]:
        dx = s["dx_base"].double()
        da, db = torch.zeros(s["a"].shape, dtype=F64, device="cuda"), torch.zeros(s["b"].shape, dtype=F64, device="cuda")
    for i in range(c["n"]):
        t = torch.nonzero(ids == i).flatten().cuda()
        if not t.numel():
            continue
        k, f = ranks[i], float(s["scale"][i])
        a, b, x = s["a"][i, :k].double(), s["b"][i, :, :k].double(), s["x"][t].double()
        v = torch.mm(x, a.t())
        out[t] += f * torch.mm(v, b.t())
        if c["train"]:
            d = s["dout"][t].double()
            dv = f * torch.mm(d, b)
            dx[t] += torch.mm(dv, a)
            da[i, :k] = torch.mm(dv.t(), x)
            db[i, :, :k] = f * torch.mm(d.t(), v)
    return {"out": out, "dx": dx, "da": da, "db": db} if c["train"] else {"out": out}


def exact(case, seed):
    s = prepare(case, seed)
    return {"sandwich": _exact_sandwich, "adapter": _exact_adapter}[case["op"]](case, s)
