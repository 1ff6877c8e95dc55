"""The expert FFN of a few tokens with MXFP4 weights on the GPU against the float64 oracle.

Tolerance, of the largest value: bf16's half step 2^-8 on out, and what a value of h near a rounding
border of MXFP8 does when fp32 and float64 put it on different sides: one e4m3 step, at most 2^-3 of that
h, one in I >= 128 of a sum. 3e-2, the layer's own mxfp4 bound, holds both."""
import numpy as np
import pytest
import torch

import combine_moe_dispatch_02_amd as moe
import oracle
from oracle import block as ob
from synth import MoEConfig, make_inputs

from _gpu import TOL, make_layer, say

pytestmark = pytest.mark.gpu


class Case:
    def __init__(self, T, H, I, E, K, seed=0, E_local=None, begin=0):
        E_local = E_local or E
        g = torch.Generator().manual_seed(seed + 31 * T + H + I)
        r = lambda *s: torch.randint(0, 256, s, generator=g, dtype=torch.uint8)  # noqa: E731
        near = lambda n, *s: torch.randint(n, n + 3, s, generator=g, dtype=torch.uint8)  # noqa: E731
        self.T, self.H, self.I, self.K, self.begin = T, H, I, K, begin
        self.w1, self.w1_s = r(E_local, 2 * I, H // 2), near(127 - int(np.log2(H) / 2 + 2), E_local, 2 * I, H // 32)
        self.w2, self.w2_s = r(E_local, H, I // 2), near(127 - int(np.log2(I) / 2 + 2), E_local, H, I // 32)
        self.x = torch.randn(T, H, generator=g).to(torch.bfloat16)
        self.idx = torch.randn(T, E, generator=g).topk(min(K, E), dim=1)[1].to(torch.int32)
        self.weights = torch.softmax(torch.randn(T, K, generator=g), 1)

    def ref(self, rows=None, quantised=None):
        rows = np.arange(self.T) if rows is None else rows
        x, xs = quantised if quantised is not None else (self.x.float().numpy(), None)
        return ob.expert_ffn_decode(x[rows], None if xs is None else xs[rows], self.idx.numpy()[rows],
                                    self.weights.numpy()[rows], *(t.numpy() for t in (self.w1, self.w1_s, self.w2, self.w2_s)),
                                    expert_begin=self.begin)

    def packed(self):
        if not hasattr(self, "_p"):
            self._p = (moe.moe_pack_weights(self.w1.cuda(), "mxfp4"), moe.moe_pack_mx_scales(self.w1_s.cuda()),
                       moe.moe_pack_weights(self.w2.cuda(), "mxfp4"), moe.moe_pack_mx_scales(self.w2_s.cuda()))
        return self._p

    def run(self, quantised=None, fill=0, rows=None):
        T = rows or self.T
        ws = torch.full((moe.expert_ffn_decode_workspace_bytes(T, self.K, self.I),), fill, dtype=torch.uint8, device="cuda")
        out = torch.full((T + 1, self.H), 7.0, dtype=torch.bfloat16, device="cuda")
        x, xs = (self.x.cuda(), None) if quantised is None else (torch.from_numpy(q).cuda() for q in quantised)
        moe.moe_expert_ffn_decode(x[:T], None if xs is None else xs[:T], self.idx[:T].cuda(), self.weights[:T].cuda(),
                                  *self.packed(), ws, out[:T], expert_begin=self.begin)
        torch.cuda.synchronize()
        assert bool((out[T] == 7.0).all())
        return out[:T]

    def quantised(self):
        return ob.quantize_rows(self.x.float().numpy(), "mxfp4")


def close(got, ref):
    return oracle.max_norm_rel_err(oracle.bf16_to_f64(got.cpu()), ref) <= TOL["mxfp4"]


SHAPES = [(1, 128, 128, 4, 1), (1, 256, 128, 8, 8), (1, 1152, 384, 6, 3), (2, 4096, 128, 5, 2), (3, 128, 1536, 7, 4),
          (15, 640, 256, 9, 3), (16, 256, 640, 6, 6), (17, 384, 128, 6, 2), (32, 256, 256, 12, 4), (33, 128, 128, 40, 7),
          (48, 512, 128, 3, 1), (63, 256, 384, 16, 16), (64, 256, 128, 64, 16), (64, 128, 256, 1, 1)]


@pytest.mark.parametrize("T,H,I,E,K", SHAPES)
def test_matches_oracle(T, H, I, E, K):
    say("decode", T, H, I, E, K)
    c = Case(T, H, I, E, K)
    got = c.run()
    assert close(got, c.ref())
    # rows that are quantised already are the same rows; the workspace's content does not matter
    again = c.run(c.quantised(), fill=255)
    assert torch.equal(got.view(torch.int16), again.view(torch.int16))


@pytest.mark.parametrize("T", [1, 5, 16, 40, 64])
def test_one_rank_of_many(T):
    """Ids of other ranks, -1 and nonsense ids add nothing; tokens without a local pair get zeros."""
    say("decode share", T)
    c = Case(T, 256, 128, 24, 4, seed=3, E_local=8, begin=8)
    c.idx[T // 2] = torch.tensor([0, -1, 23, 7])
    if T > 1:
        c.idx[0] = torch.tensor([8, 15, 2**31 - 1, -2**31])
    got, ref = c.run(), c.ref()
    assert close(got, ref)
    none = (ref == 0).all(1)
    assert none[T // 2] and bool((got[torch.from_numpy(none).cuda()] == 0).all())


@pytest.mark.parametrize("T", [1, 13, 64])
def test_nothing_local(T):
    say("decode nothing local", T)
    c = Case(T, 256, 128, 4, 2)
    c.begin = 100
    assert bool((c.run() == 0).all())


def test_every_token_to_the_same_experts_and_doubled_ids():
    say("decode crowded")
    c = Case(64, 256, 128, 6, 4, seed=5)
    c.idx[:] = torch.tensor([5, 2, 5, 5])        # an expert three times in a token: three pairs
    got = c.run()
    assert close(got, c.ref())
    c = Case(20, 128, 256, 6, 3, seed=6)
    c.idx[:, 1] = c.idx[:, 0]
    assert close(c.run(c.quantised()), c.ref())


@pytest.mark.parametrize("E", [2, 40])
@pytest.mark.parametrize("n", [7, 8, 9, 15, 16, 17, 24, 25, 31, 32, 33, 40, 41, 48, 49, 63, 64])
def test_an_expert_of_n_tokens(n, E):
    """n tokens for one expert next to one that all 64 reach: every count of column groups, whole and partly
    filled, where the experts are few and where they are many. The n tokens are spread over the batch."""
    say("decode expert of n tokens", n, E)
    c = Case(64, 384, 640, E, 2, seed=8)
    c.idx[:, 0], c.idx[:, 1] = E - 1, -1
    c.idx[torch.randperm(64, generator=torch.Generator().manual_seed(n))[:n], 1] = 0
    assert close(c.run(), c.ref())


@pytest.mark.parametrize("T,H,I,E", [(64, 512, 128, 8), (10, 1792, 128, 30), (64, 4096, 128, 16), (5, 7168, 256, 4)])
def test_no_code_of_h_is_off(T, H, I, E):
    """One expert a token with weight 1: a token's row is W2 h of one h, and a code of h beside its own puts 1/16 or
    more of that h into it, 1e-2 of the row's norm at I = 128 for one of average size. Row by row: bf16's half step 2^-8
    of each value, and 2e-4 of the sums of I magnitudes, sqrt(I) times the result: 2e-4 * 16."""
    say("decode codes of h", T, H, I)
    c = Case(T, H, I, E, 1, seed=12)
    c.weights[:] = 1.0
    got, ref = oracle.bf16_to_f64(c.run().cpu()), c.ref()
    off = np.linalg.norm(got - ref, axis=1) / np.linalg.norm(ref, axis=1)
    assert off.max() <= 2.0 ** -8 + 2e-4 * 16


def test_scales_of_all_sizes_and_nan():
    """Weight and activation scales over many powers of two (no product past fp32's range), zero blocks, and a NaN scale."""
    say("decode scales")
    c = Case(6, 256, 128, 4, 2, seed=13)
    g = torch.Generator().manual_seed(1)
    c.w1_s = torch.randint(90, 150, c.w1_s.shape, generator=g, dtype=torch.uint8)
    c.x = (torch.randn(6, 256, generator=g) * torch.exp2(torch.randint(-40, 5, (6, 8), generator=g).float()).repeat_interleave(32, 1)).bfloat16()
    c.x[0, 32:64] = 0
    c.w1_s[0, :, 0] = 0
    assert close(c.run(), c.ref())
    codes, scales = c.quantised()
    scales = scales.copy()
    scales[3, 1] = 255
    got = c.run((codes, scales)).float().cpu()
    assert bool(got[3].isnan().all()) and bool(got[[0, 1, 2, 4, 5]].isfinite().all())


def test_1024_experts():
    say("decode 1024 experts")
    c = Case(64, 128, 128, 1024, 16, seed=7)
    assert close(c.run(), c.ref())
    c.idx[0, 0], c.idx[0, 1] = 1023, 0
    assert close(c.run(rows=1), c.ref(rows=np.array([0])))


def test_tokens_do_not_depend_on_each_other():
    """A token's output is the same alone and in a batch (within the rounding of another order),
    and one token's NaN stays its own: also where another shares its experts."""
    say("decode independence")
    c = Case(24, 512, 256, 8, 2, seed=8)
    whole = c.run().float()
    one = c.run(rows=1).float()
    assert (whole[0] - one[0]).abs().max() <= 2.0 ** -7 * one.abs().max()
    c.x[3, 77] = float("nan")
    c.x[4, 5] = float("inf")
    got = c.run()
    assert bool(got[3].isnan().all()) and bool(got[4].isnan().all())
    rest = [t for t in range(24) if t not in (3, 4)]
    assert torch.equal(got[rest].float(), whole[rest])


def test_an_experts_nan_reaches_its_tokens_alone():
    say("decode NaN expert")
    c = Case(20, 256, 128, 6, 2, seed=9)
    c.w2_s[3] = 255                              # E8M0 NaN
    got = c.run().float()
    hit = (c.idx == 3).any(1)
    assert hit.any() and not hit.all()
    assert bool(got[hit.cuda()].isnan().all()) and not bool(got[~hit.cuda()].isnan().any())


def test_zero_rows_and_zero_weights():
    say("decode zeros")
    c = Case(6, 256, 128, 5, 2, seed=10)
    c.x[2] = 0
    c.weights[4] = 0
    got = c.run()
    assert bool((got[2] == 0).all()) and bool((got[4] == 0).all()) and close(got, c.ref())


def test_repeats_bit_for_bit():
    say("decode repeats")
    for T in (1, 9, 64):
        c = Case(T, 2048, 512, 24, 8, seed=11)
        first = c.run()
        for i in range(3):
            assert torch.equal(c.run(fill=i).view(torch.int16), first.view(torch.int16))


@pytest.mark.parametrize("T", [1, 7, 48])
def test_layer_decode_matches_forward(T):
    """StreamMoE.decode on the layer's prepared weights against its pooled forward."""
    say("layer decode", T)
    cfg = MoEConfig("dec", 48, 512, 256, 12, 2, 8, 4, 128, "mxfp4")
    inp = make_inputs(cfg, 17)
    layer = make_layer(cfg)
    w = layer.prepare_weights(*(t.view(torch.uint8).cuda() for t in (inp.w1, inp.w2, inp.w1_scale, inp.w2_scale)))
    x, idx, tw = inp.x.cuda(), inp.topk_idx.cuda(), inp.topk_weights.cuda()
    ref = layer.forward(x, idx, tw, *w).clone()
    got = layer.decode(x[:T], idx[:T], tw[:T], *w)
    torch.cuda.synchronize()
    layer.check_errors()
    assert got.data_ptr() == layer.out.data_ptr() and got.shape == (T, 512)
    assert oracle.max_norm_rel_err(oracle.bf16_to_f64(got.cpu()), oracle.bf16_to_f64(ref[:T].cpu())) <= TOL["mxfp4"]
    orc = oracle.moe_layer(inp, tokens=list(range(T))).out
    assert oracle.max_norm_rel_err(oracle.bf16_to_f64(got.cpu()), orc) <= TOL["mxfp4"]


def test_refusals():
    say("decode refusals")
    c = Case(4, 256, 128, 4, 2)
    w = c.packed()
    x, idx, tw = c.x.cuda(), c.idx.cuda(), c.weights.cuda()
    ws = torch.empty(moe.expert_ffn_decode_workspace_bytes(4, 2, 128), dtype=torch.uint8, device="cuda")
    out = torch.empty(4, 256, dtype=torch.bfloat16, device="cuda")
    for bad in ((x, None, idx.long(), tw, *w, ws, out), (x, None, idx, tw[:2], *w, ws, out), (x, None, idx, tw, *w, ws, out[:3]),
                (x[:, :128].contiguous(), None, idx, tw, *w, ws, out), (x, x, idx, tw, *w, ws, out),
                (x, None, idx, tw, w[0], w[1], w[0], w[3], ws, out), (x.float(), None, idx, tw, *w, ws, out)):
        with pytest.raises(ValueError):
            moe.moe_expert_ffn_decode(*bad)
    with pytest.raises(moe.MoeError):
        moe.moe_expert_ffn_decode(x, None, idx, tw, *w, ws[:16], out)
    layer = moe.StreamMoE(8, 512, 256, 2, 4, dtype="bf16")
    with pytest.raises(moe.MoeError):
        layer.decode(x, idx, tw, *w)
    layer = moe.StreamMoE(2, 512, 256, 2, 4, dtype="mxfp4")
    with pytest.raises(ValueError):
        layer.decode(torch.zeros(4, 512, dtype=torch.bfloat16, device="cuda"), idx, tw, *w)
