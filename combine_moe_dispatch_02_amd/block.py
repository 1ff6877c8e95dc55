"""Python binding of the operators around the MoE layer (include/moe355_block.h).

The residual's addition with the RMS norm and its 8-bit output, the router's choice of
experts, the dispatch of rows that are quantised already, and the expert FFN of a few
tokens. Argument marshalling only, as in ``layer``: the caller owns every tensor and the
calls are asynchronous. All tensors of a call are on one device, which need not be the
current one; ``stream`` defaults to that device's current stream.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass
from typing import Optional

import torch

from . import _abi
from ._abi import MOE_BF16, MOE_F32, MOE_FP8_E4M3_G128, MOE_MXFP4, check, load
from .layer import Plan, Workspace, _dtype_code, _need_cuda, _vp

__all__ = [
    "RouterConfig", "moe_rmsnorm", "moe_rmsnorm_backward", "rmsnorm_backward_workspace_bytes", "moe_router_topk",
    "moe_router_topk_backward", "moe_dispatch_quantized", "moe_expert_ffn_decode",
    "expert_ffn_decode_workspace_bytes", "quantized_scales",
]

_CODES = (torch.uint8, torch.float8_e4m3fn)


def _launch(name: str, tensors, stream, *args) -> None:
    """Call entry point ``name`` on the tensors' device, the stream as its last argument."""
    dev = None
    for t in tensors:
        if t is None:
            continue
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError(f"{name}: tensors are on {dev} and {t.device}")
    if stream is None:
        stream = torch.cuda.current_stream(dev)
    if isinstance(stream, torch.cuda.Stream):
        if stream.device != dev:
            raise ValueError(f"{name}: the stream is on {stream.device}, the tensors are on {dev}")
        stream = stream.cuda_stream
    fn = getattr(load(), name)
    if torch.cuda.current_device() == dev.index:
        status = fn(*args, ctypes.c_void_p(int(stream)))
    else:
        with torch.cuda.device(dev):
            status = fn(*args, ctypes.c_void_p(int(stream)))
    check(name, status)


def _shaped(t: torch.Tensor, name: str, shape, dtype) -> None:
    _need_cuda(t, name, dtype)
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _real_dtype(t: torch.Tensor, name: str) -> int:
    _need_cuda(t, name, (torch.bfloat16, torch.float32))
    return MOE_F32 if t.dtype == torch.float32 else MOE_BF16


def _scale_words(q_s: torch.Tensor, name: str, T: int, H: int, code: int) -> None:
    """Row-major scale words: fp32 [T, ceil(H/128)] (fp8) or bytes [T, 4 ceil(H/128)] (mxfp4)."""
    words = (H + 127) // 128
    if code == MOE_FP8_E4M3_G128:
        _shaped(q_s, name, (T, words), torch.float32)
    else:
        _shaped(q_s, name, (T, 4 * words), torch.uint8)


def quantized_scales(T: int, H: int, dtype, device="cuda") -> torch.Tensor:
    """An uninitialised scale tensor for quantised rows [T, H] of format ``dtype``."""
    words = (H + 127) // 128
    if _dtype_code(dtype) == MOE_FP8_E4M3_G128:
        return torch.empty(T, words, dtype=torch.float32, device=device)
    return torch.empty(T, 4 * words, dtype=torch.uint8, device=device)


def moe_rmsnorm(x: torch.Tensor, weight: torch.Tensor, eps: float, y: Optional[torch.Tensor] = None, *,
                res: Optional[torch.Tensor] = None, res_out: Optional[torch.Tensor] = None,
                rstd: Optional[torch.Tensor] = None, q: Optional[torch.Tensor] = None,
                q_s: Optional[torch.Tensor] = None, dtype="bf16", stream=None) -> None:
    """y = rms_norm(s) * weight with s = x + res (s goes to ``res_out``), and its copy (q, q_s) in
    the activation format ``dtype`` ("fp8" or "mxfp4"); rstd for the backward pass. x, res, res_out, y:
    bf16 [T, H]; weight: bf16 or fp32 [H]; q: codes [T, H]; q_s: see quantized_scales()."""
    _need_cuda(x, "x", torch.bfloat16)
    if x.dim() != 2:
        raise ValueError("x must be [T, H]")
    T, H = x.shape
    code = _dtype_code(dtype)
    wcode = _real_dtype(weight, "weight")
    if weight.shape != (H,):
        raise ValueError("weight must be [H]")
    for t, n in ((res, "res"), (res_out, "res_out"), (y, "y")):
        if t is not None:
            _shaped(t, n, (T, H), torch.bfloat16)
    if rstd is not None:
        _shaped(rstd, "rstd", (T,), torch.float32)
    if q is not None:
        _shaped(q, "q", (T, H), _CODES)
    if q_s is not None:
        _scale_words(q_s, "q_s", T, H, code)
    _launch("moe_rmsnorm", (x, res, weight, res_out, y, rstd, q, q_s), stream,
            _vp(x), _vp(res), _vp(weight), wcode, T, H, float(eps), _vp(res_out), _vp(y), _vp(rstd), code, _vp(q),
            _vp(q_s))


def rmsnorm_backward_workspace_bytes(T: int, H: int) -> int:
    return int(load().moe_rmsnorm_backward_workspace_bytes(T, H))


def moe_rmsnorm_backward(dy: torch.Tensor, s: torch.Tensor, weight: torch.Tensor, rstd: torch.Tensor,
                         dx: torch.Tensor, dweight: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                         *, d_res: Optional[torch.Tensor] = None, stream=None) -> None:
    """Gradients of moe_rmsnorm: dx (of x and of res) with the stream's own gradient d_res added, and
    dweight fp32 [H] (written, not added to), for which ws is a byte tensor of
    rmsnorm_backward_workspace_bytes(T, H). s is res_out of the forward (x where there was no residual)."""
    _need_cuda(dy, "dy", torch.bfloat16)
    if dy.dim() != 2:
        raise ValueError("dy must be [T, H]")
    T, H = dy.shape
    wcode = _real_dtype(weight, "weight")
    if weight.shape != (H,):
        raise ValueError("weight must be [H]")
    for t, n in ((s, "s"), (dx, "dx"), (d_res, "d_res")):
        if t is not None:
            _shaped(t, n, (T, H), torch.bfloat16)
    _shaped(rstd, "rstd", (T,), torch.float32)
    if dweight is not None:
        _shaped(dweight, "dweight", (H,), torch.float32)
    if ws is not None:
        _need_cuda(ws, "ws", torch.uint8)
    _launch("moe_rmsnorm_backward", (dy, s, weight, rstd, d_res, dx, dweight, ws), stream,
            _vp(dy), _vp(s), _vp(weight), wcode, _vp(rstd), _vp(d_res), T, H, _vp(dx), _vp(dweight), _vp(ws),
            0 if ws is None else ws.numel())


@dataclass(frozen=True)
class RouterConfig:
    """How experts are scored and chosen (moe_router_config)."""

    score: str = "softmax"     # or "sigmoid"
    normalize: bool = True     # weights divided by their sum over the chosen
    groups: int = 1            # groups of neighbouring experts
    topk_groups: int = 1       # groups a token may choose from
    group_top: int = 1         # a group counts as the sum of its 1 or 2 largest keys
    scale: float = 1.0         # factor of the weights

    def c(self) -> _abi.RouterConfigT:
        got = self.__dict__.get("_c")
        if got is None:
            if self.score not in ("softmax", "sigmoid"):
                raise ValueError(f"score {self.score!r}")
            got = _abi.RouterConfigT(
                _abi.MOE_SCORE_SOFTMAX if self.score == "softmax" else _abi.MOE_SCORE_SIGMOID, int(self.normalize),
                self.groups, self.topk_groups, self.group_top, self.scale)
            object.__setattr__(self, "_c", got)
        return got


def moe_router_topk(logits: torch.Tensor, topk_idx: torch.Tensor, topk_weights: torch.Tensor,
                    cfg: RouterConfig = RouterConfig(), *, bias: Optional[torch.Tensor] = None, stream=None) -> None:
    """topk_idx int32 [T, K] and topk_weights fp32 [T, K] of the experts chosen by logits [T, E]
    (fp32 or bf16) and, in the choice alone, bias fp32 [E]. -1 with weight 0 where a token's
    experts are used up (logits of -inf or NaN switch an expert off)."""
    lcode = _real_dtype(logits, "logits")
    if logits.dim() != 2 or topk_idx.dim() != 2:
        raise ValueError("logits must be [T, E], topk_idx [T, K]")
    (T, E), K = logits.shape, topk_idx.shape[1]
    _shaped(topk_idx, "topk_idx", (T, K), torch.int32)
    _shaped(topk_weights, "topk_weights", (T, K), torch.float32)
    if bias is not None:
        _shaped(bias, "bias", (E,), torch.float32)
    _launch("moe_router_topk", (logits, bias, topk_idx, topk_weights), stream,
            _vp(logits), lcode, _vp(bias), T, E, K, ctypes.byref(cfg.c()), _vp(topk_idx), _vp(topk_weights))


def moe_router_topk_backward(d_topk_weights: torch.Tensor, logits: torch.Tensor, topk_idx: torch.Tensor,
                             d_logits: torch.Tensor, cfg: RouterConfig = RouterConfig(), *, stream=None) -> None:
    """d_logits [T, E] (in logits' type, every element) from d_topk_weights fp32 [T, K], e.g.
    moe_combine_backward's, for the topk_idx that moe_router_topk wrote with the same cfg."""
    lcode = _real_dtype(logits, "logits")
    if logits.dim() != 2 or topk_idx.dim() != 2:
        raise ValueError("logits must be [T, E], topk_idx [T, K]")
    (T, E), K = logits.shape, topk_idx.shape[1]
    _shaped(topk_idx, "topk_idx", (T, K), torch.int32)
    _shaped(d_topk_weights, "d_topk_weights", (T, K), torch.float32)
    _shaped(d_logits, "d_logits", (T, E), logits.dtype)
    _launch("moe_router_topk_backward", (d_topk_weights, logits, topk_idx, d_logits), stream,
            _vp(d_topk_weights), _vp(logits), lcode, _vp(topk_idx), T, E, K, ctypes.byref(cfg.c()), _vp(d_logits))


def moe_dispatch_quantized(q: torch.Tensor, q_s: torch.Tensor, plan: Plan, pool: torch.Tensor, pool_s: torch.Tensor,
                           epoch: int, ws: Workspace, dtype, stream=None) -> None:
    """moe_dispatch of rows that are codes [T, H] with row-major scales (quantized_scales()) already."""
    code = _dtype_code(dtype)
    if q.dim() != 2 or pool.dim() != 2:
        raise ValueError("q must be [T, H], pool [pool rows, H]")
    H = q.shape[1]
    _shaped(q, "q", (plan.T, H), _CODES)
    if code != MOE_BF16:
        _scale_words(q_s, "q_s", plan.T, H, code)
    _shaped(pool, "pool", (pool.shape[0], H), _CODES)
    _need_cuda(pool_s, "pool_s", (torch.float32, torch.uint8))
    if pool_s.numel() * pool_s.element_size() < pool.shape[0] * ((H + 127) // 128) * 4:
        raise ValueError("pool_s holds fewer scale words than the pool has")
    c = plan.c()
    _launch("moe_dispatch_quantized", (q, q_s, plan.pos, pool, pool_s, ws.buf), stream,
            _vp(q), _vp(q_s), H, code, ctypes.byref(c), pool.shape[0], _vp(pool), _vp(pool_s), epoch, _vp(ws.buf),
            ws.nbytes)


def expert_ffn_decode_workspace_bytes(T: int, K: int, I: int) -> int:
    return int(load().moe_expert_ffn_decode_workspace_bytes(T, K, I))


def moe_expert_ffn_decode(x: torch.Tensor, x_s: Optional[torch.Tensor], topk_idx: torch.Tensor,
                          topk_weights: torch.Tensor, w1: torch.Tensor, w1_s: torch.Tensor, w2: torch.Tensor,
                          w2_s: torch.Tensor, ws: torch.Tensor, out: torch.Tensor, expert_begin: int = 0,
                          stream=None) -> None:
    """out [T, H] of up to 64 tokens through the MXFP4 experts, without plan or pool. x: MXFP8 codes
    [T, H] with x_s (moe_rmsnorm's q and q_s), or bf16 with x_s None. Weights and scales as
    moe_pack_weights and moe_pack_mx_scales give them: w1 [E_local, 2I, H/2], w2 [E_local, H, I/2].
    ws: a byte tensor of expert_ffn_decode_workspace_bytes(T, K, I)."""
    if x.dim() != 2 or w1.dim() != 3 or topk_idx.dim() != 2:
        raise ValueError("x must be [T, H], w1 [E_local, 2I, H/2], topk_idx [T, K]")
    (T, H), K = x.shape, topk_idx.shape[1]
    E, I = w1.shape[0], w1.shape[1] // 2
    if x_s is None:
        _need_cuda(x, "x", torch.bfloat16)
    else:
        _need_cuda(x, "x", _CODES)
        _scale_words(x_s, "x_s", T, H, MOE_MXFP4)
    _shaped(topk_idx, "topk_idx", (T, K), torch.int32)
    _shaped(topk_weights, "topk_weights", (T, K), torch.float32)
    _shaped(w1, "w1", (E, 2 * I, H // 2), torch.uint8)
    _shaped(w1_s, "w1_s", (E, 2 * I, H // 32), torch.uint8)
    _shaped(w2, "w2", (E, H, I // 2), torch.uint8)
    _shaped(w2_s, "w2_s", (E, H, I // 32), torch.uint8)
    _shaped(out, "out", (T, H), torch.bfloat16)
    _need_cuda(ws, "ws", torch.uint8)
    _launch("moe_expert_ffn_decode", (x, x_s, topk_idx, topk_weights, w1, w1_s, w2, w2_s, ws, out), stream,
            _vp(x), _vp(x_s), MOE_BF16 if x_s is None else MOE_MXFP4, T, H, I, K, expert_begin, E, _vp(topk_idx),
            _vp(topk_weights), _vp(w1), _vp(w1_s), _vp(w2), _vp(w2_s), _vp(ws), ws.numel(), _vp(out))
