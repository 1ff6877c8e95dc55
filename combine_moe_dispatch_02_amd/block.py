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
from ._abi import MOE_BF16, MOE_F32, MOE_FP8_E4M3_G128, MOE_MXFP4, MoeError, check, load
from .layer import Plan, Workspace, _dtype_code, _need_cuda

__all__ = [
    "RouterConfig", "moe_rmsnorm", "moe_rmsnorm_backward", "rmsnorm_backward_workspace_bytes", "moe_router_topk",
    "moe_router_topk_backward", "moe_dispatch_quantized", "moe_expert_ffn_decode",
    "expert_ffn_decode_workspace_bytes", "quantized_scales",
]

_CODES = (torch.uint8, torch.float8_e4m3fn)
_BF16, _F32, _I32, _U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


def _device(t: torch.Tensor, name: str) -> int:
    """The device index of a call's first tensor."""
    d = t.get_device()
    if d < 0:
        raise ValueError(f"{name} must be a device tensor")
    return d


def _ptr(t: Optional[torch.Tensor], name: str, dev: int, shape, dtype) -> Optional[int]:
    """The address of a checked tensor (None for None): on device ``dev``, dense, of shape and dtype
    (a dtype or a tuple of them). One line of cheap tests, since a token's call is all launch."""
    if t is None:
        return None
    if (t.get_device() == dev and t.is_contiguous() and t.shape == shape
            and (t.dtype is dtype or (dtype.__class__ is tuple and t.dtype in dtype))):
        return t.data_ptr()
    _need_cuda(t, name, dtype)
    if t.get_device() != dev:
        raise ValueError(f"{name} is on device {t.get_device()}, the call's first tensor on {dev}")
    raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _bytes(t: Optional[torch.Tensor], name: str, dev: int):
    """(address, bytes) of a workspace; (None, 0) for None."""
    return (None, 0) if t is None else (_ptr(t, name, dev, t.shape, _U8), t.numel())


def _i32(*sizes: int) -> None:
    """Sizes and offsets that the C ABI takes as int32; a larger one would arrive as another number."""
    if max(sizes) > 0x7FFFFFFF:
        raise ValueError(f"a size of {max(sizes)} is past 2^31 - 1")


def _launch(name: str, dev: int, stream, *args) -> None:
    """Call entry point ``name`` on device ``dev``, the stream as its last argument."""
    if stream is None:
        stream = torch._C._cuda_getCurrentRawStream(dev)
    elif isinstance(stream, torch.cuda.Stream):
        if stream.device.index != dev:
            raise ValueError(f"{name}: the stream is on {stream.device}, the tensors are on device {dev}")
        stream = stream.cuda_stream
    fn = getattr(load(), name)
    if torch._C._cuda_getDevice() == dev:
        status = fn(*args, stream)
    else:
        with torch.cuda.device(dev):
            status = fn(*args, stream)
    if status:
        check(name, status)


def _real_dtype(t: torch.Tensor, name: str) -> int:
    if t.dtype is _F32:
        return MOE_F32
    if t.dtype is _BF16:
        return MOE_BF16
    raise ValueError(f"{name} has dtype {t.dtype}, expected bf16 or fp32")


def _scales(q_s: Optional[torch.Tensor], name: str, dev: int, T: int, H: int, code: int) -> Optional[int]:
    """Row-major scale words: fp32 [T, ceil(H/128)] (fp8) or bytes [T, 4 ceil(H/128)] (mxfp4)."""
    words = (H + 127) // 128
    if code == MOE_FP8_E4M3_G128:
        return _ptr(q_s, name, dev, (T, words), _F32)
    return _ptr(q_s, name, dev, (T, 4 * words), _U8)


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
    dev = _device(x, "x")
    if x.dim() != 2:
        raise ValueError("x must be [T, H]")
    shape = x.shape
    T, H = shape
    _i32(T, H)
    code = MOE_BF16 if dtype == "bf16" else _dtype_code(dtype)
    wcode = _real_dtype(weight, "weight")
    _launch("moe_rmsnorm", dev, stream,
            _ptr(x, "x", dev, shape, _BF16), _ptr(res, "res", dev, shape, _BF16),
            _ptr(weight, "weight", dev, (H,), weight.dtype), wcode, T, H, eps,
            _ptr(res_out, "res_out", dev, shape, _BF16), _ptr(y, "y", dev, shape, _BF16),
            _ptr(rstd, "rstd", dev, (T,), _F32), code, _ptr(q, "q", dev, shape, _CODES),
            _scales(q_s, "q_s", dev, T, H, code))


def rmsnorm_backward_workspace_bytes(T: int, H: int) -> int:
    _i32(T, H)
    return int(load().moe_rmsnorm_backward_workspace_bytes(T, H))


def moe_rmsnorm_backward(dy: torch.Tensor, s: torch.Tensor, weight: torch.Tensor, rstd: torch.Tensor,
                         dx: torch.Tensor, dweight: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                         *, d_res: Optional[torch.Tensor] = None, stream=None) -> None:
    """Gradients of moe_rmsnorm: dx (of x and of res) with the stream's own gradient d_res added, and
    dweight fp32 [H] (written, not added to), for which ws is a byte tensor of
    rmsnorm_backward_workspace_bytes(T, H). s is res_out of the forward (x where there was no residual)."""
    dev = _device(dy, "dy")
    if dy.dim() != 2:
        raise ValueError("dy must be [T, H]")
    shape = dy.shape
    T, H = shape
    _i32(T, H)
    wcode = _real_dtype(weight, "weight")
    ws_ptr, ws_bytes = _bytes(ws, "ws", dev)
    _launch("moe_rmsnorm_backward", dev, stream,
            _ptr(dy, "dy", dev, shape, _BF16), _ptr(s, "s", dev, shape, _BF16),
            _ptr(weight, "weight", dev, (H,), weight.dtype), wcode, _ptr(rstd, "rstd", dev, (T,), _F32),
            _ptr(d_res, "d_res", dev, shape, _BF16), T, H, _ptr(dx, "dx", dev, shape, _BF16),
            _ptr(dweight, "dweight", dev, (H,), _F32), ws_ptr, ws_bytes)


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
        """The C struct, made once (the fields cannot change)."""
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
    dev = _device(logits, "logits")
    lcode = _real_dtype(logits, "logits")
    if logits.dim() != 2 or topk_idx.dim() != 2:
        raise ValueError("logits must be [T, E], topk_idx [T, K]")
    (T, E), K = logits.shape, topk_idx.shape[1]
    _i32(T, E, K)
    _launch("moe_router_topk", dev, stream,
            _ptr(logits, "logits", dev, logits.shape, logits.dtype), lcode, _ptr(bias, "bias", dev, (E,), _F32), T, E, K,
            cfg.c(), _ptr(topk_idx, "topk_idx", dev, (T, K), _I32), _ptr(topk_weights, "topk_weights", dev, (T, K), _F32))


def moe_router_topk_backward(d_topk_weights: torch.Tensor, logits: torch.Tensor, topk_idx: torch.Tensor,
                             d_logits: torch.Tensor, cfg: RouterConfig = RouterConfig(), *, stream=None) -> None:
    """d_logits [T, E] (in logits' type, every element) from d_topk_weights fp32 [T, K], e.g.
    moe_combine_backward's, for the topk_idx that moe_router_topk wrote with the same cfg."""
    dev = _device(logits, "logits")
    lcode = _real_dtype(logits, "logits")
    if logits.dim() != 2 or topk_idx.dim() != 2:
        raise ValueError("logits must be [T, E], topk_idx [T, K]")
    (T, E), K = logits.shape, topk_idx.shape[1]
    _i32(T, E, K)
    _launch("moe_router_topk_backward", dev, stream,
            _ptr(d_topk_weights, "d_topk_weights", dev, (T, K), _F32),
            _ptr(logits, "logits", dev, logits.shape, logits.dtype), lcode, _ptr(topk_idx, "topk_idx", dev, (T, K), _I32),
            T, E, K, cfg.c(), _ptr(d_logits, "d_logits", dev, logits.shape, logits.dtype))


def moe_dispatch_quantized(q: torch.Tensor, q_s: torch.Tensor, plan: Plan, pool: torch.Tensor, pool_s: torch.Tensor,
                           epoch: int, ws: Workspace, dtype, stream=None) -> None:
    """moe_dispatch of rows that are codes [T, H] with row-major scales (quantized_scales()) already."""
    dev = _device(q, "q")
    code = _dtype_code(dtype)
    if code == MOE_BF16:                      # a bf16 pool has no codes to take (and no scales)
        raise MoeError("moe_dispatch_quantized", _abi.MOE_ERR_INVALID)
    if q.dim() != 2 or pool.dim() != 2:
        raise ValueError("q must be [T, H], pool [pool rows, H]")
    H, rows = q.shape[1], pool.shape[0]
    _i32(H, rows)
    if epoch > 0xFFFFFFFF:
        raise ValueError(f"epoch {epoch} is past 2^32 - 1")
    for t, n in ((plan.pos, "the plan"), (ws.buf, "ws")):
        if t.get_device() != dev:
            raise ValueError(f"{n} is on device {t.get_device()}, q on {dev}")
    if pool_s.numel() * pool_s.element_size() < rows * ((H + 127) // 128) * 4:
        raise ValueError("pool_s holds fewer scale words than the pool has")
    c = plan.c()
    _launch("moe_dispatch_quantized", dev, stream,
            _ptr(q, "q", dev, (plan.T, H), _CODES), _scales(q_s, "q_s", dev, plan.T, H, code),
            H, code, ctypes.byref(c), rows, _ptr(pool, "pool", dev, (rows, H), _CODES),
            _ptr(pool_s, "pool_s", dev, pool_s.shape, (_F32, _U8)), epoch, ws.buf.data_ptr(), ws.nbytes)


def expert_ffn_decode_workspace_bytes(T: int, K: int, I: int) -> int:
    _i32(T, K, I)
    return int(load().moe_expert_ffn_decode_workspace_bytes(T, K, I))


def moe_expert_ffn_decode(x: torch.Tensor, x_s: Optional[torch.Tensor], topk_idx: torch.Tensor,
                          topk_weights: torch.Tensor, w1: torch.Tensor, w1_s: torch.Tensor, w2: torch.Tensor,
                          w2_s: torch.Tensor, ws: torch.Tensor, out: torch.Tensor, expert_begin: int = 0,
                          stream=None) -> None:
    """out [T, H] of up to 64 tokens through the MXFP4 experts, without plan or pool. x: MXFP8 codes
    [T, H] with x_s (moe_rmsnorm's q and q_s), or bf16 with x_s None. Weights and scales as
    moe_pack_weights and moe_pack_mx_scales give them: w1 [E_local, 2I, H/2], w2 [E_local, H, I/2].
    ws: a byte tensor of expert_ffn_decode_workspace_bytes(T, K, I)."""
    dev = _device(x, "x")
    if x.dim() != 2 or w1.dim() != 3 or topk_idx.dim() != 2:
        raise ValueError("x must be [T, H], w1 [E_local, 2I, H/2], topk_idx [T, K]")
    (T, H), K = x.shape, topk_idx.shape[1]
    E, I = w1.shape[0], w1.shape[1] // 2
    _i32(T, H, K, E, I, expert_begin)
    ws_ptr, ws_bytes = _bytes(ws, "ws", dev)
    _launch("moe_expert_ffn_decode", dev, stream,
            _ptr(x, "x", dev, x.shape, _BF16 if x_s is None else _CODES), _scales(x_s, "x_s", dev, T, H, MOE_MXFP4),
            MOE_BF16 if x_s is None else MOE_MXFP4, T, H, I, K, expert_begin, E,
            _ptr(topk_idx, "topk_idx", dev, (T, K), _I32), _ptr(topk_weights, "topk_weights", dev, (T, K), _F32),
            _ptr(w1, "w1", dev, (E, 2 * I, H // 2), _U8), _ptr(w1_s, "w1_s", dev, (E, 2 * I, H // 32), _U8),
            _ptr(w2, "w2", dev, (E, H, I // 2), _U8), _ptr(w2_s, "w2_s", dev, (E, H, I // 32), _U8),
            ws_ptr, ws_bytes, _ptr(out, "out", dev, (T, H), _BF16))
