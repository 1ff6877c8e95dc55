"""Python binding of the operators around the MoE layer (include/moe355_block.h).

The residual's addition with the RMS norm and its 8-bit output, the router's choice of
experts, the dispatch of rows that are quantised already, the expert FFN of a few
tokens; the norms around a block's gate and residual, and low-rank adapters. Argument
marshalling only, as in ``layer``: the caller owns every tensor and the calls are
asynchronous. All tensors of a call are on one device, which need not be the current one;
``stream`` defaults to that device's current stream.
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
    "expert_ffn_decode_workspace_bytes", "quantized_scales", "moe_sandwich_norm", "moe_sandwich_norm_backward",
    "sandwich_norm_backward_workspace_bytes", "moe_adapter", "moe_adapter_backward", "adapter_workspace_bytes",
    "adapter_backward_workspace_bytes", "adapter_tile",
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


_GATE_ACTS = {"none": _abi.MOE_GATE_IDENTITY, "sigmoid": _abi.MOE_GATE_SIGMOID, "tanh": _abi.MOE_GATE_TANH}


def _gate(gate: Optional[torch.Tensor], act: str, dev: int, T: int, H: int):
    """(kind, activation, type, shape, address) of a block's gate: [T, 1] a row, [H] a channel, [T, H] a value."""
    code = _GATE_ACTS.get(act)
    if code is None:
        raise ValueError(f"gate_act {act!r}")
    if gate is None:
        return _abi.MOE_GATE_NONE, code, MOE_BF16, None, None
    shape = gate.shape
    if shape == (T, 1):
        kind = _abi.MOE_GATE_ROW
    elif shape == (H,):
        kind = _abi.MOE_GATE_CHANNEL
    elif shape == (T, H):
        kind = _abi.MOE_GATE_FULL
    else:
        raise ValueError(f"gate has shape {tuple(shape)}, expected [T, 1], [H] or [T, H]")
    return kind, code, _real_dtype(gate, "gate"), shape, _ptr(gate, "gate", dev, shape, gate.dtype)


def _both_weights(post_weight, weight, dev: int, H: int):
    """(type, post_weight's address, weight's) of two norm weights of one type, either of them None."""
    some = weight if weight is not None else post_weight
    if some is None:
        return MOE_BF16, None, None
    return (_real_dtype(some, "weight" if weight is not None else "post_weight"),
            _ptr(post_weight, "post_weight", dev, (H,), some.dtype), _ptr(weight, "weight", dev, (H,), some.dtype))


def moe_sandwich_norm(x: torch.Tensor, res: Optional[torch.Tensor], weight: Optional[torch.Tensor], eps: float,
                      s_out: torch.Tensor, y: Optional[torch.Tensor] = None, *,
                      post_weight: Optional[torch.Tensor] = None, post_eps: Optional[float] = None,
                      gate: Optional[torch.Tensor] = None, gate_act: str = "none", res_scale: float = 1.0,
                      branch_scale: float = 1.0, post_rstd: Optional[torch.Tensor] = None,
                      rstd: Optional[torch.Tensor] = None, q: Optional[torch.Tensor] = None,
                      q_s: Optional[torch.Tensor] = None, dtype="bf16", stream=None) -> None:
    """Between two blocks: s = res * res_scale + rms_norm(x) * post_weight * (act(gate) * branch_scale), then
    y = rms_norm(s) * weight and its copy (q, q_s) in the activation format ``dtype``. x is the block's output,
    s (to ``s_out``) the residual stream. Without post_weight x is taken as it is, without weight
    only s is made. gate: bf16 or fp32, [T, 1] (a factor a row), [H] (a column) or [T, H];
    gate_act: "none", "sigmoid" or "tanh". post_eps is eps unless given; post_rstd and rstd for the backward pass."""
    dev = _device(x, "x")
    if x.dim() != 2:
        raise ValueError("x must be [T, H]")
    shape = x.shape
    T, H = shape
    _i32(T, H)
    code = MOE_BF16 if dtype == "bf16" else _dtype_code(dtype)
    wcode, wp_ptr, w_ptr = _both_weights(post_weight, weight, dev, H)
    kind, act, gcode, _, g_ptr = _gate(gate, gate_act, dev, T, H)
    cfg = _abi.SandwichConfigT(eps if post_eps is None else post_eps, eps, res_scale, branch_scale, kind, act, gcode)
    _launch("moe_sandwich_norm", dev, stream,
            _ptr(x, "x", dev, shape, _BF16), _ptr(res, "res", dev, shape, _BF16), wp_ptr, w_ptr, wcode, g_ptr, cfg, T, H,
            _ptr(s_out, "s_out", dev, shape, _BF16), _ptr(y, "y", dev, shape, _BF16),
            _ptr(post_rstd, "post_rstd", dev, (T,), _F32), _ptr(rstd, "rstd", dev, (T,), _F32), code,
            _ptr(q, "q", dev, shape, _CODES), _scales(q_s, "q_s", dev, T, H, code))


def sandwich_norm_backward_workspace_bytes(T: int, H: int) -> int:
    _i32(T, H)
    return int(load().moe_sandwich_norm_backward_workspace_bytes(T, H))


def moe_sandwich_norm_backward(dy: Optional[torch.Tensor], d_s: Optional[torch.Tensor], x: Optional[torch.Tensor],
                               s: Optional[torch.Tensor], weight: Optional[torch.Tensor],
                               rstd: Optional[torch.Tensor], dx: torch.Tensor, d_res: Optional[torch.Tensor] = None,
                               dweight: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None, *,
                               post_weight: Optional[torch.Tensor] = None, post_rstd: Optional[torch.Tensor] = None,
                               gate: Optional[torch.Tensor] = None, gate_act: str = "none", res_scale: float = 1.0,
                               branch_scale: float = 1.0, d_post_weight: Optional[torch.Tensor] = None,
                               d_gate: Optional[torch.Tensor] = None, stream=None) -> None:
    """Gradients of moe_sandwich_norm from dy (of y; with weight) and d_s (of the stream behind it): dx, d_res,
    dweight and d_post_weight (fp32 [H]) and d_gate (as the gate; of a channel gate fp32 [H]), written, not
    added to. x, s, rstd and post_rstd are the forward's. ws is a byte tensor of
    sandwich_norm_backward_workspace_bytes(T, H), needed for the sums over rows."""
    dev = _device(dx, "dx")
    if dx.dim() != 2:
        raise ValueError("dx must be [T, H]")
    shape = dx.shape
    T, H = shape
    _i32(T, H)
    wcode, wp_ptr, w_ptr = _both_weights(post_weight, weight, dev, H)
    kind, act, gcode, gshape, g_ptr = _gate(gate, gate_act, dev, T, H)
    if d_gate is not None and gate is None:
        raise ValueError("d_gate without a gate")
    cfg = _abi.SandwichConfigT(0.0, 0.0, res_scale, branch_scale, kind, act, gcode)
    ws_ptr, ws_bytes = _bytes(ws, "ws", dev)
    _launch("moe_sandwich_norm_backward", dev, stream,
            _ptr(dy, "dy", dev, shape, _BF16), _ptr(d_s, "d_s", dev, shape, _BF16), _ptr(x, "x", dev, shape, _BF16),
            _ptr(s, "s", dev, shape, _BF16), wp_ptr, w_ptr, wcode, g_ptr, cfg, _ptr(post_rstd, "post_rstd", dev, (T,), _F32),
            _ptr(rstd, "rstd", dev, (T,), _F32), T, H, _ptr(dx, "dx", dev, shape, _BF16),
            _ptr(d_res, "d_res", dev, shape, _BF16), _ptr(dweight, "dweight", dev, (H,), _F32),
            _ptr(d_post_weight, "d_post_weight", dev, (H,), _F32),
            _ptr(d_gate, "d_gate", dev, gshape, _F32 if kind == _abi.MOE_GATE_CHANNEL else gate.dtype if gate is not None else None),
            ws_ptr, ws_bytes)


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


def _rows(t: Optional[torch.Tensor], name: str, dev: int, T: int, width: int):
    """(address, row pitch) of a checked bf16 tensor [T, width] whose rows may be columns of wider ones."""
    if t is None:
        return None, 0
    if t.dtype is _BF16 and t.get_device() == dev and t.is_contiguous() and t.shape == (T, width):
        return t.data_ptr(), width
    if t.dtype is not _BF16:
        raise ValueError(f"{name} has dtype {t.dtype}, expected bf16")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on device {t.get_device()}, the call's first tensor on {dev}")
    if t.shape != (T, width):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {(T, width)}")
    if T > 1 and (t.stride(1) != 1 or t.stride(0) < width):
        raise ValueError(f"{name} must have dense rows that do not overlap")
    if T == 1 and width > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must have dense rows")
    ld = t.stride(0) if T > 1 else width
    _i32(ld)
    return t.data_ptr(), ld


def adapter_tile(T: int, n: int) -> int:
    """The tile of a plan that groups T rows by n adapters: 16, 32 or 128. Few rows need small tiles for as many workgroups as
    there are CUs, many share an adapter's factors in large ones (4096 to 4096, ranks 16 and 64, in us: 512 rows of one adapter
    11 and 13 with 16, 19 and 22 with 128; 3500 of 40 adapters 28 and 46, 29 and 44 with 32, 26 and 33 with 128; 8192 of
    256: 64 and 126, 65 and 112, 82 and 116)."""
    return 128 if T >= max(3000, 64 * n) else 32 if T >= 2048 else 16


def adapter_workspace_bytes(T: int, K: int, R: int) -> int:
    _i32(T, K, R)
    return int(load().moe_adapter_workspace_bytes(T, K, R))


def _adapters(a: torch.Tensor, b: torch.Tensor, scale, ranks, dev: int):
    """(n, K, N, R) of the adapters' tables, and their four addresses."""
    if a.dim() != 3 or b.dim() != 3:
        raise ValueError("a must be [n, R, K], b [n, N, R]")
    (n, R, K), N = a.shape, b.shape[1]
    _i32(n, R, K, N)
    return (n, K, N, R), (_ptr(a, "a", dev, (n, R, K), _BF16), _ptr(b, "b", dev, (n, N, R), _BF16),
                          _ptr(scale, "scale", dev, (n,), _F32), _ptr(ranks, "ranks", dev, (n,), _I32))


def _adapter_plan(plan: Optional[Plan], dev: int):
    if plan is None:
        return None
    if plan.pos.get_device() != dev:
        raise ValueError(f"the plan is on device {plan.pos.get_device()}, the call's first tensor on {dev}")
    return plan.c()


def moe_adapter(x: torch.Tensor, a: torch.Tensor, b: torch.Tensor, out: torch.Tensor, ws: torch.Tensor, *,
                base: Optional[torch.Tensor] = None, ids: Optional[torch.Tensor] = None, plan: Optional[Plan] = None,
                id_begin: int = 0, scale: Optional[torch.Tensor] = None, ranks: Optional[torch.Tensor] = None,
                v: Optional[torch.Tensor] = None, stream=None) -> None:
    """out[t] = base[t] + scale[e] * b[e] @ (a[e] @ x[t]) with e the adapter of row t; base[t] (or zeros) for a row
    without one. x [T, K], base and out [T, N]: bf16, their rows may be columns of wider tensors; out may be base.
    a: bf16 [n, R, K], b: bf16 [n, N, R]; scale: fp32 [n]; ranks: int32 [n], the rows of a (columns of b)
    that an adapter has. The rows' adapters: ids int32 [T] for up to 64 rows (less id_begin; outside
    [0, n): none), or a Plan with K = 1 that moe_plan made of ids [T, 1] (see adapter_tile()). v: fp32 [T, R], kept for
    moe_adapter_backward. ws: a byte tensor of adapter_workspace_bytes(T, K, R)."""
    dev = _device(x, "x")
    if x.dim() != 2:
        raise ValueError("x must be [T, K]")
    (n, K, N, R), table = _adapters(a, b, scale, ranks, dev)
    T = x.shape[0]
    _i32(T, id_begin)
    x_ptr, ldx = _rows(x, "x", dev, T, K)
    base_ptr, ld_base = _rows(base, "base", dev, T, N)
    out_ptr, ld_out = _rows(out, "out", dev, T, N)
    ws_ptr, ws_bytes = _bytes(ws, "ws", dev)
    _launch("moe_adapter", dev, stream, x_ptr, ldx, *table, n, T, K, N, R, _ptr(ids, "ids", dev, (T,), _I32), id_begin,
            _adapter_plan(plan, dev), base_ptr, ld_base, out_ptr, ld_out, _ptr(v, "v", dev, (T, R), _F32), ws_ptr, ws_bytes)


def adapter_backward_workspace_bytes(T: int, n: int, K: int, N: int, R: int) -> int:
    _i32(T, n, K, N, R)
    return int(load().moe_adapter_backward_workspace_bytes(T, n, K, N, R))


def moe_adapter_backward(dout: torch.Tensor, x: Optional[torch.Tensor], v: Optional[torch.Tensor], a: torch.Tensor,
                         b: torch.Tensor, plan: Optional[Plan], ws: Optional[torch.Tensor],
                         da: Optional[torch.Tensor] = None, db: Optional[torch.Tensor] = None,
                         dx: Optional[torch.Tensor] = None, *, dx_base: Optional[torch.Tensor] = None,
                         scale: Optional[torch.Tensor] = None, ranks: Optional[torch.Tensor] = None, stream=None) -> None:
    """Gradients of moe_adapter for rows grouped by ``plan``: da fp32 [n, R, K] and db fp32 [n, N, R], written, not
    added to, and dx = dx_base (the shared projection's own, or zeros) + the adapters', which may be
    dx_base itself. v is what moe_adapter kept. ws: a byte tensor of adapter_backward_workspace_bytes(T, n, K, N, R)."""
    dev = _device(dout, "dout")
    if dout.dim() != 2:
        raise ValueError("dout must be [T, N]")
    (n, K, N, R), table = _adapters(a, b, scale, ranks, dev)
    T = dout.shape[0]
    _i32(T)
    d_ptr, ld_dout = _rows(dout, "dout", dev, T, N)
    x_ptr, ldx = _rows(x, "x", dev, T, K)
    base_ptr, ld_base = _rows(dx_base, "dx_base", dev, T, K)
    dx_ptr, ld_dx = _rows(dx, "dx", dev, T, K)
    ws_ptr, ws_bytes = _bytes(ws, "ws", dev)
    _launch("moe_adapter_backward", dev, stream, d_ptr, ld_dout, x_ptr, ldx, _ptr(v, "v", dev, (T, R), _F32), *table, n, T, K, N,
            R, _adapter_plan(plan, dev), base_ptr, ld_base, dx_ptr, ld_dx, _ptr(da, "da", dev, (n, R, K), _F32),
            _ptr(db, "db", dev, (n, N, R), _F32), ws_ptr, ws_bytes)


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
