"""The block around the memory layer: gated norm, join and gated recurrence (thin binding of the
block operators of libgka.so; every step runs in the HIP kernels).

A block is ``norm -> mixer -> gated_norm -> product -> join``: the mixer is ``gka.fwd_chunked`` or
``recur``, and ``join`` ends the block and normalises the stream for the next one. The names mirror
include/gka.h, which holds the formulas:

  gated_norm, gated_norm_bwd        -> gka_gated_norm, gka_gated_norm_bwd
  join, join_bwd                    -> gka_join, gka_join_bwd
  recur, recur_step, recur_bwd      -> gka_recur, gka_recur_step, gka_recur_bwd

Tensors are bfloat16 or float32 device tensors; weights, scales, states and their gradients are
float32. ``x``, ``gate``, ``f``, ``y`` and the residual stream may be slices of wider rows (the
halves of a fused projection, say); everything else is dense. Work is enqueued on ``stream``
(default: the current stream of the tensors' device); with another stream the caller orders it
after the inputs' producers and before the outputs' readers. Results are plain tensors without an
autograd history: training calls the ``*_bwd`` functions (examples/block_stack.py wraps them in
autograd functions).
"""
from __future__ import annotations

import ctypes
import functools
import inspect
import math
from typing import NamedTuple, Optional

import torch

from . import gka

ACT = {"silu": 0, "sigmoid": 1}
_CODE = {torch.bfloat16: gka.GKA_BF16, torch.float32: gka.GKA_FP32}


class JoinGrads(NamedTuple):
    """Gradients of ``join``; the entries of absent arguments are None."""
    dres: torch.Tensor
    dy: torch.Tensor
    dgate: Optional[torch.Tensor]
    dw_post: Optional[torch.Tensor]
    dscale: Optional[torch.Tensor]
    dw_pre: Optional[torch.Tensor]


# ---- checks and parameter blocks, by the tensors' metadata -----------------------------------------
# A call's checks depend on shapes, strides, dtypes and devices alone. They run on those (a tuple per
# tensor) and are remembered with the parameter block they led to, so a repeated call costs one
# look-up: 1 us instead of 3 for the gated norm of one token. Scalars enter as Python numbers: a tensor
# would be looked up by its identity, whatever it holds by then.
_SHAPE, _STRIDE, _DTYPE, _DEVICE = range(4)


def _sig(t: Optional[torch.Tensor]):
    return None if t is None else (t.shape, t.stride(), t.dtype, t.get_device())


def _act(act: str) -> int:
    if act not in ACT:
        raise ValueError(f"act must be one of {sorted(ACT)}, got {act!r}")
    return ACT[act]


def _dense(sig) -> bool:
    want = 1
    for n, st in zip(reversed(sig[_SHAPE]), reversed(sig[_STRIDE])):
        if n == 0:
            return True
        if n != 1 and st != want:
            return False
        want *= n
    return True


def _rows(sig, tail: int, what: str):
    """(rows, stride) of a tensor whose last ``tail`` dims are one token: the elements of a token
    are consecutive and the tokens a constant stride apart."""
    shape, stride = sig[_SHAPE], sig[_STRIDE]
    width, rows = math.prod(shape[-tail:]), math.prod(shape[:-tail])
    if rows * width == 0:
        return rows, width
    want = 1
    for d in range(len(shape) - 1, len(shape) - 1 - tail, -1):
        if shape[d] != 1 and stride[d] != want:
            raise ValueError(f"the elements of one token of {what} must be consecutive")
        want *= shape[d]
    token = None
    for d in range(len(shape) - tail - 1, -1, -1):
        if shape[d] == 1:
            continue
        if token is None:
            token = want = stride[d]
        if stride[d] != want:
            raise ValueError(f"the tokens of {what} must be a constant stride apart")
        want *= shape[d]
    return rows, width if token is None else token


def _on_same_device(x, t, what: str):
    if t[_DEVICE] != x[_DEVICE]:
        raise ValueError(f"{what} must be on cuda:{x[_DEVICE]}")


def _same(x, t, what: str, dense: bool):
    """``t`` has x's shape, dtype and device (and is dense)."""
    if t[_SHAPE] != x[_SHAPE] or t[_DTYPE] != x[_DTYPE]:
        raise ValueError(f"{what} must have shape {tuple(x[_SHAPE])} and dtype {x[_DTYPE]}")
    if dense and not _dense(t):
        raise ValueError(f"{what} must be dense")
    _on_same_device(x, t, what)


def _float32(x, t, shape, what: str):
    """``t`` is None or a dense float32 tensor of ``shape`` on x's device."""
    if t is None:
        return
    if t[_DTYPE] != torch.float32 or tuple(t[_SHAPE]) != tuple(shape) or not _dense(t):
        raise ValueError(f"{what} must be a dense float32 tensor of shape {tuple(shape)}")
    _on_same_device(x, t, what)


def _on_device(fn):
    """Runs ``fn`` with the device of its first argument current and ``stream`` as the current
    stream of it. On another stream than the caller's current one, what the call allocates comes
    from that stream's pool, and inputs and outputs are marked as used on both streams, so that the
    allocator hands none of their memory out while either still uses it."""
    first = next(iter(inspect.signature(fn).parameters))

    @functools.wraps(fn)
    def call(*args, stream=None, **kw):
        if not args and first not in kw:
            return fn(**kw)  # raises the TypeError that names it
        x = args[0] if args else kw[first]
        device = x.get_device() if isinstance(x, torch.Tensor) else -1
        if device < 0:
            raise ValueError("libgka takes GPU (device) tensors")
        if stream is None and device == torch.cuda.current_device():
            return fn(*args, **kw)
        outer = torch.cuda.current_stream(x.device)
        inner = outer if stream is None else stream
        if inner.device != x.device:
            raise ValueError(f"stream must belong to {x.device}")
        with torch.cuda.device(x.device), torch.cuda.stream(inner):
            out = fn(*args, **kw)
        if inner != outer:
            for t in (*args, *kw.values()):
                if isinstance(t, torch.Tensor) and t.is_cuda:  # (a scalar may be a host tensor)
                    t.record_stream(inner)
            for t in out if isinstance(out, tuple) else (out,):
                if isinstance(t, torch.Tensor):
                    t.record_stream(outer)
        return out
    return call


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


# The current stream's handle. torch.cuda.current_stream() builds a Stream object for it, which
# takes 2 us of a call of 7; this is the accessor that torch's own generated code uses.
_raw_stream = torch._C._cuda_getCurrentRawStream


def _stream(x: torch.Tensor) -> int:
    return _raw_stream(x.get_device())


def _scratch(x: torch.Tensor, given: Optional[torch.Tensor], need: int):
    """The workspace: the given one, or a new one of ``need`` bytes (none for 0)."""
    if given is None:
        return x.new_empty(need, dtype=torch.uint8) if need else None
    if given.get_device() != x.get_device() or not given.is_contiguous():
        raise ValueError(f"the workspace must be a dense tensor on {x.device}")
    return given


def _bytes(t: Optional[torch.Tensor]) -> int:
    return 0 if t is None else t.numel() * t.element_size()


def _new(x: torch.Tensor):
    """A new dense tensor of x's shape and dtype."""
    return torch.empty_like(x) if x.is_contiguous() else x.new_empty(x.shape)


def _out(x: torch.Tensor, out: Optional[torch.Tensor], what: str):
    if out is None:
        return _new(x)
    _same(_sig(x), _sig(out), what, True)
    return out


# ---- gated norm ------------------------------------------------------------------------------
@functools.lru_cache(maxsize=4096)
def _norm_plan(x, gate, weight, dy, eps, act):
    """(parameter block, workspace bytes of the backward)"""
    shape = x[_SHAPE]
    if len(shape) < 2:
        raise ValueError("x must be [..., H, D]")
    H, D = shape[-2:]
    rows, xs = _rows(x, 2, "x")
    gs = xs
    if gate is not None:
        _same(x, gate, "gate", False)
        gs = _rows(gate, 2, "gate")[1]
    per_head = 0
    if weight is not None:
        per_head = int(len(weight[_SHAPE]) == 2)
        _float32(x, weight, (H, D) if per_head else (D,), "weight")
    if dy is not None:
        _same(x, dy, "dy", True)
    p = ctypes.byref(gka.GkaGatedNormParams(rows, H, D, per_head, _act(act),
                                            _CODE.get(x[_DTYPE], -1), eps, xs, gs))
    return p, int(gka.load().gka_gated_norm_bwd_workspace_bytes(p))


@_on_device
def gated_norm(x: torch.Tensor, gate: Optional[torch.Tensor] = None,
               weight: Optional[torch.Tensor] = None, eps: float = 1e-6, act: str = "silu",
               out: Optional[torch.Tensor] = None):
    """gka_gated_norm: x / rms(x) * weight * act(gate) over the last dim of x [..., H, D].

    ``gate`` has x's shape (None: no gate), ``weight`` is float32 [D], or [H, D] with weights per
    head (None: ones), ``act`` "silu" or "sigmoid". Also takes ``stream``. Returns a dense tensor of
    x's shape and dtype."""
    p, _ = _norm_plan(_sig(x), _sig(gate), _sig(weight), None, float(eps), act)
    y = _out(x, out, "out")
    gka._check(gka.load().gka_gated_norm(p, x.data_ptr(), _ptr(gate), _ptr(weight), y.data_ptr(),
                                         _stream(x)))
    return y


@_on_device
def gated_norm_bwd(x: torch.Tensor, gate: Optional[torch.Tensor], weight: Optional[torch.Tensor],
                   dy: torch.Tensor, eps: float = 1e-6, act: str = "silu",
                   workspace: Optional[torch.Tensor] = None):
    """gka_gated_norm_bwd: (dx, dgate, dweight) of gated_norm, given dy (dense, x's shape). dgate
    and dweight are None without a gate or weight. Also takes ``stream``."""
    p, need = _norm_plan(_sig(x), _sig(gate), _sig(weight), _sig(dy), float(eps), act)
    dx = _new(x)
    dgate = None if gate is None else torch.empty_like(dx)
    dweight = None if weight is None else torch.empty_like(weight)
    ws = _scratch(x, workspace, 0 if weight is None else need)
    gka._check(gka.load().gka_gated_norm_bwd(
        p, x.data_ptr(), _ptr(gate), _ptr(weight), dy.data_ptr(), dx.data_ptr(), _ptr(dgate),
        _ptr(dweight), _ptr(ws), _bytes(ws), _stream(x)))
    return dx, dgate, dweight


# ---- join --------------------------------------------------------------------------------------
@functools.lru_cache(maxsize=4096)
def _join_plan(res, y, gate, w_post, scale, w_pre, dres_out, dn, alpha, eps, act):
    """(parameter block, workspace bytes of the backward)"""
    shape = res[_SHAPE]
    if len(shape) < 1 or y[_SHAPE] != shape:
        raise ValueError("res and y must be [..., C] of the same shape")
    _on_same_device(res, y, "y")
    C = shape[-1]
    rows, rs = _rows(res, 1, "res")
    ys = gs = _rows(y, 1, "y")[1]
    if gate is not None:
        _same(y, gate, "gate", False)
        gs = _rows(gate, 1, "gate")[1]
    for t, what in ((w_post, "w_post"), (scale, "scale"), (w_pre, "w_pre")):
        _float32(res, t, (C,), what)
    if dres_out is not None:  # the backward
        _same(res, dres_out, "dres_out", True)
        if (dn is None) != (w_pre is None):
            raise ValueError("dn must be given exactly when w_pre is")
        if dn is not None:
            _same(y, dn, "dn", True)
    p = ctypes.byref(gka.GkaJoinParams(rows, C, _act(act), _CODE.get(y[_DTYPE], -1),
                                       _CODE.get(res[_DTYPE], -1), eps, alpha, rs, ys, gs))
    return p, int(gka.load().gka_join_bwd_workspace_bytes(p))


@_on_device
def join(res: torch.Tensor, y: torch.Tensor, gate: Optional[torch.Tensor] = None,
         w_post: Optional[torch.Tensor] = None, scale: Optional[torch.Tensor] = None,
         w_pre: Optional[torch.Tensor] = None, alpha: float = 1.0, eps: float = 1e-6,
         act: str = "silu", out: Optional[torch.Tensor] = None,
         n_out: Optional[torch.Tensor] = None):
    """gka_join on [..., C]: res_out = res + alpha * scale * (y / rms(y) * w_post * act(gate)) and
    n = res_out / rms(res_out) * w_pre, the terms of absent arguments left out.

    ``res`` is in y's dtype or float32; ``w_post``, ``scale`` and ``w_pre`` are float32 [C].
    ``out`` may be ``res`` itself (dense), which updates the stream in place. Also takes
    ``stream``. Returns (res_out, n); n, in y's dtype, is None without ``w_pre``."""
    p, _ = _join_plan(_sig(res), _sig(y), _sig(gate), _sig(w_post), _sig(scale), _sig(w_pre), None,
                      None, float(alpha), float(eps), act)
    res_out = _out(res, out, "out")
    n = None if w_pre is None else _out(y, n_out, "n_out")
    gka._check(gka.load().gka_join(
        p, res.data_ptr(), y.data_ptr(), _ptr(gate), _ptr(w_post), _ptr(scale), _ptr(w_pre),
        res_out.data_ptr(), _ptr(n), _stream(res)))
    return res_out, n


@_on_device
def join_bwd(res: torch.Tensor, y: torch.Tensor, dres_out: torch.Tensor,
             dn: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None,
             w_post: Optional[torch.Tensor] = None, scale: Optional[torch.Tensor] = None,
             w_pre: Optional[torch.Tensor] = None, alpha: float = 1.0, eps: float = 1e-6,
             act: str = "silu", workspace: Optional[torch.Tensor] = None) -> JoinGrads:
    """gka_join_bwd: the gradients of ``join`` from its inputs (``res`` as it was before the join)
    and the gradients ``dres_out`` (dense, res's shape and dtype) and ``dn`` (dense, y's; exactly
    when ``w_pre`` is given) to its two results. Also takes ``stream``."""
    p, need = _join_plan(_sig(res), _sig(y), _sig(gate), _sig(w_post), _sig(scale), _sig(w_pre),
                         _sig(dres_out), _sig(dn), float(alpha), float(eps), act)
    dres, dy = _new(res), _new(y)
    dgate = None if gate is None else torch.empty_like(dy)
    dws = [None if w is None else torch.empty_like(w) for w in (w_post, scale, w_pre)]
    ws = _scratch(res, workspace, need if any(w is not None for w in dws) else 0)
    gka._check(gka.load().gka_join_bwd(
        p, res.data_ptr(), y.data_ptr(), _ptr(gate), _ptr(w_post), _ptr(scale), _ptr(w_pre),
        dres_out.data_ptr(), _ptr(dn), dres.data_ptr(), dy.data_ptr(), _ptr(dgate),
        *(_ptr(w) for w in dws), _ptr(ws), _bytes(ws), _stream(res)))
    return JoinGrads(dres, dy, dgate, *dws)


# ---- recurrence ----------------------------------------------------------------------------------
@functools.lru_cache(maxsize=4096)
def _recur_plan(x, f, state, dh, dstate, complement, step):
    """(parameter block, bytes of the carry, of the workspace, of the backward's workspace)"""
    shape = x[_SHAPE]
    if len(shape) != (2 if step else 3):
        raise ValueError("x must be [B, C]" if step else "x must be [B, T, C]")
    if max(shape) > 0x7fffffff:  # the parameter block would hold it modulo 2^32
        raise ValueError(f"x of shape {tuple(shape)}: its dimensions must be below 2^31")
    _same(x, f, "f", False)
    B, C = shape[0], shape[-1]
    T = 1 if step else shape[1]
    strides = []
    for t, what in ((x, "x"), (f, "f")):
        st = t[_STRIDE]
        if C > 1 and st[-1] != 1:
            raise ValueError(f"the channels of one token of {what} must be consecutive")
        ts = C if step or T <= 1 else st[1]
        strides += [st[0] if B > 1 else T * ts, ts]
    _float32(x, state, (B, C), "state")
    _float32(x, dstate, (B, C), "dstate")
    if dh is not None:
        _same(x, dh, "dh", True)
    lib = gka.load()
    p = ctypes.byref(gka.GkaRecurParams(B, T, C, int(complement), _CODE.get(x[_DTYPE], -1),
                                        *strides))
    return (p, int(lib.gka_recur_carry_bytes(p)), int(lib.gka_recur_workspace_bytes(p)),
            int(lib.gka_recur_bwd_workspace_bytes(p)))


@_on_device
def recur(x: torch.Tensor, f: torch.Tensor, state: Optional[torch.Tensor] = None,
          complement: bool = True, return_carry: bool = False,
          out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
    """gka_recur: h_t = gamma_t h_{t-1} + beta_t x_t over [B, T, C], gamma = sigmoid(f), beta =
    1 - gamma (``complement``) or 1.

    ``state`` (optional, float32 [B, C]) is read as the initial state and overwritten with the
    final one. With ``return_carry`` the call returns (h, carry), carry being what ``recur_bwd``
    takes. Also takes ``stream``."""
    p, carry_bytes, need, _ = _recur_plan(_sig(x), _sig(f), _sig(state), None, None,
                                          bool(complement), False)
    h = _out(x, out, "out")
    carry = x.new_empty(carry_bytes // 4, dtype=torch.float32) if return_carry else None
    ws = _scratch(x, workspace, need)
    gka._check(gka.load().gka_recur(p, x.data_ptr(), f.data_ptr(), h.data_ptr(), _ptr(state),
                                    _ptr(carry), _ptr(ws), _bytes(ws), _stream(x)))
    return (h, carry) if return_carry else h


@_on_device
def recur_step(x: torch.Tensor, f: torch.Tensor, state: torch.Tensor, complement: bool = True,
               out: Optional[torch.Tensor] = None):
    """gka_recur_step: one token, x and f [B, C]; updates ``state`` (float32 [B, C]) in place and
    returns h [B, C]. Also takes ``stream``."""
    p = _recur_plan(_sig(x), _sig(f), _sig(state), None, None, bool(complement), True)[0]
    h = _out(x, out, "out")
    gka._check(gka.load().gka_recur_step(p, x.data_ptr(), f.data_ptr(), h.data_ptr(), _ptr(state),
                                         _stream(x)))
    return h


@_on_device
def recur_bwd(x: torch.Tensor, f: torch.Tensor, dh: torch.Tensor, carry: torch.Tensor,
              dstate: Optional[torch.Tensor] = None, complement: bool = True,
              workspace: Optional[torch.Tensor] = None):
    """gka_recur_bwd: (dx, df, dstate) given dh (dense, x's shape), the ``carry`` of the forward
    call and ``dstate``, the gradient to the final state (float32 [B, C], None: zero; it is left as
    it is). The returned dstate is the gradient to the initial state. Also takes ``stream``."""
    p, carry_bytes, _, need = _recur_plan(_sig(x), _sig(f), None, _sig(dh), _sig(dstate),
                                          bool(complement), False)
    _float32(_sig(x), _sig(carry), (carry_bytes // 4,), "carry")
    dx, df = _new(x), _new(x)
    ds = x.new_empty((x.shape[0], x.shape[2]), dtype=torch.float32)
    ws = _scratch(x, workspace, need)
    gka._check(gka.load().gka_recur_bwd(p, x.data_ptr(), f.data_ptr(), dh.data_ptr(),
                                        carry.data_ptr(), _ptr(dstate), dx.data_ptr(),
                                        df.data_ptr(), ds.data_ptr(), _ptr(ws), _bytes(ws),
                                        _stream(x)))
    return dx, df, ds
