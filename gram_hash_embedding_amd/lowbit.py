"""The module in narrow formats: the ctypes binding of libengram.so's 4-bit weights and 8-bit checkpoints
(include/engram.h), under the same rules as the rest of the package -- GPU tensors in, dtype / shape / contiguity checked,
no fallback.

    engram_mx4_quant        -- bf16 rows -> OCP MX fp4 (E2M1 + E8M0 scale per 32 columns)
    engram_mx4_pack_weight  -- MX fp4 weights -> the layout the products read (one-off)
    engram_wkv_mx4          -- the wkv projection of MX fp8 or MX fp4 rows on MX fp4 weights
    engram_wkv_mx4_gate     -- engram_wkv_mx4 fused with the gate dot (keys reduced in the projection)
    engram_ckpt_save, engram_ckpt_load -- bf16 rows to 8-bit checkpoints (OCP MX int8) and back
    engram_gate_output_ckpt -- engram_gate_output keeping its stream, keys and value in 8 bits
    engram_gate_output_backward_ckpt -- engram_gate_output_backward from what was kept
"""
from __future__ import annotations

import ctypes
import math
from typing import NamedTuple

from . import _check, lib
from . import training as _t

RECORD_BYTES = 4352  # of the weight layout: 64 rows x 128 columns


def declare(L: ctypes.CDLL) -> None:
    """Argument and result types of these entry points."""
    i64, i32, p, f32 = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p, ctypes.c_float
    L.engram_mx4_quant.argtypes = [p, i64, i32, p, p, p]
    L.engram_mx4_weight_bytes.argtypes = [i32, i32]
    L.engram_mx4_weight_bytes.restype = i64
    L.engram_mx4_pack_weight.argtypes = [p, p, i32, i32, p, p]
    L.engram_wkv_mx4.argtypes = [p, p, i32, p, p, i64, i32, i32, p]
    L.engram_wkv_mx4_gate.argtypes = [p, p, i32, p, p, p, p, f32, p, i64, p, p, i64, i64, i32, i32, i32, p]
    L.engram_ckpt_save.argtypes = [p, i64, i32, p, p, p]
    L.engram_ckpt_load.argtypes = [p, p, i64, i32, p, p]
    L.engram_gate_output_ckpt.argtypes = [p, p, i64, p, p, f32, p, p, p, p, p, p, p, i64, i32, i32, p]
    L.engram_gate_output_backward_ckpt.argtypes = [p, p, p, p, p, p, f32, p, p, p, p, p, p, p, p, i64, i64, i32, i32, p]


class GateCheckpoint(NamedTuple):
    """What engram_gate_output_ckpt keeps of its rows."""

    x: "torch.Tensor"          # int8 [T, hc, dim]
    x_scale: "torch.Tensor"    # uint8 [T, hc, ceil(dim / 32)]
    kv: "torch.Tensor"         # int8 [T, hc + 1, dim]: the keys, then the value
    kv_scale: "torch.Tensor"   # uint8 [T, hc + 1, ceil(dim / 32)]


def _scale_shape(rows: int, K: int):
    return (K // 128, (rows + 3) // 4 * 4, 4)


def _scale_bytes(rows: int, K: int) -> int:
    """engram_mx_scale_bytes; a K that is no multiple of 128 is left to the entry point's own check."""
    return K // 128 * ((rows + 3) // 4 * 16)


def engram_mx4_quant(x, q=None, scale=None, stream=None):
    """(q uint8 [rows, K/2], scale uint8 [K/128, ceil4(rows), 4]): bf16 rows x [rows, K] in OCP MX fp4 (E2M1, two elements
    a byte, the even column in the low half; an E8M0 scale per 32 columns in the layout of engram_mx_quant's)."""
    on = _t._On(stream, x, "x")
    torch = _t.torch
    xp = on.ptr(x, "x", torch.bfloat16, 2)
    rows, K = x.shape
    if K < 128 or K % 128:
        raise ValueError(f"K={K} must be a positive multiple of 128")
    q, qp = _out(on, q, "q", (rows, K // 2), torch.uint8)
    if scale is None:
        scale, sp = _out(on, None, "scale", _scale_shape(rows, K), torch.uint8)
    elif scale.numel() != _scale_bytes(rows, K):
        raise ValueError(f"scale must hold {_scale_bytes(rows, K)} bytes")
    else:
        sp = on.ptr(scale, "scale", torch.uint8)
    _check(lib().engram_mx4_quant(xp, rows, K, qp, sp, on.handle))
    return q, scale


def _out(on, t, name, shape, dtype):
    """(tensor, address) of an output: the given one, checked, or a new one."""
    if t is None:  # (sizes as arguments are parsed faster than as a tuple)
        t = _t.torch.empty(*shape, dtype=dtype, device=on.index) if on.side is None else on.empty(shape, dtype)
        return t, t.data_ptr()
    if t.shape != shape:
        raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
    return t, on.ptr(t, name, dtype)


def _out_like(on, t, name, like, dtype):
    """_out of the shape of `like`, a contiguous tensor of the call's device."""
    if t is None and on.side is None:
        t = _t.torch.empty_like(like, dtype=dtype)
        return t, t.data_ptr()
    return _out(on, t, name, like.shape, dtype)


def engram_mx4_weight_bytes(nout: int, K: int) -> int:
    n = lib().engram_mx4_weight_bytes(int(nout), int(K))
    if n < 0:
        raise ValueError(f"engram_wkv_mx4: Nout={nout} K={K} outside the limits")
    return n


def engram_mx4_pack_weight(q, scale, out=None, stream=None):
    """Weights uint8 [ceil(Nout / 64), K / 128, 4352] in the layout the products read, from MX fp4 rows q uint8 [Nout, K/2]
    and their scales (engram_mx4_quant's).  A one-off conversion."""
    on = _t._On(stream, q, "q")
    u8 = _t.torch.uint8
    qp = on.ptr(q, "q", u8, 2)
    N, K = q.shape[0], 2 * q.shape[1]
    engram_mx4_weight_bytes(N, K)
    if scale.numel() != _scale_bytes(N, K):
        raise ValueError("scale must be the MX scale array of q")
    out, op = _out(on, out, "out", ((N + 63) // 64, K // 128, RECORD_BYTES), u8)
    _check(lib().engram_mx4_pack_weight(qp, on.ptr(scale, "scale", u8), N, K, op, on.handle))
    return out


def _operands(on, a, a_scale, w):
    """(a address, scale address, bits, weight address, T, K, rows of the weight's records)."""
    u8 = _t.torch.uint8
    ap = on.ptr(a, "a", _t.torch.float8_e4m3fn if a.dtype is _t.torch.float8_e4m3fn else u8, 2)
    wp = on.ptr(w, "w", u8, 3)
    groups, steps, record = w.shape
    if record != RECORD_BYTES:
        raise ValueError("w must be packed weights (engram_mx4_pack_weight)")
    T, row = a.shape
    K = 128 * steps
    if row != K and (row != K // 2 or a.dtype is not u8):
        raise ValueError(f"a must be [T, K={K}] (MX fp8) or [T, K/2] (MX fp4), got {tuple(a.shape)}")
    if a_scale.numel() != steps * ((T + 3) // 4 * 16):  # _scale_bytes
        raise ValueError("a_scale must be the MX scale array of a")
    return ap, on.ptr(a_scale, "a_scale", u8), 8 if row == K else 4, wp, T, K, 64 * groups


def engram_wkv_mx4(a, a_scale, w, nout=None, out=None, stream=None):
    """kv bf16 [T, nout] of rows a -- MX fp8 (uint8 or float8_e4m3fn [T, K]: engram_mx_quant's, engram_gather_mx's) or MX fp4
    (uint8 [T, K/2]: engram_mx4_quant's) with their scales -- on packed MX fp4 weights w.  nout: out's columns, or by default
    all of the weight's rows, counted in whole records of 64."""
    on = _t._On(stream, a, "a")
    ap, sp, bits, wp, T, K, rows = _operands(on, a, a_scale, w)
    if nout is None:
        nout = rows if out is None else out.shape[-1]
    if not rows - 64 < nout <= rows:
        raise ValueError(f"nout={nout} is not the row count of weights of {rows // 64} records")
    out, op = _out(on, out, "out", (T, nout), _t.torch.bfloat16)
    _check(lib().engram_wkv_mx4(ap, sp, bits, wp, op, T, K, nout, on.handle))
    return out


def engram_wkv_mx4_gate(a, a_scale, w, x, q_weight, k_weight, eps, value=None, dot=None, workspace=None, stream=None):
    """(value bf16 [T, dim], dot float32 [T, hc]) from rows a with their scales and packed MX fp4 weights w of (hc+1)*dim
    rows (as engram_wkv_mx4 takes them) and the stream x bf16 [T, hc, dim] (or [B, L, hc, dim]); `value`, `dot` and
    `workspace` as engram_wkv_gate."""
    on = _t._On(stream, a, "a")
    torch = _t.torch
    bf, f32 = torch.bfloat16, torch.float32
    ap, sp, bits, wp, T, K, rows = _operands(on, a, a_scale, w)
    hc, dim = x.shape[-2:]
    if x.dim() < 3 or x.numel() != T * hc * dim:
        raise ValueError("x must be [T, hc, dim] (or [B, L, hc, dim]) with a's T")
    if rows != (hc + 1) * dim:
        raise ValueError("w must have (hc+1)*dim rows")
    if q_weight.shape != (hc, dim) or k_weight.shape != (hc, dim):
        raise ValueError("q_weight and k_weight must be [hc, dim]")
    if value is None:
        value, vp = _out(on, None, "value", (T, dim), bf)
    elif value.dim() != 2 or value.shape[0] != T or value.shape[1] < dim or value.stride(1) != 1:
        raise ValueError("value must be [T, >= dim] with unit column stride")
    elif value.dtype != bf or value.get_device() != on.index:
        raise TypeError("value must be a bf16 tensor of the call's GPU")
    else:
        vp = value.data_ptr()
    dot, dp = _out(on, dot, "dot", (T, hc), f32)
    _ws, sw, sn = on.workspace(workspace, hc * (dim // 128) * 3 * T * 4)  # engram_wkv_gate_workspace_bytes
    _check(lib().engram_wkv_mx4_gate(ap, sp, bits, wp, on.ptr(x, "x", bf), on.ptr(q_weight, "q_weight", bf),
                                     on.ptr(k_weight, "k_weight", bf), float(eps), vp, value.stride(0), dp, sw,
                                     sn, T, K, hc, dim, on.handle))
    return value, dot


def engram_ckpt_save(x, q=None, scale=None, stream=None):
    """(q int8 of x's shape, scale uint8 [..., ceil(D/32)]): the rows of bf16 x [..., D] in OCP MX int8."""
    on = _t._On(stream, x, "x")
    torch = _t.torch
    xp = on.ptr(x, "x", torch.bfloat16)
    if x.dim() < 1:
        raise ValueError("x must have a dimension")
    shape = x.shape
    D = shape[-1]
    q, qp = _out_like(on, q, "q", x, torch.int8)
    scale, sp = _out(on, scale, "scale", (*shape[:-1], (D + 31) // 32), torch.uint8)
    _check(lib().engram_ckpt_save(xp, math.prod(shape[:-1]), D, qp, sp, on.handle))
    return q, scale


def engram_ckpt_load(q, scale, out=None, stream=None):
    """bf16 rows of q's shape: exactly what the checkpoint (engram_ckpt_save's q and scale) stands for."""
    on = _t._On(stream, q, "q")
    torch = _t.torch
    qp = on.ptr(q, "q", torch.int8)
    if q.dim() < 1:
        raise ValueError("q must have a dimension")
    shape = q.shape
    *lead, D = shape
    if scale.shape != (*lead, (D + 31) // 32):
        raise ValueError("scale must hold a byte per 32 columns of each row of q")
    out, op = _out_like(on, out, "out", q, torch.bfloat16)
    _check(lib().engram_ckpt_load(qp, on.ptr(scale, "scale", torch.uint8), math.prod(lead), D, op, on.handle))
    return out


def _mask(on, token_mask, T):
    if token_mask is None:
        return None
    if token_mask.numel() != T:
        raise ValueError("token_mask must hold one entry per token")
    if token_mask.dtype == _t.torch.bool:
        token_mask = token_mask.view(_t.torch.uint8)
    return on.ptr(token_mask, "token_mask", _t.torch.uint8)


def engram_gate_output_ckpt(x, kv, q_weight, k_weight, eps, token_mask=None, out=None, dot=None, checkpoint=None,
                            stream=None):
    """(out, dot, GateCheckpoint): engram_gate_output of x bf16 [T, hc, dim] (or [B, L, hc, dim]) and kv [T, >= (hc+1)*dim],
    with x, the keys and the value kept in 8 bits (engram_ckpt_save's, of their rows of dim) for
    engram_gate_output_backward_ckpt.  out (x's shape; x itself is allowed), dot (float32 [T, hc]) and `checkpoint`, or those
    of its tensors that are None, are allocated if not given."""
    on = _t._On(stream, x, "x")
    torch = _t.torch
    bf, f32 = torch.bfloat16, torch.float32
    if x.dim() < 3:
        raise ValueError("x must be [T, hc, dim] (or [B, L, hc, dim])")
    hc, dim = x.shape[-2:]
    T = x.numel() // (hc * dim) if hc * dim else 0
    if kv.dim() != 2 or kv.shape[0] != T or kv.shape[1] < (hc + 1) * dim:
        raise ValueError("kv must be [T, >= (hc+1)*dim]")
    if q_weight.shape != (hc, dim) or k_weight.shape != (hc, dim):
        raise ValueError("q_weight and k_weight must be [hc, dim]")
    xp = on.ptr(x, "x", bf)
    mp = _mask(on, token_mask, T)
    out, op = _out_like(on, out, "out", x, bf)
    dot, dp = _out(on, dot, "dot", (T, hc), f32)
    checkpoint, c = _checkpoint(on, checkpoint, T, hc, dim)
    _check(lib().engram_gate_output_ckpt(
        xp, on.ptr(kv, "kv", bf, 2), kv.shape[1], on.ptr(q_weight, "q_weight", bf),
        on.ptr(k_weight, "k_weight", bf), float(eps), mp, op, dp, *c, T, hc, dim, on.handle))
    return out, dot, checkpoint


def _checkpoint(on, given, T, hc, dim):
    """(GateCheckpoint, its addresses): the given one's tensors, checked, and new ones where it has none."""
    i8, u8, nb = _t.torch.int8, _t.torch.uint8, (dim + 31) // 32
    x, xs, kv, kvs = given if given is not None else (None, None, None, None)
    x, p0 = _out(on, x, "checkpoint.x", (T, hc, dim), i8)
    xs, p1 = _out(on, xs, "checkpoint.x_scale", (T, hc, nb), u8)
    kv, p2 = _out(on, kv, "checkpoint.kv", (T, hc + 1, dim), i8)
    kvs, p3 = _out(on, kvs, "checkpoint.kv_scale", (T, hc + 1, nb), u8)
    return GateCheckpoint(x, xs, kv, kvs), (p0, p1, p2, p3)


def engram_gate_output_backward_ckpt(checkpoint, q_weight, k_weight, eps, dot, dout, token_mask=None, dx=None, dkv=None,
                                     dq=None, dk=None, workspace=None, stream=None):
    """(dx bf16 of dout's shape, dkv bf16 [T, (hc+1)*dim], dq, dk float32 [hc, dim]) from dout bf16 [T, hc, dim] (or [B, L,
    hc, dim]) and what engram_gate_output_ckpt kept: engram_gate_output_backward of the x and kv that engram_ckpt_load gives,
    bit for bit.  `dx` may be dout itself."""
    on = _t._On(stream, dout, "dout")
    bf, f32 = _t.torch.bfloat16, _t.torch.float32
    if dout.dim() < 3:
        raise ValueError("dout must be [T, hc, dim] (or [B, L, hc, dim])")
    hc, dim = dout.shape[-2:]
    T = dout.numel() // (hc * dim) if hc * dim else 0
    if checkpoint is None or any(t is None for t in checkpoint):
        raise ValueError("the gradient needs the checkpoint of engram_gate_output_ckpt")
    _, c = _checkpoint(on, checkpoint, T, hc, dim)
    if q_weight.shape != (hc, dim) or k_weight.shape != (hc, dim):
        raise ValueError("q_weight and k_weight must be [hc, dim]")
    if dot.shape != (T, hc):
        raise ValueError("dot must be [T, hc]")
    gp = on.ptr(dout, "dout", bf)
    mp = _mask(on, token_mask, T)
    dx, xp = _out_like(on, dx, "dx", dout, bf)
    dkv, kvp = _out(on, dkv, "dkv", (T, (hc + 1) * dim), bf)
    dq, qp = _out(on, dq, "dq", (hc, dim), f32)
    dk, kp = _out(on, dk, "dk", (hc, dim), f32)
    _ws, wp, wn = on.workspace(workspace, _t.engram_gate_output_backward_workspace_bytes(T, hc, dim))
    _check(lib().engram_gate_output_backward_ckpt(
        *c, on.ptr(q_weight, "q_weight", bf), on.ptr(k_weight, "k_weight", bf), float(eps), on.ptr(dot, "dot", f32),
        gp, mp, xp, kvp, qp, kp, wp, wn, T, hc, dim, on.handle))
    return dx, dkv, dq, dk


__all__ = ["GateCheckpoint", "engram_mx4_quant", "engram_mx4_weight_bytes", "engram_mx4_pack_weight", "engram_wkv_mx4",
           "engram_wkv_mx4_gate", "engram_ckpt_save", "engram_ckpt_load", "engram_gate_output_ckpt",
           "engram_gate_output_backward_ckpt"]
