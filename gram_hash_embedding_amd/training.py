"""The gradients that train the Engram module and its embeddings: the ctypes binding of libengram.so's training entry
points (include/engram.h), under the same rules as the rest of the package -- GPU tensors in, dtype / shape /
contiguity checked, no fallback.

    engram_embed           -- rows of a trainable table by id, scaled
    engram_embed_grad      -- its gradient, a row per table row
    engram_embed_grad_rows -- its gradient as the distinct rows (hashed tables)
    engram_gate_output_backward -- the gradient of engram_gate_output
    engram_wkv_backward    -- the gradient of engram_wkv
    engram_grad_norm       -- the 2-norm of many gradients together
    engram_clip_grads      -- every gradient times min(1, max_norm / (norm + 1e-6))

Outputs and workspaces that are not given are allocated on the stream the call runs on, so that the caching allocator
does not hand their memory on before that stream is done with it.
"""
from __future__ import annotations

import contextlib
import ctypes

from . import _check, _dev, lib

BF16, F32 = 0, 1  # ENGRAM_BF16, ENGRAM_F32


def declare(L: ctypes.CDLL) -> None:
    """Argument and result types of the training entry points."""
    i64, i32, p, f32 = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p, ctypes.c_float
    L.engram_embed.argtypes = [p, i32, i64, p, i32, i64, i64, i32, f32, p, i32, p]
    L.engram_embed_grad.argtypes = [p, i32, i64, i64, i32, p, i32, i64, i64, i32, f32, p, i32, i32, p, i64, p]
    L.engram_embed_grad_rows.argtypes = [p, i32, i64, i64, i32, p, i32, i64, i64, i32, f32, p, p, i32, p, p, i64, p]
    L.engram_embed_grad_workspace_bytes.argtypes = [i64, i32, i64]
    L.engram_gate_output_backward.argtypes = [p, p, i64, p, p, f32, p, p, p, p, p, p, p, p, i64, i64, i32, i32, p]
    L.engram_gate_output_backward_workspace_bytes.argtypes = [i64, i32, i32]
    L.engram_wkv_backward.argtypes = [p, p, p, p, p, i32, i32, p, i64, i64, i32, i32, p]
    L.engram_wkv_backward_workspace_bytes.argtypes = [i64, i32, i32]
    L.engram_grad_norm.argtypes = [i32, p, p, p, p, p, i64, p]
    L.engram_grad_norm_workspace_bytes.argtypes = [i32, p, p]
    L.engram_clip_grads.argtypes = [i32, p, p, p, p, p, f32, p]
    for f in (L.engram_embed_grad_workspace_bytes, L.engram_gate_output_backward_workspace_bytes,
              L.engram_wkv_backward_workspace_bytes, L.engram_grad_norm_workspace_bytes):
        f.restype = i64


class _On:
    """The call's stream: `handle` for the C side, `empty` for what the call allocates."""

    def __init__(self, stream):
        import torch

        self.torch = torch
        self.current = torch.cuda.current_stream()
        self.stream = self.current if stream is None else stream
        self.other = stream is not None and stream.cuda_stream != self.current.cuda_stream
        self.handle = ctypes.c_void_p(self.stream.cuda_stream)

    def empty(self, shape, dtype, device, keep=True):
        """An uninitialised tensor of the call's stream; `keep`: the caller gets it (and may use it on its own)."""
        if not self.other:
            return self.torch.empty(shape, dtype=dtype, device=device)
        with self.torch.cuda.stream(self.stream):
            t = self.torch.empty(shape, dtype=dtype, device=device)
        if keep:
            t.record_stream(self.current)
        return t


def _float_type(dtype, name):
    import torch

    if dtype == torch.bfloat16:
        return BF16
    if dtype == torch.float32:
        return F32
    raise TypeError(f"{name} must be bfloat16 or float32, got {dtype}")


def _any_float(t, name, ndim=None):
    """(pointer, element type) of a contiguous bf16 or float32 GPU tensor."""
    return _dev(t, name, t.dtype, ndim), _float_type(t.dtype, name)


def _ids(ids):
    import torch

    if ids.dtype not in (torch.int64, torch.int32):
        raise TypeError(f"ids must be int64 or int32, got {ids.dtype}")
    return _dev(ids, "ids", ids.dtype), ids.element_size()


def engram_embed(ids, table, scale=1.0, row_start=0, out=None, out_dtype=None, stream=None):
    """out [*ids.shape, D] = scale * table[ids - row_start] (zeros for ids outside the table's rows).

    ids: int64 or int32 of any shape; table: bf16 or float32 [R, D]; out in `out_dtype` (the table's by default)."""
    on = _On(stream)
    tp, td = _any_float(table, "table", 2)
    ip, ib = _ids(ids)
    R, D = table.shape
    if out is None:
        out = on.empty((*ids.shape, D), table.dtype if out_dtype is None else out_dtype, ids.device)
    elif tuple(out.shape) != (*ids.shape, D) or (out_dtype is not None and out.dtype != out_dtype):
        raise ValueError("out must be [*ids.shape, D] of out_dtype")
    op, od = _any_float(out, "out")
    _check(lib().engram_embed(ip, ib, ids.numel(), tp, td, R, int(row_start), D, float(scale), op, od, on.handle))
    return out


def _lookup(ids, grad, layer):
    """(ids pointer, id bytes, T, token stride, C, D) of ids [*] with grad [*, D], or of layer `layer` of ids
    [B, L, E, C] with grad [B*L, C, D] or [B*L, C*D]."""
    ip, ib = _ids(ids)
    if layer is not None:
        if ids.dim() != 4 or not 0 <= layer < ids.shape[2]:
            raise ValueError("`layer` needs ids [B, L, E, C] with that layer")
        B, L, E, C = ids.shape
        T, stride = B * L, E * C
        ip = ctypes.c_void_p(ids.data_ptr() + ids.element_size() * layer * C)
        n = T * C
        if grad.dim() == 2 and T > 0 and grad.shape[0] == T and grad.shape[1] % C == 0 and C > 1:
            D = grad.shape[1] // C
        else:
            D = grad.shape[-1]
    else:
        T, stride, C, n, D = ids.numel(), 1, 1, ids.numel(), grad.shape[-1]
    if D < 1 or grad.numel() != n * D:
        raise ValueError(f"grad must hold a row of D elements for each of the {n} ids, got shape {tuple(grad.shape)}")
    return ip, ib, T, stride, C, n, D


def engram_embed_grad_workspace_bytes(n: int, D: int, num_rows: int) -> int:
    b = lib().engram_embed_grad_workspace_bytes(int(n), int(D), int(num_rows))
    if b < 0:
        raise ValueError(f"engram_embed_grad: n={n} D={D} num_rows={num_rows} outside the limits")
    return b


def _workspace(on, workspace, need, device):
    import torch

    if workspace is None:
        workspace = on.empty(max(need, 16), torch.uint8, device, keep=False)
    return _dev(workspace, "workspace", torch.uint8), workspace.numel()


def engram_embed_grad(ids, grad, num_rows, scale=1.0, row_start=0, layer=None, out=None, out_dtype=None, accumulate=False,
                      workspace=None, stream=None):
    """The gradient of a lookup: out [num_rows, D], row r = scale * (sum of grad's rows whose id is row_start + r).

    ids: int64 or int32 of any shape with grad [*ids.shape, D] (bf16 or float32); or engram_hash's [B, L, E, C] with
    `layer` and grad [B*L, C, D] or [B*L, C*D].  out is float32 unless `out_dtype` says bf16; with `accumulate` the sum
    is added to the given `out`, whose other rows are not touched."""
    import torch

    on = _On(stream)
    ip, ib, T, stride, C, n, D = _lookup(ids, grad, layer)
    gp, gd = _any_float(grad, "grad")
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs the out to add to")
        out = on.empty((num_rows, D), torch.float32 if out_dtype is None else out_dtype, ids.device)
    elif tuple(out.shape) != (num_rows, D) or (out_dtype is not None and out.dtype != out_dtype):
        raise ValueError("out must be [num_rows, D] of out_dtype")
    op, od = _any_float(out, "out", 2)
    wp, wn = _workspace(on, workspace, engram_embed_grad_workspace_bytes(n, D, num_rows), ids.device)
    _check(lib().engram_embed_grad(ip, ib, T, stride, C, gp, gd, int(num_rows), int(row_start), D, float(scale), op, od,
                                   int(bool(accumulate)), wp, wn, on.handle))
    return out


def engram_embed_grad_rows(ids, grad, num_rows, scale=1.0, row_start=0, layer=None, unique=None, rows=None, count=None,
                           out_dtype=None, workspace=None, stream=None):
    """The same gradient as its distinct rows: (unique int64 [n] ascending, -1 past the last; rows [n, D], zeros past
    the last; count int32 [1]), n the number of ids.  Arguments as engram_embed_grad; rows float32 unless `out_dtype`
    says bf16."""
    import torch

    on = _On(stream)
    ip, ib, T, stride, C, n, D = _lookup(ids, grad, layer)
    gp, gd = _any_float(grad, "grad")
    if unique is None:
        unique = on.empty((n,), torch.int64, ids.device)
    if rows is None:
        rows = on.empty((n, D), torch.float32 if out_dtype is None else out_dtype, ids.device)
    elif out_dtype is not None and rows.dtype != out_dtype:
        raise ValueError("rows must be of out_dtype")
    if count is None:
        count = on.empty((1,), torch.int32, ids.device)
    if tuple(unique.shape) != (n,) or tuple(rows.shape) != (n, D) or count.numel() != 1:
        raise ValueError("unique must be [n], rows [n, D] and count [1]")
    rp, rd = _any_float(rows, "rows", 2)
    wp, wn = _workspace(on, workspace, engram_embed_grad_workspace_bytes(n, D, num_rows), ids.device)
    _check(lib().engram_embed_grad_rows(ip, ib, T, stride, C, gp, gd, int(num_rows), int(row_start), D, float(scale),
                                        _dev(unique, "unique", torch.int64), rp, rd, _dev(count, "count", torch.int32),
                                        wp, wn, on.handle))
    return unique, rows, count


def engram_gate_output_backward_workspace_bytes(T: int, hc: int, dim: int) -> int:
    b = lib().engram_gate_output_backward_workspace_bytes(int(T), int(hc), int(dim))
    if b < 0:
        raise ValueError(f"engram_gate_output_backward: T={T} hc={hc} dim={dim} outside the limits")
    return b


def engram_gate_output_backward(x, kv, q_weight, k_weight, eps, dot, dout, token_mask=None, dx=None, dkv=None, dq=None,
                                dk=None, workspace=None, stream=None):
    """(dx bf16 of x's shape, dkv bf16 [T, (hc+1)*dim], dq, dk float32 [hc, dim]) from dout, the gradient of
    engram_gate_output's out (or engram_gate_residual's), and the forward's x, kv [T, >= (hc+1)*dim] and dot float32
    [T, hc]; token_mask as the forward's.  `dx` may be dout itself."""
    import torch

    on = _On(stream)
    x3 = x.reshape(-1, x.shape[-2], x.shape[-1])
    T, hc, dim = x3.shape
    if kv.dim() != 2 or kv.shape[0] != T or kv.shape[1] < (hc + 1) * dim:
        raise ValueError("kv must be [T, >= (hc+1)*dim]")
    if tuple(q_weight.shape) != (hc, dim) or tuple(k_weight.shape) != (hc, dim):
        raise ValueError("q_weight and k_weight must be [hc, dim]")
    if tuple(dot.shape) != (T, hc):
        raise ValueError("dot must be [T, hc]")
    if dout.shape != x.shape:
        raise ValueError("dout must have x's shape")
    mask_p = None
    if token_mask is not None:
        if token_mask.numel() != T:
            raise ValueError("token_mask must hold one entry per token")
        if token_mask.dtype == torch.bool:
            token_mask = token_mask.view(torch.uint8)
        mask_p = _dev(token_mask, "token_mask", torch.uint8)
    if dx is None:
        dx = on.empty(x.shape, torch.bfloat16, x.device)
    if dkv is None:
        dkv = on.empty((T, (hc + 1) * dim), torch.bfloat16, x.device)
    if dq is None:
        dq = on.empty((hc, dim), torch.float32, x.device)
    if dk is None:
        dk = on.empty((hc, dim), torch.float32, x.device)
    if dx.shape != x.shape or tuple(dkv.shape) != (T, (hc + 1) * dim):
        raise ValueError("dx must have x's shape and dkv be [T, (hc+1)*dim]")
    if tuple(dq.shape) != (hc, dim) or tuple(dk.shape) != (hc, dim):
        raise ValueError("dq and dk must be [hc, dim]")
    wp, wn = _workspace(on, workspace, engram_gate_output_backward_workspace_bytes(T, hc, dim), x.device)
    bf = torch.bfloat16
    _check(lib().engram_gate_output_backward(
        _dev(x, "x", bf), _dev(kv, "kv", bf, 2), kv.shape[1], _dev(q_weight, "q_weight", bf, 2),
        _dev(k_weight, "k_weight", bf, 2), float(eps), _dev(dot, "dot", torch.float32, 2), _dev(dout, "dout", bf), mask_p,
        _dev(dx, "dx", bf), _dev(dkv, "dkv", bf, 2), _dev(dq, "dq", torch.float32, 2), _dev(dk, "dk", torch.float32, 2),
        wp, wn, T, hc, dim, on.handle))
    return dx, dkv, dq, dk


def engram_wkv_backward_workspace_bytes(T: int, K: int, Nout: int) -> int:
    b = lib().engram_wkv_backward_workspace_bytes(int(T), int(K), int(Nout))
    if b < 0:
        raise ValueError(f"engram_wkv_backward: T={T} K={K} Nout={Nout} outside the limits")
    return b


def engram_wkv_backward(dkv, a, w, da=None, dw=None, dw_dtype=None, accumulate=False, need_da=True, need_dw=True,
                        workspace=None, stream=None):
    """(da bf16 [T, K], dw [Nout, K]) = (dkv w, dkv^T a) of bf16 dkv [T, Nout], a [T, K] (or [T, C, D]) and w [Nout, K].

    dw is float32 unless `dw_dtype` says bf16; with `accumulate` the product is added to the given `dw`.  With
    need_da / need_dw False that product is not computed (None) and the operand only it reads (w / a) may be None."""
    import torch

    on = _On(stream)
    if not (need_da or need_dw):
        raise ValueError("neither da nor dw is asked for")
    if (need_da and w is None) or (need_dw and a is None):
        raise ValueError("da needs w, dw needs a")
    bf = torch.bfloat16
    dp = _dev(dkv, "dkv", bf, 2)
    T, N = dkv.shape
    ap = wp_ = dap = dwp = None
    K = None
    if w is not None:
        wp_ = _dev(w, "w", bf, 2)
        K = w.shape[1]
        if w.shape[0] != N:
            raise ValueError(f"w must be [Nout={N}, K], got {tuple(w.shape)}")
    if a is not None:
        ap = _dev(a, "a", bf)
        Ka = a.shape[1] * a.shape[2] if a.dim() == 3 else a.shape[-1]
        if a.dim() not in (2, 3) or a.shape[0] != T or (K is not None and Ka != K):
            raise ValueError(f"a must be [T={T}, K={K}], got {tuple(a.shape)}")
        K = Ka
    if need_da:
        if da is None:
            da = on.empty((T, K), bf, dkv.device)
        if da.numel() != T * K:
            raise ValueError("da must hold T * K elements")
        dap = _dev(da, "da", bf)
    else:
        da = None
    dwt = F32
    if need_dw:
        if dw is None:
            if accumulate:
                raise ValueError("accumulate needs the dw to add to")
            dw = on.empty((N, K), torch.float32 if dw_dtype is None else dw_dtype, dkv.device)
        if tuple(dw.shape) != (N, K) or (dw_dtype is not None and dw.dtype != dw_dtype):
            raise ValueError("dw must be [Nout, K] of dw_dtype")
        dwp, dwt = _any_float(dw, "dw", 2)
    else:
        dw = None
    wsp, wsn = _workspace(on, workspace, engram_wkv_backward_workspace_bytes(T, K, N), dkv.device)
    _check(lib().engram_wkv_backward(dp, ap, wp_, dap, dwp, dwt, int(bool(accumulate)), wsp, wsn, T, K, N, on.handle))
    return da, dw


def _tensor_list(grads):
    """(count, host arrays of pointers, element counts and element types) of contiguous bf16 / float32 tensors."""
    n = len(grads)
    got = [_any_float(g, f"grads[{i}]") for i, g in enumerate(grads)]
    return (n, (ctypes.c_void_p * n)(*[p.value for p, _ in got]), (ctypes.c_int64 * n)(*[g.numel() for g in grads]),
            (ctypes.c_int32 * n)(*[d for _, d in got]))


def engram_grad_norm(grads, out=None, workspace=None, stream=None):
    """float32 [1]: the 2-norm of all elements of `grads` (a list of contiguous bf16 / float32 tensors) together."""
    import torch

    on = _On(stream)
    n, ptrs, sizes, types = _tensor_list(grads)
    if out is None:
        out = on.empty((1,), torch.float32, grads[0].device if n else "cuda")
    if out.numel() != 1:
        raise ValueError("out must hold one element")
    need = lib().engram_grad_norm_workspace_bytes(n, sizes, types)
    wp, wn = _workspace(on, workspace, need, out.device)
    _check(lib().engram_grad_norm(n, ptrs, sizes, types, _dev(out, "out", torch.float32), wp, wn, on.handle))
    return out


def engram_clip_grads(grads, norm, max_norm, outs=None, stream=None):
    """Every gradient times min(1, max_norm / (norm + 1e-6)): into `outs` (tensors of the gradients' types and sizes), or
    in place.  `norm`: float32 [1] on the GPU (engram_grad_norm's).  Returns the clipped tensors."""
    import torch

    on = _On(stream)
    n, ptrs, sizes, types = _tensor_list(grads)
    if outs is None:
        outs, optrs = grads, ptrs
    else:
        if len(outs) != n or any(o.dtype != g.dtype or o.numel() != g.numel() for o, g in zip(outs, grads)):
            raise ValueError("outs must match grads in number, types and sizes")
        optrs = (ctypes.c_void_p * n)(*[_dev(o, f"outs[{i}]", o.dtype).value for i, o in enumerate(outs)])
    if norm.numel() != 1:
        raise ValueError("norm must hold one element")
    _check(lib().engram_clip_grads(n, ptrs, optrs, sizes, types, _dev(norm, "norm", torch.float32), float(max_norm),
                                   on.handle))
    return outs


__all__ = ["engram_embed", "engram_embed_grad", "engram_embed_grad_rows", "engram_embed_grad_workspace_bytes",
           "engram_gate_output_backward", "engram_gate_output_backward_workspace_bytes", "engram_wkv_backward",
           "engram_wkv_backward_workspace_bytes", "engram_grad_norm", "engram_clip_grads"]
