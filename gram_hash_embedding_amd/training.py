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

import ctypes

from . import _check, lib

torch = None  # imported by the first call, as in the rest of the package
_current_device = _raw_stream = None


def _load():
    global torch, _current_device, _raw_stream
    import torch as t

    torch = t
    _current_device, _raw_stream = t._C._cuda_getDevice, t._C._cuda_getCurrentRawStream


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
    """Where a call runs: the device of its tensors (which has to be the current one) and its stream.  At the smallest
    sizes this binding is most of a call's time, so it asks for the raw stream and passes plain integers."""

    __slots__ = ("index", "handle", "side")

    def __init__(self, stream, like=None, name="tensor"):
        if torch is None:
            _load()
        if like is None:
            self.index = torch.cuda.current_device()
        else:
            if not isinstance(like, torch.Tensor):
                raise TypeError(f"{name} must be a torch.Tensor")
            if not like.is_cuda:
                raise ValueError(f"{name} must be a GPU tensor")
            self.index = like.get_device()
            if self.index != _current_device():
                raise ValueError(f"{name} is on GPU {self.index}, the current device is {torch.cuda.current_device()}")
        current = _raw_stream(self.index)
        self.handle, self.side = current, None
        if stream is not None and stream.cuda_stream != current:
            self.handle, self.side = stream.cuda_stream, stream

    def ptr(self, t, name, dtype, ndim=None):
        """Address of a contiguous tensor of the call's device."""
        try:
            if (t.dtype is dtype and t.get_device() == self.index and t.is_contiguous() and
                    (ndim is None or t.dim() == ndim)):
                return t.data_ptr()
        except AttributeError:  # no tensor
            pass
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if not t.is_cuda:
            raise ValueError(f"{name} must be a GPU tensor")
        if t.dtype is not dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
        if t.get_device() != self.index:
            raise ValueError(f"{name} is on GPU {t.get_device()}, the call runs on GPU {self.index}")
        if ndim is not None and t.dim() != ndim:
            raise ValueError(f"{name} must have {ndim} dims, got shape {tuple(t.shape)}")
        raise ValueError(f"{name} must be contiguous")

    def real(self, t, name, ndim=None):
        """(address, element type) of a contiguous bf16 or float32 tensor."""
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        kind = BF16 if t.dtype is torch.bfloat16 else F32
        if kind == F32 and t.dtype is not torch.float32:
            raise TypeError(f"{name} must be bfloat16 or float32, got {t.dtype}")
        return self.ptr(t, name, t.dtype, ndim), kind

    def ids(self, ids):
        """(address, bytes per id)."""
        if not isinstance(ids, torch.Tensor) or ids.dtype not in (torch.int64, torch.int32):
            raise TypeError("ids must be an int64 or int32 tensor")
        return self.ptr(ids, "ids", ids.dtype), ids.element_size()

    def empty(self, shape, dtype, keep=True):
        """An uninitialised tensor of the call's stream; `keep`: the caller gets it (and may use it on its own)."""
        if self.side is None:
            return torch.empty(shape, dtype=dtype, device=self.index)
        with torch.cuda.stream(self.side):
            t = torch.empty(shape, dtype=dtype, device=self.index)
        if keep:
            t.record_stream(torch.cuda.current_stream())
        return t

    def workspace(self, given, need):
        """(tensor, address, bytes) of the call's scratch; (None, None, 0) where it needs none and none is given."""
        if given is None:
            if need == 0:
                return None, None, 0
            given = self.empty(need, torch.uint8, keep=False)
            return given, given.data_ptr(), need
        return given, self.ptr(given, "workspace", torch.uint8), given.numel()


def engram_embed(ids, table, scale=1.0, row_start=0, out=None, out_dtype=None, stream=None):
    """out [*ids.shape, D] = scale * table[ids - row_start] (zeros for ids outside the table's rows).

    ids: int64 or int32 of any shape; table: bf16 or float32 [R, D]; out in `out_dtype` (the table's by default)."""
    on = _On(stream, table, "table")
    tp, td = on.real(table, "table", 2)
    ip, ib = on.ids(ids)
    R, D = table.shape
    if out is None:
        out = on.empty((*ids.shape, D), table.dtype if out_dtype is None else out_dtype)
    elif tuple(out.shape) != (*ids.shape, D) or (out_dtype is not None and out.dtype != out_dtype):
        raise ValueError("out must be [*ids.shape, D] of out_dtype")
    op, od = on.real(out, "out")
    _check(lib().engram_embed(ip, ib, ids.numel(), tp, td, R, int(row_start), D, float(scale), op, od, on.handle))
    return out


def _lookup(on, ids, grad, layer):
    """(ids pointer, id bytes, T, token stride, C, D) of ids [*] with grad [*, D], or of layer `layer` of ids
    [B, L, E, C] with grad [B*L, C, D] or [B*L, C*D]."""
    ip, ib = on.ids(ids)
    if layer is not None:
        if ids.dim() != 4 or not 0 <= layer < ids.shape[2]:
            raise ValueError("`layer` needs ids [B, L, E, C] with that layer")
        B, L, E, C = ids.shape
        T, stride = B * L, E * C
        ip += ib * layer * C
        n = T * C
        if grad.dim() == 2 and grad.shape[0] == T and grad.shape[1] % C == 0:
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


def engram_embed_grad(ids, grad, num_rows, scale=1.0, row_start=0, layer=None, out=None, out_dtype=None, accumulate=False,
                      workspace=None, stream=None):
    """The gradient of a lookup: out [num_rows, D], row r = scale * (sum of grad's rows whose id is row_start + r).

    ids: int64 or int32 of any shape with grad [*ids.shape, D] (bf16 or float32); or engram_hash's [B, L, E, C] with
    `layer` and grad [B*L, C, D] or [B*L, C*D].  out is float32 unless `out_dtype` says bf16; with `accumulate` the sum
    is added to the given `out`, whose other rows are not touched."""
    on = _On(stream, grad, "grad")
    ip, ib, T, stride, C, n, D = _lookup(on, ids, grad, layer)
    gp, gd = on.real(grad, "grad")
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs the out to add to")
        out = on.empty((num_rows, D), torch.float32 if out_dtype is None else out_dtype)
    elif tuple(out.shape) != (num_rows, D) or (out_dtype is not None and out.dtype != out_dtype):
        raise ValueError("out must be [num_rows, D] of out_dtype")
    op, od = on.real(out, "out", 2)
    _ws, wp, wn = on.workspace(workspace, engram_embed_grad_workspace_bytes(n, D, num_rows))
    _check(lib().engram_embed_grad(ip, ib, T, stride, C, gp, gd, int(num_rows), int(row_start), D, float(scale), op, od,
                                   int(bool(accumulate)), wp, wn, on.handle))
    return out


def engram_embed_grad_rows(ids, grad, num_rows, scale=1.0, row_start=0, layer=None, unique=None, rows=None, count=None,
                           out_dtype=None, workspace=None, stream=None):
    """The same gradient as its distinct rows: (unique int64 [n] ascending, -1 past the last; rows [n, D], zeros past
    the last; count int32 [1]), n the number of ids.  Arguments as engram_embed_grad; rows float32 unless `out_dtype`
    says bf16."""
    on = _On(stream, grad, "grad")
    ip, ib, T, stride, C, n, D = _lookup(on, ids, grad, layer)
    gp, gd = on.real(grad, "grad")
    if unique is None:
        unique = on.empty((n,), torch.int64)
    if rows is None:
        rows = on.empty((n, D), torch.float32 if out_dtype is None else out_dtype)
    elif out_dtype is not None and rows.dtype != out_dtype:
        raise ValueError("rows must be of out_dtype")
    if count is None:
        count = on.empty((1,), torch.int32)
    if tuple(unique.shape) != (n,) or tuple(rows.shape) != (n, D) or count.numel() != 1:
        raise ValueError("unique must be [n], rows [n, D] and count [1]")
    rp, rd = on.real(rows, "rows", 2)
    _ws, wp, wn = on.workspace(workspace, engram_embed_grad_workspace_bytes(n, D, num_rows))
    _check(lib().engram_embed_grad_rows(ip, ib, T, stride, C, gp, gd, int(num_rows), int(row_start), D, float(scale),
                                        on.ptr(unique, "unique", torch.int64), rp, rd, on.ptr(count, "count", torch.int32),
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
    on = _On(stream, x, "x")
    if x.dim() < 3:
        raise ValueError("x must be [T, hc, dim] (or [B, L, hc, dim])")
    hc, dim = x.shape[-2:]
    T = x.numel() // (hc * dim) if hc * dim else 0
    if kv.dim() != 2 or kv.shape[0] != T or kv.shape[1] < (hc + 1) * dim:
        raise ValueError("kv must be [T, >= (hc+1)*dim]")
    if q_weight.shape != (hc, dim) or k_weight.shape != (hc, dim):
        raise ValueError("q_weight and k_weight must be [hc, dim]")
    if dot.shape != (T, hc):
        raise ValueError("dot must be [T, hc]")
    if dout.shape != x.shape:
        raise ValueError("dout must have x's shape")
    mask_p = None
    if token_mask is not None:
        if token_mask.numel() != T:
            raise ValueError("token_mask must hold one entry per token")
        if token_mask.dtype == torch.bool:
            token_mask = token_mask.view(torch.uint8)
        mask_p = on.ptr(token_mask, "token_mask", torch.uint8)
    need = engram_gate_output_backward_workspace_bytes(T, hc, dim)
    bf, f32 = torch.bfloat16, torch.float32
    if dx is None:
        dx = on.empty(x.shape, bf)
    elif dx.shape != x.shape:
        raise ValueError("dx must have x's shape")
    if dkv is None:
        dkv = on.empty((T, (hc + 1) * dim), bf)
    elif dkv.shape != (T, (hc + 1) * dim):
        raise ValueError("dkv must be [T, (hc+1)*dim]")
    if dq is None:
        dq = on.empty((hc, dim), f32)
    if dk is None:
        dk = on.empty((hc, dim), f32)
    if dq.shape != (hc, dim) or dk.shape != (hc, dim):
        raise ValueError("dq and dk must be [hc, dim]")
    _ws, wp, wn = on.workspace(workspace, need)
    _check(lib().engram_gate_output_backward(
        on.ptr(x, "x", bf), on.ptr(kv, "kv", bf, 2), kv.shape[1], on.ptr(q_weight, "q_weight", bf, 2),
        on.ptr(k_weight, "k_weight", bf, 2), float(eps), on.ptr(dot, "dot", f32, 2), on.ptr(dout, "dout", bf), mask_p,
        on.ptr(dx, "dx", bf), on.ptr(dkv, "dkv", bf, 2), on.ptr(dq, "dq", f32, 2), on.ptr(dk, "dk", f32, 2),
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
    on = _On(stream, dkv, "dkv")
    if not (need_da or need_dw):
        raise ValueError("neither da nor dw is asked for")
    if (need_da and w is None) or (need_dw and a is None):
        raise ValueError("da needs w, dw needs a")
    bf = torch.bfloat16
    dp = on.ptr(dkv, "dkv", bf, 2)
    T, N = dkv.shape
    ap = wp = dap = dwp = K = None
    if w is not None:
        wp = on.ptr(w, "w", bf, 2)
        if w.shape[0] != N:
            raise ValueError(f"w must be [Nout={N}, K], got {tuple(w.shape)}")
        K = w.shape[1]
    if a is not None:
        ap = on.ptr(a, "a", bf)
        Ka = a.shape[1] * a.shape[2] if a.dim() == 3 else a.shape[-1]
        if a.dim() not in (2, 3) or a.shape[0] != T or (K is not None and Ka != K):
            raise ValueError(f"a must be [T={T}, K={K}], got {tuple(a.shape)}")
        K = Ka
    need = engram_wkv_backward_workspace_bytes(T, K, N)
    if not need_da:
        da = None
    else:
        if da is None:
            da = on.empty((T, K), bf)
        elif da.numel() != T * K:
            raise ValueError("da must hold T * K elements")
        dap = on.ptr(da, "da", bf)
    kind = F32
    if not need_dw:
        dw = None
    else:
        if dw is None:
            if accumulate:
                raise ValueError("accumulate needs the dw to add to")
            dw = on.empty((N, K), torch.float32 if dw_dtype is None else dw_dtype)
        elif dw.shape != (N, K) or (dw_dtype is not None and dw.dtype != dw_dtype):
            raise ValueError("dw must be [Nout, K] of dw_dtype")
        dwp, kind = on.real(dw, "dw", 2)
    _ws, sp, sn = on.workspace(workspace, need)
    _check(lib().engram_wkv_backward(dp, ap, wp, dap, dwp, kind, int(bool(accumulate)), sp, sn, T, K, N, on.handle))
    return da, dw


def _tensor_list(on, grads, name):
    """(count, host arrays of addresses, element counts and element types) of contiguous bf16 / float32 tensors."""
    n, index, bf16, fp32 = len(grads), on.index, torch.bfloat16, torch.float32
    ptrs, sizes, types = (ctypes.c_void_p * n)(), (ctypes.c_int64 * n)(), (ctypes.c_int32 * n)()
    for i, g in enumerate(grads):
        if not isinstance(g, torch.Tensor) or g.get_device() != index or not g.is_contiguous() or (
                g.dtype is not bf16 and g.dtype is not fp32):
            on.real(g, f"{name}[{i}]")  # says what is wrong
        ptrs[i], sizes[i], types[i] = g.data_ptr(), g.numel(), BF16 if g.dtype is bf16 else F32
    return n, ptrs, sizes, types


def engram_grad_norm(grads, out=None, workspace=None, stream=None):
    """float32 [1]: the 2-norm of all elements of `grads` (a list of contiguous bf16 / float32 tensors) together."""
    on = _On(stream, grads[0] if len(grads) else None, "grads[0]")
    n, ptrs, sizes, types = _tensor_list(on, grads, "grads")
    if out is None:
        out = on.empty((1,), torch.float32)
    elif out.numel() != 1:
        raise ValueError("out must hold one element")
    _ws, wp, wn = on.workspace(workspace, lib().engram_grad_norm_workspace_bytes(n, sizes, types))
    _check(lib().engram_grad_norm(n, ptrs, sizes, types, on.ptr(out, "out", torch.float32), wp, wn, on.handle))
    return out


def engram_clip_grads(grads, norm, max_norm, outs=None, stream=None):
    """Every gradient times min(1, max_norm / (norm + 1e-6)): into `outs` (tensors of the gradients' types and sizes), or
    in place.  `norm`: float32 [1] on the GPU (engram_grad_norm's).  Returns the clipped tensors."""
    on = _On(stream, norm, "norm")
    n, ptrs, sizes, types = _tensor_list(on, grads, "grads")
    if outs is None:
        outs, optrs = grads, ptrs
    else:
        m, optrs, osizes, otypes = _tensor_list(on, outs, "outs")
        if m != n or bytes(osizes) != bytes(sizes) or bytes(otypes) != bytes(types):
            raise ValueError("outs must match grads in number, types and sizes")
    if norm.numel() != 1:
        raise ValueError("norm must hold one element")
    _check(lib().engram_clip_grads(n, ptrs, optrs, sizes, types, on.ptr(norm, "norm", torch.float32), float(max_norm),
                                   on.handle))
    return outs


__all__ = ["engram_embed", "engram_embed_grad", "engram_embed_grad_rows", "engram_embed_grad_workspace_bytes",
           "engram_gate_output_backward", "engram_gate_output_backward_workspace_bytes", "engram_wkv_backward",
           "engram_wkv_backward_workspace_bytes", "engram_grad_norm", "engram_clip_grads"]
