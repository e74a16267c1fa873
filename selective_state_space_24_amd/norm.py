"""Python binding of layer norm (``include/ssm_norm.h``): argument marshalling only.

x, y and their gradients are bfloat16 or float32 tensors of any number of dimensions, normalised
over the last; weight, bias, the statistics and the parameter gradients are float32. As with the scan,
the calls record no autograd graph: ``layer_norm_bwd`` is called for the gradients.
"""
from __future__ import annotations

import ctypes

from . import _abi


class NormDesc(ctypes.Structure):
    """Mirror of ``ssm_norm_desc``."""
    _fields_ = [("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("io_dtype", ctypes.c_int32),
                ("reserved", ctypes.c_int32), ("x_stride", ctypes.c_int64),
                ("y_stride", ctypes.c_int64), ("dx_stride", ctypes.c_int64)]


_lib = None


def _norm_lib():
    global _lib
    if _lib is None:
        h = _abi.lib()
        vp, sz, f = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_float
        dp = ctypes.POINTER(NormDesc)
        h.ssm_norm_desc_init_contiguous.argtypes = [dp, ctypes.c_int64, ctypes.c_int64, ctypes.c_int32]
        h.ssm_layer_norm_fwd.argtypes = [dp, vp, vp, vp, f, vp, vp, vp, vp]
        h.ssm_layer_norm_bwd_workspace_size.argtypes = [dp, ctypes.POINTER(sz)]
        h.ssm_layer_norm_bwd.argtypes = [dp] + [vp] * 9 + [sz, vp]
        for fn in (h.ssm_norm_desc_init_contiguous, h.ssm_layer_norm_fwd,
                   h.ssm_layer_norm_bwd_workspace_size, h.ssm_layer_norm_bwd):
            fn.restype = ctypes.c_int
        _lib = h
    return _lib


def norm_desc_contiguous(rows, cols, io_dtype=_abi.SSM_DTYPE_BF16) -> NormDesc:
    d = NormDesc()
    _abi.check(_norm_lib().ssm_norm_desc_init_contiguous(ctypes.byref(d), rows, cols, io_dtype),
               "ssm_norm_desc_init_contiguous")
    return d


def layer_norm_fwd_raw(desc, x, weight, bias, eps, y, mean, rstd, stream) -> int:
    """Direct call of ``ssm_layer_norm_fwd`` with integer device addresses (or None); returns the
    status without raising."""
    return int(_norm_lib().ssm_layer_norm_fwd(ctypes.byref(desc), x, weight, bias, eps, y, mean,
                                              rstd, stream))


def layer_norm_bwd_workspace_size(desc: NormDesc) -> int:
    out = ctypes.c_size_t(0)
    _abi.check(_norm_lib().ssm_layer_norm_bwd_workspace_size(ctypes.byref(desc), ctypes.byref(out)),
               "ssm_layer_norm_bwd_workspace_size")
    return int(out.value)


def layer_norm_bwd_raw(desc, dy, x, weight, mean, rstd, dx, dweight, dbias, workspace,
                       workspace_bytes, stream) -> int:
    """Direct call of ``ssm_layer_norm_bwd``; returns the status without raising."""
    return int(_norm_lib().ssm_layer_norm_bwd(ctypes.byref(desc), dy, x, weight, mean, rstd, dx,
                                              dweight, dbias, workspace, int(workspace_bytes),
                                              stream))


# ---------------------------------------------------------------------------------------------
# torch front end

def _row_stride(name, t, rows, cols) -> int:
    """The stride between the rows of t seen as (rows, cols)."""
    if t.dim() == 2:
        st = t.stride()
        if cols > 1 and st[1] != 1:
            raise ValueError(f"{name} must have unit stride along its last dimension")
        return st[0] if rows > 1 else cols
    if t.is_contiguous():
        return cols
    try:
        return _row_stride(name, t.view(rows, cols), rows, cols)
    except RuntimeError:
        raise ValueError(f"{name} cannot be seen as rows of one stride; make it contiguous") from None


def _shape(x):
    if x.dim() == 0 or x.shape[-1] == 0:
        raise ValueError("x must have a last dimension to normalise over")
    cols = x.shape[-1]
    return x.numel() // cols, cols


def layer_norm_fwd(x, weight=None, bias=None, eps: float = 1e-5, *, stats: bool = False, out=None,
                   stream=None):
    """Layer norm of x over its last dimension. ``weight`` and ``bias`` default to ones and zeros.
    ``out`` receives y if given. With ``stats`` returns (y, mean, rstd), what ``layer_norm_bwd``
    takes, float32 of shape x.shape[:-1]."""
    torch = _abi.torch()
    rows, cols = _shape(x)
    io = _abi.io_dtype("x", x)
    for name, t in (("weight", weight), ("bias", bias)):
        if t is not None:
            _abi.check_f32(name, t, (cols,), x.device)
    if out is not None and (out.dtype != x.dtype or out.shape != x.shape or out.device != x.device):
        raise ValueError("out must have the shape, dtype and device of x")
    with _abi.launch(x, stream) as sp:
        y = out if out is not None else torch.empty_like(x, memory_format=torch.contiguous_format)
        mean = rstd = None
        if stats:
            mean = (torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
                    if weight is None else weight.new_empty(x.shape[:-1]))
            rstd = torch.empty_like(mean)
        desc = NormDesc(rows, cols, io, 0, _row_stride("x", x, rows, cols),
                        _row_stride("out", y, rows, cols) if out is not None else cols, cols)
        _abi.check(layer_norm_fwd_raw(desc, x.data_ptr(), _abi.ptr(weight), _abi.ptr(bias), eps,
                                      y.data_ptr(), _abi.ptr(mean), _abi.ptr(rstd), sp),
                   "ssm_layer_norm_fwd")
    return (y, mean, rstd) if stats else y


def layer_norm_bwd(dy, x, weight, mean, rstd, *, params: bool = True, workspace=None, stream=None) -> dict:
    """Gradients of ``layer_norm_fwd`` from its x, weight (None: ones) and statistics: a dict of dx
    (like x, contiguous) and, with ``params``, dweight and dbias (float32). A dy that was expanded
    (stride 0) is copied first."""
    torch = _abi.torch()
    rows, cols = _shape(x)
    io = _abi.io_dtype("x", x)
    if dy.dtype != x.dtype or dy.shape != x.shape or dy.device != x.device:
        raise ValueError("dy must have the shape, dtype and device of x")
    if weight is not None:
        _abi.check_f32("weight", weight, (cols,), x.device)
    for name, t in (("mean", mean), ("rstd", rstd)):
        _abi.check_f32(name, t, x.shape[:-1], x.device)
    expanded = 0 in dy.stride()
    desc = NormDesc(rows, cols, io, 0, _row_stride("x", x, rows, cols),
                    cols if expanded else _row_stride("dy", dy, rows, cols), cols)
    need = layer_norm_bwd_workspace_size(desc) if params else 0
    with _abi.launch(x, stream) as sp:
        if expanded:
            dy = dy.contiguous()
        g = {"dx": torch.empty_like(x, memory_format=torch.contiguous_format)}
        if params:
            g["dweight"] = mean.new_empty(cols)
            g["dbias"] = mean.new_empty(cols)
        ws = _abi.workspace(workspace, need, x)
        _abi.check(layer_norm_bwd_raw(
            desc, dy.data_ptr(), x.data_ptr(), _abi.ptr(weight), mean.data_ptr(), rstd.data_ptr(),
            g["dx"].data_ptr(), _abi.ptr(g.get("dweight")), _abi.ptr(g.get("dbias")), _abi.ptr(ws),
            need, sp), "ssm_layer_norm_bwd")
    return g
