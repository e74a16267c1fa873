"""Python binding of the gated delta rule (``include/ssm_delta.h``): argument marshalling only.

Tensors: q, k (batch, L, ngroups, dstate); v, y (batch, L, nheads, headdim); g, beta
(batch, L, nheads), all bfloat16 or all float32, any strides with a unit innermost one. States are
(batch, nheads, headdim, dstate) float32, contiguous. As with the scan, the calls record no autograd
graph: ``gated_delta_bwd`` is called for the gradients.
"""
from __future__ import annotations

import ctypes
from typing import Optional

from . import _abi

SSM_DELTA_MAX_DSTATE = 128
SSM_DELTA_OPERANDS_24, SSM_DELTA_OPERANDS_16 = 0, 1


class DeltaDesc(ctypes.Structure):
    """Mirror of ``ssm_delta_desc``."""
    _fields_ = ([(n, ctypes.c_int64) for n in
                 ("batch", "seqlen", "nheads", "ngroups", "dstate", "headdim")]
                + [("io_dtype", ctypes.c_int32), ("operands", ctypes.c_int32)]
                + [(f"{t}_stride_{d}", ctypes.c_int64) for t, inner in
                   (("q", "group"), ("k", "group"), ("v", "head"), ("g", "head"),
                    ("beta", "head"), ("y", "head")) for d in ("batch", "step", inner)])


_lib = None


def _delta_lib():
    global _lib
    if _lib is None:
        h = _abi.lib()
        vp, i64, sz, f = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
        dp, szp = ctypes.POINTER(DeltaDesc), ctypes.POINTER(ctypes.c_size_t)
        h.ssm_delta_desc_init_contiguous.argtypes = [dp] + [i64] * 6 + [ctypes.c_int32]
        h.ssm_gated_delta_workspace_size.argtypes = [dp, szp]
        h.ssm_gated_delta_fwd.argtypes = [dp] + [vp] * 5 + [f] + [vp] * 4 + [sz, vp]
        h.ssm_gated_delta_update.argtypes = [dp] + [vp] * 6 + [f, vp, vp]
        h.ssm_gated_delta_bwd_workspace_size.argtypes = [dp, szp]
        h.ssm_gated_delta_bwd.argtypes = [dp] + [vp] * 5 + [f] + [vp] * 10 + [sz, vp]
        for fn in (h.ssm_delta_desc_init_contiguous, h.ssm_gated_delta_workspace_size,
                   h.ssm_gated_delta_fwd, h.ssm_gated_delta_update,
                   h.ssm_gated_delta_bwd_workspace_size, h.ssm_gated_delta_bwd):
            fn.restype = ctypes.c_int
        _lib = h
    return _lib


def delta_desc_contiguous(batch, seqlen, nheads, ngroups, dstate, headdim,
                          io_dtype=_abi.SSM_DTYPE_BF16) -> DeltaDesc:
    d = DeltaDesc()
    _abi.check(_delta_lib().ssm_delta_desc_init_contiguous(
        ctypes.byref(d), batch, seqlen, nheads, ngroups, dstate, headdim, io_dtype),
        "ssm_delta_desc_init_contiguous")
    return d


def gated_delta_workspace_size(desc: DeltaDesc) -> int:
    out = ctypes.c_size_t(0)
    _abi.check(_delta_lib().ssm_gated_delta_workspace_size(ctypes.byref(desc), ctypes.byref(out)),
               "ssm_gated_delta_workspace_size")
    return int(out.value)


def gated_delta_fwd_raw(desc, q, k, v, g, beta, scale, s0, y, s_final, workspace, workspace_bytes,
                        stream) -> int:
    """Direct call of ``ssm_gated_delta_fwd`` with integer device addresses (or None); returns the
    status without raising."""
    return int(_delta_lib().ssm_gated_delta_fwd(ctypes.byref(desc), q, k, v, g, beta, scale, s0, y,
                                                s_final, workspace, int(workspace_bytes), stream))


def gated_delta_update_raw(desc, state, q, k, v, g, beta, scale, y, stream) -> int:
    """Direct call of ``ssm_gated_delta_update``; returns the status without raising."""
    return int(_delta_lib().ssm_gated_delta_update(ctypes.byref(desc), state, q, k, v, g, beta,
                                                   scale, y, stream))


def gated_delta_bwd_workspace_size(desc: DeltaDesc) -> int:
    out = ctypes.c_size_t(0)
    _abi.check(_delta_lib().ssm_gated_delta_bwd_workspace_size(ctypes.byref(desc),
                                                               ctypes.byref(out)),
               "ssm_gated_delta_bwd_workspace_size")
    return int(out.value)


def gated_delta_bwd_raw(desc, q, k, v, g, beta, scale, s0, dy, ds_final, dq, dk, dv, dg, dbeta,
                        ds0, workspace, workspace_bytes, stream) -> int:
    """Direct call of ``ssm_gated_delta_bwd``; returns the status without raising."""
    return int(_delta_lib().ssm_gated_delta_bwd(
        ctypes.byref(desc), q, k, v, g, beta, scale, s0, dy, ds_final, dq, dk, dv, dg, dbeta, ds0,
        workspace, int(workspace_bytes), stream))


# ---------------------------------------------------------------------------------------------
# torch front end

def _check_like(v, keys, values, steps, q, k, g, beta, y, y_name):
    """Raises for the first tensor that has not v's dtype and device and its shape."""
    for name, t, shape in (("q", q, keys), ("k", k, keys), ("g", g, steps), ("beta", beta, steps),
                           (y_name, y, values)):
        if t is None:
            continue
        if t.dtype != v.dtype:
            raise TypeError(f"{name} has dtype {t.dtype}, expected {v.dtype}")
        if t.shape != shape:
            raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
        if t.device != v.device:
            raise ValueError(f"{name} is on {t.device}, v on {v.device}")


def _alike(v, keys, steps, q, k, g, beta):
    """What _check_like looks at, in one expression: it is most of a short call's time."""
    dt, dev = v.dtype, v.get_device()
    return (q.dtype is dt and k.dtype is dt and g.dtype is dt and beta.dtype is dt
            and q.shape == keys and k.shape == keys and g.shape == steps and beta.shape == steps
            and q.get_device() == dev and k.get_device() == dev and g.get_device() == dev
            and beta.get_device() == dev)


def _unit(name, st, n):
    if n > 1 and st[-1] != 1:
        raise ValueError(f"{name} must have unit stride along its last dimension")


def describe_delta(q, k, v, g, beta, y=None, y_name: str = "y") -> DeltaDesc:
    """Descriptor of torch tensors (shapes as in the module's docstring); ``y_name`` is what an error
    calls y."""
    if v.dim() != 4 or q.dim() != 4:
        raise ValueError("expected q, k (batch, L, ngroups, dstate) and v (batch, L, nheads, headdim)")
    batch, L, nheads, dv = values = v.shape
    groups, dk = q.shape[2:]
    io = _abi.io_dtype("v", v)
    keys, steps = (batch, L, groups, dk), (batch, L, nheads)
    if y is not None or not _alike(v, keys, steps, q, k, g, beta):
        _check_like(v, keys, values, steps, q, k, g, beta, y, y_name)
    qs, ks, vs = q.stride(), k.stride(), v.stride()
    ys = y.stride() if y is not None else (L * nheads * dv, nheads * dv, dv, 1)
    if qs[3] != 1 or ks[3] != 1 or vs[3] != 1 or ys[3] != 1:
        for name, st, n in (("q", qs, dk), ("k", ks, dk), ("v", vs, dv), (y_name, ys, dv)):
            _unit(name, st, n)
    return DeltaDesc(batch, L, nheads, groups, dk, dv, io, 0, *qs[:3], *ks[:3], *vs[:3],
                     *g.stride(), *beta.stride(), *ys[:3])


def describe_delta_step(q, k, v, g, beta, y=None, y_name: str = "y") -> DeltaDesc:
    """Descriptor (seqlen 1) of one step: q, k (batch, ngroups, dstate), v, y (batch, nheads,
    headdim), g, beta (batch, nheads)."""
    if v.dim() != 3 or q.dim() != 3:
        raise ValueError("expected q, k (batch, ngroups, dstate) and v (batch, nheads, headdim)")
    batch, nheads, dv = values = v.shape
    groups, dk = q.shape[1:]
    io = _abi.io_dtype("v", v)
    keys, steps = (batch, groups, dk), (batch, nheads)
    if y is not None or not _alike(v, keys, steps, q, k, g, beta):
        _check_like(v, keys, values, steps, q, k, g, beta, y, y_name)
    (qb, qg, q1), (kb, kg, k1), (vb, vh, v1) = q.stride(), k.stride(), v.stride()
    yb, yh, y1 = y.stride() if y is not None else (nheads * dv, dv, 1)
    if q1 != 1 or k1 != 1 or v1 != 1 or y1 != 1:
        for name, st, n in (("q", (q1,), dk), ("k", (k1,), dk), ("v", (v1,), dv), (y_name, (y1,), dv)):
            _unit(name, st, n)
    gb, gh = g.stride()
    bb, bh = beta.stride()
    return DeltaDesc(batch, 1, nheads, groups, dk, dv, io, 0, qb, 0, qg, kb, 0, kg, vb, 0, vh,
                     gb, 0, gh, bb, 0, bh, yb, 0, yh)


def _check_state(name, t, desc, device):
    _abi.check_f32(name, t, (desc.batch, desc.nheads, desc.headdim, desc.dstate), device)


def _operands(bits: int) -> int:
    if bits == 24:
        return SSM_DELTA_OPERANDS_24
    if bits == 16:
        return SSM_DELTA_OPERANDS_16
    raise ValueError(f"operand_bits must be 24 or 16, got {bits}")


def gated_delta_fwd(q, k, v, g, beta, scale: Optional[float] = None, *, s0=None, final_state=None,
                    out=None, operand_bits: int = 24, workspace=None, stream=None):
    """y of the gated delta rule, with S_t = exp(g_t) S_(t-1) + u_t k_t^T, u_t = beta_t (v_t -
    exp(g_t) S_(t-1) k_t) and y_t = scale S_t q_t.

    ``scale`` defaults to dstate ** -0.5. ``s0`` is the initial state. ``final_state`` is True
    (allocate) or a tensor that receives the state after the last step; the call then returns
    ``(y, final_state)``; y is the same either way. ``out`` receives y if given. ``operand_bits`` is
    how many bits of a value computed in fp32 enter the matrix products of a call on bfloat16 tensors:
    all 24, or 16, which is faster and leaves y before its rounding, and the states, good to about
    2^-17. ``workspace`` may be a uint8 device tensor
    of at least ``gated_delta_workspace_size`` bytes; otherwise one is allocated. ``stream``
    defaults to the current torch stream. Raises ScanError with the library's status on failure.
    """
    torch = _abi.torch()
    desc = describe_delta(q, k, v, g, beta, out, "out")
    desc.operands = _operands(operand_bits)
    if s0 is not None:
        _check_state("s0", s0, desc, v.device)
    if final_state is not None and not isinstance(final_state, bool):
        _check_state("final_state", final_state, desc, v.device)
    need = gated_delta_workspace_size(desc)
    with _abi.launch(v, stream) as sp:
        y = out if out is not None else torch.empty_like(v, memory_format=torch.contiguous_format)
        if final_state is True:
            final_state = torch.empty((desc.batch, desc.nheads, desc.headdim, desc.dstate),
                                      dtype=torch.float32, device=v.device)
        elif final_state is False:
            final_state = None
        ws = _abi.workspace(workspace, need, v)
        _abi.check(gated_delta_fwd_raw(
            desc, q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(),
            desc.dstate ** -0.5 if scale is None else scale, _abi.ptr(s0), y.data_ptr(),
            _abi.ptr(final_state), _abi.ptr(ws), need, sp), "ssm_gated_delta_fwd")
    return y if final_state is None else (y, final_state)


def gated_delta_update(state, q, k, v, g, beta, scale: Optional[float] = None, *, out=None,
                       stream=None):
    """One step per batch entry: updates ``state`` in place and returns y (batch, nheads, headdim).
    q, k are (batch, ngroups, dstate), v (batch, nheads, headdim), g and beta (batch, nheads)."""
    torch = _abi.torch()
    desc = describe_delta_step(q, k, v, g, beta, out, "out")
    _check_state("state", state, desc, v.device)
    with _abi.launch(v, stream) as sp:
        y = out if out is not None else torch.empty_like(v, memory_format=torch.contiguous_format)
        _abi.check(gated_delta_update_raw(
            desc, state.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(),
            beta.data_ptr(), desc.dstate ** -0.5 if scale is None else scale, y.data_ptr(), sp),
            "ssm_gated_delta_update")
    return y


def gated_delta_bwd(q, k, v, g, beta, dy, scale: Optional[float] = None, *, s0=None, ds_final=None,
                    want_ds0: bool = False, operand_bits: int = 24, workspace=None, stream=None) -> dict:
    """Gradients of ``gated_delta_fwd`` for dy, the gradient of y, and ``ds_final``, that of its
    final state if given. A dy that was expanded (stride 0) is copied first. Returns a dict of dq, dk
    (summed over the heads of a group), dv, dg, dbeta (the inputs' dtype, contiguous) and, with
    ``want_ds0``, ds0 (float32). ``operand_bits`` as for ``gated_delta_fwd``, for the states and the
    gradients."""
    torch = _abi.torch()
    operands = _operands(operand_bits)
    expanded = 0 in dy.stride()
    desc = describe_delta(q, k, v, g, beta, None if expanded else dy, "dy")
    for name, t in (("s0", s0), ("ds_final", ds_final)):
        if t is not None:
            _check_state(name, t, desc, v.device)
    with _abi.launch(v, stream) as sp:
        if expanded:
            dy = dy.contiguous()
            desc = describe_delta(q, k, v, g, beta, dy, "dy")
        desc.operands = operands
        need = gated_delta_bwd_workspace_size(desc)
        out = {n: torch.empty_like(t, memory_format=torch.contiguous_format) for n, t in
               (("dq", q), ("dk", k), ("dv", v), ("dg", g), ("dbeta", beta))}
        if want_ds0:
            out["ds0"] = torch.empty((desc.batch, desc.nheads, desc.headdim, desc.dstate),
                                     dtype=torch.float32, device=v.device)
        ws = _abi.workspace(workspace, need, v)
        _abi.check(gated_delta_bwd_raw(
            desc, q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(),
            desc.dstate ** -0.5 if scale is None else scale, _abi.ptr(s0), dy.data_ptr(),
            _abi.ptr(ds_final), out["dq"].data_ptr(), out["dk"].data_ptr(), out["dv"].data_ptr(),
            out["dg"].data_ptr(), out["dbeta"].data_ptr(), _abi.ptr(out.get("ds0")), _abi.ptr(ws),
            need, sp), "ssm_gated_delta_bwd")
    return out
