"""The gated delta rule and layer norm on the host: every declared symbol is exported, bad
arguments are refused before the GPU is touched, and the reference the GPU tests use is itself
checked (against a closed form and against differences)."""
import ctypes
import os
import re

import pytest
import torch

import selective_state_space_24_amd as ssm
from delta_cases import double, make, reference, reference_grads

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

if not os.path.exists(ssm.LIB_PATH):
    from selective_state_space_24_amd import build as _b
    _b.build()

GB = 1 << 30
FAKE = 1 << 40  # never dereferenced: every call below fails validation first


@pytest.mark.parametrize("header", ["ssm_delta.h", "ssm_norm.h"])
def test_exports_every_declared_symbol(header):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", header)).read(), flags=re.S)
    names = set(re.findall(r"^\s*int\s+(ssm_\w+)\s*\(", text, re.M))
    assert len(names) >= 4
    lib = ctypes.CDLL(ssm.LIB_PATH)
    for n in names:
        assert hasattr(lib, n), n


def test_descriptor_sizes_match_the_headers():
    assert ctypes.sizeof(ssm.DeltaDesc) == 6 * 8 + 2 * 4 + 18 * 8
    assert ctypes.sizeof(ssm.NormDesc) == 2 * 8 + 2 * 4 + 3 * 8


def _at(n):
    return FAKE + n * GB


DELTA_IN = {"q": _at(0), "k": _at(1), "v": _at(2), "g": _at(3), "beta": _at(4)}


def _fwd(d, ws=_at(8), wsb=1 << 40, s0=None, y=_at(6), s_final=None, **over):
    a = dict(DELTA_IN, **over)
    return ssm.gated_delta_fwd_raw(d, a["q"], a["k"], a["v"], a["g"], a["beta"], 0.1, s0, y,
                                   s_final, ws, wsb, None)


def _bwd(d, ws=_at(20), wsb=1 << 45, dy=_at(5), **over):
    a = dict(DELTA_IN, dq=_at(10), dk=_at(11), dv=_at(12), dg=_at(13), dbeta=_at(14), ds0=None,
             s0=None, ds_final=None)
    a.update(over)
    return ssm.gated_delta_bwd_raw(d, a["q"], a["k"], a["v"], a["g"], a["beta"], 0.1, a["s0"], dy,
                                   a["ds_final"], a["dq"], a["dk"], a["dv"], a["dg"], a["dbeta"],
                                   a["ds0"], ws, wsb, None)


def _desc(**over):
    d = ssm.delta_desc_contiguous(2, 100, 8, 4, 64, 48)
    for n, v in over.items():
        setattr(d, n, v)
    return d


@pytest.mark.parametrize("call", [_fwd, _bwd], ids=["fwd", "bwd"])
@pytest.mark.parametrize("over,status", [
    (dict(batch=-1), -2), (dict(seqlen=-1), -2), (dict(nheads=0), -2), (dict(ngroups=0), -2),
    (dict(ngroups=3), -2), (dict(dstate=0), -2), (dict(dstate=129), -2), (dict(headdim=0), -2),
    (dict(seqlen=1 << 61), -2), (dict(io_dtype=2), -3), (dict(v_stride_step=-1), -4),
    (dict(y_stride_head=47), -4), (dict(y_stride_step=0), -4), (dict(q_stride_batch=1 << 62), -2),
], ids=str)
def test_delta_refuses_bad_descriptors(call, over, status):
    d = _desc(**over)
    assert call(d) == status


def test_delta_refuses_more_workgroups_than_a_launch_takes():
    d = ssm.delta_desc_contiguous(1 << 19, 1, 1 << 13, 1 << 13, 1, 1)
    room = {n: (i + 1) << 50 for i, n in enumerate(
        ("q", "k", "v", "g", "beta", "y", "dy", "dq", "dk", "dv", "dg", "dbeta", "ws"))}
    inputs = {n: room[n] for n in DELTA_IN}
    assert _fwd(d, y=room["y"], ws=room["ws"], wsb=1 << 62, **inputs) == -9
    grads = {n: room[n] for n in ("dy", "dq", "dk", "dv", "dg", "dbeta")}
    assert _bwd(d, ws=room["ws"], wsb=1 << 62, **grads, **inputs) == -9


def test_delta_refuses_bad_buffers():
    d = _desc()
    for n in DELTA_IN:
        assert _fwd(d, **{n: None}) == -1
        assert _bwd(d, **{n: None}) == -1
        assert _fwd(d, **{n: _at(30) + 1}) == -5
    assert _fwd(d, y=None) == -1
    for n in ("dy", "dq", "dk", "dv", "dg", "dbeta"):
        assert _bwd(d, **{n: None}) == -1
    need = ssm.gated_delta_workspace_size(d)
    assert need > 0 and need % 16 == 0
    assert _fwd(d, ws=None) == -7
    assert _fwd(d, wsb=need - 1) == -7
    assert _fwd(d, ws=_at(8) + 8) == -5
    assert _fwd(d, s0=_at(7) + 2) == -5
    assert _fwd(d, y=_at(2) + 64) == -6           # y over v
    assert _fwd(d, s_final=_at(6)) == -6          # state over y
    assert _fwd(d, s0=_at(7), s_final=_at(7)) == -6
    assert _fwd(d, ws=_at(4)) == -6               # workspace over beta
    need = ssm.gated_delta_bwd_workspace_size(d)
    assert _bwd(d, wsb=need - 1) == -7
    assert _bwd(d, dq=_at(11) + 64) == -6         # dq over dk
    assert _bwd(d, dv=_at(5)) == -6               # dv over dy
    assert _bwd(d, ds_final=_at(15), ds0=_at(15)) == -6
    assert _bwd(d, dg=_at(13) + 1) == -5


def test_workspace_sizes():
    for batch, L in ((0, 100), (2, 0), (0, 0)):
        d = ssm.delta_desc_contiguous(batch, L, 8, 4, 64, 48)
        assert ssm.gated_delta_workspace_size(d) == 0
        assert ssm.gated_delta_bwd_workspace_size(d) == 0
    sizes = [ssm.gated_delta_workspace_size(ssm.delta_desc_contiguous(2, n, 8, 4, 64, 48))
             for n in (1, 64, 65, 1000, 100000)]
    assert sizes[0] == sizes[1] and sorted(sizes) == sizes and sizes[1] < sizes[2]


def test_delta_update_refusals():
    d = ssm.delta_desc_contiguous(2, 1, 8, 4, 64, 48)

    def step(d, state=_at(7), y=_at(6), **over):
        a = dict(DELTA_IN, **over)
        return ssm.gated_delta_update_raw(d, state, a["q"], a["k"], a["v"], a["g"], a["beta"], 0.1,
                                          y, None)

    assert step(_desc()) == -2                    # more than one step
    assert step(d, state=None) == -1
    assert step(d, k=None) == -1
    assert step(d, state=_at(7) + 2) == -5
    assert step(d, y=_at(7) + 64) == -6
    assert step(d, state=_at(2)) == -6
    d.dstate = 200
    assert step(d) == -2


def test_norm_refusals():
    def fwd(d, x=_at(0), w=_at(1), b=_at(2), eps=1e-5, y=_at(3), mean=_at(4), rstd=_at(5)):
        return ssm.layer_norm_fwd_raw(d, x, w, b, eps, y, mean, rstd, None)

    def bwd(d, dy=_at(0), x=_at(1), w=_at(2), mean=_at(3), rstd=_at(4), dx=_at(5), dw=_at(6),
            db=_at(7), ws=_at(8), wsb=1 << 40):
        return ssm.layer_norm_bwd_raw(d, dy, x, w, mean, rstd, dx, dw, db, ws, wsb, None)

    def desc(**over):
        d = ssm.norm_desc_contiguous(10, 100)
        for n, v in over.items():
            setattr(d, n, v)
        return d

    for call in (fwd, bwd):
        assert call(desc(rows=-1)) == -2
        assert call(desc(cols=0)) == -2
        assert call(desc(cols=16385)) == -9
        assert call(desc(io_dtype=5)) == -3
        assert call(desc(x_stride=-1)) == -4
        assert call(desc(rows=1 << 40, x_stride=1 << 40)) == -2
        assert call(desc(), x=None) == -1
        assert call(desc(), x=_at(9) + 1) == -5
    assert fwd(desc(y_stride=99)) == -4
    assert fwd(desc(), eps=-1.0) == -2
    assert fwd(desc(), eps=float("nan")) == -2
    assert fwd(desc(), y=None) == -1
    assert fwd(desc(), y=_at(0)) == -6
    assert fwd(desc(), rstd=_at(4)) == -6
    assert bwd(desc(dx_stride=99)) == -4
    assert bwd(desc(), dx=None) == -1
    assert bwd(desc(), rstd=None) == -1
    assert bwd(desc(), ws=None) == -7
    assert bwd(desc(), wsb=ssm.layer_norm_bwd_workspace_size(desc()) - 1) == -7
    assert bwd(desc(), dx=_at(1) + 64) == -6
    assert bwd(desc(), db=_at(6)) == -6


def test_python_refuses_what_does_not_fit():
    ins = make(2, 10, 4, 2, 16, 8, torch.float32)
    args = [ins[n] for n in ("q", "k", "v", "g", "beta")]
    with pytest.raises(ValueError, match="GPU"):
        ssm.gated_delta_fwd(*args)
    with pytest.raises(TypeError, match="k has dtype"):
        ssm.gated_delta_fwd(args[0], args[1].bfloat16(), *args[2:])
    with pytest.raises(TypeError, match="bfloat16 or float32"):
        ssm.gated_delta_fwd(*[t.half() for t in args])
    with pytest.raises(ValueError, match="beta must be"):
        ssm.gated_delta_fwd(*args[:4], args[4][:, :9])
    with pytest.raises(ValueError, match="unit stride"):
        ssm.gated_delta_fwd(torch.empty(2, 10, 2, 32)[..., ::2], *args[1:])
    with pytest.raises(TypeError, match="s0 must be"):
        ssm.gated_delta_fwd(*args, s0=torch.zeros(2, 4, 16, 8))
    with pytest.raises(ssm.ScanError) as e:
        ssm.gated_delta_workspace_size(_desc(dstate=129))
    assert e.value.status == -2
    with pytest.raises(ValueError, match="expected q"):
        ssm.gated_delta_update(torch.zeros(2, 4, 8, 16), *args)
    with pytest.raises(TypeError, match="weight must be"):
        ssm.layer_norm_fwd(torch.zeros(3, 8), torch.zeros(9))
    with pytest.raises(ValueError, match="last dimension"):
        ssm.layer_norm_fwd(torch.zeros(3, 0))
    with pytest.raises(ValueError, match="one stride"):
        ssm.layer_norm_bwd(torch.zeros(3, 3, 8), torch.zeros(3, 4, 16)[:, :3, :8], None,
                           torch.zeros(3, 3), torch.zeros(3, 3))


def test_reference_closed_forms():
    """Without decay and with beta 1 and orthonormal keys the state is the table sum v_t k_t^T; a
    key written again replaces what was there."""
    L, d = 8, 8
    k = torch.eye(d, dtype=torch.float64)[None, :, None]
    v = torch.arange(L * 3, dtype=torch.float64).reshape(1, L, 1, 3)
    z = torch.zeros(1, L, 1, dtype=torch.float64)
    y, S = reference(k, k, v, z, z + 1, 1.0)
    assert torch.allclose(y, v) and torch.allclose(S[0, 0], v[0, :, 0].T)
    same = k[:, :1].expand(1, L, 1, d)
    y, S = reference(same, same, v, z, z + 1, 1.0)
    assert torch.allclose(y, v) and torch.allclose(S[0, 0, :, 0], v[0, -1, 0])


@pytest.mark.parametrize("name", ["q", "k", "v", "g", "beta", "s0"])
def test_reference_gradients_against_differences(name):
    ins = double(make(1, 9, 4, 2, 5, 3, torch.float32, seed=3, s0=True))
    gen = torch.Generator().manual_seed(4)
    dy = torch.randn(1, 9, 4, 3, generator=gen, dtype=torch.float64)
    ds = torch.randn(1, 4, 3, 5, generator=gen, dtype=torch.float64)
    d = torch.randn(ins[name].shape, generator=gen, dtype=torch.float64)
    got = float((reference_grads(ins, 0.4, dy, ds)["d" + name] * d).sum())

    def loss(e):
        moved = dict(ins, **{name: ins[name] + e * d})
        y, S = reference(moved["q"], moved["k"], moved["v"], moved["g"], moved["beta"], 0.4,
                         moved["s0"])
        return float((y * dy).sum() + (S * ds).sum())

    e = 1e-5  # error of a central difference: e^2 f''' / 6 + 1e-16 f / e, both about 1e-10
    assert abs((loss(e) - loss(-e)) / (2 * e) - got) <= 1e-7 * max(1.0, abs(got))


@pytest.mark.parametrize("call", [_fwd, _bwd], ids=["fwd", "bwd"])
def test_delta_refuses_operands_that_do_not_exist(call):
    assert call(_desc(operands=2)) == -3
    assert call(_desc(operands=-1)) == -3
    assert call(_desc(operands=ssm.SSM_DELTA_OPERANDS_16), ws=None) == -7
    with pytest.raises(ValueError, match="operand_bits"):
        ins = make(2, 10, 4, 2, 16, 8, torch.float32)
        ssm.gated_delta_fwd(*[ins[n] for n in ("q", "k", "v", "g", "beta")], operand_bits=32)


def test_backward_refuses_operand_bits_that_do_not_exist():
    ins = make(2, 10, 4, 2, 16, 8, torch.float32)
    with pytest.raises(ValueError, match="operand_bits"):
        ssm.gated_delta_bwd(*[ins[n] for n in ("q", "k", "v", "g", "beta")], ins["v"], operand_bits=8)


def test_delta_refuses_launches_past_32_bits_of_threads():
    """A launch's threads along a dimension are a 32-bit number: 2^24 workgroups of 512, 2^26 of 64."""
    names = ("q", "k", "v", "g", "beta", "y", "dy", "dq", "dk", "dv", "dg", "dbeta", "ws", "state")
    room = {n: (i + 1) << 50 for i, n in enumerate(names)}
    inputs = {n: room[n] for n in DELTA_IN}
    grads = {n: room[n] for n in ("dy", "dq", "dk", "dv", "dg", "dbeta")}
    d = ssm.delta_desc_contiguous(1 << 12, 1, 1 << 12, 1 << 12, 1, 65)  # 2^24 heads, eight wavefronts each
    assert _fwd(d, y=room["y"], ws=room["ws"], wsb=1 << 62, **inputs) == -9
    assert _bwd(d, ws=room["ws"], wsb=1 << 62, **grads, **inputs) == -9
    d = ssm.delta_desc_contiguous(1 << 12, 1, 1 << 11, 1 << 11, 1, 1)  # scans of half as many; gradients not
    assert _bwd(d, ws=room["ws"], wsb=1 << 62, **grads, **inputs) == -9
    d = ssm.delta_desc_contiguous(1, (1 << 30) + 1, 1, 1, 1, 1)  # 2^24 chunks and one
    assert _fwd(d, y=room["y"], ws=room["ws"], wsb=1 << 62, **inputs) == -9
    d = ssm.delta_desc_contiguous(1 << 14, 1, 1 << 13, 1 << 13, 1, 1)
    assert ssm.gated_delta_update_raw(d, room["state"], *[room[n] for n in DELTA_IN], 0.1, room["y"], None) == -9


@pytest.mark.parametrize("seqlen", [1 << 40, 1 << 50, (1 << 54) - 65, (1 << 54) + 64, 1 << 55])
@pytest.mark.parametrize("dtype", [0, 1])
def test_delta_workspace_sizes_do_not_wrap(seqlen, dtype):
    """Either the size that is needed (the records of the chunks alone take over 200 bytes a step) or a
    refusal."""
    d = ssm.delta_desc_contiguous(1, seqlen, 1, 1, 1, 1, dtype)
    for size in (ssm.gated_delta_workspace_size, ssm.gated_delta_bwd_workspace_size):
        try:
            assert size(d) >= 200 * seqlen
        except ssm.ScanError as e:
            assert e.status == -2


def test_python_names_the_tensor_that_does_not_fit():
    ins = make(2, 10, 4, 2, 16, 8, torch.float32)
    args = [ins[n] for n in ("q", "k", "v", "g", "beta")]
    v = ins["v"]
    wide = torch.empty(2, 10, 4, 16)[..., ::2]
    with pytest.raises(TypeError, match="^dy has dtype"):
        ssm.gated_delta_bwd(*args, v.bfloat16())
    with pytest.raises(ValueError, match="^dy must be"):
        ssm.gated_delta_bwd(*args, v[:, :9])
    with pytest.raises(ValueError, match="^dy must have unit stride"):
        ssm.gated_delta_bwd(*args, wide)
    with pytest.raises(TypeError, match="^out has dtype"):
        ssm.gated_delta_fwd(*args, out=v.bfloat16())
    with pytest.raises(ValueError, match="^out must have unit stride"):
        ssm.gated_delta_fwd(*args, out=wide)
    one = [t[:, 0] for t in args]
    with pytest.raises(ValueError, match="^out must be"):
        ssm.gated_delta_update(torch.zeros(2, 4, 8, 16), *one, out=v[:, 0, :, :4])
