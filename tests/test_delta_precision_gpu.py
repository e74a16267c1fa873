"""bf16 calls of the gated delta rule round once: what is computed in between carries fp32's 24 bits
(needs an MI355X).

Each case is made so that a value which one product takes as an operand is 1 + 2^-10 and m 2^-23 (or
m 2^-22) more, all inputs exact in bf16 (or fp32, a state), and the rest of the sum takes the 1 and the
2^-10 away: what is left is m times a power of two, which two terms of 8 bits each do not hold. The
results fit in 8 bits, so the tolerance is one rounding of bf16, 2^-8.
"""
import pytest

from delta_cases import double, make, reference, reference_grads, rel

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
BF16 = torch.bfloat16
ONE = 2.0 ** -8
NAMES = ("q", "k", "v", "g", "beta")
M = (1, 3, 5, 15, 21, 35, 63, 105, 127, 165, 195, 231, 3, 7, 9, 255)  # of the columns of v
A, B = 3 * 2.0 ** -11, 5 * 2.0 ** -11  # their product is 15 2^-22
C, D = 2.0 ** -5, 2.0 ** -10  # C^2 and D are the middle of the value


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import selective_state_space_24_amd as ssm
    ssm.lib()  # fails loudly if the HIP library is not built


def _blank(L, dk):
    """Zeros everywhere (no writes, no decay)."""
    return {"q": torch.zeros(1, L, 1, dk), "k": torch.zeros(1, L, 1, dk),
            "v": torch.zeros(1, L, 1, len(M)), "g": torch.zeros(1, L, 1), "beta": torch.zeros(1, L, 1),
            "s0": torch.zeros(1, 1, len(M), dk)}


def _row(x, t, **at):
    for i, v in at.items():
        x[0, t, 0, int(i[1:])] = v


def _m():
    return torch.tensor(M) * 2.0 ** -23


def _state_to_y(dk):
    """Q S: entries 1 + 2^-10 + m 2^-23 and 1 + 2^-10 of the state."""
    ins = _blank(2, dk)
    ins["s0"][0, 0, :, 0] = 1 + D + _m()
    ins["s0"][0, 0, :, 1] = 1 + D
    _row(ins["q"], 1, _0=1, _1=-1)
    return ins, [1]


def _state_to_write(dk):
    """K S, read back by another entry of the key."""
    ins = _blank(2, dk)
    ins["s0"][0, 0, :, 0] = 1 + D + _m()
    ins["s0"][0, 0, :, 1] = 1 + D
    _row(ins["k"], 0, _0=1, _1=-1, _2=1)
    ins["beta"][0, 0] = 1
    _row(ins["q"], 1, _2=1)
    return ins, [1]


def _writes_of(dk, values, L=4):
    ins = _blank(L, dk)
    for t, v in enumerate(values):
        ins["v"][0, t], ins["beta"][0, t] = v, 1
    return ins


def _weights_of_writes(dk):
    """P U: q.k of 1 + 2^-10 + 15 2^-22 and 1 + 2^-10."""
    ins = _writes_of(dk, (1, -1))
    _row(ins["k"], 0, _0=1, _1=C, _2=A)
    _row(ins["k"], 1, _3=1, _4=C)
    _row(ins["q"], 3, _0=1, _1=C, _2=B, _3=1, _4=C)
    return ins, [3]


def _writes(dk):
    """P U: writes of 1, -(1 + 2^-10 + 15 2^-22) and 2^-10."""
    ins = _writes_of(dk, (1, -1, D))
    _row(ins["k"], 0, _0=1, _1=C, _2=A)
    _row(ins["k"], 1, _1=C, _2=B, _3=1)
    _row(ins["k"], 2, _4=1)
    _row(ins["q"], 3, _0=1, _3=1, _4=1)
    return ins, [3]


def _solve(dk):
    """T R: k.k of 1 + 2^-10 + 15 2^-22; the second write takes back the first, the third the 2^-10."""
    ins = _writes_of(dk, (1, 1, D))
    _row(ins["k"], 0, _0=1, _1=C, _2=A)
    _row(ins["k"], 1, _0=1, _1=C, _2=B, _3=1)
    _row(ins["k"], 2, _4=1)
    _row(ins["q"], 3, _3=1, _4=1)
    return ins, [3]


def _corrected(dk):
    """T R: what the first write puts right is 1 + 2^-10 + m 2^-23."""
    ins = _writes_of(dk, (1, 1, D))
    ins["s0"][0, 0, :, 0] = -(D + _m())
    _row(ins["k"], 0, _0=1, _1=1)
    _row(ins["k"], 1, _1=1, _2=1)
    _row(ins["k"], 2, _3=1)
    _row(ins["q"], 3, _2=1, _3=1)
    return ins, [3]


def _kept(dk, L=200, at=130):
    """K^T U, read two chunks later: writes of 1 + 2^-10 + m 2^-23, -1 and -2^-10 with keys at right
    angles."""
    ins = _writes_of(dk, (1, -1, -D), L)
    ins["s0"][0, 0, :, 0] = -(D + _m())
    _row(ins["k"], 0, _0=1, _1=1)
    _row(ins["k"], 1, _2=1)
    _row(ins["k"], 2, _3=1)
    _row(ins["q"], at, _1=1, _2=1, _3=1)
    return ins, [at]


def _kept_over_segments(dk):
    return _kept(dk, 1500, 1400)


CASES = [_state_to_y, _state_to_write, _weights_of_writes, _writes, _solve, _corrected, _kept,
         _kept_over_segments]


def _inputs(ins, heads=1):
    """The case in bf16 on the GPU, over `heads` equal heads."""
    for n in NAMES:
        assert torch.equal(ins[n].to(BF16).float(), ins[n])  # exact
    dev = {n: ins[n].to(BF16).cuda().expand(-1, -1, heads, *ins[n].shape[3:]).contiguous() for n in NAMES}
    return dev, ins["s0"].cuda().expand(-1, heads, -1, -1).contiguous()


@pytest.mark.parametrize("dk", [24, 64, 128])
@pytest.mark.parametrize("case", CASES, ids=lambda f: f.__name__[1:])
def test_forward_carries_24_bits(case, dk):
    import selective_state_space_24_amd as ssm
    ins, rows = case(dk)
    want = reference(*[ins[n].double() for n in NAMES], 1.0, ins["s0"].double())[0][:, rows]
    assert want.abs().min() > 0 and torch.equal(want.to(BF16).double(), want)
    dev, s0 = _inputs(ins, 2)
    for fin in (False, True):
        y = ssm.gated_delta_fwd(*[dev[n] for n in NAMES], 1.0, s0=s0, final_state=fin)
        y = (y[0] if fin else y)[:, rows]
        assert rel(y, want.expand_as(y)) <= ONE


SHAPES = [(1, 200, 2, 1, 128, 128), (2, 70, 4, 2, 40, 24), (64, 130, 4, 2, 128, 128),
          (1, 2100, 1, 1, 128, 40), (1, 1100, 4, 2, 64, 64)]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)))
@pytest.mark.parametrize("bits", [24, 16])
def test_y_does_not_depend_on_the_state_being_asked_for(shape, bits):
    import selective_state_space_24_amd as ssm
    ins = {n: None if t is None else t.cuda() for n, t in make(*shape, BF16, seed=3, s0=True).items()}
    a = [ins[n] for n in NAMES]
    y, _ = ssm.gated_delta_fwd(*a, 0.3, s0=ins["s0"], final_state=True, operand_bits=bits)
    assert torch.equal(y, ssm.gated_delta_fwd(*a, 0.3, s0=ins["s0"], operand_bits=bits))


@pytest.mark.parametrize("shape", SHAPES[:2] + SHAPES[3:], ids=lambda s: "-".join(map(str, s)))
def test_sixteen_bits_by_choice(shape):
    """Operands of 16 bits: y as for 24 bits (one rounding to 8 bits and 2^-12 before it); the state
    within 2^-17 of each of the values that enter a product, four products one after the other."""
    import selective_state_space_24_amd as ssm
    cpu = make(*shape, BF16, seed=4, s0=True)
    ins = {n: t.cuda() for n, t in cpu.items()}
    yr, Sr = reference(*[cpu[n].double() for n in NAMES], 0.3, cpu["s0"].double())
    y, S = ssm.gated_delta_fwd(*[ins[n] for n in NAMES], 0.3, s0=ins["s0"], final_state=True, operand_bits=16)
    assert rel(y, yr) <= 2.0 ** -8 + 2.0 ** -12
    assert rel(S, Sr) <= 4 * 2.0 ** -17


# --- the backward pass ---------------------------------------------------------------------------
# dy and ds_final beside the inputs; what is read back: a gradient's name and an index into it (after
# the batch). P0 and P1 are two columns of v.
P0, P1 = 0, 1


def _blank_grads(L, dk):
    ins = _blank(L, dk)
    return dict(ins, dy=torch.zeros_like(ins["v"]), ds=torch.zeros_like(ins["s0"]))


def _entries(dk):
    """m 2^-23 along the entries of a key but the last two."""
    m = torch.tensor(M) * 2.0 ** -23
    return torch.cat([m.repeat(dk // len(M) + 1)[:dk - 2], torch.zeros(2)])


def _read_state(dk):
    """dq = S dY."""
    ins = _blank_grads(2, dk)
    ins["s0"][0, 0, P0] = 1 + D + _entries(dk)
    ins["s0"][0, 0, P1] = 1 + D
    ins["dy"][0, 1, 0, P0], ins["dy"][0, 1, 0, P1] = 1, -1
    return ins, "dq", (1, 0, slice(0, dk - 2))


def _write_of_the_state(dk):
    """dv = beta dS k."""
    ins = _blank_grads(2, dk)
    ins["ds"][0, 0, :, 0] = 1 + D + _m()
    ins["ds"][0, 0, :, 1] = 1 + D
    _row(ins["k"], 0, _0=1, _1=-1)
    ins["beta"][0, 0] = 1
    return ins, "dv", (0, 0)


def _key_of_the_state(dk):
    """dk = dS u."""
    ins = _blank_grads(2, dk)
    ins["ds"][0, 0, P0] = 1 + D + _entries(dk)
    ins["ds"][0, 0, P1] = 1 + D
    ins["v"][0, 0, 0, P0], ins["v"][0, 0, 0, P1] = 1, -1
    ins["beta"][0, 0] = 1
    return ins, "dk", (0, 0, slice(0, dk - 2))


def _key_of_the_correction(dk):
    """dk = -S dr."""
    ins = _blank_grads(2, dk)
    ins["s0"][0, 0, P0] = 1 + D + _entries(dk)
    ins["s0"][0, 0, P1] = 1 + D
    ins["s0"][..., dk - 2:] = 0
    ins["ds"][0, 0, P0, dk - 1], ins["ds"][0, 0, P1, dk - 1] = 1, -1
    ins["k"][0, 0, 0, dk - 1] = 1
    ins["beta"][0, 0] = 1
    return ins, "dk", (0, 0, slice(0, dk - 2))


def _read_writes(dk):
    """dq = sum of E k: E of m 2^-23 from writes of 1 + 2^-10 + m 2^-23 and -(1 + 2^-10) in two columns."""
    ins = _blank_grads(3, dk)
    ins["s0"][0, 0, P0, 2], ins["s0"][0, 0, P1, 2] = -(D + 21 * 2.0 ** -23), D
    _row(ins["k"], 0, _0=1, _2=1)
    ins["beta"][0, 0] = 1
    ins["v"][0, 0, 0, P0], ins["v"][0, 0, 0, P1] = 1, -1
    ins["dy"][0, 2, 0, P0] = ins["dy"][0, 2, 0, P1] = 1
    return ins, "dq", (2, 0, 0)


def _weights_of_read_writes(dk):
    """dq = sum of E k: E of 1 + 2^-10 + m 2^-23 and -(1 + 2^-10)."""
    ins = _blank_grads(3, dk)
    ins["s0"][0, 0, P0, 2], ins["s0"][0, 0, P0, 3] = -(D + 21 * 2.0 ** -23), D
    _row(ins["k"], 0, _0=1, _1=1, _2=1)
    _row(ins["k"], 1, _0=1, _1=-1, _3=1)
    ins["beta"][0, :2] = 1
    ins["v"][0, 0, 0, P0], ins["v"][0, 1, 0, P0] = 1, -1
    ins["dy"][0, 2, 0, P0] = 1
    return ins, "dq", (2, 0, 0)


def _weights_of_reads(dk):
    """dk = sum of E q."""
    ins = _blank_grads(3, dk)
    ins["s0"][0, 0, P0, 2], ins["s0"][0, 0, P1, 2] = -(D + 21 * 2.0 ** -23), -D
    _row(ins["k"], 0, _2=1)
    ins["beta"][0, 0] = 1
    ins["v"][0, 0, 0, P0] = ins["v"][0, 0, 0, P1] = 1
    _row(ins["q"], 1, _0=1, _1=1)
    _row(ins["q"], 2, _0=1, _1=-1)
    ins["dy"][0, 1, 0, P0], ins["dy"][0, 2, 0, P1] = 1, -1
    return ins, "dk", (0, 0, 0)


def _weights_of_corrections(dk):
    """dk = sum of M k."""
    ins = _blank_grads(3, dk)
    ins["s0"][0, 0, P0, 2], ins["s0"][0, 0, P1, 2] = -(D + 21 * 2.0 ** -23), -D
    _row(ins["k"], 0, _2=1)
    _row(ins["k"], 1, _0=1, _1=1, _4=1)
    _row(ins["k"], 2, _0=1, _1=-1, _5=1)
    ins["beta"][0] = 1
    ins["v"][0, 0, 0, P0] = ins["v"][0, 0, 0, P1] = 1
    ins["ds"][0, 0, P0, 4], ins["ds"][0, 0, P1, 5] = -1, 1
    return ins, "dk", (0, 0, 0)


def _strength(dk):
    """dbeta = dr.v."""
    ins = _blank_grads(2, dk)
    ins["ds"][0, 0, P0, 0], ins["ds"][0, 0, P1, 0] = 1 + D + 21 * 2.0 ** -23, -(1 + D)
    _row(ins["k"], 0, _0=1)
    ins["beta"][0, 0] = 1
    ins["v"][0, 0, 0, P0] = ins["v"][0, 0, 0, P1] = 1
    return ins, "dbeta", (0, 0)


def _decay(dk):
    """dg = <S, dS>."""
    ins = _blank_grads(2, dk)
    ins["s0"][0, 0, P0, 0], ins["s0"][0, 0, P1, 0] = 1 + D + 21 * 2.0 ** -23, 1 + D
    ins["ds"][0, 0, P0, 0], ins["ds"][0, 0, P1, 0] = 1, -1
    return ins, "dg", (0, 0)


def _passed_back(dk, L=200, at=150):
    """dS <- dS - k dr, read chunks before: dr of 1 + 2^-10 + m 2^-23 beside an entry of 1 + 2^-10."""
    ins = _blank_grads(L, dk)
    ins["ds"][0, 0, :, 0], ins["ds"][0, 0, :, 1] = 1 + D, _m()
    _row(ins["k"], at, _0=1, _1=1)
    _row(ins["k"], 0, _0=1)
    ins["beta"][0, 0] = ins["beta"][0, at] = 1
    return ins, "dv", (0, 0)


def _passed_back_over_segments(dk):
    return _passed_back(dk, 1500, 1400)


GRAD_CASES = [_read_state, _write_of_the_state, _key_of_the_state, _key_of_the_correction, _read_writes,
              _weights_of_read_writes, _weights_of_reads, _weights_of_corrections, _strength, _decay,
              _passed_back, _passed_back_over_segments]


@pytest.mark.parametrize("dk", [24, 64, 128])
@pytest.mark.parametrize("case", GRAD_CASES, ids=lambda f: f.__name__[1:])
def test_backward_carries_24_bits(case, dk):
    import selective_state_space_24_amd as ssm
    ins, name, at = case(dk)
    wide = {n: ins[n].double() for n in NAMES + ("s0",)}
    want = reference_grads(wide, 1.0, ins["dy"].double(), ins["ds"].double())[name][(0,) + at]
    assert want.abs().min() > 0 and torch.equal(want.to(BF16).double(), want)
    dev, s0 = _inputs(ins)
    dy, ds = ins["dy"].to(BF16).cuda(), ins["ds"].cuda()
    for ds0 in (False, True):
        got = ssm.gated_delta_bwd(*[dev[n] for n in NAMES], dy, 1.0, s0=s0, ds_final=ds, want_ds0=ds0)
        assert rel(got[name][(0,) + at], want) <= ONE


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)))
@pytest.mark.parametrize("bits", [24, 16])
def test_gradients_do_not_depend_on_the_states_being_asked_for(shape, bits):
    import selective_state_space_24_amd as ssm
    ins = {n: t.cuda() for n, t in make(*shape, BF16, seed=5, s0=True).items()}
    a = [ins[n] for n in NAMES]
    dy = torch.randn(ins["v"].shape, device="cuda", generator=torch.Generator("cuda").manual_seed(6)).to(BF16)
    one = ssm.gated_delta_bwd(*a, dy, 0.3, s0=ins["s0"], operand_bits=bits)
    two = ssm.gated_delta_bwd(*a, dy, 0.3, s0=ins["s0"], want_ds0=True, operand_bits=bits)
    assert all(torch.equal(one[n], two[n]) for n in one)


@pytest.mark.parametrize("shape", SHAPES[:2] + SHAPES[3:], ids=lambda s: "-".join(map(str, s)))
def test_sixteen_bits_by_choice_in_the_backward_pass(shape):
    """One rounding to 8 bits and 2^-12 before it, 8 times that for dg, a sum over the later steps of a
    chunk; ds0 as the state in the forward pass."""
    import selective_state_space_24_amd as ssm
    cpu = make(*shape, BF16, seed=7, s0=True)
    ins = {n: t.cuda() for n, t in cpu.items()}
    gen = torch.Generator().manual_seed(8)
    dy = torch.randn(cpu["v"].shape, generator=gen).to(BF16)
    ds = torch.randn(cpu["s0"].shape, generator=gen)
    want = reference_grads(double(cpu), 0.3, dy.double(), ds.double())
    got = ssm.gated_delta_bwd(*[ins[n] for n in NAMES], dy.cuda(), 0.3, s0=ins["s0"], ds_final=ds.cuda(),
                              want_ds0=True, operand_bits=16)
    for n in want:
        bound = 4 * 2.0 ** -17 if n == "ds0" else 2.0 ** -8 + (8 if n == "dg" else 1) * 2.0 ** -12
        assert rel(got[n], want[n]) <= bound, n
