"""The gated delta rule where it runs in workgroups of eight wavefronts (columns of v enough for more
than four, and heads enough to fill the chip), against the recurrence in 64 bits on the GPU (needs an
MI355X).

Keys of each padded length, several chunks (so that the next chunk's operands are loaded beside the
one that is worked on), whole sequences and split ones, with and without the states, both types and
both operand widths. Tolerances are those of the narrow cases: on the 2-norm, bf16 outputs one rounding
to 8 bits and 2^-12 before it, fp32 outputs 3.4e-6, dg 8 times what stands before the rounding (a sum
over the later steps of a chunk); with 16-bit operands the states 4 products of 2^-17.
"""
import pytest

from delta_cases import double, make, reference, reference_grads, rel

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
F32 = 3.4e-6
NAMES = ("q", "k", "v", "g", "beta")
KINDS = [(torch.bfloat16, 24), (torch.bfloat16, 16), (torch.float32, 24)]
WHOLE = [  # batch, L, heads, groups, dstate, headdim
    (64, 130, 4, 2, 128, 128), (64, 200, 4, 4, 64, 72), (130, 130, 2, 1, 24, 80), (32, 150, 4, 1, 100, 200),
]
SPLIT = [(1, 2000, 32, 32, 24, 72), (1, 2000, 32, 32, 64, 80), (1, 3300, 32, 16, 128, 72)]
kind = pytest.mark.parametrize("dtype,bits", KINDS, ids=["bf16", "bf16-16", "f32"])


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import selective_state_space_24_amd as ssm
    ssm.lib()  # fails loudly if the HIP library is not built


def _bound(name, dtype, bits):
    grow = 8.0 if name == "dg" else 1.0
    if name in ("s_final", "ds0"):
        return 4 * 2.0 ** -17 if bits == 16 else F32
    return 2.0 ** -8 + grow * 2.0 ** -12 if dtype == torch.bfloat16 else grow * F32


def _inputs(shape, dtype, seed):
    ins = {n: t.cuda() for n, t in make(*shape, dtype, seed=seed, s0=True, decay=0.3).items()}
    gen = torch.Generator().manual_seed(seed + 1)
    dy = torch.randn(ins["v"].shape, generator=gen).to(dtype).cuda()
    ds = torch.randn(ins["s0"].shape, generator=gen).cuda()
    return ins, dy, ds


@kind
@pytest.mark.parametrize("shape", WHOLE + SPLIT, ids=lambda s: "-".join(map(str, s)))
def test_forward(shape, dtype, bits):
    import selective_state_space_24_amd as ssm
    ins, _, _ = _inputs(shape, dtype, shape[1])
    yr, Sr = reference(*[double(ins)[n] for n in NAMES], 0.3, ins["s0"].double())
    a = [ins[n] for n in NAMES]
    y, S = ssm.gated_delta_fwd(*a, 0.3, s0=ins["s0"], final_state=True, operand_bits=bits)
    alone = ssm.gated_delta_fwd(*a, 0.3, s0=ins["s0"], operand_bits=bits)
    off = rel(y, yr), rel(alone, yr), rel(S, Sr)
    print(" ".join(f"{e:.2e}" for e in off), flush=True)
    assert off[0] <= _bound("y", dtype, bits) and off[1] <= _bound("y", dtype, bits)
    assert off[2] <= _bound("s_final", dtype, bits)


@kind
@pytest.mark.parametrize("shape", WHOLE + SPLIT, ids=lambda s: "-".join(map(str, s)))
def test_backward(shape, dtype, bits):
    import selective_state_space_24_amd as ssm
    ins, dy, ds = _inputs(shape, dtype, shape[1] + 7)
    want = reference_grads(double(ins), 0.3, dy.double(), ds.double())
    got = ssm.gated_delta_bwd(*[ins[n] for n in NAMES], dy, 0.3, s0=ins["s0"], ds_final=ds, want_ds0=True,
                              operand_bits=bits)
    assert set(got) == set(want)
    off = {n: rel(got[n], want[n]) for n in want}
    print(" ".join(f"{n} {e:.2e}" for n, e in off.items()), flush=True)
    for n, e in off.items():
        assert e <= _bound(n, dtype, bits), n
