"""The gradient of the decays of heads that forget fast (needs an MI355X).

With every g at -10 a head's dg is e^-10 of the products it is made of, in each of its terms: what
the terms without that factor add and take away again must not stay behind as their rounding. dg is
compared head by head, since slow heads beside fast ones would hide them in one norm. The tolerances
are those of the backward pass for any decay: fp32 3.4e-6, 8 times that for dg, a sum over the later
steps of a chunk; bf16 one rounding to 8 bits and 8 times 2^-12.
"""
import pytest

from delta_cases import double, make, reference_grads, rel

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
NAMES = ("q", "k", "v", "g", "beta")
BOUND = {torch.float32: 8 * 3.4e-6, torch.bfloat16: 2.0 ** -8 + 8 * 2.0 ** -12}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import selective_state_space_24_amd as ssm
    ssm.lib()  # fails loudly if the HIP library is not built


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape", [(1, 64, 2, 2, 32, 32), (2, 150, 4, 2, 128, 64), (1, 37, 2, 1, 64, 40)],
                         ids=lambda s: "-".join(map(str, s)))
def test_gradient_of_strong_decays(shape, dtype):
    import selective_state_space_24_amd as ssm
    cpu = make(*shape, dtype, seed=shape[1], s0=True)
    cpu["g"][:, :, 0] = -10.0  # the other heads keep their slow decays
    cpu["g"][:, :, 1] = -6.0
    gen = torch.Generator().manual_seed(1)
    dy = torch.randn(cpu["v"].shape, generator=gen).to(dtype)
    ds = torch.randn(cpu["s0"].shape, generator=gen)
    want = reference_grads(double(cpu), 0.3, dy.double(), ds.double())["dg"]
    got = ssm.gated_delta_bwd(*[cpu[n].cuda() for n in NAMES], dy.cuda(), 0.3, s0=cpu["s0"].cuda(),
                              ds_final=ds.cuda())["dg"]
    off = [rel(got[:, :, h], want[:, :, h]) for h in range(shape[2])]
    print(" ".join(f"{e:.1e}" for e in off), flush=True)
    assert max(off) <= BOUND[dtype]
