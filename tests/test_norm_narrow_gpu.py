"""Layer norm of narrow rows, every output (needs an MI355X). Tolerances as for wider rows: fp32 sums
and a few products, 2e-6 of the 2-norm, 4e-6 for sums over rows; bf16 one rounding, 2^-8, and 2^-16
before it; dx, whose terms cancel in such rows, against the size of its terms."""
import pytest

from delta_cases import rel

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
OUT = {torch.bfloat16: 2.0 ** -8 + 2.0 ** -16, torch.float32: 2e-6}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import selective_state_space_24_amd as ssm
    ssm.lib()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape", [(5, 2), (200, 2), (5, 3), (7, 4), (3, 5)], ids=lambda s: "-".join(map(str, s)))
def test_every_output_of_narrow_rows(shape, dtype):
    import selective_state_space_24_amd as ssm
    gen = torch.Generator(device="cuda").manual_seed(shape[1])
    r = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    x, w, b, dy = (2 * r(*shape) + 0.5).to(dtype), 1 + 0.3 * r(shape[1]), r(shape[1]), r(*shape).to(dtype)
    eps = 1e-3
    y, mean, rstd = ssm.layer_norm_fwd(x, w, b, eps, stats=True)
    xd, wd, bd, d = (t.double().cpu() for t in (x, w, b, dy))
    mr = xd.mean(-1, keepdim=True)
    rr = 1 / ((xd - mr).square().mean(-1, keepdim=True) + eps).sqrt()
    assert rel(y, (xd - mr) * rr * wd + bd) <= OUT[dtype]
    assert float((mean.double().cpu() - mr[:, 0]).abs().max()) <= 1e-6 * float(xd.square().mean().sqrt())
    assert rel(rstd, rr[:, 0]) <= 2e-6
    got = ssm.layer_norm_bwd(dy, x, w, mean, rstd)
    m, s = mean.double().cpu()[:, None], rstd.double().cpu()[:, None]  # the statistics that were passed
    xh, h = (xd - m) * s, d * wd
    dx = s * (h - h.mean(1, keepdim=True) - xh * (h * xh).mean(1, keepdim=True))
    assert float((got["dx"].double().cpu() - dx).norm()) <= OUT[dtype] * float((s * h).norm())
    assert rel(got["dweight"], (d * xh).sum(0)) <= 4e-6
    assert rel(got["dbias"], d.sum(0)) <= 4e-6
