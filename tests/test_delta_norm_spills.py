"""Spills of the gated delta rule's and layer norm's kernels, read from the built library (CPU only):
none, but for the kernels below, which are held to what they have. The fp32 scan with keys of 128 and
128 columns of v a workgroup is faster so than in workgroups of half the columns; layer norm's backward
pass over rows of more than 8192 entries keeps two sums an entry beside the row, which do not fit the
128 registers that sixteen wavefronts leave a lane."""
import pytest

from test_kernel_resources import _kernel_metadata

SPILLS = {  # mangled-name fragment: VGPRs, bytes of scratch a lane
    "delta_scan_kernelINS_5delta3F32ELi4ELi8ELNS0_4ModeE0E": (7, 32),
    "norm_bwd_kernelItLi8ELi2ELi16E": (66, 148),
    "norm_bwd_kernelIfLi4ELi4ELi16E": (96, 188),
    "norm_bwd_kernelItLi1ELi16ELi16E": (119, 280),
    "norm_bwd_kernelIfLi1ELi16ELi16E": (105, 224),
}


@pytest.fixture(scope="module")
def kernels():
    return {n: k for n, k in _kernel_metadata().items()
            if any(x in n for x in ("12_GLOBAL__N_117delta_", "12_GLOBAL__N_118delta_",
                                    "12_GLOBAL__N_119delta_", "12_GLOBAL__N_120delta_",
                                    "norm_fwd_kernel", "norm_bwd_"))}


def test_known_spills(kernels):
    for frag, (vgprs, scratch) in SPILLS.items():
        hits = [k for n, k in kernels.items() if frag in n]
        assert len(hits) == 1, frag
        assert hits[0]["spill"] <= vgprs and hits[0]["scratch"] <= scratch, frag


def test_no_other_spills(kernels):
    assert len(kernels) > 100
    assert not [n for n, k in kernels.items()
                if (k["spill"] or k["scratch"]) and not any(f in n for f in SPILLS)]
