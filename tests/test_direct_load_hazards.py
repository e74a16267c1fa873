"""Wait states before the direct loads into LDS, read from the built library (CPU only).

A direct load takes its LDS base from M0, and gfx9 wants one wait state between a scalar write of M0
and the load; where the load's address is a scalar pair written by a vector instruction (a
v_readfirstlane), five. The compiler puts them in for its own loads. The kernels' loads are inline
assembly, which it does not look into, so that the assembly itself has to hold them. An instruction
between the two counts as one wait state, ``s_nop n`` as n + 1.
"""
import os
import re
import subprocess

import pytest

import selective_state_space_24_amd as ssm
from test_kernel_resources import LLVM


def _disassembly(tmp):
    for t in ("llvm-objcopy", "clang-offload-bundler", "llvm-objdump"):
        if not os.path.exists(os.path.join(LLVM, t)):
            pytest.skip(f"{t} not found under {LLVM}")
    if not os.path.exists(ssm.LIB_PATH):
        pytest.skip("library not built")
    fat = os.path.join(tmp, "fatbin.bin")
    subprocess.run([os.path.join(LLVM, "llvm-objcopy"), f"--dump-section=.hip_fatbin={fat}",
                    ssm.LIB_PATH, os.path.join(tmp, "copy.so")], check=True)
    data = open(fat, "rb").read()
    at = [m.start() for m in re.finditer(b"__CLANG_OFFLOAD_BUNDLE__", data)] + [len(data)]
    text = []
    for i in range(len(at) - 1):
        part, co = os.path.join(tmp, f"{i}.bin"), os.path.join(tmp, f"{i}.co")
        with open(part, "wb") as f:
            f.write(data[at[i]:at[i + 1]])
        subprocess.run([os.path.join(LLVM, "clang-offload-bundler"), "--type=o",
                        "--targets=hipv4-amdgcn-amd-amdhsa--gfx950", f"--input={part}",
                        f"--output={co}", "--unbundle"], check=True)
        text.append(subprocess.run([os.path.join(LLVM, "llvm-objdump"), "-d", "--no-show-raw-insn", co],
                                   capture_output=True, text=True, check=True).stdout)
    return "\n".join(text)


def _scalars(operand):
    """The numbers of the scalar registers an operand names."""
    m = re.fullmatch(r"s\[(\d+):(\d+)\]", operand) or re.fullmatch(r"s(\d+)()", operand)
    return set(range(int(m[1]), int(m[2] or m[1]) + 1)) if m else set()


def _faults(text):
    """kernel -> [direct loads, those too near M0's write, those too near their address's]."""
    found, kernel, past = {}, None, []
    for line in text.splitlines():
        head = re.match(r"[0-9a-f]+ <(\S+)>:", line)
        if head:
            kernel, past = head[1], []
            continue
        code = line.split("//")[0].strip()
        if kernel is None or not line.startswith(("\t", " ")) or not code:
            continue
        op, _, rest = code.partition(" ")
        args = [a.strip() for a in rest.split(",")]
        if re.match(r"(global|scratch)_load_lds_", op) or (op.startswith("buffer_load") and re.search(r"\blds\b", rest)):
            count = found.setdefault(kernel, [0, 0, 0])
            count[0] += 1
            base = set().union(*(_scalars(a.split()[0]) for a in args if a))
            states = 0
            for before, to in reversed(past):
                if before.startswith("s_") and "m0" in to[:1] and states < 1:
                    count[1] += 1
                if before.startswith("v_") and base & set().union(*(_scalars(a) for a in to[:2])) and states < 5:
                    count[2] += 1
                states += 1 + (int(to[0], 0) if before == "s_nop" else 0)
                if states >= 5:
                    break
        past = past[-8:] + [(op, args)]
    return found


@pytest.fixture(scope="module")
def found(tmp_path_factory):
    return _faults(_disassembly(str(tmp_path_factory.mktemp("co"))))


@pytest.mark.parametrize("kernel", ["delta_scan_kernel", "delta_combine_kernel", "delta_back_kernel",
                                    "delta_grad_kernel"])
def test_direct_loads_of_the_gated_delta_rule(found, kernel):
    hits = {k: v for k, v in found.items() if kernel in k}
    assert hits and all(n[0] > 0 for n in hits.values())
    assert not {k: n for k, n in hits.items() if n[1] or n[2]}


def test_direct_loads_of_the_chunked_scan(found):
    hits = {k: v for k, v in found.items() if "ssd_fwd_kernel" in k}
    assert hits and all(n[0] > 0 for n in hits.values())
    assert not {k: n for k, n in hits.items() if n[1] or n[2]}


def test_the_check_itself():
    lines = ["0 <k>:", "\ts_mov_b32 m0, s4", "\tglobal_load_lds_dwordx4 v[0:1], off",
             "\ts_mov_b32 m0, s4", "\ts_nop 0", "\tglobal_load_lds_dwordx4 v[0:1], off",
             "\tv_readfirstlane_b32 s7, v3", "\ts_mov_b32 m0, s4", "\ts_nop 2",
             "\tglobal_load_lds_dwordx4 v0, s[6:7]", "\tv_readfirstlane_b32 s7, v3",
             "\ts_mov_b32 m0, s4", "\ts_nop 3", "\tglobal_load_lds_dwordx4 v0, s[6:7]"]
    assert _faults("\n".join(lines)) == {"k": [4, 1, 1]}
