"""The built library's loads straight to LDS (no GPU needed): the address that such a load takes from M0
has to be written at least one wait state before it."""
import os
import re
import subprocess

import pytest

from w4a4_quantized_gemm_rudder_amd import build as b
from w4a4_quantized_gemm_rudder_amd import rudder as r

OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"


@pytest.fixture(scope="module")
def listings(tmp_path_factory):
    """The instructions of every code object in the library."""
    if not os.path.exists(OBJDUMP):
        pytest.skip("no disassembler")
    r.load_library()
    folder = tmp_path_factory.mktemp("objects")
    lib = folder / "librudder.so"
    lib.symlink_to(b.LIB_PATH)
    subprocess.run([OBJDUMP, "--offloading", str(lib)], cwd=folder, check=True,
                   capture_output=True)
    out = []
    for path in sorted(folder.glob("*amdgcn*")):
        text = subprocess.run([OBJDUMP, "-d", str(path)], check=True, capture_output=True,
                              text=True).stdout
        out.append([line.split("//")[0].strip() for line in text.splitlines()
                    if line.startswith("\t")])
    assert out
    return out


def _without_wait(instructions):
    """(loads to LDS, those right behind a scalar write of M0)"""
    writes = re.compile(r"s_(?!cmp|bitcmp|nop|waitcnt|branch|cbranch|barrier)\w+ m0,")
    loads = [i for i, x in enumerate(instructions)
             if re.match(r"global_load_lds_|(buffer|scratch)_load_\w+ .*\blds\b", x)]
    return len(loads), [instructions[i - 1] for i in loads if writes.match(instructions[i - 1])]


def test_a_wait_state_behind_writes_of_m0(listings):
    counts = [_without_wait(x) for x in listings]
    assert sum(n for n, _ in counts) > 0
    assert not [x for _, bad in counts for x in bad]


def test_the_check_itself():
    load = "global_load_lds_dwordx4 v1, s[2:3]"
    assert _without_wait(["s_mov_b32 m0, s4", "s_nop 0", load, load]) == (2, [])
    assert _without_wait(["s_mov_b32 m0, s4", load]) == (1, ["s_mov_b32 m0, s4"])
    assert _without_wait(["s_lshl_b32 m0, s4, 4", load])[1]
    assert not _without_wait(["s_cmp_eq_u32 m0, s4", load])[1]
