"""What the built library's device code has to keep to, read from its own disassembly."""
import os
import re
import shutil
import subprocess

import pytest

from trellis_coded_gemv_amd import binding as tg
from trellis_coded_gemv_amd import build

OBJDUMP = os.path.join(os.path.dirname(build.ROCM_LIB), "llvm", "bin", "llvm-objdump")
LOAD_TO_LDS = re.compile(r"(global|buffer|scratch)_load_.*lds")


@pytest.fixture(scope="module")
def instructions(tmp_path_factory):
    """The device instructions of each source, in order, as text."""
    if not os.path.exists(OBJDUMP):
        pytest.skip("no llvm-objdump")
    d = tmp_path_factory.mktemp("device_code")
    shutil.copy(tg.LIB_PATH, d / "lib.so")
    subprocess.run([OBJDUMP, "--offloading", "lib.so"], cwd=d, check=True, capture_output=True)
    out = {}
    for name in sorted(os.listdir(d)):
        if name.endswith(build.ARCH):
            p = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", "--no-leading-addr", name], cwd=d, check=True, capture_output=True, text=True)
            out[name] = [s for s in (line.split("//")[0].strip() for line in p.stdout.splitlines()) if s]
    assert len(out) == len(build.SOURCES)
    return out


def test_loads_to_lds_wait_for_m0(instructions):
    """A load to LDS takes its base from m0, and needs one wait state after a scalar instruction that writes it."""
    loads = 0
    for name, code in instructions.items():
        for before, load in zip(code, code[1:]):
            if LOAD_TO_LDS.match(load):
                loads += 1
                assert not re.match(r"s_\w+\s+m0\b", before), (name, before, load)
    assert loads > 0


def test_asm_declares_m0():
    """Inline assembly that writes m0 says so, or the compiler may keep a value of its own there."""
    found = 0
    for name in sorted(os.listdir(build.CSRC)):
        with open(os.path.join(build.CSRC, name)) as f:
            text = f.read()
        for asm in re.findall(r"\basm(?:\s+volatile)?\s*\(.*?\);", text, flags=re.S):
            if re.search(r"\bs_\w+\s+m0\b", asm):
                found += 1
                assert re.search(r':\s*(?:"\w+",\s*)*"m0"', asm), (name, asm)
    assert found > 0
