"""What the built library's device code has to keep to, read from its own disassembly."""
import functools
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


def _registers(operand):
    """Scalar registers that an operand's text names, as numbers; vcc is -1 and -2."""
    operand = operand.strip().strip("-|")
    if operand in ("vcc", "vcc_lo", "vcc_hi"):
        return {"vcc": {-1, -2}, "vcc_lo": {-1}, "vcc_hi": {-2}}[operand]
    m = re.fullmatch(r"s(\d+)", operand)
    if m:
        return {int(m[1])}
    m = re.fullmatch(r"s\[(\d+):(\d+)\]", operand)
    return set(range(int(m[1]), int(m[2]) + 1)) if m else set()


@functools.lru_cache(maxsize=None)
def _vector_alu(text):
    """(scalar registers written, scalar registers read) of a vector ALU instruction."""
    op, _, rest = text.partition(" ")
    operands = [o.split(" ")[0] for o in re.split(r",\s*", rest.strip())]
    writes = 1 + bool(re.match(r"v_(add|sub|subrev|addc|subb|subbrev)_co_u32|v_div_scale|v_mad_[ui]64", op))
    wrote = set().union(*(_registers(o) for o in operands[:writes]))
    read = set().union(*(_registers(o) for o in operands[writes:])) if len(operands) > writes else set()
    return wrote, read | ({-1, -2} if op.startswith("v_div_fmas") else set())


def _late_readers(code, needed, reads, writes):
    """(writer, reader) pairs in straight-line code with fewer than `needed` wait states between them."""
    recent = []                                                      # (wait states since, registers, text)
    for text in code:
        op = text.split(" ")[0]
        use = reads(text)
        if use:
            for since, regs, writer in recent:
                if regs & use:
                    yield writer, text
        states = int(text.split()[1]) + 1 if op == "s_nop" else 1
        recent = [(since + states, regs, writer) for since, regs, writer in recent if since + states < needed]
        regs = writes(text)
        if regs:
            recent.append((0, regs, text))
        if op in ("s_branch", "s_endpgm", "s_setpc_b64"):
            recent = []


def _valu(text):
    return text.startswith("v_") and not text.startswith(("v_mfma", "v_accvgpr"))


def test_scalar_results_of_vector_instructions_are_waited_for(instructions):
    """A vector instruction that writes scalar registers (a comparison, a carry, a lane read) is two wait states ahead of a vector
    instruction that reads them, and five ahead of a memory instruction that takes its address from them."""
    writes = lambda t: _vector_alu(t)[0] if _valu(t) else set()
    for name, code in instructions.items():
        found = list(_late_readers(code, 2, lambda t: _vector_alu(t)[1] if _valu(t) else set(), writes))
        assert not found, (name, len(found), found[0])
        memory = lambda t: set().union(*map(_registers, re.split(r",\s*|\s+", t)[1:])) if re.match(r"(global|buffer|scratch|flat)_", t) else set()
        found = list(_late_readers(code, 5, memory, writes))
        assert not found, (name, len(found), found[0])


def test_word_writes_are_waited_for(instructions):
    """The result of a vector instruction that writes a part of its register is read one wait state later at the earliest."""
    for name, code in instructions.items():
        for write, after in zip(code, code[1:]):
            if "dst_sel:" in write and "dst_sel:DWORD" not in write and _valu(after):
                register = write.split()[1].rstrip(",")
                sources = re.split(r",\s*", after.partition(" ")[2])[1:] + ([after.split()[1].rstrip(",")] if re.match(r"v_(dot2c|fmac|mac)", after) else [])
                assert register not in [s.split(" ")[0] for s in sources], (name, write, after)
