"""The loads that expert_i8.hip's tile kernel makes by hand, in the library as it was
built, on the CPU.

A scalar register that a vector instruction wrote may be read by a load five wait states
later at the earliest.  The compiler keeps to that for its own loads, but does not look
into blocks of assembly, and it brings scalars back from vector lanes (v_readlane)
wherever it has run out of registers.  So each block has to hold the wait states itself,
whatever the compiler puts before it.  An instruction is one, s_nop n is n + 1."""
import glob
import os
import re
import shutil
import subprocess

import pytest

from combine_get_dispatch_02_amd import build

OBJDUMP = os.path.join(os.path.dirname(os.path.dirname(build.HIPCC)), "llvm", "bin", "llvm-objdump")
WAITS = 5


def scalars(operand):
    """Scalar registers of an operand."""
    m = re.fullmatch(r"s(\d+)|s\[(\d+):(\d+)\]", operand)
    if not m:
        return {operand} & {"vcc", "m0", "exec"}
    a, b = (m[1], m[1]) if m[1] else (m[2], m[3])
    return {f"s{i}" for i in range(int(a), int(b) + 1)}


def parse(line):
    """(mnemonic, operands) of a line of the listing."""
    name, _, rest = line.split("//")[0].strip().partition(" ")
    return name, [o.strip() for o in rest.split(",")]


def states(name, operands):
    return int(operands[0]) + 1 if name == "s_nop" else 1


def written(name, operands):
    """What a vector instruction writes of scalar registers."""
    if not name.startswith("v_"):
        return set()
    second = scalars(operands[1]) if ("_co_" in name or "div_scale" in name) and len(operands) > 1 else set()
    return scalars(operands[0]) | second


def by_hand(listing):
    """Loads past the registers, as indexes into the listing."""
    return [i for i, (name, ops) in enumerate(listing) if name.startswith("buffer_load") and ops[-1].endswith(" lds")]


def read(ops):
    """Scalar registers that a load reads: its buffer, its offset, m0."""
    return scalars(ops[1]) | scalars(ops[2].split()[0]) | {"m0"}


def too_early(listing):
    bad = []
    for i in by_hand(listing):
        need, waits, at = read(listing[i][1]), 0, i - 1
        while at >= 0 and waits < WAITS:
            name, ops = listing[at]
            if written(name, ops) & need:
                bad.append(listing[at: i + 1])
            if name.startswith("s_") and not name.startswith(("s_cmp", "s_nop")):
                need = need - scalars(ops[0])       # what it held before is not read
            waits += states(name, ops)
            at -= 1
    return bad


def own_waits(listing, i):
    """Wait states between a block's first instruction, which sets m0, and its load,
    that one among them."""
    waits, at = 0, i - 1
    while at >= 0 and (listing[at][0] == "s_nop" or (listing[at][0] == "s_mov_b32" and listing[at][1][0] == "m0")):
        waits += states(*listing[at])
        if listing[at][0] == "s_mov_b32":
            break
        at -= 1
    return waits


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    """The instructions of each tile kernel."""
    if not os.path.exists(OBJDUMP):
        pytest.skip("no llvm-objdump")
    room = tmp_path_factory.mktemp("code")
    lib = shutil.copy(build.LIB, room)
    subprocess.run([OBJDUMP, "--offloading", lib], check=True, cwd=room, stdout=subprocess.DEVNULL)
    found = {}
    for code in glob.glob(str(room / "*gfx950*")):
        with open(code, "rb") as f:
            if b"tile_i8_kernel" not in f.read():
                continue
        text = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", "--no-leading-addr", code], check=True, cwd=room,
                              stdout=subprocess.PIPE, text=True).stdout
        name = None
        for line in text.splitlines():
            if line.startswith("<"):
                name = line
            elif name and "tile_i8_kernel" in name and line.strip():
                found.setdefault(name, []).append(parse(line))
    assert len(found) == 2, "a tile kernel for each epilogue"
    return found


def test_no_load_reads_a_scalar_too_early(kernels):
    for listing in kernels.values():
        assert len(by_hand(listing)) > 100
        assert too_early(listing) == []


def test_every_block_waits_by_itself(kernels):
    for listing in kernels.values():
        assert {own_waits(listing, i) for i in by_hand(listing)} == {WAITS}


def test_the_check_sees_a_scalar_written_too_late():
    def block(between):
        return [parse(s) for s in ("v_readlane_b32 s21, v254, 3", *between, "buffer_load_dwordx4 v105, s[20:23], s8 offen lds")]
    assert too_early(block(["s_mov_b32 m0, s2", "s_nop 0"])) and too_early(block(["s_mov_b32 m0, s2", "s_nop 2"]))
    assert not too_early(block(["s_mov_b32 m0, s2", "s_nop 3"]))
    late = block(["v_readfirstlane_b32 s8, v1", "s_mov_b32 m0, s2", "s_nop 0"])
    assert len(too_early(late)) == 2
    assert too_early([parse("v_cmp_lt_i32_e64 s[22:23], v1, v2")] + late[2:])
    assert not too_early([parse("v_readlane_b32 s24, v254, 3")] + late[2:])
    assert not too_early(block(["s_lshl_b32 s21, s3, 7", "s_mov_b32 m0, s2", "s_nop 0"]))
