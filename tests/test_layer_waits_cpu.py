"""The layer operators' product kernels meet at raw workgroup barriers, which wait for nothing by
themselves. Before each of them a wave has to have waited for its own LDS operations: after it other
waves' loads may fill the places that it read or wrote (a workgroup that walks tiles loads the next
tile's operands over the rows of the last tile's epilogue).

Read off the machine code that the build put into the library: along every path from an LDS operation
to an s_barrier there is an s_waitcnt that lets none stay in flight. No GPU is needed."""
import os
import re
import subprocess

import pytest

from test_kernel_resources import LIB, _bundles

OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"
FAMILIES = ["layer_pp256_kernel", "layer_pp128_kernel", "layer_ring_kernel"]
LINE = re.compile(r"^\t(\S+)\s*(.*?)\s*// ([0-9A-F]+):")


def code(family, tmp):
    """{kernel: [(address, mnemonic, operands)]} of the kernels whose name holds `family`."""
    if not os.path.exists(LIB):
        import test_kernel_resources
        test_kernel_resources._kernels()  # builds the library
    with open(LIB, "rb") as f:
        data = f.read()
    kernels = {}
    for triple, obj in _bundles(data):
        if "gfx950" not in triple or family.encode() not in obj:
            continue
        path = tmp / "code.co"
        path.write_bytes(obj)
        text = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", str(path)], capture_output=True, text=True,
                              check=True).stdout
        here = None
        for line in text.splitlines():
            if line.endswith(">:"):
                name = line[line.index("<") + 1:-2]
                here = kernels.setdefault(name, []) if family in name else None
            elif here is not None and (m := LINE.match(line)):
                here.append((int(m[3], 16), m[1], m[2]))
    return kernels


def follows(at, op, arg):
    """The addresses that control can go to, of an instruction of 4 or 8 bytes: None stands for the next."""
    if op == "s_endpgm":
        return []
    if op.startswith(("s_branch", "s_cbranch")):
        to = at + 4 + 4 * ((int(arg) ^ 0x8000) - 0x8000)
        return [to] if op == "s_branch" else [to, None]
    assert not op.startswith(("s_setpc", "s_swappc", "s_call")), op
    return [None]


def barriers_with_lds_in_flight(insns):
    """Addresses of the barriers that some path reaches with an LDS operation of its wave in flight,
    counted from a write on (a fragment that is only read is waited for by the product that takes it).
    The states of an instruction are whether a write came since the last barrier, and whether
    anything since then is in flight."""
    index = {a: i for i, (a, _, _) in enumerate(insns)}
    seen, bad, todo = set(), set(), [(0, False, False)]
    while todo:
        if (at := todo.pop()) in seen:
            continue
        seen.add(at)
        i, wrote, flying = at
        addr, op, arg = insns[i]
        if op.startswith("ds_write"):
            wrote = flying = True
        elif op.startswith("ds_"):
            flying = flying or wrote
        elif op == "s_waitcnt" and "lgkmcnt(0)" in arg:
            flying = False
        elif op == "s_barrier":
            if flying:
                bad.add(addr)
            wrote = False
        todo += [(i + 1 if to is None else index[to], wrote, flying) for to in follows(addr, op, arg)]
    return [hex(a) for a in sorted(bad)]


def test_the_reading_itself():
    """On a few instructions: a barrier after an LDS write, with a wait, without, and round a loop."""
    def run(*ops):
        return barriers_with_lds_in_flight([(4 * i, *o) for i, o in enumerate(ops)])
    write, wait, meet, end = ("ds_write_b32", "v0, v1"), ("s_waitcnt", "lgkmcnt(0)"), ("s_barrier", ""), ("s_endpgm", "")
    assert run(write, wait, meet, end) == []
    assert run(write, meet, end) == ["0x4"]
    assert run(write, ("s_waitcnt", "vmcnt(0)"), meet, end) == ["0x8"]
    back = ("s_cbranch_scc1", str(0x10000 - 3))  # to the first instruction of three
    assert run(meet, write, back, end) == ["0x0"]
    assert run(meet, write, wait, ("s_cbranch_scc1", str(0x10000 - 4)), end) == []
    assert run(write, ("s_cbranch_execz", "1"), wait, meet, end) == ["0xc"]
    read = ("ds_read_b32", "v0, v1")
    assert run(write, wait, read, meet, end) == ["0xc"]
    assert run(read, meet, end) == []


@pytest.mark.skipif(not os.path.exists(OBJDUMP), reason="no llvm-objdump")
@pytest.mark.parametrize("family", FAMILIES)
def test_no_lds_operation_is_in_flight_at_a_barrier(family, tmp_path):
    kernels = code(family, tmp_path)
    assert kernels, family
    bad = {}
    for name, insns in kernels.items():
        assert any(op == "s_barrier" for _, op, _ in insns), name
        if found := barriers_with_lds_in_flight(insns):
            bad[name] = found
    assert not bad, f"{len(bad)} of {len(kernels)} kernels, e.g. {list(bad.items())[0]}"
