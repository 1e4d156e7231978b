"""The built library's gfx950 machine code: no instruction touches a matrix
product's result before the matrix cores have written it.

The hardware does not hold back a vector instruction that reads or overwrites
the result of a v_mfma too early; the compiler puts s_nop in between.  Where it
moved the reads behind a conditional branch it has left them out on the taken
side: paged attention over an 8-bit cache with 256 columns then gave wrong
scores, the same ones every time.  The test walks every kernel from each v_mfma
over both sides of every branch and counts the issue slots up to the first other
instruction that names a register of its result.  Slots needed: 4 passes (16 x 16
bf16) 8, 8 passes (32 x 32 bf16) 12, 16 x 16 fp32 10.
"""
import os
import re
import subprocess
import tempfile

import pytest

import bench

LIB = os.path.join(bench.ROOT, "gated_deltanet_recurrent_decode_amd", "libgdn.so")
OBJDUMP = os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "llvm", "bin", "llvm-objdump")
REG = re.compile(r"\b([va])(?:\[(\d+):(\d+)\]|(\d+)\b)")
NEED = {"v_mfma_f32_16x16x32_bf16": 8, "v_mfma_f32_32x32x16_bf16": 12, "v_mfma_f32_16x16x4_f32": 10,
        "v_mfma_f32_32x32x2_f32": 18}


def _regs(text):
    got = set()
    for m in REG.finditer(text):
        a, b = (m.group(2), m.group(3)) if m.group(2) else (m.group(4), m.group(4))
        got |= {(m.group(1), i) for i in range(int(a), int(b) + 1)}
    return got


def parse(text):
    """[(function, address, opcode, operands)] and the index of every address."""
    out, func = [], None
    for line in text.splitlines():
        m = re.match(r"^[0-9a-f]+ <(\S+)>:", line)
        if m:
            func = m.group(1)
            continue
        m = re.match(r"^\s+(\S+)\s*(.*?)\s*//\s*([0-9A-F]+):", line)
        if m and func:
            out.append((func, int(m.group(3), 16), m.group(1), m.group(2)))
    return out, {(f, a): i for i, (f, a, _, _) in enumerate(out)}


def early(insts, where):
    """Every (product, instruction, slots between) that comes too early."""
    bad = []
    for i, (f, _, op, args) in enumerate(insts):
        if not op.startswith("v_mfma"):
            continue
        need = NEED.get(op, 20)
        result = _regs(args.split(",")[0])
        todo, seen = [(i + 1, 0)], set()
        while todo:
            j, w = todo.pop()
            while j < len(insts) and w < need and insts[j][0] == f and (j, w) not in seen:
                seen.add((j, w))
                _, at, o, a = insts[j]
                if not o.startswith(("v_mfma", "s_")) and _regs(a) & result:
                    bad.append((f, f"{op} {args}", f"{o} {a}", w))
                    break
                if o in ("s_endpgm", "s_setpc_b64"):
                    break
                if o.startswith("s_cbranch") or o == "s_branch":
                    words = int(a.split()[0])
                    to = where.get((f, at + 4 + 4 * (words - 65536 if words > 32767 else words)))
                    if to is not None and (to, w + 1) not in seen:
                        todo.append((to, w + 1))
                    if o == "s_branch":
                        break
                w += int(a.split()[0]) + 1 if o == "s_nop" else 1
                j += 1
    return bad


def test_the_walk_finds_an_early_read_behind_a_branch():
    code = """
0000000000000000 <k>:
\tv_mfma_f32_16x16x32_bf16 a[4:7], v[0:3], v[4:7], a[4:7]    // 000000000000: D3B58004
\ts_cbranch_scc1 2                                           // 000000000008: BF850002 <k+0x14>
\ts_nop 7                                                    // 00000000000C: BF800007
\ts_nop 0                                                    // 000000000010: BF800000
\tv_accvgpr_read_b32 v1, a7                                  // 000000000014: D3D84001
\ts_endpgm                                                   // 00000000001C: BF810000
"""
    assert [(b[2].split()[0], b[3]) for b in early(*parse(code))] == [("v_accvgpr_read_b32", 1)]
    assert early(*parse(code.replace("s_cbranch_scc1 2 ", "s_nop 7 "))) == []


def test_products_are_awaited_on_every_path():
    if not os.path.exists(LIB):
        pytest.skip("libgdn.so is not built")
    if not os.path.exists(OBJDUMP):
        pytest.skip("llvm-objdump is not available")
    products, bad = 0, []
    with tempfile.TemporaryDirectory() as d:
        for i, co in enumerate(bench.device_code_objects(LIB)):
            path = os.path.join(d, f"co{i}.elf")
            with open(path, "wb") as f:
                f.write(co)
            text = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", path], capture_output=True, text=True,
                                  check=True).stdout
            insts, where = parse(text)
            products += sum(x[2].startswith("v_mfma") for x in insts)
            bad += early(insts, where)
    assert products > 500, "expected the library's matrix products in the disassembly"
    assert not bad, "results read too early:\n" + "\n".join(f"{f}: {a} | {b} after {w}" for f, a, b, w in bad[:10])
