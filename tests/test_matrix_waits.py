"""CPU test of the built kernels: on every way through a kernel, between a matrix
instruction and the next that reads its result (or writes over it) otherwise than as a sum
to go on with, lie the wait states that the unit needs.  The compiler has left them out on
a loop's way out; what it leaves in straight lines is what is asked for here.
"""
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BUILD = os.path.join(ROOT, "_build")
LLVM = "/opt/rocm/llvm/bin/"
TOOLS = [LLVM + "llvm-objdump", LLVM + "llvm-objcopy", LLVM + "clang-offload-bundler"]
STATES = {"v_mfma_f32_16x16x32_bf16": 8, "v_mfma_f32_16x16x32_f16": 8, "v_mfma_f32_16x16x4_f32": 10,
          "v_mfma_f32_4x4x1_16b_f32": 4}
# kernels with matrix products in loops
OBJECTS = ["delta_bwd", "delta_fwd", "delta_grad", "delta_prep", "selective_scan_bwd", "selective_scan_fwd", "ssd_bf16_t128",
           "ssd_bf16_t256", "ssd_bf16_t32", "ssd_bf16_t64", "ssd_fused"]

REG = re.compile(r"\b([va])(?:\[(\d+):(\d+)\]|(\d+))")


def registers(text):
    out = set()
    for file, lo, hi, one in REG.findall(text):
        lo = int(one or lo)
        out.update((file, r) for r in range(lo, int(hi or lo) + 1))
    return out


def disassemble(obj, tmp):
    fat, code = str(tmp / "fat"), str(tmp / "code")
    subprocess.run([TOOLS[1], "-O", "binary", "--only-section=.hip_fatbin", obj, fat], check=True)
    subprocess.run([TOOLS[2], "--unbundle", "--type=o", "--targets=hipv4-amdgcn-amd-amdhsa--gfx950", "--input=" + fat,
                    "--output=" + code], check=True)
    return subprocess.run([TOOLS[0], "-d", code], check=True, capture_output=True, text=True).stdout


def kernels(text):
    """(name, [(address, instruction, target or None)]) of each function."""
    name, out = None, []
    for line in text.splitlines():
        m = re.match(r"^([0-9a-f]+) <(.*)>:$", line)
        if m:
            if name:
                yield name, out
            name, start, out = m.group(2), int(m.group(1), 16), []
            continue
        m = re.match(r"^\s+(\S.*?)\s*// ([0-9A-F]+):.*?(?:<(.*?)(?:\+0x([0-9a-f]+))?>)?$", line)
        if name and m:
            out.append((int(m.group(2), 16), m.group(1), start + int(m.group(4) or "0", 16) if m.group(3) == name else None))
    if name:
        yield name, out


def too_soon(code, states=STATES):
    """[(wait states, product, reader)] below what the product needs."""
    at = {a: i for i, (a, _, _) in enumerate(code)}
    text = [t for _, t, _ in code]
    found = []

    def following(i):
        op = text[i].split()[0]
        if op in ("s_endpgm", "s_setpc_b64"):
            return []
        to = [at[code[i][2]]] if op.startswith(("s_cbranch", "s_branch")) else []
        return to if op == "s_branch" else to + ([i + 1] if i + 1 < len(text) else [])

    for i, product in enumerate(text):
        if not product.startswith("v_mfma"):
            continue
        op, operands = product.split(None, 1)
        result, need = registers(operands.split(",")[0]), states[op]
        seen, todo = {}, [(j, 0) for j in following(i)]
        while todo:
            j, d = todo.pop()
            if d >= need or seen.get(j, need) <= d:
                continue
            seen[j] = d
            op, _, operands = text[j].partition(" ")
            if op.startswith("v_mfma"):
                a, *read = re.split(r",\s*(?![^\[]*\])", operands)
                if registers(a) & result:  # goes on with the sum, or starts another: the unit keeps them apart
                    if registers(read[0] + " " + read[1]) & result:
                        found.append((d, product, text[j]))
                    continue
                hit = registers(read[0] + " " + read[1]) & result
            else:
                hit = op.startswith(("v_", "ds_", "buffer_", "global_", "scratch_", "flat_")) and registers(operands) & result
            if hit:
                found.append((d, product, text[j]))
                continue
            todo += [(n, d + (int(operands) + 1 if op == "s_nop" else 1)) for n in following(j)]
    return found


def test_the_check_itself():
    code = [(0, "v_mfma_f32_16x16x32_bf16 v[0:3], v[8:11], v[12:15], v[0:3]", None), (8, "s_cbranch_scc1 4", 24),
            (12, "s_nop 7", None), (16, "v_mov_b64_e32 v[4:5], v[2:3]", None), (20, "s_endpgm", None),
            (24, "v_mov_b64_e32 v[6:7], v[2:3]", None), (28, "s_endpgm", None)]
    assert too_soon(code) == [(1, code[0][1], code[5][1])]  # the branch's way; the other has its nine
    code[1] = (8, "s_nop 6", None)
    code[2] = (12, "s_nop 0", None)
    assert too_soon(code) == []
    assert registers("v[2:4], a7, s[2:3], v9") == {("v", 2), ("v", 3), ("v", 4), ("a", 7), ("v", 9)}


@pytest.mark.skipif(not all(map(os.path.exists, TOOLS)), reason="no LLVM tools")
@pytest.mark.parametrize("name", OBJECTS)
def test_results_are_read_when_they_are_written(name, tmp_path):
    obj = os.path.join(BUILD, name + ".hip.o")
    if not os.path.exists(obj):
        pytest.skip("not built here")
    products = 0
    for kernel, code in kernels(disassemble(obj, tmp_path)):
        products += sum(t.startswith("v_mfma") for _, t, _ in code)
        found = too_soon(code)
        assert not found, (kernel, min(found))
    assert products
