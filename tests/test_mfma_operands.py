"""The scaled matrix instructions of the microscaled products are written in assembly, which the compiler does not keep apart
from what writes their operands and reads their sums.  The built library is checked for it: a vector instruction that writes an
operand is at least two instructions away, one that writes the execution mask four, and what touches a sum 19 (no GPU needed)."""

import os
import re
import struct
import subprocess

import pytest

import bit_blockwise_weight_amd as qk

OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"
OPERAND, EXEC, SUM = 2, 4, 19


def _registers(text):
    """Vector and accumulation registers named in operands."""
    out = set()
    for kind, lo, hi, one in re.findall(r"\b([va])(?:\[(\d+):(\d+)\]|(\d+))", text):
        out |= {kind + one} if one else {f"{kind}{i}" for i in range(int(lo), int(hi) + 1)}
    return out


def _read(listing):
    """(function, [(address, name, operands, target address of a branch or None)]) of a disassembly."""
    functions = []
    for line in listing.splitlines():
        head = re.match(r"^([0-9a-f]+) <(.+)>:$", line)
        if head:
            functions.append((head.group(2), []))
            continue
        code = re.match(r"^\s+(\S+)\s*(.*?)\s*// ([0-9A-F]+): ([0-9A-F]{8})", line)
        if not code:
            continue
        name, operands, at, word = code.group(1), code.group(2), int(code.group(3), 16), int(code.group(4), 16)
        target = None
        if name == "s_branch" or name.startswith("s_cbranch"):
            jump = word & 0xFFFF
            target = at + 4 + 4 * (jump - 0x10000 if jump & 0x8000 else jump)
        functions[-1][1].append((at, name, operands, target))
    return functions


def _is_vector(name):
    return name.startswith("v_") and not name.startswith("v_mfma")


def _written(name, operands):
    parts = operands.split(",")
    return _registers(",".join(parts[:2]) if "swap" in name else parts[0])


def hazards(code, tile):
    """What stands too close to a scaled matrix instruction in a function; tile: sums are looked at, too."""
    at = {c[0]: i for i, c in enumerate(code)}
    jumps = {}
    for i, c in enumerate(code):
        if c[3] is not None and c[3] in at:
            jumps.setdefault(at[c[3]], []).append(i)

    def before(i):
        if i > 0 and code[i - 1][1] not in ("s_branch", "s_endpgm"):
            yield i - 1
        yield from jumps.get(i, ())

    def walk(i, most, wrong):
        """Instructions before i with fewer than `most` states in between, as far as wrong(instruction) is true of one."""
        best, todo = {}, [(p, 0) for p in before(i)]
        while todo:
            p, states = todo.pop()
            if states >= most or best.get(p, most) <= states:
                continue
            best[p] = states
            name, operands = code[p][1], code[p][2]
            if wrong(name, operands, states):
                yield code[p]
            states += 1 + (int(operands, 0) if name == "s_nop" else 0)
            todo += [(q, states) for q in before(p)]

    found = []
    for i, (_, name, operands, _) in enumerate(code):
        if name.startswith("v_mfma_scale"):
            read = set().union(*(_registers(o) for o in operands.split(",")[1:]))
            found += [(c, code[i]) for c in walk(i, EXEC, lambda n, o, s: n.startswith("v_cmpx") or (
                s < OPERAND and _is_vector(n) and bool(_written(n, o) & read)))]
        elif tile and not name.startswith("s_"):
            used = {r for r in _registers(operands) if r[0] == "a"}
            if used and not name.startswith("v_mfma"):
                found += [(c, code[i]) for c in walk(i, SUM, lambda n, o, s: n.startswith("v_mfma_scale") and bool(
                    _written(n, o) & used))]
    return found


def _code_object(path, holding):
    """The gfx950 code object of the library that holds a kernel."""
    data, at = open(path, "rb").read(), 0
    while True:
        at = data.find(b"__CLANG_OFFLOAD_BUNDLE__", at)
        if at < 0:
            return None
        count, p = struct.unpack_from("<Q", data, at + 24)[0], at + 32
        for _ in range(count):
            off, size, length = struct.unpack_from("<QQQ", data, p)
            blob = data[at + off:at + off + size]
            if b"gfx950" in data[p + 24:p + 24 + length] and holding in blob:
                return blob
            p += 24 + length
        at += 24


def test_operands_and_sums_of_the_scaled_products(tmp_path):
    if not os.path.exists(qk.LIB_PATH):
        pytest.fail("libqk.so is not built; run python -m bit_blockwise_weight_amd.build")
    if not os.path.exists(OBJDUMP):
        pytest.skip("no disassembler")
    blob = _code_object(qk.LIB_PATH, b"mx4_tile_kernel")
    assert blob, "no code object with the products"
    path = tmp_path / "products.co"
    path.write_bytes(blob)
    listing = subprocess.run([OBJDUMP, "-d", str(path)], capture_output=True, text=True, check=True).stdout
    products = 0
    for name, code in _read(listing):
        products += sum(c[1].startswith("v_mfma_scale") for c in code)
        bad = hazards(code, "mx4_tile_kernel" in name)
        assert not bad, (name, len(bad), bad[:4])
    assert products > 1000


MFMA = "v_mfma_scale_f32_16x16x128_f8f6f4 a[0:3], v[4:7], v[8:11], a[0:3], v12, v13 cbsz:4 blgp:4"


@pytest.mark.parametrize("lines,wrong", [
    (["v_mov_b32_e32 v12, v1", MFMA], 1), (["v_mov_b32_e32 v9, v1", "s_mov_b32 s0, 0", MFMA], 1),
    (["v_mov_b32_e32 v9, v1", "s_nop 1", MFMA], 0), (["v_mov_b32_e32 v14, v1", MFMA], 0),
    (["v_permlane32_swap_b32 v1, v4", MFMA], 1), (["v_accvgpr_write_b32 a2, 0", MFMA], 1),
    (["ds_read_b128 v[4:7], v1", "s_waitcnt lgkmcnt(0)", MFMA], 0), (["v_cmpx_gt_u32_e32 v1, v2", "s_nop 2", MFMA], 1),
    ([MFMA, MFMA, "s_nop 15", "v_accvgpr_read_b32 v1, a3"], 2), ([MFMA, "s_nop 15", "s_nop 15", "v_accvgpr_read_b32 v1, a3"], 0),
    ([MFMA, "global_store_dwordx4 v[0:1], a[0:3], off"], 1)])
def test_the_check_itself(lines, wrong):
    code = [(4 * i, line.split()[0], line.split(" ", 1)[1], None) for i, line in enumerate(lines)]
    assert len(hazards(code, True)) == wrong


def test_the_check_follows_branches():
    text = "0000000000000000 <f>:\n" + "\n".join(f"\t{t} // {4 * i:012X}: {w:08X}" for i, (t, w) in enumerate(
        [(MFMA, 0), ("s_nop 3", 0), ("v_mov_b32_e32 v12, v1", 0), ("s_cbranch_scc1 65532", 0xBF85FFFC), ("s_endpgm", 0)]))
    (_, code), = _read(text)
    assert code[3][3] == 0 and len(hazards(code, True)) == 1
