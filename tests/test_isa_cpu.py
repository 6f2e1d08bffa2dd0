"""Wait states around the direct global->LDS loads, in the machine code that was built.

The loads are written in inline asm, which the compiler's own hazard pass does
not look into, so what it guarantees elsewhere is checked here on libmoe.so's
gfx950 code:
  * a scalar write of m0, then a load that takes its LDS address from it: at
    least one wait state between them;
  * a VALU write of a scalar register (v_readfirstlane, a comparison), then a
    vector memory instruction that reads it: at least five.
Every instruction is one wait state, s_nop N is N + 1.  Paths through branches
count as well as straight code.
"""
import os
import re
import shutil
import subprocess

import pytest

from mixture_experts_transformer_moe_amd import binding, build

OBJDUMP = os.path.join(os.path.dirname(os.path.realpath(build.hipcc())), "..", "llvm", "bin", "llvm-objdump")
_INSN = re.compile(r"^\s+([a-z]\w*)\s*(.*?)\s*// ([0-9A-F]+):")
_LABEL = re.compile(r"^([0-9a-f]+) <(.+)>:$")
_TARGET = re.compile(r"<.+\+0x([0-9a-f]+)>$")
_SREG = re.compile(r"\bs(?:(\d+)\b|\[(\d+):(\d+)\])|\b(vcc)\b|\b(m0)\b")
_VMEM = ("global_", "buffer_", "flat_", "scratch_")


def sregs(text):
    out = set()
    for one, lo, hi, vcc, m0 in _SREG.findall(text):
        if one:
            out.add(f"s{one}")
        elif lo:
            out |= {f"s{k}" for k in range(int(lo), int(hi) + 1)}
        else:
            out.add(vcc or m0)
    return out


def functions(text):
    """{name: [(address, mnemonic, operands, branch target or None)]} of a disassembly."""
    found, cur, base = {}, None, 0
    for line in text.splitlines():
        if label := _LABEL.match(line):
            base = int(label[1], 16)
            cur = found.setdefault(label[2], [])
        elif cur is not None and (m := _INSN.match(line)):
            to = _TARGET.search(line) if m[1].startswith(("s_cbranch", "s_branch")) else None
            cur.append((int(m[3], 16), m[1], m[2], base + int(to[1], 16) if to else None))
    return found


def predecessors(code):
    at = {a: i for i, (a, *_) in enumerate(code)}
    pred = [[] for _ in code]
    for i, (_, name, _, to) in enumerate(code):
        if i + 1 < len(code) and name not in ("s_branch", "s_endpgm", "s_setpc_b64"):
            pred[i + 1].append(i)
        if to is not None:
            pred[at[to]].append(i)
    return pred


def hazards(code):
    """Descriptions of the loads of one function that come too early."""
    pred = predecessors(code)

    def reached(i, waits, breaks):
        # an instruction for which breaks() holds with fewer than `waits` wait states before instruction i
        seen, todo = {}, [(p, 0) for p in pred[i]]
        while todo:
            j, passed = todo.pop()
            if seen.get(j, waits) <= passed:
                continue
            seen[j] = passed
            _, name, ops, _ = code[j]
            if breaks(name, ops):
                return j
            passed += int(ops, 0) + 1 if name == "s_nop" else 1
            if passed < waits:
                todo += [(p, passed) for p in pred[j]]
        return None

    bad = []
    for i, (addr, name, ops, _) in enumerate(code):
        if not name.startswith(_VMEM):
            continue
        if "_lds_" in name or re.search(r"\blds\b", ops):
            j = reached(i, 1, lambda n, o: n.startswith("s_") and o.split(",")[0] == "m0")
            if j is not None:
                bad.append(f"{addr:x}: {code[j][1]} {code[j][2]}; {name} {ops}")
        read = sregs(ops)
        if read:
            j = reached(i, 5, lambda n, o: n.startswith("v_") and sregs(o.split(",")[0]) & read)
            if j is not None:
                bad.append(f"{addr:x}: {code[j][1]} {code[j][2]} ... {name} {ops}")
    return bad


def lines(*code):
    return "0000000000000100 <f>:\n" + "\n".join(
        f"\t{c:<40}// {0x100 + 4 * i:012X}: 00000000" + (" <f+0x0>" if "branch" in c else "") for i, c in enumerate(code)) + "\n"


@pytest.mark.parametrize("code,count", [
    (("s_mov_b32 m0, s5", "global_load_lds_dwordx4 v1, s[2:3]"), 1),
    (("s_mov_b32 m0, s5", "s_nop 0", "global_load_lds_dwordx4 v1, s[2:3]"), 0),
    (("s_add_u32 m0, s5, 0x400", "global_load_lds_dword v1, s[2:3]"), 1),
    (("v_readfirstlane_b32 s3, v0", "s_nop 3", "global_load_dword v1, v2, s[2:3]"), 1),
    (("v_readfirstlane_b32 s3, v0", "s_nop 4", "global_load_dword v1, v2, s[2:3]"), 0),
    (("v_readfirstlane_b32 s4, v0", "global_load_dword v1, v2, s[2:3]"), 0),
    (("global_load_dword v1, v2, s[2:3]", "v_cmp_gt_u32 s[2:3], v0, v1", "s_cbranch_scc1 0"), 1),     # round the loop
    (("s_nop 4", "global_load_dword v1, v2, s[2:3]", "v_cmp_gt_u32 s[2:3], v0, v1", "s_cbranch_scc1 0"), 0),
])
def test_scan_finds_what_it_looks_for(code, count):
    (f,) = functions(lines(*code)).values()
    assert len(f) == len(code)
    assert len(hazards(f)) == count


def test_wait_states_of_lds_loads(tmp_path):
    if not os.path.exists(binding.LIB_PATH):
        build.build(verbose=False)
    lib = shutil.copy(binding.LIB_PATH, tmp_path)
    subprocess.run([OBJDUMP, "--offloading", lib], check=True, capture_output=True)
    objects = sorted(p for p in tmp_path.iterdir() if "gfx950" in p.name)
    assert len(objects) >= len(build.SOURCES) - 1          # (api.hip holds no kernel)
    bad, loads = [], 0
    for o in objects:
        text = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", "--mcpu=gfx950", str(o)], check=True,
                              capture_output=True, text=True).stdout
        for name, code in functions(text).items():
            loads += sum("_lds_" in n for _, n, _, _ in code)
            bad += [f"{name[:100]} {b}" for b in hazards(code)]
    assert loads > 100                                     # the scan sees the kernels
    assert not bad, f"{len(bad)} of {loads} loads:\n" + "\n".join(bad[:20])
