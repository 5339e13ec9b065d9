"""The wait states that gfx950 leaves to the program, in the device code of the built library (CPU only: the code objects
built here, disassembled).

The compiler keeps them between its own instructions, but does not look into inline asm.  Between a vector instruction
that writes a scalar register and a memory instruction that reads it lie five; between a scalar write of m0 and a load that
goes to LDS lies one.  Every instruction is one, s_nop N is N + 1.  Looked for backwards along every path, branches
included."""
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "sparse_weight_direct_amd", "libsparseconv.so")
OBJDUMP = next((p for p in (shutil.which("llvm-objdump"), "/opt/rocm/llvm/bin/llvm-objdump") if p and os.path.exists(p)), None)

LINE = re.compile(r"^\s+([a-z]\w*)(?: (.*?))?\s+// ([0-9A-F]{12}): ")
SCALAR = re.compile(r"(?<![\w\[])(?:s(\d+)|s\[(\d+):(\d+)\]|(vcc)(?:_lo|_hi)?)(?!\w)")
MEMORY = ("buffer_", "global_", "flat_", "scratch_")
ENDS = ("s_branch", "s_endpgm", "s_setpc_b64")


def scalars(text):
    """Numbers of the scalar registers that a piece of operands names."""
    found = set()
    for one, lo, hi, vcc in SCALAR.findall(text):
        found |= {106, 107} if vcc else {int(one)} if one else set(range(int(lo), int(hi) + 1))
    return found


def vector_writes(op, args):
    """Scalar registers that a vector instruction writes."""
    parts = args.split(", ")
    if op.startswith(("v_readfirstlane", "v_readlane", "v_cmp")):
        return scalars(parts[0])
    if "_co_" in op or op.startswith(("v_div_scale", "v_mad_u64", "v_mad_i64")):
        return scalars(parts[1])
    return set()


def violations(listing):
    """(function, address, instruction) of every memory instruction that comes too soon."""
    code, name, names = [], "", {}
    for line in listing.splitlines():
        if line.endswith(">:"):
            name = line.split("<")[1][:-2]
        m = LINE.match(line)
        if m:
            names[len(code)] = name
            code.append((m[1], (m[2] or "").strip(), int(m[3], 16)))
    at = {c[2]: i for i, c in enumerate(code)}
    into = {}
    for i, (op, args, address) in enumerate(code):
        if op.startswith(("s_cbranch", "s_branch")):
            offset = int(args.split()[0])
            target = at.get(address + 4 + 4 * (offset - 65536 if offset >= 32768 else offset))
            if target is not None:
                into.setdefault(target, []).append(i)

    def before(i):
        if i and code[i - 1][0] not in ENDS and names[i - 1] == names[i]:
            yield i - 1
        yield from into.get(i, ())

    found = []
    for i, (op, args, address) in enumerate(code):
        if not op.startswith(MEMORY):
            continue
        read = scalars(args)
        to_lds = "_lds_" in op or args.endswith(" lds")
        if not read and not to_lds:
            continue
        todo, seen = [(j, 0) for j in before(i)], set()
        while todo:
            j, waited = todo.pop()
            if (j, waited) in seen:
                continue
            seen.add((j, waited))
            o, a, _ = code[j]
            wrote_m0 = to_lds and waited < 1 and o.startswith("s_") and a.split(", ")[0] == "m0"
            if wrote_m0 or (o.startswith("v_") and vector_writes(o, a) & read):
                found.append((names[i], hex(address), f"{o} {a}; +{waited}: {op} {args}"))
                break
            waited += int(a, 0) + 1 if o == "s_nop" else 1
            if waited < 5:
                todo += [(k, waited) for k in before(j)]
    return found


def test_the_search_finds_what_it_looks_for():
    def listing(*lines):
        return "0 <f>:\n" + "\n".join(f"\t{s:60}// {4 * i:012X}: 00000000" for i, s in enumerate(lines))

    load = "global_load_lds_dwordx4 v1, s[2:3]"
    first = "v_readfirstlane_b32 s3, v0"
    m0 = "s_mov_b32 m0, s9"
    assert len(violations(listing(first, m0, "s_nop 0", load))) == 1
    assert len(violations(listing(first, m0, "s_nop 2", load))) == 1  # four
    assert violations(listing(first, m0, "s_nop 3", load)) == []
    assert violations(listing("v_readfirstlane_b32 s4, v0", m0, "s_nop 0", load)) == []
    assert len(violations(listing("s_nop 0", m0, load))) == 1
    assert len(violations(listing("v_cmp_eq_u32_e64 s[2:3], v0, v1", "global_load_dword v1, v2, s[2:3]"))) == 1
    assert len(violations(listing("v_cmp_eq_u32_e32 vcc, v0, v1", "global_load_dword v1, v2, vcc"))) == 1
    # over a branch: from the end of the loop to its beginning
    assert len(violations(listing(load, "s_nop 7", first, "s_cbranch_scc1 65532", "s_endpgm"))) == 1
    assert violations(listing(load, "s_nop 7", first, "s_nop 3", "s_cbranch_scc1 65531", "s_endpgm")) == []


@pytest.mark.skipif(OBJDUMP is None, reason="no llvm-objdump")
def test_wait_states_of_the_built_kernels(tmp_path):
    lib = shutil.copy(LIB, tmp_path / "lib.so")
    subprocess.run([OBJDUMP, "--offloading", lib], check=True, capture_output=True, cwd=tmp_path)
    objects = sorted(p for p in os.listdir(tmp_path) if p.endswith("gfx950"))
    assert len(objects) >= 9, objects
    found, loads = [], 0
    for o in objects:
        listing = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", o], check=True, capture_output=True, text=True, cwd=tmp_path).stdout
        loads += listing.count("global_load_lds_dwordx4")
        found += violations(listing)
    assert loads > 100  # the listing is what it is taken for
    assert not found, f"{len(found)} too soon, first: {found[:5]}"
