"""Wait states that the hardware does not keep by itself, in the compiled
kernels (CPU only: the built library is disassembled).

A vector memory instruction that reads a scalar register (a buffer's
descriptor, a scalar offset or base) must come at least five wait states behind
the vector instruction that wrote the register: every instruction between is
one, s_nop n is n + 1. The compiler keeps this for its own instructions, not for
those written as asm. And what asm writes without saying so."""
import glob
import os
import re
import shutil
import subprocess

import pytest

import routing_grouped_expert_amd as moe

OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"
STATES = 5

pytestmark = pytest.mark.skipif(not os.path.exists(OBJDUMP), reason="llvm-objdump not available")


def kernels(tmp):
    """(name, [(address, mnemonic, operands, branch target or None)]) of every
    function of the library's device code."""
    moe.lib()
    so = os.path.join(tmp, "lib.so")
    shutil.copy(moe.LIB_PATH, so)
    subprocess.run([OBJDUMP, "--offloading", so], check=True, capture_output=True, cwd=tmp)
    for code in sorted(glob.glob(os.path.join(tmp, "lib.so.*gfx950"))):
        text = subprocess.run([OBJDUMP, "-d", code], check=True, capture_output=True, text=True).stdout
        name, start, ins = None, 0, []
        for line in text.splitlines():
            m = re.match(r"([0-9a-f]+) <(.+)>:$", line)
            if m:
                if name:
                    yield name, ins
                start, name, ins = int(m[1], 16), m[2], []
                continue
            m = re.match(r"\t(\w+)\s*(.*?)\s*// ([0-9A-F]+):(.*)$", line)
            if m:
                to = re.search(r"<\S+?(?:\+0x([0-9a-f]+))?>\s*$", m[4]) if m[1].startswith(("s_branch", "s_cbranch")) else None
                ins.append((int(m[3], 16), m[1], m[2], start + int(to[1] or "0", 16) if to else None))
        if name:
            yield name, ins


def scalars(operand):
    """The scalar registers an operand names."""
    operand = operand.strip()
    m = re.fullmatch(r"s\[(\d+):(\d+)\]", operand)
    if m:
        return {f"s{i}" for i in range(int(m[1]), int(m[2]) + 1)}
    m = re.match(r"(s\d+|vcc_lo|vcc_hi)\b", operand)
    if m:
        return {m[1]}
    return {"vcc_lo", "vcc_hi"} if re.match(r"vcc\b", operand) else set()


def written(op, operands):
    """The scalar registers a vector instruction writes: its first operand, or
    the second where that is the carry (the first being a vector register)."""
    if not op.startswith("v_"):
        return set()
    parts = operands.split(",")
    out = scalars(parts[0])
    if not out and len(parts) > 1 and re.match(r"v_(add|sub|subrev)b?(_co|c_co)|v_div_scale|v_mad_[iu]64", op):
        out = scalars(parts[1])
    return out


def too_early(ins):
    """The vector memory instructions that read a scalar register fewer than
    STATES wait states behind its vector write, along any path."""
    at = {a: i for i, (a, *_) in enumerate(ins)}
    into = [[] for _ in ins]
    for i, (_, op, _, to) in enumerate(ins):
        if i + 1 < len(ins) and op not in ("s_branch", "s_endpgm", "s_setpc_b64"):
            into[i + 1].append(i)
        if to in at:
            into[at[to]].append(i)
    bad = []
    for i, (a, op, operands, _) in enumerate(ins):
        if not re.match(r"(buffer|tbuffer|global|flat|scratch)_", op):
            continue
        reads = set().union(*(scalars(w) for p in operands.split(",") for w in p.split()))
        work, seen = [(j, 0) for j in into[i]], set()
        while reads and work:
            j, states = work.pop()
            if states >= STATES or (j, states) in seen:
                continue
            seen.add((j, states))
            _, o, w, _ = ins[j]
            if written(o, w) & reads:
                bad.append((hex(a), op, operands, o, w, states))
                break
            more = int(w, 0) + 1 if o == "s_nop" else 1
            work += [(p, states + more) for p in into[j]]
    return bad


def test_scalar_operands_of_vector_memory(tmp_path):
    checked, bad = 0, {}
    for name, ins in kernels(str(tmp_path)):
        checked += sum(op.startswith("buffer_load") for _, op, _, _ in ins)
        found = too_early(ins)
        if found:
            bad[name] = (len(found), found[0])
    assert checked > 500
    assert not bad, "\n".join(f"{k}: {v}" for k, v in bad.items())


def test_the_check_finds_them():
    """The walk over instructions by itself: straight, behind s_nop, and round
    a loop."""
    load = ("buffer_load_dwordx4", "v1, s[4:7], s9 offen lds", None)
    first = ("v_readfirstlane_b32", "s6, v2", None)

    def run(*body):
        return too_early([(4 * i, *b) for i, b in enumerate(body)])

    def nop(n):
        return "s_nop", str(n), None

    assert run(first, load) and run(first, nop(3), load) and not run(first, nop(4), load)
    assert run(first, ("s_mov_b32", "m0, s3", None), nop(0), load)
    assert not run(first, ("s_mov_b32", "m0, s3", None), nop(3), load)
    assert run(("v_readlane_b32", "s9, v2, 3", None), load)
    assert run(("v_cmp_lt_u32_e64", "s[4:5], v0, v1", None), load)
    assert not run(("v_readfirstlane_b32", "s8, v2", None), load)
    assert run(load, nop(0), first, ("s_cbranch_scc1", "65000", 0))
    assert not run(load, first, nop(3), ("s_cbranch_scc1", "65000", 0))


def test_asm_names_m0():
    """asm that writes m0 says so (as a clobber or as an operand that it
    changes): the compiler may keep an index or an LDS address
    there."""
    src = os.path.join(moe.PKG, "csrc")
    found = 0
    for f in sorted(os.listdir(src)):
        text = re.sub(r"//[^\n]*", "", open(os.path.join(src, f)).read())
        for m in re.finditer(r"\basm volatile\s*\((.*?)\);", text, re.S):
            code, *rest = re.split(r"\n\s*:", m[1])
            rest = "".join(rest)
            found += "m0" in m[1]
            if re.search(r"\bm0\s*,", code):
                assert '"m0"' in rest or '"+{m0}"' in rest, f"{f}: {code.strip()}"
    assert found >= 4


def test_no_stores_that_no_call_reaches(tmp_path):
    """The few-row kernel stores single elements for microscaled operands only:
    bf16 calls without whole 16-byte pieces of y go to another kernel."""
    seen = 0
    for name, ins in kernels(str(tmp_path)):
        m = re.search(r"skinny_kernelILi(\d+)ELi\dE(\w)E", name)
        if m:
            single = "global_store_short" if m[2] == "t" else "global_store_dword"
            stores = sum(op == single for _, op, _, _ in ins)
            assert (stores > 0) == (m[1] != "16"), name
            seen += 1
    assert seen == 12
