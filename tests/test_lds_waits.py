"""No wave of the built kernels passes a workgroup barrier with LDS accesses of its
own in flight (no GPU needed).

s_barrier waits for no memory access.  A write still on its way at the barrier may
land after another wave's read of it, and a read may return what another wave wrote
after it; neither shows in results reliably, so the instructions are checked.  The
library's own code objects are listed, and along every path through a kernel the LDS
accesses since the last sufficient s_waitcnt lgkmcnt are followed: a wave's LDS
accesses complete in order, so lgkmcnt(n) leaves at most its n newest in flight.
(Direct loads into LDS count in vmcnt and stay in flight across barriers by design.)
"""
import os
import re
import struct
import subprocess

import pytest

import w8a8_fp8_block_amd as fp8q

OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"
MAGIC = b"__CLANG_OFFLOAD_BUNDLE__"
READ, WRITE = 0, 1


def _code_objects(blob):
    """The gfx950 code objects of the library's offload bundles."""
    at = blob.find(MAGIC)
    while at >= 0:
        entry = at + len(MAGIC) + 8
        for _ in range(struct.unpack_from("<Q", blob, entry - 8)[0]):
            off, size, n = struct.unpack_from("<QQQ", blob, entry)
            if b"gfx950" in blob[entry + 24:entry + 24 + n]:
                yield blob[at + off:at + off + size]
            entry += 24 + n
        at = blob.find(MAGIC, at + len(MAGIC))


def _kernels(listing):
    """(name, [(address, mnemonic, operands, branch target address or None)])."""
    name, base, body = None, 0, []
    for line in listing.splitlines():
        m = re.match(r"^([0-9a-f]+) <(.+)>:$", line)
        if m:
            if body:
                yield name, body
            name, base, body = m.group(2), int(m.group(1), 16), []
            continue
        m = re.match(r"^\s+(\S+)(.*?)\s*// ([0-9A-F]+):(.*)$", line)
        if m and name:
            t = re.search(r"<%s(?:\+0x([0-9a-f]+))?>" % re.escape(name), m.group(4))
            body.append((int(m.group(3), 16), m.group(1), m.group(2), base + int(t.group(1) or "0", 16) if t else None))
    if body:
        yield name, body


def _step(state, op, args):
    """state: per kind, how many LDS accesses ago (1: the newest) the newest one in
    flight was issued, 0 if none is."""
    if op.startswith("ds_") and not op.startswith(("ds_bpermute", "ds_permute", "ds_swizzle")):
        kinds = (READ,) if op.startswith("ds_read") else (WRITE,)
        return tuple(1 if k in kinds else (p + 1 if p else 0) for k, p in enumerate(state))
    if op.startswith("ds_"):  # crosses lanes, touches no LDS, counts in lgkmcnt
        return tuple(p + 1 if p else 0 for p in state)
    if op == "s_waitcnt":
        m = re.search(r"lgkmcnt\((\d+)\)", args)
        if m:
            return tuple(p if p <= int(m.group(1)) else 0 for p in state)
    return state


def _join(a, b):
    return tuple(min(p, q) if p and q else p or q for p, q in zip(a, b))


def in_flight_at_barriers(body):
    """[(address, kind)] of the barriers that some path reaches with an LDS access in
    flight."""
    index = {a: i for i, (a, *_) in enumerate(body)}
    states, todo, found = {0: (0, 0)}, [0], set()
    while todo:
        i = todo.pop()
        s = states[i]
        while i < len(body):
            addr, op, args, target = body[i]
            if op == "s_barrier":
                found |= {(addr, k) for k in (READ, WRITE) if s[k]}
            s = _step(s, op, args)
            ends = op in ("s_endpgm", "s_branch")
            nexts = [index[target]] if target is not None else []
            if not ends and (nexts or i + 1 in states):
                nexts.append(i + 1)
            if nexts or ends:
                for n in nexts:
                    j = _join(states[n], s) if n in states else s
                    if states.get(n) != j:
                        states[n] = j
                        todo.append(n)
                break
            i += 1
    return sorted(found)


def test_the_check_itself():
    """On written listings: a missing wait, a partial one, one on a single path."""
    def found(*ops):
        body = []
        for i, o in enumerate(ops):
            op, _, args = o.partition(" ")
            m = re.search(r"->(\d+)", args)
            body.append((i, op, args, int(m.group(1)) if m else None))
        return in_flight_at_barriers(body)

    assert found("ds_write_b32 v0, v1", "s_barrier", "s_endpgm") == [(1, WRITE)]
    assert found("ds_write_b32 v0, v1", "s_waitcnt lgkmcnt(0)", "s_barrier", "s_endpgm") == []
    assert found("ds_write_b32 v0, v1", "s_waitcnt vmcnt(0)", "s_barrier", "s_endpgm") == [(2, WRITE)]
    assert found("ds_write_b32 v0, v1", "ds_read_b32 v2, v3", "s_waitcnt vmcnt(0) lgkmcnt(1)", "s_barrier",
                 "s_endpgm") == [(3, READ)]
    assert found("s_cbranch_scc0 ->2", "ds_read_b32 v2, v3", "s_barrier", "s_endpgm") == [(2, READ)]
    # a loop: the access follows the barrier and reaches it again
    assert found("s_barrier", "ds_read_b32 v2, v3", "s_cbranch_scc0 ->0", "s_endpgm") == [(0, READ)]
    assert found("s_branch ->2", "ds_read_b32 v2, v3", "s_barrier", "s_endpgm") == []


@pytest.mark.skipif(not os.path.exists(OBJDUMP), reason="no llvm-objdump")
def test_no_lds_access_in_flight_at_a_barrier(tmp_path):
    fp8q.lib()
    faults, barriers = [], 0
    for i, code in enumerate(_code_objects(open(fp8q.LIB_PATH, "rb").read())):
        path = tmp_path / f"{i}.co"
        path.write_bytes(code)
        listing = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", path], capture_output=True, text=True,
                                 check=True).stdout
        for name, body in _kernels(listing):
            barriers += sum(op == "s_barrier" for _, op, *_ in body)
            faults += [f"{name}+{a - body[0][0]:#x}: {('read', 'write')[k]}" for a, k in in_flight_at_barriers(body)]
    assert barriers > 100
    assert not faults, "\n".join(faults)
