"""No store of the built gradient kernels reads the result of a matrix instruction before
it is there (no GPU needed).

The hardware does not hold a memory instruction back for a matrix instruction's result:
the wait states between the two are the program's.  The compiler counts them for the
instructions it makes itself, but knows nothing of a store that stands in inline assembly.
So the built kernels are listed, and along every path the wait states since each register
was last written by a matrix instruction are followed to the stores that read it: an
instruction counts one, s_nop n counts n + 1.  A 32 x 32 x 64 FP8 product takes 16 passes,
and a memory instruction may read its result 20 wait states behind it."""
import os
import re
import subprocess

import pytest

import w8a8_fp8_block_amd as fp8q
from test_lds_waits import OBJDUMP, _code_objects, _kernels

ENOUGH = 20
PRODUCTS = ("v_mfma_f32_32x32x64_f8f6f4", "v_mfma_scale_f32_32x32x64_f8f6f4")


def _regs(text):
    """VGPRs and AGPRs that operands name."""
    out = set()
    for kind, lo, hi, single_kind, single in re.findall(r"\b([va])\[(\d+):(\d+)\]|\b([va])(\d+)\b", text):
        out |= {(kind, i) for i in range(int(lo), int(hi) + 1)} if kind else {(single_kind, int(single))}
    return frozenset(out)


def _decode(body):
    """Per instruction: wait states, registers it stores, registers it writes as a product,
    registers it writes otherwise, successors."""
    index = {a: i for i, (a, *_) in enumerate(body)}
    code = []
    for i, (_, op, args, target) in enumerate(body):
        operands = args.split(",")
        states = int(operands[0], 0) + 1 if op == "s_nop" else 1
        store = op.startswith(("global_store", "buffer_store", "flat_store", "scratch_store"))
        vector = op.startswith(("v_", "ds_read", "global_load", "buffer_load", "scratch_load")) and not store
        dest = _regs(operands[0]) if vector and not args.rstrip().endswith(" lds") else frozenset()
        nxt = [] if op.startswith(("s_endpgm", "s_branch")) else [i + 1]
        if target is not None:
            nxt.append(index[target])
        code.append((states, _regs(args) if store else frozenset(), dest if op in PRODUCTS else frozenset(),
                     frozenset() if op in PRODUCTS else dest, [n for n in nxt if n < len(body)]))
    return code


def _too_soon(body):
    """[(address, wait states)] of the stores that read a product's result too soon."""
    code = _decode(body)
    state = [None] * len(code)  # register -> wait states since its product, below ENOUGH
    state[0] = {}
    todo, found = [0], {}
    while todo:
        i = todo.pop()
        s = state[i]
        states, stored, product, other, nxt = code[i]
        for r in stored & s.keys():
            found[body[i][0]] = min(s[r], found.get(body[i][0], ENOUGH))
        out = {r: n + states for r, n in s.items() if n + states < ENOUGH and r not in other}
        out.update((r, 1) for r in product)
        for n in nxt:
            old = state[n]
            new = out if old is None else {**old, **{r: min(c, old.get(r, ENOUGH)) for r, c in out.items()}}
            if new != old:
                state[n] = dict(new)
                todo.append(n)
    return sorted(found.items())


def test_the_check_itself():
    """On written listings: too few wait states, enough, too few on one of two paths."""
    product = PRODUCTS[1] + " v[0:15], v[16:23], v[24:31], v[0:15], v32, v33"
    store = "global_store_dwordx4 v50, v[12:15], s[0:1]"

    def found(*ops):
        body = []
        for i, o in enumerate(ops):
            op, _, args = o.partition(" ")
            m = re.search(r"->(\d+)", args)
            body.append((i, op, args, int(m.group(1)) if m else None))
        return _too_soon(body)

    assert found(product, "s_nop 0", "v_mov_b32_e32 v40, v41", store, "s_endpgm") == [(3, 3)]
    assert found(product, "s_nop 15", "s_nop 2", store, "s_endpgm") == []
    assert found(product, "s_nop 15", "s_nop 1", store, "s_endpgm") == [(3, 19)]
    assert found(product, "v_mov_b32_e32 v12, v13", store, "s_endpgm") == [(2, 2)]  # v13 is still the product's
    assert found(product, "s_cbranch_scc0 ->4", "s_nop 15", "s_nop 15", store, "s_endpgm") == [(4, 2)]
    assert found(product, "global_store_dwordx4 v50, v[40:43], s[0:1]", "s_endpgm") == []


@pytest.mark.skipif(not os.path.exists(OBJDUMP), reason="no llvm-objdump")
def test_stores_wait_for_products(tmp_path):
    fp8q.lib()
    faults, seen = [], 0
    for i, code in enumerate(_code_objects(open(fp8q.LIB_PATH, "rb").read())):
        path = tmp_path / f"{i}.co"
        path.write_bytes(code)
        listing = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", path], capture_output=True, text=True,
                                 check=True).stdout
        for name, body in _kernels(listing):
            if any(op in PRODUCTS for _, op, *_ in body):
                seen += 1
                faults += [f"{name}+{a - body[0][0]:#x}: {n} wait states" for a, n in _too_soon(body)]
    assert seen == 6  # dx: two tiles, whole and in ranges; dW: whole and in ranges
    assert not faults, "\n".join(faults)
