"""Read gfx950 assembly text and find instructions that touch a matrix-core
instruction's result too early.

The result of an MFMA may be read or overwritten by an instruction that is not
an MFMA only after a number of wait states: 7 for the forms of 4 passes (bf16 16x16x32), 11
for those of 8 (16x16x128).
The compiler inserts them after MFMAs written as builtins; after those in
inline assembly it sees an ordinary instruction, so a register copy that it
adds itself (where a kernel runs short of registers, say) can read the
accumulator while the MFMA still runs.  Every path from an MFMA is followed
until they have passed: an instruction counts one, ``s_nop N``
counts N + 1, another MFMA as many as its issue takes, 4."""
import re

import asm_hazards

MFMA_ISSUE = 4


def need(op):
    return 7 if "16x16x32" in op else 11


def _touched(ops):
    out = set()
    for o in ops:
        if o:
            out |= asm_hazards._regs(o.split()[0])
    return out


def find(text):
    """[(function, line, instruction, the MFMA's line, wait states seen)] for every violation."""
    ins, labels = asm_hazards._instructions(text)
    found = set()
    for i, (func, line, op, ops, _) in enumerate(ins):
        if not op.startswith("v_mfma"):
            continue
        result, limit = asm_hazards._regs(ops[0]), need(op)
        todo, seen = [(i + 1, 0)], {}
        while todo:
            k, waited = todo.pop()
            while k < len(ins) and ins[k][0] == func and waited < limit:
                if seen.get(k, limit) <= waited:
                    break
                seen[k] = waited
                _, ln, o, args, full = ins[k]
                if o.startswith("v_mfma"):
                    if args and asm_hazards._regs(args[0]) == result:
                        break                      # the next product on the same accumulator: in order
                    waited += MFMA_ISSUE
                elif o in ("s_endpgm", "s_setpc_b64"):
                    break
                elif o.startswith(("s_cbranch", "s_branch")):
                    to = labels.get((func, args[0])) if args else None
                    waited += 1
                    if to is not None:
                        todo.append((to, waited))
                    if o == "s_branch":
                        break
                elif o == "s_nop":
                    waited += int(args[0], 0) + 1
                else:
                    if not o.startswith("s_") and _touched(args) & result:
                        found.add((func, ln, full, line, waited))
                        break
                    waited += 1
                k += 1
    return sorted(found)
