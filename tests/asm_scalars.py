"""Read gfx950 assembly text and find global -> LDS copies that read a scalar
register too early after a vector-ALU instruction wrote it.

A vector-ALU write of a scalar register (a lane read into it, a comparison's
mask) followed by a vector-memory instruction that reads it as its buffer
resource or offset needs 5 wait states in between.  The compiler inserts them
where it knows the instruction; behind inline assembly the kernel itself has to
keep to it, and a register that the compiler spilled comes back with a lane
read of its own.  Every path from the write is followed until the wait states
have passed: an instruction counts one, ``s_nop N`` counts N + 1."""
import re

import asm_hazards

NEED = 5


def _scalars(tok):
    tok = tok.strip().rstrip(",")
    m = re.fullmatch(r"s\[(\d+):(\d+)\]", tok)
    if m:
        return set(range(int(m.group(1)), int(m.group(2)) + 1))
    m = re.fullmatch(r"s(\d+)", tok)
    return {int(m.group(1))} if m else set()


def _written(op, ops):
    """Scalar registers that a vector-ALU instruction writes."""
    if not op.startswith("v_") or not ops:
        return set()
    out = _scalars(ops[0].split()[0])                       # lane reads, comparisons (VOP3)
    if len(ops) > 1 and ("_co_" in op or op.startswith(("v_div_scale", "v_mad_u64", "v_mad_i64"))):
        out |= _scalars(ops[1].split()[0])                  # carry and mask outputs
    return out


def find(text):
    """[(function, line of the copy, instruction, line of the write, wait states seen)] for every violation."""
    ins, labels = asm_hazards._instructions(text)
    found = set()
    for i, (func, line, op, ops, _) in enumerate(ins):
        regs = _written(op, ops)
        if not regs:
            continue
        todo, seen = [(i + 1, 0)], {}
        while todo:
            k, waited = todo.pop()
            if k >= len(ins) or waited >= NEED or ins[k][0] != func or seen.get(k, NEED) <= waited:
                continue
            seen[k] = waited
            _, at, kop, kops, full = ins[k]
            if kop.startswith("buffer_load") and full.split()[-1] == "lds":
                read = set().union(*(_scalars(t) for o in kops for t in o.split())) & regs
                if read:
                    found.add((func, at, full, line, waited))
            after = waited + (int(kops[0], 0) + 1 if kop == "s_nop" else 1)
            if kop.startswith("s_cbranch") or kop == "s_branch":
                target = labels.get((func, kops[0]))
                if target is not None:
                    todo.append((target, after))
            if kop not in ("s_branch", "s_endpgm"):
                todo.append((k + 1, after))
    return sorted(found)
