"""Read gfx950 assembly text and find barriers that certify an asynchronous
global -> LDS copy which the wait before them does not cover.

The large-tile kernels copy A a few k-tiles ahead and wait, with a count of
the loads that may still be outstanding (``s_waitcnt vmcnt(N)``, vector-memory
loads complete in order), before the barrier that lets every wave read a
k-tile.  The count is written from the kernel's own order of loads; where the
compiler removes one of them (a reload of B past the last k-tile, whose
register nothing reads), fewer loads follow the copy than the count assumes,
and the wait ends before it has landed.  From every such barrier each path is
followed backwards: past the copies of later k-tiles (`newer` of them), the
next one has to have at least N loads behind it, or an earlier wait that
covers it."""
import re

import asm_hazards


def is_load(op):
    return op.startswith(("buffer_load", "global_load", "buffer_store", "global_store", "flat_"))


def is_copy(ins):
    return ins[2] == "buffer_load_dwordx4" and ins[4].endswith(" lds")


def _vmcnt(ins):
    m = re.search(r"vmcnt\((\d+)\)", ins[4]) if ins[2] == "s_waitcnt" else None
    return int(m.group(1)) if m else None


def find(text, newer):
    """[(function, line of the wait, line of the copy)]; newer(function name)
    -> the copies that may be outstanding, None: not such a kernel."""
    ins, labels = asm_hazards._instructions(text)
    preds = {}
    for k, (func, _, op, ops, _) in enumerate(ins):
        if op.startswith(("s_cbranch", "s_branch")):
            to = labels.get((func, ops[0])) if ops else None
            if to is not None:
                preds.setdefault(to, []).append(k)
        if op not in ("s_branch", "s_endpgm", "s_setpc_b64") and k + 1 < len(ins) and ins[k + 1][0] == func:
            preds.setdefault(k + 1, []).append(k)
    found, checked = [], 0
    for b in range(1, len(ins)):
        func = ins[b][0]
        n = _vmcnt(ins[b - 1]) if ins[b][2] == "s_barrier" else None
        skip = newer(func) if n else None
        if skip is None:
            continue
        checked += 1
        todo, seen = [(p, 0, 0, n) for p in preds.get(b - 1, [])], set()
        while todo:
            k, loads, copies, limit = todo.pop()
            if (k, loads, copies, limit) in seen or loads >= limit:
                continue
            seen.add((k, loads, copies, limit))
            w = _vmcnt(ins[k])
            if w is not None:
                limit = min(limit, loads + w)
            elif is_copy(ins[k]):
                if copies == skip:
                    found.append((func, ins[b - 1][1], ins[k][1]))
                    break
                loads, copies = loads + 1, copies + 1
            elif is_load(ins[k][2]):
                loads += 1
            todo += [(p, loads, copies, limit) for p in preds.get(k, [])]
    return found, checked
