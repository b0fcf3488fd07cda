"""asm_copies for the large-tile kernels that stage E8M0 scales for several
k-tiles at once: there two kinds of asynchronous global -> LDS copies, A's of
every k-tile and those of a scale stage, go through the same instruction and
are told apart by the buffer resource they read (A's is the one with the most
copies; every k-tile has some).

A's copies are followed as in asm_copies, with the scale copies among the loads
behind them.  A stage's copies are first read `ahead` barriers after the one
they are issued behind, those in front of the loop at the first barrier: from
every barrier each path is followed backwards, and where it has passed that
many barriers the scale copies on it have to have at least as many loads
behind them as the wait lets be outstanding, or an earlier wait that covers
them."""
import collections
import re

import asm_hazards
from asm_copies import _vmcnt, is_copy, is_load


def _resource(ins):
    return re.search(r"s\[\d+:\d+\]", ins[4]).group(0)


def find(text, plan):
    """([(function, line of the wait, line of the copy)], waits checked, scale
    copies followed); plan(function name) -> (A copies that may be outstanding,
    ahead), None: not such a kernel."""
    ins, labels = asm_hazards._instructions(text)
    preds, quads, first = {}, {}, {}
    for k, (func, _, op, ops, _) in enumerate(ins):
        if op.startswith(("s_cbranch", "s_branch")):
            to = labels.get((func, ops[0])) if ops else None
            if to is not None:
                preds.setdefault(to, []).append(k)
        if op not in ("s_branch", "s_endpgm", "s_setpc_b64") and k + 1 < len(ins) and ins[k + 1][0] == func:
            preds.setdefault(k + 1, []).append(k)
        if is_copy(ins[k]):
            quads.setdefault(func, collections.Counter())[_resource(ins[k])] += 1

    def wait(b):   # the count of a barrier that lets a k-tile be read, else None
        n = _vmcnt(ins[b - 1]) if ins[b][2] == "s_barrier" and ins[b - 1][0] == ins[b][0] else None
        return n or None

    waits = {b: wait(b) for b in range(1, len(ins)) if wait(b)}
    for b in sorted(waits, reverse=True):
        first[ins[b][0]] = b
    found, scales = [], set()
    for b, n in waits.items():
        func = ins[b][0]
        p = plan(func)
        if p is None:
            continue
        newer, ahead = p
        a_quad = quads[func].most_common(1)[0][0]
        todo, seen, bad = [(k, 0, 0, 0, n) for k in preds.get(b - 1, [])], set(), False
        while todo and not bad:
            state = todo.pop()
            k, loads, copies, passed, limit = state
            if state in seen or loads >= limit:
                continue
            seen.add(state)
            w = _vmcnt(ins[k])
            if w is not None:
                limit = min(limit, loads + w)
            elif ins[k][2] == "s_barrier" and k in waits:
                passed = min(passed + 1, ahead)
            elif is_copy(ins[k]) and _resource(ins[k]) == a_quad:
                bad = copies == newer
                loads, copies = loads + 1, copies + 1
            elif is_copy(ins[k]):
                scales.add(k)
                bad = passed >= (0 if k < first[func] else ahead)
                loads += 1
            elif is_load(ins[k][2]):
                loads += 1
            if bad:
                found.append((func, ins[b - 1][1], ins[k][1]))
            todo += [(q, loads, copies, passed, limit) for q in preds.get(k, [])]
    return found, sum(plan(ins[b][0]) is not None for b in waits), len(scales)
