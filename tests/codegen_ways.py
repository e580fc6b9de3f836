"""Compiled kernels as blocks and ways between them, and what can go wrong around
matrix instructions in inline assembly, whose waits the compiler does not know.

A matrix instruction's result must not be read or written for LATENCY wait
states, except by a matrix instruction that adds to it in place, and no vector
instruction may write a register OPERAND wait states or less before a matrix
instruction reads it.  Both are followed along every way through a kernel.
An instruction counts as one wait state, s_nop n as n + 1: no instruction takes
less.

The loops end in a piece of assembly that waits in the last turn only:
    s_cmp_lt_i32 at, end;  s_cbranch_scc1 .Lturn;  s_nop ..;  .Lturn:
It is followed by the loop's own branch on the same comparison, so a way that
skipped the wait goes on with the next turn, and one that waited leaves.
"""
import re

LATENCY = 19  # the longest of them: 16 passes of a 32 x 32 result; these have 8
OPERAND = 2


def parse(text):
    """{kernel: (instructions, {label: position}, {position of an instruction in inline assembly})}."""
    found = {}
    for m in re.finditer(r"^(_ZN\S+):\s*;.*?\n(.*?)\.Lfunc_end", text, re.S | re.M):
        code, labels, inline, inside = [], {}, set(), False
        for line in m[2].split("\n"):
            if "#ASMSTART" in line or "#ASMEND" in line:
                inside = "#ASMSTART" in line
                continue
            line = line.split(";")[0].strip()
            at = re.match(r"(\.L\w+):", line)
            if at:
                labels[at[1]] = len(code)
            elif line and not line.startswith("."):
                if inside:
                    inline.add(len(code))
                code.append(line)
        found[m[1]] = (code, labels, inline)
    return found


def registers(text):
    """Vector registers and accumulators that an operand list names."""
    got = set()
    for kind, lo, hi in re.findall(r"\b([av])\[(\d+):(\d+)\]", text):
        got |= {kind + str(i) for i in range(int(lo), int(hi) + 1)}
    return got | {k + n for k, n in re.findall(r"\b([av])(\d+)\b", text)}


def operands(line):
    """The operands of an instruction, each as text."""
    parts = line.split(None, 1)
    return [x.strip() for x in parts[1].split(",")] if len(parts) > 1 else []


def blocks_of(code, labels):
    """First positions of blocks: labels and what follows a branch."""
    starts = {0} | {p for p in labels.values() if p < len(code)}
    starts |= {i + 1 for i, x in enumerate(code) if re.match(r"s_c?branch|s_endpgm|s_setpc", x) and i + 1 < len(code)}
    return sorted(starts)


def _ways(code, labels, at, end):
    """Blocks that may follow code[at:end], as (position, taken)."""
    last = code[end - 1]
    m = re.match(r"s_(c?)branch\S*\s+(\S+)", last)
    if m:
        to = [(labels[m[2]], True)]
        return to + [(end, False)] if m[1] else to
    if last.startswith("s_setpc"):  # a branch too long for one instruction: its target was added to the position
        m = [re.search(r"\(?(\.LBB\w+)-\.Lpost_getpc", x) for x in code[at:end]]
        return [(labels[x[1]], True) for x in m if x][:1]
    return [] if last.startswith("s_endpgm") else [(end, False)]


def _step(line, inline, now, busy, written, report):
    """The state after one instruction: busy and written hold when a register is free again."""
    op = line.split()[0]
    args = operands(line)
    if op == "s_nop":
        return now + int(args[0]) + 1
    named = registers(" ".join(args))
    if op.startswith("v_mfma"):
        result = registers(args[0])
        in_place = args[0] == args[3]
        early = {r for r in named if busy.get(r, now) > now and not (in_place and r in result)}
        early |= {r for r in registers(args[1] + " " + args[2]) & result if busy.get(r, now) > now}
        if inline:
            late = {r for r in named if written.get(r, now) > now}
            if late:
                report(line, "written right before", late)
        if early:
            report(line, "not there yet", early)
        for r in result:
            written.pop(r, None)
            if inline:
                busy[r] = now + 1 + LATENCY
            else:
                busy.pop(r, None)
        return now + 1
    early = {r for r in named if busy.get(r, now) > now}
    if early:
        report(line, "not there yet", early)
    if op.startswith("v_") and args:
        for r in registers(args[0]) | (registers(args[1]) if "swap" in op and len(args) > 1 else set()):
            written[r] = now + 1 + OPERAND
    return now + 1


def hazards(kernel):
    """Every (instruction, what, registers) that some way through a kernel leads to."""
    code, labels, inline = kernel
    starts = blocks_of(code, labels)
    ends = dict(zip(starts, starts[1:] + [len(code)]))
    found = set()
    states = {(0, None): ({}, {})}  # (block, comparison that the turn's end decided, and how): states on entry
    todo = [(0, None)]
    while todo:
        key = todo.pop()
        at, turn = key
        end = ends[at]
        busy, written = (dict(s) for s in states[key])
        now = 0
        for i in range(at, end):
            now = _step(code[i], i in inline, now, busy, written,
                        lambda line, what, regs, i=i: found.add((i, line, what, tuple(sorted(regs)))))
        left = tuple({r: t - now for r, t in s.items() if t > now} for s in (busy, written))
        last, before = code[end - 1], code[max(at, end - 2)]
        ways = _ways(code, labels, at, end)
        if (end - 1) in inline and last.startswith("s_cbranch_scc1 .Lturn"):  # taken: another turn
            compared = operands(before)
            ways = [(p, (tuple(compared), taken)) for p, taken in ways]
        elif turn is not None and last.startswith("s_cbranch_scc"):
            m = re.match(r"s_cmp_(ge|lt)_i32", before)
            if not m or tuple(operands(before)) != turn[0]:
                found.add((end - 1, last, "another branch behind a turn's end", ()))
            jump_is_more = (m is not None) and (m[1] == "lt") == (last.split()[0] == "s_cbranch_scc1")
            ways = [(p, None) for p, taken in ways if (taken == jump_is_more) == turn[1]]
        else:
            ways = [(p, turn) for p, _ in ways]
        for to in ways:
            if to[0] >= len(code):
                continue
            old = states.get(to)
            new = left if old is None else tuple({r: max(a.get(r, 0), b.get(r, 0)) for r in a.keys() | b.keys()}
                                                 for a, b in zip(old, left))
            if old is None or new != old:
                states[to] = new
                if to not in todo:
                    todo.append(to)
    return sorted(found)


def loops(kernel):
    """The innermost loops that multiply, as lists of their blocks' (first, last) positions: what leads back to a
    block that every way to it passes."""
    code, labels, _ = kernel
    starts = blocks_of(code, labels)
    ends = dict(zip(starts, starts[1:] + [len(code)]))
    to = {b: sorted({p for p, _ in _ways(code, labels, b, ends[b]) if p < len(code)}) for b in starts}
    order, seen, stack = [], {0}, [(0, iter(to[0]))]  # blocks, each after those it leads to
    while stack:
        b, rest = stack[-1]
        nxt = next((p for p in rest if p not in seen), None)
        if nxt is None:
            order.append(b)
            stack.pop()
        else:
            seen.add(nxt)
            stack.append((nxt, iter(to[nxt])))
    order.reverse()
    number = {b: i for i, b in enumerate(order)}
    ahead = {b: [] for b in order}
    for b in order:
        for p in to[b]:
            ahead[p].append(b)
    every = (1 << len(order)) - 1
    passed = {b: every for b in order}  # as bits: the blocks on every way to one
    passed[0] = 1
    changed = True
    while changed:
        changed = False
        for b in order[1:]:
            bits = every
            for p in ahead[b]:
                bits &= passed[p]
            bits |= 1 << number[b]
            changed |= bits != passed[b]
            passed[b] = bits
    bodies = {}
    for b in order:
        for head in to[b]:
            if passed[b] >> number[head] & 1:
                body, todo = bodies.setdefault(head, {head}), [b]
                while todo:
                    x = todo.pop()
                    if x not in body:
                        body.add(x)
                        todo += ahead[x]
    found = [body for body in bodies.values()
             if sum(code[i].startswith("v_mfma") for b in body for i in range(b, ends[b])) >= 16]
    return [[(b, ends[b] - 1) for b in sorted(body)] for body in found if not any(o < body for o in found)]
