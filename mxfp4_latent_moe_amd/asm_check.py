"""Check of gfx950 assembly built here: registers that an LDS read is still to fill.

Kernels that pace their LDS reads by hand issue them in inline assembly, one
block for a read and another, later, for the wait.  The compiler takes such a
register as written where the read stands: a copy or a spill that it puts before
the wait would carry the old value on, with no error.  Whether it did is plain
from the assembly: along every path through a kernel, no instruction may name a
register between the read that fills it and the wait that covers the read.
"""
from __future__ import annotations

import re

_REG = re.compile(r"\b([av])(?:(\d+)\b|\[(\d+):(\d+)\])")
_FILLS = re.compile(r"ds_(?:read|load|bpermute|permute|swizzle|consume|append|\w+_rtn)")
_COUNTED = 15  # the most that a wait can leave in flight
_MOST_STATES = 4096


def _regs(text):
    return [(m[1], int(m[2] or m[3]), int(m[2] or m[4])) for m in _REG.finditer(text)]


def _meets(a, b):
    return a is not None and a[0] == b[0] and a[1] <= b[2] and b[1] <= a[2]


def _kernels(asm):
    """(name, [(line number, text)]) of each function."""
    name, lines = None, []
    for no, line in enumerate(asm.splitlines(), 1):
        text = line.split(";")[0].strip()
        label = re.match(r"(\w\S*):$", text)
        if label and not text.startswith(".L"):
            if name is not None:
                yield name, lines
            name, lines = label[1], []
        elif text and (not text.startswith(".") or text.startswith(".LBB")):
            lines.append((no, text))
    if name is not None:
        yield name, lines


def _blocks(lines):
    """Straight pieces of code, and the piece that each label begins."""
    blocks, at = [[]], {}
    for no, text in lines:
        label = re.match(r"(\.LBB\S+):$", text)
        if label:
            blocks.append([])
            at[label[1]] = len(blocks) - 1
            continue
        blocks[-1].append((no, text))
        if text.startswith(("s_branch", "s_cbranch", "s_endpgm")):
            blocks.append([])
    return blocks, at


def _step(text, flight, no, name, found):
    """The reads in flight behind an instruction.  LDS operations end in their order, so `flight` is the newest
    _COUNTED of them, oldest first, and the set of those before, which any wait covers."""
    old, new = flight
    wait = re.search(r"lgkmcnt\((\d+)\)", text)
    if wait:
        return frozenset(), new[max(0, len(new) - int(wait[1])):]
    if text.startswith("s_waitcnt"):
        return (frozenset(), ()) if re.fullmatch(r"s_waitcnt\s+(0|0x0)", text) else flight
    if text.startswith("s_"):
        return flight
    regs = _regs(text)
    if any(_meets(p, r) for p in (*old, *new) for r in regs):
        found.add((name, no, text))
    if text.startswith("ds_"):
        new += (regs[0] if _FILLS.match(text) and regs else None,)
        return old | {p for p in new[:-_COUNTED] if p is not None}, new[-_COUNTED:]
    return flight


def unsafe_reads(asm: str) -> list:
    """(function, line, instruction) for every use of a register that an LDS read in flight is to fill."""
    found = set()
    for name, lines in _kernels(asm):
        if not any(text.startswith("ds_") for _, text in lines):
            continue
        blocks, at = _blocks(lines)
        seen = [set() for _ in blocks]
        work = [(0, (frozenset(), ()))]
        while work:
            i, flight = work.pop()
            if i >= len(blocks) or flight in seen[i]:
                continue
            seen[i].add(flight)
            if len(seen[i]) > _MOST_STATES:
                raise RuntimeError(f"{name}: too many states of reads in flight")
            follows = [i + 1]
            for no, text in blocks[i]:
                if text.startswith("s_branch"):
                    follows = [at[text.split()[1]]]
                elif text.startswith("s_cbranch"):
                    follows = [i + 1, at[text.split()[1]]]
                elif text.startswith("s_endpgm"):
                    follows = []
                flight = _step(text, flight, no, name, found)
            work += [(j, flight) for j in follows]
    return sorted(found)
