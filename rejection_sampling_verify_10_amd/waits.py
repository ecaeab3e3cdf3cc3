"""Checks compiled kernels for reads of matrix sums that nothing waited for.

Where a kernel issues its matrix products in inline assembly, the compiler sees no matrix instruction and places no wait
states before what reads their result; the kernel does, in assembly of its own.  Whether every path has them depends on
where the compiler puts copies of those registers, so each build is looked over (:func:`unwaited`): after such a product, no
instruction but another one may touch the registers it wrote before 32 wait states (``s_nop``) have passed.  A product of
sixteen passes needs 18.
"""

from __future__ import annotations

import re
from typing import Dict, FrozenSet, List, Set, Tuple

WAIT_STATES = 32

_RANGE, _ONE = re.compile(r"\b([av])\[(\d+):(\d+)\]"), re.compile(r"\b([av])(\d+)\b")


def _registers(text: str) -> Set[Tuple[str, int]]:
    out = {(m[1], i) for m in _RANGE.finditer(text) for i in range(int(m[2]), int(m[3]) + 1)}
    return out | {(m[1], int(m[2])) for m in _ONE.finditer(text)}


def _blocks(lines: List[str]) -> Tuple[List[List[Tuple[str, bool]]], List[Set[int]]]:
    """Basic blocks of a function, (instruction, whether it stands in inline assembly), and their successors."""
    blocks: List[List[Tuple[str, bool]]] = [[]]
    label: Dict[str, int] = {}
    inline = False
    for line in lines:
        m = re.match(r"(\.L\w+):", line)
        if m:
            blocks.append([])
            label[m[1]] = len(blocks) - 1
            continue
        text = line.strip()
        if text.startswith((";APP", ";;#ASMSTART", "#APP", "; APP")):
            inline = True
        elif text.startswith((";NO_APP", ";;#ASMEND", "#NO_APP", "; NO_APP")):
            inline = False
        text = text.split(";")[0].strip()
        if text and not text.startswith((".", "#")):
            blocks[-1].append((text, inline))
    succ = []
    for k, block in enumerate(blocks):
        to, falls = set(), True
        for text, _ in block:
            m = re.match(r"s_(c?branch\w*)\s+(\.L\w+)", text)
            if m:
                to.add(label[m[2]])
            falls = not text.startswith(("s_branch", "s_endpgm"))
        if falls and k + 1 < len(blocks):
            to.add(k + 1)
        succ.append(to)
    return blocks, succ


def unwaited(assembly: str) -> Tuple[int, List[str]]:
    """(products in inline assembly, accesses of their results that come too early), over all functions of a device assembly."""
    found, early = 0, []
    for m in re.finditer(r"^(\w+):.*?^\.Lfunc_end\w*:", assembly, re.M | re.S):
        body = m[0]
        if "v_mfma" not in body:
            continue
        blocks, succ = _blocks(body.split("\n")[1:])
        if not any(inline and "v_mfma" in text for b in blocks for text, inline in b):
            continue
        found += sum(inline and "v_mfma" in text for b in blocks for text, inline in b)
        # registers written by a product and not waited for, with the wait states passed, at each block's start
        start: List[Dict[Tuple[str, int], int]] = [{} for _ in blocks]
        seen: List[bool] = [False] * len(blocks)
        work, bad = [0], {}
        seen[0] = True
        while work:
            k = work.pop()
            open_: Dict[Tuple[str, int], int] = dict(start[k])
            for text, inline in blocks[k]:
                if text.startswith("s_nop"):
                    n = int(text.split()[1], 0) + 1
                    open_ = {r: w + n for r, w in open_.items() if w + n < WAIT_STATES}
                    continue
                regs = _registers(text)
                if inline and "v_mfma" in text:
                    result = _registers(text.split(",")[0])
                    operands = _registers(",".join(text.split(",")[1:3]))
                    if operands & open_.keys():
                        bad[(k, text)] = True
                    open_.update((r, 0) for r in result)
                    continue
                if regs & open_.keys():
                    bad[(k, text)] = True
            for x in succ[k]:
                merged = dict(start[x])
                for r, w in open_.items():
                    merged[r] = min(w, merged.get(r, WAIT_STATES))
                if merged != start[x] or not seen[x]:
                    start[x], seen[x] = merged, True
                    work.append(x)
        early += [f"{m[1]}: {text}" for _, text in bad]
    return found, early
