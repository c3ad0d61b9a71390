"""Numeric labels of inline assembly, and vector-ALU results on their way into
an inline matrix instruction, for the checks of mfma_hazards.

``named_labels`` gives every numeric label ("1:") a name of its own and points
the branches to it ("1f", "1b") there, so that a scan follows them.

``scan_sources`` finds matrix instructions that read a register which a
vector-ALU instruction wrote fewer than SOURCE_WAIT wait states before. The
compiler keeps that distance for its own matrix instructions, not for those
written as inline assembly.
"""
from __future__ import annotations

import re

import mfma_hazards as mh

SOURCE_WAIT = 2


def named_labels(lines: list[str]) -> list[str]:
    out = list(lines)
    last: dict[str, str] = {}
    waiting: dict[str, list[int]] = {}
    for i, line in enumerate(lines):
        label = re.match(r"^(\d+):$", line)
        branch = re.match(r"^(s_c?branch\w*\s+)(\d+)([fb])$", line)
        if label:
            name = f".Lnumeric{i}"
            out[i] = name + ":"
            last[label.group(1)] = name
            for j in waiting.pop(label.group(1), []):
                out[j] = out[j].rsplit(None, 1)[0] + " " + name
        elif branch and branch.group(3) == "f":
            waiting.setdefault(branch.group(2), []).append(i)
        elif branch:
            out[i] = branch.group(1) + last[branch.group(2)]
    assert not waiting, "a branch to a numeric label that does not follow"
    return out


def scan_sources(lines: list[str], wait: int = SOURCE_WAIT) -> list[tuple[int, str, str]]:
    def step(i, ins, state, report):
        op = ins.split()[0]
        parts = [p.strip() for p in ins[len(op):].split(",")]
        if op.startswith("v_mfma"):
            for r in set().union(*(mh._regs(p) for p in parts[1:])):
                if state.get(r, 0) > 0:
                    report.append((i, ins, r))
        paid = int(ins.split()[1], 0) + 1 if op == "s_nop" else 1
        state = {r: w - paid for r, w in state.items() if w - paid > 0}
        if op.startswith("v_") and not op.startswith("v_mfma"):
            for r in mh._regs(parts[0]):
                state[r] = wait
        return state

    return mh._flow(lines, step)
