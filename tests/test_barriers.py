"""No block barrier of the kernels stands under the outcome of a bounded wait.

A wait that runs out does so for each warp by itself.  A barrier that only the
warps whose wait succeeded come to would keep them there for good, so barriers
are reached whatever came of the waits before them (read from the sources)."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sparse_long_context_min_b200", "csrc")
BARRIER = re.compile(r"\b(bar_\w+|__syncthreads\w*|cluster_sync|cluster_arrive|cluster_wait)\s*\(")
WAIT = re.compile(r"\b(ok|go|dead|pfx_wait|mbar_\w*wait\w*)\b")


def guarded_barriers(text, call=BARRIER, outcome=WAIT):
    """(line, barrier, condition) of every barrier inside an `if` on a wait's outcome."""
    text = re.sub(r"//[^\n]*", "", text)
    found, stack, i, pending, parens = [], [], 0, None, 0   # stack: the condition in front of each open brace
    while i < len(text):
        m = re.compile(r"\b(?:else\s+)?if\s*(?:constexpr\s*)?\(").match(text, i) if text[i] in "ei" else None
        if m and (i == 0 or not (text[i - 1].isalnum() or text[i - 1] == "_")):
            depth, j = 1, m.end()
            while depth:
                depth += {"(": 1, ")": -1}.get(text[j], 0)
                j += 1
            pending, i = text[m.end():j - 1], j
            continue
        c = text[i]
        b = call.match(text, i) if c.isalpha() or c == "_" else None
        if b and not (text[i - 1].isalnum() or text[i - 1] == "_"):
            for cond in [x for x, _ in stack] + [pending]:
                if cond and outcome.search(cond):
                    found.append((text.count("\n", 0, i) + 1, b.group().rstrip("( "), " ".join(cond.split())))
            i, parens = b.end(), parens + 1
            continue
        if c == "{":
            stack.append((pending, parens))              # (a lambda may stand in an argument list)
            pending, parens = None, 0
        elif c == "}":
            pending, parens = None, stack.pop()[1] if stack else 0
        elif c in "()":
            parens += 1 if c == "(" else -1
        elif c == ";" and parens == 0:                   # (not those of a `for`)
            pending = None
        i += 1
    return found


@pytest.mark.parametrize("path", sorted(glob.glob(os.path.join(CSRC, "*.cu*"))), ids=os.path.basename)
def test_no_barrier_under_a_wait(path):
    with open(path) as f:
        assert guarded_barriers(f.read()) == []


# the loops in which a producer waits for the last loads it issued
LANDED = re.compile(r"mbar_wait\s*\((?=&(?:full|k_full|v_full)\[i )")


@pytest.mark.parametrize("name,loops", [("window.cu", 1), ("prefix.cu", 3)])
def test_loads_have_landed_whoever_gave_up(name, loops):
    """A CTA does not end with loads under way, be it that another role than the
    producer gave up: the producer waits for its last loads in any case."""
    with open(os.path.join(CSRC, name)) as f:
        text = f.read()
    assert len(LANDED.findall(text)) == loops
    assert guarded_barriers(text, LANDED, re.compile(r"\b(stop|go|ok|dead)\b")) == []


def test_the_reading_finds_them():
    bad = "void f() { const bool ok = mbar_wait(b); if (ok && x) { g(); if (y) { bar_halves(3); } } }"
    assert [x[1] for x in guarded_barriers(bad)] == ["bar_halves"]
    assert [x[1] for x in guarded_barriers("{ if (!dead) __syncthreads(); }")] == ["__syncthreads"]
    assert guarded_barriers("{ if (ok) { g(); } bar_halves(3); if (y) __syncthreads(); else { cluster_sync(); } }") == []
