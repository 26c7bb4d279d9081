"""Order of the tree attention's accesses to tensor memory in a softmax step, read from the kernel's source (CPU).

A store to tensor memory is done for the thread that issued it only behind a wait for its stores.  A row's reference
may move in the first half of a unit and another row's of the same warp in the second: the result's columns, stored by
the first move, are then loaded again.  The statements of one half are read from the source and run for every
combination of moves, each store pending until the next wait; a load of columns with a store pending is a fault.
"""
import itertools
import os
import re

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
SOURCE = os.path.join(HERE, "..", "position_independent_kv_critical_gb300", "csrc", "kernel_tree.cuh")


def text_of_a_half():
    """Source of the loop over a unit's halves, and of what follows it up to the weights' hand-over."""
    with open(SOURCE) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    start = text.index("for (int h = 0; h < 2; ++h)")
    return text[start: text.index("tc_fence_before();", text.index("l_run += sum", start))]


TOKENS = re.compile(r"(?P<open>\{)|(?P<close>\})|(?P<half>if \(h == 1\))|(?P<cols>for \(int cc = q > 0 [^{]*)"
                    r"|(?P<again>for \(bool again[^{]*)|(?P<vote>if \(again \|\| [^;]*break;)"
                    r"|(?P<wait>tmem_st_wait\(\))|(?P<access>tmem_(?:ld|st)(?:16|32)\(t[SO][^;]*;)")


def statements(text):
    """Nested lists of (kind, text): what is in braces behind a condition or loop is its body."""
    def block(tokens):
        out, head = [], None
        for kind, value in tokens:
            if kind == "close":
                return out
            if kind == "open":
                body = block(tokens)
                out.append((head or "plain", body))
                head = None
            elif kind in ("half", "cols", "again"):
                head = kind
            else:
                out.append((kind, value))
        return out
    return block(iter([(m.lastgroup, m.group()) for m in TOKENS.finditer(text)]))


def faults(program, moves):
    """Loads of a unit behind the first whose halves in `moves` move the reference that meet a pending store."""
    pending, found = set(), []

    class Done(Exception):
        pass

    def access(value, h):
        if value.startswith("tmem_ld"):
            # (scores of half h: columns 32 h ..; weights of half h: columns 16 h .., on the first half's scores)
            place = {"result"} if "tO" in value else {("s", x) for x in (range(2 * h, 2 * h + 2) if "32 * h" in value else (0,))}
            found.extend((value, h) for x in place if x in pending)
        else:
            pending.update({"result"} if "tO" in value else {("s", h if "16 * h" in value else 0)})

    def run(body, h, again):
        for kind, value in body:
            if kind == "wait":
                pending.clear()
            elif kind == "access":
                access(value, h)
            elif kind == "vote":
                if again or h not in moves:
                    raise Done
            elif kind == "half":
                if h == 1:
                    run(value, h, again)
            elif kind == "again":
                try:
                    for turn in (False, True):
                        run(value, h, turn)
                except Done:
                    pass
            else:
                run(value, h, again)

    (kind, unit), *behind = [s for s in program if isinstance(s[1], list)][:1] + [s for s in program if not isinstance(s[1], list)]
    for h in range(2):
        run(unit, h, False)
    run(behind, 1, False)
    if pending:
        found.append(("weights or result handed over before they are stored", 1))
    return found


def test_the_source_is_read_whole():
    text = text_of_a_half()
    kinds = [m.lastgroup for m in TOKENS.finditer(text)]
    assert kinds.count("again") == kinds.count("vote") == kinds.count("half") == kinds.count("cols") == 1
    assert len(re.findall(r"tmem_(?:ld|st)(?:16|32)\(", text)) == kinds.count("access") == 7


@pytest.mark.parametrize("moves", [m for n in range(3) for m in itertools.combinations(range(2), n)])
def test_no_load_meets_a_pending_store(moves):
    assert faults(statements(text_of_a_half()), moves) == []


def test_a_missing_wait_is_found():
    text = text_of_a_half()
    at = [m.start() for m in re.finditer(r"tmem_st_wait\(\);", text)]
    for i in at:
        cut = text[:i] + text[i + len("tmem_st_wait();"):]
        assert any(faults(statements(cut), m) for m in ((), (0,), (1,), (0, 1)))
