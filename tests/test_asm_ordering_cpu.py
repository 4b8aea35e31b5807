"""Inline assembly that orders memory is ordered for the compiler as well.

A barrier or an asynchronous copy without a "memory" clobber holds the threads
but not the compiler, which may move ordinary shared-memory accesses across it;
whether it does is not visible in results, so the sources themselves are
checked."""
import glob
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "gated_delta_rule_156_b200", "csrc")


def asm_statements(text):
    """(line, statement) of every asm(...) in a source text."""
    for m in re.finditer(r"\basm\b\s*(?:volatile\b)?\s*\(", text):
        depth, quoted, i = 1, False, m.end()
        while depth:
            c = text[i]
            if c == "\\":
                i += 1
            elif c == '"':
                quoted = not quoted
            elif not quoted:
                depth += (c == "(") - (c == ")")
            i += 1
        yield text.count("\n", 0, m.start()) + 1, text[m.start():i]


def without_clobber(pattern):
    bad, seen = [], 0
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))):
        with open(path) as f:
            for line, stmt in asm_statements(f.read()):
                if re.search(pattern, stmt):
                    seen += 1
                    if '"memory"' not in stmt:
                        bad.append(f"{os.path.basename(path)}:{line}")
    assert seen, pattern
    return bad


def test_the_parser_finds_statements():
    text = 'asm volatile("a; // )" ::"r"(f(x)) : "memory");\n  asm("b" : "=r"(y));'
    got = list(asm_statements(text))
    assert [n for n, _ in got] == [1, 2]
    assert got[0][1].endswith('"memory")') and got[1][1].endswith("(y))")


def test_barriers_clobber_memory():
    assert without_clobber(r"\bbar\.sync|\bbarrier\.|\bmbarrier\.|\bfence\.") == []


def test_asynchronous_copies_clobber_memory():
    # a copy into a buffer must stay behind the last reads of what it held
    assert without_clobber(r"\bcp\.async") == []
