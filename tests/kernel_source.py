"""The kernels' source as tests read it: functions by name, comments taken out, calls to a header's own functions in place."""

import re
from pathlib import Path

CSRC = Path(__file__).resolve().parents[1] / "dsa_sparse_attention_fp8_gb300" / "csrc"
HEAD = re.compile(r"\b(__global__|__device__)\b[^;{}]*?\b(\w+)\s*\((?=[^;{}]*\)\s*\{)")


def _matching(text, at, pair):
    depth = 0
    for i in range(at, len(text)):
        depth += (text[i] == pair[0]) - (text[i] == pair[1])
        if depth == 0:
            return i
    raise ValueError("brackets do not match")


def functions(name):
    """{function: (is a kernel, body)} of a file of csrc, `name`."""
    text = re.sub(r"//[^\n]*|__launch_bounds__\([^)]*\)", "", (CSRC / name).read_text())
    found = {}
    for m in HEAD.finditer(text):
        closed = _matching(text, text.index("(", m.end() - 1), "()")
        opened = text.index("{", closed)
        body = text[opened:_matching(text, opened, "{}") + 1]
        kernel, old = m.group(1) == "__global__", found.get(m.group(2), (False, ""))
        found[m.group(2)] = (kernel or old[0], old[1] + body)          # overloads one after the other
    return found


def kernels(name):
    """{kernel: body} of a file of csrc with the file's own device functions in the place of their calls."""
    parts = functions(name)

    def inlined(body, inside=()):
        def put(m):
            called = m.group(1)
            return m.group(0) + inlined(parts[called][1], inside + (called,)) if called not in inside else m.group(0)
        own = [n for n, (kernel, _) in parts.items() if not kernel]
        return re.sub(rf"\b({'|'.join(own)})\b(?=\s*[(<])", put, body) if own else body
    return {n: inlined(body) for n, (kernel, body) in parts.items() if kernel}
