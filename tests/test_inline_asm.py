"""Inline assembly of the kernels leaves the compiler's registers as they were
(no GPU needed): one that a statement names itself is in its clobber list or
put back from a copy, and loads do not return to registers, which the compiler
would take as written at once."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "combine_ep_get_dispatch_amd", "csrc")


def statements():
    """(file, lines of code, output operands, clobbers) of each statement."""
    for f in sorted(glob.glob(os.path.join(CSRC, "*"))):
        text = re.sub(r"//[^\n]*", "", open(f).read())
        for m in re.finditer(r"\basm\s+volatile\s*\(", text):
            depth, i = 1, m.end()
            while depth:
                depth += {"(": 1, ")": -1}.get(text[i], 0)
                i += 1
            body = text[m.end():i - 1]
            lits = re.match(r'(\s*"(?:[^"\\]|\\.)*")+', body)
            code = "".join(re.findall(r'"((?:[^"\\]|\\.)*)"', lits.group(0))).replace("\\n", "\n").replace("\\t", " ")
            lists = [p.strip() for p in body[lits.end():].replace("::", ": :").split(":")[1:]]
            yield (os.path.basename(f), [c.strip() for c in code.split("\n")], lists[0] if lists else "",
                   lists[2] if len(lists) > 2 else "")


def test_named_registers():
    found = 0
    for f, code, _, clobbers in statements():
        writes = {}
        for line in code:
            w = re.match(r"[vs]_\w+\s+(m0|vcc|exec|scc|[vs]\d+|[vs]\[\d+:\d+\])\s*,\s*(\S+)", line)
            if w:
                writes.setdefault(w.group(1), []).append(w.group(2))
        for reg, sources in writes.items():
            found += 1
            put_back = code[0] == f"s_mov_b32 {sources[-1]}, {reg}" and code[-1] == f"s_mov_b32 {reg}, {sources[-1]}"
            # the compiler reserves m0 and warns that it may not mind a clobber of it
            assert put_back or (reg != "m0" and f'"{reg}"' in clobbers), f"{f}: {reg} in {code}"
    assert found


def test_loads_do_not_return_to_registers():
    for f, code, outputs, _ in statements():
        for line in code:
            if re.match(r"(buffer|global|flat|ds|s)_(load|read)", line):
                assert re.search(r"\blds$", line) and "v\"" not in outputs, f"{f}: {line}"
