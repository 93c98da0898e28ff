"""Inline assembly of the kernels declares what it writes (no GPU needed): a
register that a statement names itself is in its clobber list, and loads do not
return to registers, which the compiler would take as written at once."""
import glob
import os
import re
import subprocess

from combine_ep_get_dispatch_amd.build import hipcc

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
        for line in code:
            w = re.match(r"[vs]_\w+\s+(m0|vcc|exec|scc|[vs]\d+|[vs]\[\d+:\d+\])\s*,", line)
            if w:
                found += 1
                assert f'"{w.group(1)}"' in clobbers, f"{f}: {line} writes {w.group(1)}, not in its clobbers"
    assert found


PROBE = """
#include <hip/hip_runtime.h>
typedef __attribute__((address_space(3))) void lds;
__global__ void k(const char* p, int off, int* o) {
    __shared__ int s[256];
    auto rs = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(p), (short)0, 0x7FFFFFFF, 0x00020000);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds*)s, 4, off, 0, 0, 0);
    asm volatile("s_mov_b32 m0, %0" ::"s"(off) : "memory", "m0");
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds*)s, 4, off + 64, 0, 0, 0);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    o[threadIdx.x] = s[threadIdx.x];
}
"""


def test_the_compiler_minds_a_clobber_of_m0(tmp_path):
    """It warns that m0 is reserved; what counts is that it sets m0 anew for a
    load into LDS after the statement."""
    src = tmp_path / "m0.hip"
    src.write_text(PROBE)
    asm = subprocess.run([hipcc(), "--offload-arch=gfx950", "-O3", "--cuda-device-only", "-S", "-o", "-", str(src)],
                         check=True, capture_output=True, text=True).stdout
    lines = [ln.split()[0] if ln.split()[-1] == "lds" else ln.strip() for ln in asm.splitlines()
             if re.search(r"\bs_mov_b32 m0,|\blds$", ln)]
    assert lines[0] == lines[3] == "s_mov_b32 m0, 0" and lines[2].startswith("s_mov_b32 m0, s"), lines
    assert lines[1] == lines[4] == "buffer_load_dword", lines


def test_loads_do_not_return_to_registers():
    for f, code, outputs, _ in statements():
        for line in code:
            if re.match(r"(buffer|global|flat|ds|s)_(load|read)", line):
                assert re.search(r"\blds$", line) and "v\"" not in outputs, f"{f}: {line}"
