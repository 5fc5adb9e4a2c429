"""CPU: inline assembly of the kernels.  A direct copy to LDS takes its LDS address from m0,
and the instruction after a scalar write of m0 may still read the old value: gfx9 wants a
wait state between the two, which the compiler inserts for its own code and nobody does
inside an asm string."""
import glob
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCES = sorted(glob.glob(os.path.join(ROOT, "w4a8_gemm_amd", "csrc", "*.*")))


def asm_strings(text):
    """The instructions of every asm statement, one list each."""
    out = []
    for m in re.finditer(r'\basm\b(?:\s+volatile)?\s*\(((?:\s*"(?:[^"\\]|\\.)*")+)', text):
        s = "".join(re.findall(r'"((?:[^"\\]|\\.)*)"', m.group(1)))
        out.append([i.strip() for i in re.split(r"\\n|\\t|;", s) if i.strip()])
    return out


def reads_m0(i):
    return "load_lds" in i or re.search(r"\blds\b", i) is not None and i.startswith("buffer_load")


def unwaited(text):
    """Copies to LDS whose m0 the instruction before them wrote, or that write no m0 of their own."""
    found = []
    for code in asm_strings(text):
        for at, i in enumerate(code):
            if reads_m0(i) and (at < 2 or not code[at - 1].startswith("s_nop") or not re.match(r"s_mov_b32 m0\b", code[at - 2])):
                found.append(i)
    return found


def test_the_scan_sees_a_missing_wait():
    bad = r'asm volatile("s_mov_b32 m0, %1\n\tglobal_load_lds_dword %0, off" ::"v"(p), "s"(b) : "memory", "m0");'
    good = bad.replace(r"%1\n\t", r"%1\n\ts_nop 0\n\t")
    assert unwaited(bad) == ["global_load_lds_dword %0, off"] and unwaited(good) == []
    bad = 'asm volatile("s_mov_b32 m0, %3\\n\\t"\n "buffer_load_dword %0, %1, %2 offen lds" :: );'
    assert len(unwaited(bad)) == 1


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_copies_to_lds_wait_for_m0(path):
    with open(path) as f:
        assert unwaited(f.read()) == []
