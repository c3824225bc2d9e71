"""Inline PTX that touches memory, or waits, must be tied to its place: without `volatile` and a "memory"
clobber the compiler may take it for a function of its operands alone and move it over a wait that it
has to come after (a kernel's first is for the kernel before it, whose output it reads).  Loads of shared
memory may do with `volatile`, which keeps their order among the waits and stores written like them."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "pointwise_conv_cnn_gb300", "csrc")
SOURCES = sorted(p for p in glob.glob(os.path.join(CSRC, "*")) if p.endswith((".cu", ".cuh")))
# loads, stores, copies, atomics, fences, barriers and grid waits, by the instruction's first part; shuffles,
# moves between registers and address conversions are none
TOUCHES = re.compile(r"(?<![\w.])(ld|st|cp|red|atom|ldmatrix|stmatrix|fence|membar|bar|barrier|mbarrier|griddepcontrol|"
                     r"tcgen05|prefetch)\.")


def statements(text):
    """(line, qualifiers, body) of each asm statement."""
    for m in re.finditer(r"\basm\b\s*(volatile|__volatile__)?\s*\(", text):
        depth, i, quoted = 1, m.end(), False
        while depth:
            ch = text[i]
            if ch == '"' and text[i - 1] != "\\":
                quoted = not quoted
            elif not quoted:
                depth += (ch == "(") - (ch == ")")
            i += 1
        yield text.count("\n", 0, m.start()) + 1, m.group(1) or "", text[m.end():i - 1]


def unordered(text):
    found = []
    for line, volatile, body in statements(text):
        code = " ".join(re.findall(r'"((?:[^"\\]|\\.)*)"', body)).replace("\\n", " ").replace("\\t", " ")
        clobber = re.search(r':\s*"memory"\s*$', body.strip()) or code.startswith("ld.shared.")
        if TOUCHES.search(code) and not (volatile and clobber):
            found.append((line, code[:60]))
    return found


def test_the_search_sees_what_it_should():
    assert unordered('asm("{\\n\\t@p ld.global.v4.u32 {%0}, [%1];\\n\\t}" : "+r"(v) : "l"(p));')
    assert unordered('asm volatile("ld.global.u32 %0, [%1];" : "=r"(v) : "l"(f(p)));')
    assert unordered('asm("griddepcontrol.wait;" ::: "memory");')
    assert not unordered('asm volatile("ld.global.u32 %0, [%1];" : "=r"(v) : "l"(f(p)) : "memory");')
    assert unordered('asm("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(p));')
    assert not unordered('asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(p));')
    assert not unordered('asm("fma.rn.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));')


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_memory_is_touched_in_order(path):
    assert not unordered(open(path).read())
