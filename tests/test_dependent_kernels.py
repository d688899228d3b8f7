"""Source rule of the kernels that are launched while the kernel ahead of them still runs, checked on the text
(no GPU): what that kernel writes changes during their lifetime, so where they join its partial sums they read
them by ld_after_wait() alone.  __ldg, and a const __restrict__ pointer that lets the compiler choose the same
load, promise memory that nobody writes meanwhile; such a load may also be moved ahead of the wait."""

import re

import pytest

from test_kernel_rules import SOURCES, _text


def kernels(src):
    """(name, parameters, body) of every __global__ function, the body found by brace matching."""
    for m in re.finditer(r"__global__\s+void\s+(?:__launch_bounds__\((?:[^()]|\([^()]*\))*\)\s*)?(\w+)\s*\(([^)]*)\)\s*\{", src):
        i, depth = m.end(), 1
        while depth:
            depth += {"{": 1, "}": -1}.get(src[i], 0)
            i += 1
        yield m.group(1), m.group(2), src[m.end():i]


def faults(params, body):
    """What a joining kernel (one that reads `partial` results of the kernel ahead) does wrong."""
    found = []
    if "grid_dep_wait" not in body:
        found.append("no wait")
    if re.search(r"const[^,]*\*\s*__restrict__", params):
        found.append("const __restrict__")
    if "__ldg" in body:
        found.append("__ldg")
    if re.search(r"\b(partial|from)\s*\[", body):
        found.append("plain index")
    if "ld_after_wait" in body and "grid_dep_wait" in body and body.index("ld_after_wait") < body.index("grid_dep_wait"):
        found.append("read ahead of the wait")
    return found


def joining():
    return [(n, *k) for n in SOURCES for k in kernels(_text(n)) if re.search(r"\*[^,]*\bpartial\b", k[1])]


def test_the_joining_kernels_are_found():
    assert {k[1] for k in joining()} >= {"layer_norm_sum_kernel", "wgrad_sum_kernel"}


@pytest.mark.parametrize("kernel", joining(), ids=lambda k: k[1])
def test_partial_results_are_read_behind_the_wait(kernel):
    assert faults(*kernel[2:]) == []


def test_the_rule_sees_planted_faults():
    wait = "grid_dep_wait(); "
    assert faults("const float* __restrict__ partial, float* G", wait + "ld_after_wait(partial);") == ["const __restrict__"]
    assert faults("const float* partial, float* G", wait + "v = __ldg(partial + i);") == ["__ldg"]
    assert faults("const float* partial, float* G", wait + "v = partial[i];") == ["plain index"]
    assert faults("const float* partial, float* G", "v = ld_after_wait(partial); " + wait) == ["read ahead of the wait"]
    assert faults("const float* partial, float* G", "v = ld_after_wait(partial);") == ["no wait"]
