"""Kernels that start under programmatic launch while the kernel ahead of them may still run, by their source: what
a GPU shows only where two kernels meet on an SM at the wrong time."""
import glob
import os
import re

import pytest

import variable_length_flash_gb300 as vlf

CSRC = os.path.join(os.path.dirname(os.path.abspath(vlf.__file__)), "csrc")
FILES = sorted(os.path.basename(f) for f in glob.glob(os.path.join(CSRC, "*.cu*")))


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def kernels(text):
    """(name, body) of each __global__ function with one."""
    for m in re.finditer(r"__global__", text):
        at, depth = m.end(), 0
        while text[at] != "{" or depth:  # the body's brace: behind the parameters' parentheses
            depth += {"(": 1, ")": -1}.get(text[at], 0)
            if text[at] == ";" and not depth:
                break
            at += 1
        if text[at] != "{":
            continue
        end, depth = at, 0
        while True:
            depth += {"{": 1, "}": -1}.get(text[end], 0)
            end += 1
            if not depth:
                break
        yield re.findall(r"(\w+)\s*\(", text[m.end():at])[-1], text[at:end]


def test_the_kernels_are_found():
    names = [name for f in FILES for name, _ in kernels(source(f))]
    assert {"pages_tc_kernel", "pages_rows_kernel", "pages_join_kernel", "norm_rope_kernel", "pages_write_kernel"} <= set(names)


@pytest.mark.parametrize("name", FILES)
def test_no_tensor_memory_is_held_ahead_of_the_wait(name):
    """A kernel's CTAs trigger the next launch before they allocate; if the next one's CTAs held columns while they
    wait, neither would end."""
    for kernel, body in kernels(source(name)):
        if "pdl_wait()" in body and "tmem_alloc(" in body:
            assert body.index("pdl_wait()") < body.index("tmem_alloc("), kernel


SERVING = ["norm_rope.cu", "pages.cu", "pages_tc.cu", "pages_tc.cuh", "pages_rows.cu", "rope.cuh", "e4m3.cuh"]


@pytest.mark.parametrize("name", SERVING)
def test_what_the_kernel_ahead_writes_is_not_read_as_constant(name):
    """__ldg asks that nobody writes the memory from the kernel's start on; these start before the one ahead ends."""
    assert not re.search(r"__ldg\b|ld\.global\.nc|__restrict__", source(name))


@pytest.mark.parametrize("name", ["tc_fwd.cu", "prefix.cu", "key_weights.cu", "common.cuh", "tc_common.cuh"])
def test_nor_by_the_forward_and_the_decoding_kernels(name):
    """The forward, shared-prefix attention and key weights start so where their grids are small.  (The others' __ldg is
    right: their first kernel is launched plainly, and reads inputs.)"""
    assert not re.search(r"__ldg\b|ld\.global\.nc|__restrict__", source(name))
