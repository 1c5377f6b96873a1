"""The copies into LDS are inline assembly, so the compiler knows neither the
LDS address register nor the wait states they need.  Small kernels around them
are compiled here, and the assembly of each copy is followed back to what it
depends on (nothing runs)."""
import os
import re
import subprocess

import pytest

from combine_ep_get_layout_amd import build

pytestmark = pytest.mark.skipif(not os.path.exists(build.HIPCC), reason="no hipcc")

SOURCE = r"""
#include <type_traits>
#include "ep_expert_device.h"
using namespace ep;
__shared__ __align__(1024) uint8_t lds[65536];

// descriptors that come from vector registers right before the copies
extern "C" __global__ void fresh_descriptor(const uint64_t *p, const int *n, uint32_t v) {
    const int w = threadIdx.x;
    const ep_i32x4 r = buffer_of((const void *)p[w], n[w]);
    dma16(r, 0x1000, v, 0);
    dma1(buffer_of((const void *)p[w + 1], n[w + 1]), 0x2000, v, n[w + 2]);
    ep_i32x4 four = buffer_of((const void *)p[w + 2], n[w + 3]);
    uint32_t soff = n[w + 4];
    dma16_of4<0>(four, 0x3000, v, soff);
    dma16_of4<1>(four, 0x3000, v, soff);
    dma16_of4<2>(four, 0x3000, v, soff);
    dma16_of4<3>(four, 0x3000, v, soff);
}

// other copies between the first and the others of four
extern "C" __global__ void other_copies_between(const void *p, int n, uint32_t v) {
    ep_i32x4 r = buffer_of(p, n);
    uint32_t soff = 0;
    dma16_of4<0>(r, 0x1000, v, soff);
    dma1(r, 0x2000, v, 0);
    dma16_of4<1>(r, 0x1000, v, soff);
    dma16(r, 0x3000, v, 0);
    dma16_of4<2>(r, 0x1000, v, soff);
    dma16_of4<3>(r, 0x1000, v, soff);
}
"""


def assembly(source, out):
    """Instructions of each kernel of a source file."""
    subprocess.run([build.HIPCC, *build.CFLAGS, "-I", build.CSRC, "--cuda-device-only", "-S",
                    str(source), "-o", str(out)], check=True, capture_output=True)
    found, name = {}, None
    for line in out.read_text().splitlines():
        line = line.split(";")[0].strip()
        m = re.match(r"(\w+):$", line)
        if m and not line.startswith("."):
            name = m.group(1)
            found[name] = []
        elif line.startswith(".Lfunc_end"):
            name = None
        elif name and line and not line.startswith("."):
            found[name].append(line)
    return found


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    d = tmp_path_factory.mktemp("copies")
    (d / "copies.hip").write_text(SOURCE)
    return assembly(d / "copies.hip", d / "copies.s")


def is_copy(line):
    return line.startswith("buffer_load") and line.endswith(" lds")


def registers(operand):
    m = re.match(r"s\[(\d+):(\d+)\]$", operand) or re.match(r"s(\d+)$", operand)
    return set(range(int(m.group(1)), int(m.groups()[-1]) + 1)) if m else set()


def wait_states(line):
    return int(line.split()[1], 0) + 1 if line.startswith("s_nop") else 1


def check_waits(code):
    """A memory instruction reads a scalar register no sooner than five wait
    states after a vector instruction has written it, and the LDS address one
    after its write; the hardware holds neither.  Returns the copies seen."""
    copies = [i for i, line in enumerate(code) if is_copy(line)]
    for at in copies:
        words = code[at].replace(",", " ").split()
        needed = set().union(*(registers(w) for w in words[2:]))
        waited, i = 0, at - 1
        while i >= 0 and waited < 5:
            op, target = (code[i].replace(",", " ").split() + [""])[:2]
            assert not (op.startswith(("v_readfirstlane", "v_readlane", "v_cmp"))
                        and registers(target) & needed), (code[i], code[at], waited)
            assert not (target == "m0" and waited < 1), (code[i], code[at])
            waited += wait_states(code[i])
            i -= 1
    return len(copies)


def test_scalars_from_vector_instructions_are_waited_for(kernels):
    code = kernels["fresh_descriptor"]
    assert any(line.startswith("v_readfirstlane") for line in code)
    assert check_waits(code) == 6


def test_every_copy_finds_its_own_lds_address(kernels):
    scalars, seen = {}, []
    for line in kernels["other_copies_between"]:
        m = re.match(r"s_mov(?:k_i32|_b32) (\w+), (\w+)$", line)
        if m:
            to, what = m.groups()
            scalars[to] = int(what, 0) if what[0].isdigit() else scalars.get(what)
        elif is_copy(line):
            seen.append(scalars.get("m0"))
    assert seen == [0x1000, 0x2000, 0x1000, 0x3000, 0x1000, 0x1000]


@pytest.mark.parametrize("name", ["ep_expert_linear", "ep_expert_wgrad"])
def test_waits_of_the_kernels(name, tmp_path):
    code = assembly(os.path.join(build.CSRC, name + ".hip"), tmp_path / "kernels.s")
    assert sum(check_waits(c) for c in code.values()) >= 100
