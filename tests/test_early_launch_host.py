"""Kernels that may begin while the one before them on the stream still runs, in
their source (no GPU needed)."""
import os
import re

import pytest

from tiled_online_softmax_02_gb300 import build

# files whose kernels are all launched so, one with such a kernel and a fill, and the headers that those share with others
EARLY = ["cache4.cu", "rope.cu", "attn_paged4_dec.cu", "attn_paged4_tc.cu", "attn_paged4_join.cu", "attn_paged_join.cu"]
SHARED = ["attn_merge.cu", "early_load.cuh", "paged4.cuh", "paged_join.cuh", "paged_mma.cuh"]


def code(name):
    """A source file without its comments."""
    with open(os.path.join(build.CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_the_list_is_whole():
    for f in os.listdir(build.CSRC):
        if f.endswith(".cu") and "launch_early(" in code(f):
            assert f in EARLY, f


@pytest.mark.parametrize("name", EARLY + SHARED)
def test_no_read_only_loads(name):
    """The read-only path is for memory that nobody writes while the kernel lives."""
    assert not re.search(r"__ldg\b|ld\.global\.nc|__restrict__", code(name))


def test_no_read_only_loads_in_the_shares():
    """The lengths' reader chooses by the kernel, and such kernels ask for another load.  (The 8-bit kernels' scales,
    behind the walk, are theirs alone.)"""
    text = code("paged_sched.cuh")
    text = text[:text.index("struct ScaleFeed")]
    chosen = "if constexpr (LOAD == kReadOnly) return __ldg(x);"
    assert text.count(chosen) == 1 and not re.search(r"__ldg\b|ld\.global\.nc|__restrict__", text.replace(chosen, ""))
    for name in EARLY[2:4]:
        made = re.findall(r"(?:PagedWalk|paged_share|paged_share_long)<[^;(]*?>(?=[ (;])", code(name))
        assert len(made) >= 3 and all(re.search(r", (kWritten|kOrdinary)>$", m) for m in made), made


@pytest.mark.parametrize("name", EARLY)
def test_every_kernel_waits(name):
    kernels = re.findall(r"__global__[^{;]*\{(.*?)\n\}", code(name), re.S)
    assert kernels
    for body in kernels:
        assert re.search(r"after_earlier_kernels\(\);|griddepcontrol\.wait", body), body[:200]


@pytest.mark.parametrize("name", ["attn_paged4_tc.cu", "attn_paged_tc.cu", "attn_paged_dec.cu"])
def test_later_kernels_come_in_once_tensor_memory_is_held(name):
    """A CTA whose columns a later kernel had taken would wait for that one, which waits for this grid."""
    text = code(name)
    alloc, sync = text.index("tmem_alloc("), text.index("__syncthreads();", text.index("tmem_alloc("))
    assert text.count("launch_dependents") == 1 and alloc < sync < text.index("launch_dependents")
