"""Memory-ordering rules that the products' kernels have to keep, checked in their sources. A break of one of
them is not seen in results on every run, so it is looked for where it is written."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "latentmoe_layer_b200", "csrc")


def code(name):
    """A source file without its comments."""
    with open(os.path.join(CSRC, name)) as f:
        text = f.read()
    return re.sub(r"/\*.*?\*/", "", re.sub(r"//[^\n]*", "", text), flags=re.S)


@pytest.mark.parametrize("name", ["grouped.cu", "few.cu", "fp8.cu"])
def test_dependent_kernels_do_not_use_the_read_only_path(name):
    """A kernel launched as a dependent is resident while the kernel before it still writes. Non-coherent
    loads are for data that is read-only as long as the kernel lives, and a compiler may move them ahead of
    the wait; operands, counts and scales are none of that."""
    text = code(name)
    assert "dependent_wait_and_release()" in text
    assert not re.search(r"__ldg\b|ld_global_nc|ld\.global\.nc|__restrict__", text)


def test_relaxed_arrivals_hand_over_tmem_only():
    """An arrival without a release orders no earlier read of shared memory. It is allowed where a buffer of
    TMEM is given back: wait::ld has completed the reads, and the fence before the arrival orders them."""
    text = code("grouped.cu")
    arrivals = [m.start() for m in re.finditer(r"arrive\.relaxed", text)]
    assert len(arrivals) == 1
    before = text[:arrivals[0]]
    body = before[before.rindex("__device__"):]
    assert "tc_fence_before();" in body and "__syncwarp();" in body and body.index("tc_fence_before") < body.index("__syncwarp")


@pytest.mark.parametrize("name", ["grouped.cu", "ptx.cuh"])
def test_arrivals_on_another_cta_name_their_scope(name):
    """Without a scope an arrival releases to its own CTA alone; on a shared::cluster address the waiting
    thread may be in another one."""
    for m in re.finditer(r'"[^"\n]*mbarrier\.arrive[^"\n]*shared::cluster[^"\n]*"', code(name)):
        assert re.search(r"arrive(\.expect_tx)?\.(release|relaxed)\.cluster", m.group()) or "tcgen05.commit" in m.group(), m.group()


def test_a_warp_gives_up_a_wait_as_a_whole():
    """A wait that runs out for some lanes of a warp and not for others would send them different ways before
    an instruction that needs all of them. Waits of single elected threads may decide alone; the others vote."""
    text = code("grouped.cu")
    roles = ["elect_one()) {", "warp >= 2 &&", "setmaxnreg.inc", "void epilogue_rows"]
    single = [m.start() for m in re.finditer(r"\bif \(!?(?:mbar_)?wait_\w+\(|\b(?:mbar_)?wait_\w+\(&", text)]
    checked = 0
    for at in single:
        name = re.search(r"(\w*wait_\w+)\(", text[at:]).group(1)
        place = max((text.rfind(r, 0, at), r) for r in roles)
        if place[0] < 0:
            continue  # inside the waits themselves
        checked += 1
        assert ("warp" in name) == (place[1] != "elect_one()) {"), (name, place[1], text[at:at + 80])
    assert checked >= 12
    body = text[text.index("wait_warp("):]
    assert "__all_sync" in body[:body.index("\n}\n")]
