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
    roles = ["elect_one()) {", "void drain_loads", "warp >= 2 &&", "setmaxnreg.inc", "void epilogue_rows"]
    waits = [(m.start(), m.group(1)) for m in re.finditer(r"\b(\w*wait\w*)(?:<\w+>)?\(&S\.", text)]
    assert len(waits) >= 10
    for at, name in waits:
        role = max((text.rfind(r, 0, at), r) for r in roles)[1]
        assert ("warp" in name) == (role not in roles[:2]), (name, role, text[at:at + 80])
    body = text[text.index("wait_warp("):]
    assert "__all_sync" in body[:body.index("\n}\n")]


def test_waits_leave_on_a_word_of_their_own_launch():
    """A kernel that gave up its waits because of a word shared by the process would be cut short by another
    stream's failure, and once more at every replay of a graph. The word that reports to the host is written
    by kernels and read by the host only."""
    text = code("grouped.cu")
    assert "*(volatile int*)err" not in text and "mbar_wait_bounded" not in text
    assert "gave_up" in text[text.index("struct alignas(1024) GgShared"):text.index("constexpr size_t kGgSmem")]


def test_final_drains_do_not_leave_early():
    """The waits for MMAs and copies in flight, ahead of freeing TMEM and leaving, go on after a timeout."""
    text = code("grouped.cu")
    body = text[text.index("drain_wait("):]
    body = body[:body.index("\n}\n")]
    assert "try_wait" in body and "gave_up" not in body
    for bar in ("S.done", "S.landed", "S.full"):
        assert re.search(r"drain_wait\(&%s\b" % bar, text), bar


def test_the_host_only_reads_the_count_of_timeouts():
    """Taking the word (an exchange) would give one caller's report to another."""
    text = code("ops.cu")
    assert "__atomic_exchange" not in text and "thread_local" in text
    assert len(re.findall(r"\*st\.herr\s*=", text)) == 1  # its initial zero


def test_the_sm_count_is_kept_by_device():
    """Grids and the few-row kernel's share of an SM follow the current device, and two threads may ask at once."""
    text = code("gemm_tc.cu")
    body = text[text.index("int tc_num_sms()"):]
    body = body[:body.index("\n}\n")]
    assert re.search(r"std::atomic<int>\s+g_num_sms\[", text) and "cudaGetDevice" in body and "[dev]" in body
