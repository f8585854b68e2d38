"""Rules of memory ordering that the kernels' sources keep (no GPU needed): no run shows a breach reliably."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "lut_dequant_gemv_b200", "csrc")


def code(name):
    """The file without its comments."""
    return re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())


def test_kernels_launched_early_read_through_the_coherent_path():
    """The 8-bit quantizer and product start before the previous kernel of the stream has ended, and read what it
    writes: not through the non-coherent path, which requires memory that nobody writes while the kernel lives."""
    for name in ("kernels_fp8.cuh", "fp8_common.cuh"):
        assert not re.search(r"__ldg\(|ldg_stream_u128|ldg_u128|ldg_u32|\.nc\b", code(name)), name
    for name in ("kernels_tc.cuh", "kernels_pd.cuh"):  # (their weights never change)
        assert not re.search(r"(__ldg|ldg_\w+)\(p\.x\b", code(name)), name


def test_a_barrier_hands_on_what_one_thread_acquired_from_the_grid():
    """One thread waits for the grid's barrier; the threads that then read what other CTAs wrote are ordered behind it
    by a barrier, which a warp vote is not."""
    text = code("kernels_moe.cuh")
    calls = [m.start() for m in re.finditer(r"&& grid_wait\(|\) grid_wait\(", text)]
    assert len(calls) == 2
    for at in calls:
        after = [line.strip() for line in text[at:].split("\n")[1:] if line.strip()]
        assert re.match(r"__sync(threads|warp)\(\);", after[0]), after[0]
