"""Orders between threads and launches that a run cannot show to be kept: a
missing one gives wrong results only at rare timings. So the sources are read."""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "mtp_speculative_decoding_step_gb300", "csrc")


def source(name):
    """A source without its comments."""
    return re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())


def test_partial_results_are_cleared_by_the_lane_that_hands_out_shares():
    """The softmax warps write a block's two entries of part_meta after they have been given a share. Only the lane that
    arrives on the share's barrier orders its own stores before theirs; the other lanes' may come later."""
    src = source("attn_q4.cuh")
    clears = [line for line in src.splitlines() if "part_meta" in line and "make_int4(0, 0, 0, 0)" in line]
    assert len(clears) == 1 and clears[0].strip().startswith("if (lane == 0)"), clears
    shares = src[src.index("part_meta[2 * blockIdx.x"):]
    gives = re.findall(r"if \(([^)]*lane == 0)\) \{[^}]*mbar_arrive\(smem_u32\(&M\.run_full", shares)
    assert gives == ["left == 0 && lane == 0", "lane == 0"]


def test_no_read_only_loads_in_kernels_that_start_before_their_predecessor_ends():
    """These kernels are launched with programmatic serialisation: what they read (tables, lengths, K and V, logits) may
    still be written between their start and griddepcontrol.wait. A load through the read-only path (ld.global.nc) is for
    data that does not change while the kernel runs, and may be moved to before the wait."""
    for name in ("kv_page.cu", "kv_q4.cu", "q4.cuh", "attn_q4.cu", "attn_q4.cuh", "logprobs.cu"):
        assert not re.findall(r"__ldg|ldg_stream|global\.nc|__restrict__", source(name)), name
    common = source("common.cuh")
    body = common[common.index("uint4 ld_stream("):]
    assert "ld.global.L1::no_allocate" in body[:body.index("}\n")]
