"""Copies to shared memory, read from the sources: a block fetches its own tiles. The library is one for every rank of a
run on several GPUs, and nothing ties a call's tensors to the memory of the GPU that it runs on, which copies to several
blocks of a cluster ask for."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mtp_speculative_decoding_step_gb300", "csrc")


def test_no_copy_goes_to_several_blocks():
    for name in sorted(os.listdir(CSRC)):
        # strings that the compiler joins, as one
        src = re.sub(r'"\s*\n?\s*"', "", open(os.path.join(CSRC, name)).read())
        for copy in re.findall(r"cp\.async\.bulk[^;]*", src):
            assert "multicast" not in copy, (name, copy)
