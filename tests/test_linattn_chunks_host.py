"""The decay's gradient sums rows by the chunks of the kernel that wrote them (no GPU needed): each chunk's
length is defined once."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fft_signal_processing_gb300", "csrc")


def test_chunks_have_one_length():
    src = "".join(open(f).read() for f in glob.glob(os.path.join(CSRC, "linattn*")))
    for name in ("kTcChunk", "kAttnChunk"):
        assert len(re.findall(rf"constexpr int {name} *=", src)) == 1
