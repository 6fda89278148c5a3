"""The error word of linear attention is read and cleared in one operation (no GPU needed: the source is
read, since the time between two operations is not one that a test can hit)."""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_the_word_is_taken_in_one_operation():
    src = open(os.path.join(ROOT, "fft_signal_processing_gb300", "csrc", "linattn_api.cu")).read()
    body = src[src.index("int fft_linattn_check("):]
    body = body[:body.index("\n}\n")]
    assert "cudaMemset" not in body
    kernel = re.search(r"(\w+)<<<", body).group(1)
    start = src.index(f"void {kernel}(")
    assert "atomicExch(&g_attn_error, 0)" in src[start:src.index("}", start)]
