"""The check of outputs over inputs (csrc/seq_overlap.h) against sets of addresses, for random sizes
and strides: no shared value is missed, and tensors of the same strides are never refused without one."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHECK = r"""
#include <stdio.h>
#include <random>
#include <set>
#include "seq_overlap.h"
using namespace gbfft;
int main() {
    std::mt19937 rng(3);
    auto pick = [&](int lo, int hi) { return lo + (int)(rng() % (hi - lo)); };
    long seen[2] = {0, 0}, missed = 0, refused = 0;
    for (int n = 0; n < 400000; ++n) {
        const int nseq = pick(1, 5), length = pick(1, 6), width = pick(1, 5), other = pick(1, 5);
        const bool same = pick(0, 3) != 0, packed = pick(0, 4) == 0;
        const int tok = pick(0, 14), seq = pick(0, 60), first[2] = {pick(0, 80), pick(0, 80)};
        const int btok = same ? tok : pick(0, 14), bseq = same ? seq : pick(0, 60);
        char* base = (char*)0x100000;  // never read
        const fft_seq a = {base + 4 * first[0], seq, tok}, b = {base + 4 * first[1], bseq, btok};
        std::set<int> values;
        bool meet = false;
        for (int q = 0; q < (packed ? 1 : nseq); ++q)
            for (int t = 0; t < length; ++t)
                for (int c = 0; c < width; ++c) values.insert(first[0] + q * seq + t * tok + c);
        for (int q = 0; q < (packed ? 1 : nseq); ++q)
            for (int t = 0; t < length; ++t)
                for (int c = 0; c < other; ++c) meet |= values.count(first[1] + q * bseq + t * btok + c);
        const bool got = seqs_meet(a, b, width, other, nseq, length, packed, 4);
        ++seen[meet];
        missed += meet && !got;
        refused += same && got && !meet;
    }
    printf("%ld %ld %ld %ld", seen[0], seen[1], missed, refused);
    return 0;
}
"""


def test_against_sets_of_addresses(tmp_path):
    src, exe = tmp_path / "check.cpp", tmp_path / "check"
    src.write_text(CHECK)
    csrc = os.path.join(ROOT, "fft_signal_processing_gb300", "csrc")
    subprocess.run(["g++", "-O2", "-std=c++17", "-I", csrc, str(src), "-o", str(exe)], check=True)
    apart, meet, missed, refused = map(int, subprocess.run([str(exe)], capture_output=True, text=True,
                                                           check=True).stdout.split())
    assert min(apart, meet) > 100000 and missed == 0 and refused == 0
