"""Rules of the scan, the convolution and the group norm that are decided on the host
and that no result shows on every machine (CPU only)."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "linear_rnn_sequence_wkv7_amd", "csrc")
ROCM = "/opt/rocm/include"

# Every place where a kernel that moves whole words starts a run of channels, in each type that it moves
# them in, and of states: the rows of 3 tokens, each group, blocks of 16 channels, `e` channels to a lane.
WORDS = r"""
#include <cstdio>
#include "seq_internal.h"
using namespace wkv7;
static int bad = 0;
static void at(long off, const char* what, const SsmParams& p, int a) {
    if (off % 4 && bad++ < 10)
        std::printf("%s at byte %ld: C=%d G=%d N=%d in_bf16=%d y_bf16=%d (%d)\n", what, off, p.C, p.G, p.N, int(p.in_bf16), int(p.y_bf16), a);
}
static void channels(const SsmParams& p, int e) {
    const int Cg = p.C / p.G;
    for (int t = 0; t < 3; ++t)
        for (int g = 0; g < p.G; ++g)
            for (int c = 0; c + e <= Cg; c += e) {
                const long i = long(t) * p.C + g * Cg + c;
                if (e * (p.in_bf16 ? 2 : 4) >= 4) at(i * (p.in_bf16 ? 2 : 4), "channels of the inputs", p, e);
                if (e * (p.y_bf16 ? 2 : 4) >= 4) at(i * (p.y_bf16 ? 2 : 4), "channels of y or dy", p, e);
            }
}
static void states(const SsmParams& p, int npl) {
    for (int t = 0; t < 3; ++t)
        for (int g = 0; g < p.G; ++g)
            for (int n = 0; n < p.N; n += npl) {
                if (npl * (p.in_bf16 ? 2 : 4) >= 4) at((long(t) * p.G * p.N + g * p.N + n) * (p.in_bf16 ? 2 : 4), "states", p, npl);
                if (n + npl > p.N && bad++ < 10) std::printf("a lane has some of its states: N=%d, %d\n", p.N, npl);
            }
}
int main() {
    long words = 0;
    SsmParams p{};
    for (p.C = 1; p.C <= 36; ++p.C)
        for (p.G = 1; p.G <= p.C; ++p.G) {
            if (p.C % p.G) continue;
            for (p.N = 1; p.N <= 64; ++p.N)
                for (int ty = 0; ty < 4; ++ty) {
                    p.in_bf16 = ty & 1;
                    p.y_bf16 = ty & 2;
                    const int npl = p.N <= 4 ? 1 : p.N <= 8 ? 2 : p.N <= 16 ? 4 : p.N <= 32 ? 8 : 16;
                    if (ssm_forward_words(p, npl)) {
                        ++words;
                        channels(p, 4);
                        states(p, npl);
                    }
                    if (ssm_backward_words(p)) {
                        ++words;
                        for (int e = 1; e <= 4; e *= 2) channels(p, e);
                        states(p, 2);
                    }
                }
        }
    std::printf("%ld %d\n", words, bad);
    return bad != 0;
}
"""


@pytest.mark.skipif(not os.path.isdir(ROCM), reason="no HIP headers")
def test_words_start_on_4_bytes(tmp_path):
    """The scan's kernels load and store runs of channels and of states as whole words only where every run,
    of the inputs and of y or dy, in each of their types, starts on 4 bytes."""
    src, exe = tmp_path / "words.cpp", tmp_path / "words"
    src.write_text(WORDS)
    subprocess.run(["g++", "-std=c++17", "-D__HIP_PLATFORM_AMD__", "-I", CSRC, "-I", ROCM, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
    assert int(r.stdout.split()[-2]) > 1000   # and there are such sizes
