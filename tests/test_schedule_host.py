"""The work split's window arithmetic (csrc/schedule.cuh, csrc/window.cuh), compiled for the host and compared
with unbounded integers over the largest windows and the shortest sequences."""
import subprocess

import pytest

from mla_kv_cache_b200 import build as kbuild

SOURCE = r"""
#include <cstdio>
#include "window.cuh"
int main() {
    int align, len, q_len, window;
    while (std::scanf("%d %d %d %d", &align, &len, &q_len, &window) == 4) {
        const int s = kvattn::active_start_on(align, len, q_len, window);
        std::printf("%d %d %d\n", s, kvattn::tiles_of(len - s, 128), kvattn::window_start(len - q_len + 1, window));
    }
}
"""
MAX = 2 ** 31 - 1
WINDOWS = [1, 2, 127, 128, 129, 4096, MAX - 4097, MAX - 1, MAX]
LENS = [0, 1, 2, 4, 5, 127, 128, 129, 300, 4096, 100000]
Q_LENS = [1, 2, 3, 4, 5, 64, 4096]


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    d = tmp_path_factory.mktemp("schedule")
    src, exe = d / "split.cu", d / "split"
    src.write_text(SOURCE)
    subprocess.run([kbuild.NVCC, "-gencode", "arch=compute_100a,code=sm_100a", "-std=c++17", "-I", kbuild.CSRC, str(src), "-o",
                    str(exe)], check=True, capture_output=True)
    return str(exe)


def test_windows_up_to_the_largest(program):
    cases = [(a, n, q, w) for a in (0, 128) for n in LENS for q in Q_LENS for w in [0] + WINDOWS]
    text = "\n".join(" ".join(map(str, c)) for c in cases)
    lines = subprocess.run([program], input=text, capture_output=True, text=True, check=True).stdout.split("\n")
    for (align, n, q, w), line in zip(cases, lines):
        start = max(n - q + 1 - w, 0) if w else 0
        if align:
            start -= start % align
        got = list(map(int, line.split()))
        assert got[:2] == [start, -(-(n - start) // 128)], (align, n, q, w)
        if w:
            assert got[2] == max(n - q + 1 - w, 0)
