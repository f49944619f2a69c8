"""The list of candidates of qmv_logprobs for rows of up to 8192, counted on
the host (logprob_host_driver.cpp): the kernel's shared memory holds 4 * top *
E of them for E elements a thread, which no row may pass."""
import os
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "block_quant_weight_amd", "csrc")


@pytest.fixture(scope="module")
def driver(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("logprobs") / "driver")
    subprocess.check_call(["g++", "-O2", "-std=c++17", "-Wall", "-Wno-unknown-pragmas", "-I", CSRC, "-o", exe,
                           os.path.join(HERE, "logprob_host_driver.cpp")])
    return exe


def cases(vocab):
    """(NaN, -infinity) of a row: none, one, around a thread's, a wave's and the row's size."""
    parts = sorted({0, 1, 3, vocab // 8, vocab // 2, vocab - vocab // 8, vocab - 1, vocab})
    return [(a, b) for a in parts for b in parts if a + b <= vocab]


@pytest.mark.parametrize("vocab", [1, 2, 5, 33, 64, 1000, 1023, 1024, 1025, 2047, 2048, 3001, 4096, 4097, 8191, 8192])
def test_no_row_lists_more_than_there_is_room_for(driver, vocab):
    want = [(vocab, top, a, b, order, 7 * a + b) for top in {1, min(20, vocab), min(32, vocab)}
            for a, b in cases(vocab) for order in range(4)]
    out = subprocess.run([driver], input="".join("%d %d %d %d %d %d\n" % c for c in want), capture_output=True,
                         text=True, check=True, timeout=300).stdout.split("\n")
    assert len(out) == len(want) + 1
    for c, line in zip(want, out):
        e, listed, wrong, missing = map(int, line.split())
        assert listed <= 4 * c[1] * e and wrong == 0 and missing == 0, (c, line)
