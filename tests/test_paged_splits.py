"""How far the key axis of a chunk is cut for the kernel whose blocks run one per
SM, 148 at a time: the rule itself, compiled for the host."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SMS = 148

MAIN = """
#include <cstdio>
#include "paged_splits.h"
int main() {
    long long blocks, keys, bytes;
    while (scanf("%lld %lld %lld", &blocks, &keys, &bytes) == 3)
        printf("%lld\\n", (long long)dit::tc_splits(blocks, keys, bytes));
}
"""


@pytest.fixture(scope="module")
def splits(tmp_path_factory):
    d = tmp_path_factory.mktemp("splits")
    (d / "main.cpp").write_text(MAIN)
    exe = str(d / "main")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I",
                    os.path.join(ROOT, "dit_token_b200", "csrc"), str(d / "main.cpp"), "-o", exe], check=True)

    def ask(cases):
        text = "\n".join(" ".join(str(v) for v in c) for c in cases)
        return [int(v) for v in subprocess.run([exe], input=text, capture_output=True, text=True,
                                               check=True).stdout.split()]
    return ask


CASES = [(b, k, 520 * 256 * b) for b in (1, 2, 3, 7, 16, 32, 40, 74, 75, 80, 100, 147, 148, 149, 150, 296, 600, 5000,
                                         10**6) for k in (1, 500, 1023, 1024, 2000, 8000, 30000, 10**6, 2**31 - 1)]


def rounds(blocks):
    return -(-blocks // SMS)


def test_a_cut_shortens_the_rounds(splits):
    """Time goes with the rounds of blocks times the length of a run: a cut that
    leaves it as long only adds parts (80 blocks in 2 runs each are two rounds
    of half the length)."""
    for (b, k, _), s in zip(CASES, splits(CASES)):
        assert 1 <= s <= max(1, k // 512) and s <= 8 * SMS
        assert s == 1 or rounds(b * s) / s < 0.86 * rounds(b), (b, k, s)


def test_few_blocks_fill_one_round(splits):
    """Runs of a whole round where the next one would be nearly empty."""
    for b, s in ((16, 9), (32, 4), (37, 4), (74, 2)):
        got = splits([(b, 6000, 520 * 256 * b)])[0]
        assert rounds(b * got) * s <= got, (b, got)  # as short as s runs of one round, or shorter


def test_more_keys_never_ask_for_fewer_splits(splits):
    for b in (1, 5, 16, 33, 80, 110, 150, 290):
        for part in (0, 10**6, 10**8):
            got = splits([(b, k, part) for k in range(1, 60000, 97)])
            assert got == sorted(got)
