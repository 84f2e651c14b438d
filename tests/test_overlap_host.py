"""The host's test for buffers that share a byte (csrc/overlap.h) against sets of
addresses, and against known answers at sizes that no set holds."""
import os
import random
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "speculative_decode_verify_paged_gb300", "csrc")


@pytest.fixture(scope="module")
def overlap(tmp_path_factory):
    at = tmp_path_factory.mktemp("overlap")
    src, exe = at / "overlap.cpp", at / "overlap"
    src.write_text('''#include "overlap.h"
        #include <stdio.h>
        int main() {
            unsigned long long v[8];
            for (;;) {
                for (auto& x : v)
                    if (scanf("%llu", &x) != 1) return 0;
                const spec_attn::ByteRows a = {(const void*)v[0], v[1], v[2], v[3]}, b = {(const void*)v[4], v[5], v[6], v[7]};
                printf("%d", spec_attn::overlap(a, b) ? 1 : 0);
            }
        }''')
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-I", CSRC, str(src), "-o", str(exe)], check=True)

    def ask(pairs):
        text = "\n".join(" ".join(str(x) for x in (*a, *b)) for a, b in pairs)
        out = subprocess.run([str(exe)], input=text, capture_output=True, text=True, check=True).stdout
        assert len(out) == len(pairs)
        return [c == "1" for c in out]
    return ask


def test_small_rows_against_sets(overlap):
    rng = random.Random(4)
    pairs, want = [], []
    for _ in range(20000):
        def rows():
            width = rng.randint(0, 6)
            return rng.randint(1, 90), width, width + rng.choice((0, 0, 1, rng.randint(0, 20))), rng.randint(0, 7)
        a, b = rows(), rows()
        sets = [{at + i * step + k for i in range(n) for k in range(width)} for at, width, step, n in (a, b)]
        pairs.append((a, b))
        want.append(bool(sets[0] & sets[1]))
    assert 3000 < sum(want) < 17000
    got = overlap(pairs)
    assert [p for p, g, w in zip(pairs, got, want) if g != w] == []
    assert overlap([(b, a) for a, b in pairs]) == want


def test_large_rows(overlap):
    base, n = 2 ** 46, 2 ** 31 - 1
    q, k, v = ((base + at, w, 12288, n) for at, w in ((0, 8192), (8192, 2048), (10240, 2048)))
    assert overlap([(q, k), (k, v), (q, v), (q, q), (q, (base + 8191, 2, 12288, n))]) == [False, False, False, True, True]
    # rows 64 and 96 bytes apart: all offsets modulo 32 come up, and nothing else
    assert overlap([((base, 16, 64, n), (base + 16, 16, 96, n)), ((base, 17, 64, n), (base + 16, 16, 96, n))]) == [False, True]
    # steps without a common divisor meet after 2^20 rows at the latest, and not among the first ones
    a, far = (base, 1, 2 ** 20, n), (base + 2 ** 19, 1, 2 ** 20 + 1, n)
    assert overlap([(a, far), ((base, 1, 2 ** 20, 2 ** 18), far), (a, (far[0], 1, far[2], 2 ** 19))]) == [True, False, False]
    # behind each other, and one inside a gap
    assert overlap([(a, (base + 2 ** 20 * (n - 1) + 1, 5, 5, 1)), (a, (base + 1, 2 ** 20 - 1, 7, 1)),
                    (a, (base + 1, 2 ** 20, 7, 1))]) == [False, False, True]


def test_no_buffer_and_no_rows(overlap):
    a = (1000, 64, 64, 10)
    assert overlap([(a, (0, 2 ** 40, 1, 1)), (a, (1000, 0, 64, 10)), (a, (1000, 64, 64, 0))]) == [False] * 3
