"""What the rotated append takes for an overlap of its output with its inputs (share_bytes of overlap.h, compiled for the host),
against the bytes counted one by one."""
import os
import random
import subprocess
import time

import pytest

from int2_rotated_kv_rotate_gb300 import build

PROGRAM = """
#include <cstdio>
#include "overlap.h"
int main() {
  oscar::Pieces a, b;
  long long x, y;
  while (std::scanf("%lld %lld %lld %lld %lld %lld %lld %lld %lld %lld %lld %lld", &x, &a.n, &a.heads, &a.row, &a.head, &a.bytes,
                    &y, &b.n, &b.heads, &b.row, &b.head, &b.bytes) == 12) {
    a.at = x, b.at = y;
    std::printf("%d\\n", int(oscar::share_bytes(a, b)));
  }
}
"""


@pytest.fixture(scope="module")
def answers(tmp_path_factory):
    d = tmp_path_factory.mktemp("overlap")
    (d / "overlap.cpp").write_text(PROGRAM)
    subprocess.run(["g++", "-O1", "-std=c++17", "-Wall", "-Werror", "-I", build.CSRC, "-o", str(d / "overlap"), str(d / "overlap.cpp")],
                   check=True)

    def run(cases):
        text = "\n".join(" ".join(map(str, a + b)) for a, b in cases)
        out = subprocess.run([str(d / "overlap")], input=text, check=True, capture_output=True, text=True).stdout.split()
        assert len(out) == len(cases)
        return [x == "1" for x in out]

    return run


def held(p):
    at, n, heads, row, head, size = p
    return {at + r * row + h * head + i for r in range(n) for h in range(heads) for i in range(size)}


def test_against_every_byte(answers):
    r = random.Random(1)
    cases = []
    while len(cases) < 20000:
        pieces = []
        for output in (True, False):
            n, heads, size = r.choice([1, 1, 2, 3, 5]), r.choice([1, 1, 2, 3, 4]), r.choice([1, 2, 3, 4])
            if not output:
                row, head = r.choice([0, r.randrange(40)]), r.choice([0, size, r.randrange(12)])
            elif r.random() < 0.5:  # heads inside their row
                head = size + r.choice([0, 0, r.randrange(4)])
                row = (heads - 1) * head + size + r.choice([0, 0, r.randrange(12)])
            else:
                row = size + r.choice([0, 0, r.randrange(4)])
                head = (n - 1) * row + size + r.choice([0, 0, r.randrange(12)])
            pieces.append([100 + r.randrange(60), n, heads, row, head, size])
        if r.random() < 0.4:
            pieces[1][3] = pieces[0][3]  # slices of the same rows
        cases.append(tuple(map(tuple, pieces)))
    got = answers(cases)
    want = [bool(held(a) & held(b)) for a, b in cases]
    assert 2000 < sum(want) < 18000
    wrong = [c for c, g, w in zip(cases, got, want) if g != w]
    assert not wrong, wrong[:5]


def test_slices_of_a_projection(answers):
    """q turned in place beside k and v of the same rows, of any number, in no time; a row further is an overlap."""
    q, k = 64 * 256, 8 * 256
    row, n = q + 2 * k, 1 << 30
    base = 1 << 40
    out = (base, n, 64, row, 256, 256)
    cases = [(out, (base + q, n, 8, row, 256, 256)), (out, (base + q + k, n, 8, row, 256, 256)), (out, (base + q - 16, n, 8, row, 256, 256)),
             (out, (base + q + 2 * k - 255, n, 8, row, 256, 256)), (out, (base - 2 * k, n, 8, row, 256, 256)),
             (out, (base - 2 * k + 1, n, 8, row, 256, 256)), (out, (base - 2 * k - 1, n, 8, row, 256, 256)), (out, (base + n * row, n, 8, row, 256, 256)), (out, (base - n * 4, n, 1, 4, 0, 4))]
    t = time.perf_counter()
    # (a row from base - 2 k + x on begins at base + q + x)
    assert answers(cases) == [False, False, True, True, False, False, True, False, False]
    assert time.perf_counter() - t < 5


def test_heads_apart_in_the_rows_of_a_projection(answers):
    """Heads of 192 channels of which 128 are turned, their values behind: no slower for any number of rows."""
    n, base = 1 << 30, 1 << 40
    row = 64 * 384 + 16 * 384
    out = (base, n, 64, row, 384, 256)
    rest = (base + 256, n, 64, row, 384, 128)  # the channels between
    k = (base + 64 * 384, n, 8, row, 384, 256)
    cases = [(out, rest), (out, k), (out, (base + 255, n, 64, row, 384, 128)), (out, (base + 256, n, 64, row, 384, 129)),
             (out, (base + 64 * 384 - 129, n, 8, row, 384, 256)), (out, (base - 16 * 384 - 128, n, 16, row, 384, 128)),
             (out, (base - 16 * 384 + 1, n, 16, row, 384, 384))]
    t = time.perf_counter()
    # (a row from base - 16 x 384 + x on begins at base + 64 x 384 + x; the last ends 383 bytes past the next row's first)
    assert answers(cases) == [False, False, True, True, True, False, True]
    assert time.perf_counter() - t < 5
