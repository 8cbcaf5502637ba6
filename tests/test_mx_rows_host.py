"""The integer rules for rows sorted by expert (csrc/mx_rows.h), compiled for the
host, against plain Python: offsets of any value, partitions and none."""
import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

MAIN = r'''
#include <cstdio>
#include <cstring>

#include "mx_rows.h"

int main() {
    char what[16];
    long long a, b, c, d, e;
    while (scanf("%15s %lld %lld %lld %lld %lld", what, &a, &b, &c, &d, &e) == 6)
        if (!strcmp(what, "end"))
            printf("%lld\n", (long long)qg::mx_span_end(a, b, c, d, (int)e));
        else if (!strcmp(what, "blocks")) printf("%d\n", qg::mx_add_blocks((int)a, (int)b, (int)c, (int)d, (int)e));
}
'''

LOW, TOP = -2 ** 31, 2 ** 31 - 1


@pytest.fixture(scope="module")
def rules(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("no host C++ compiler")
    d = tmp_path_factory.mktemp("rows")
    (d / "m.cpp").write_text(MAIN)
    subprocess.check_call(["g++", "-O1", "-std=c++17", "-fsanitize=undefined", "-fno-sanitize-recover", "-I",
                           os.path.join(ROOT, "quantized_gemm_tcgen05_gb300", "csrc"), str(d / "m.cpp"), "-o", str(d / "m")])

    def ask(name, rows):
        text = "".join(f"{name} {' '.join(map(str, r))}\n" for r in rows)
        out = subprocess.run([str(d / "m")], input=text, capture_output=True, text=True, check=True).stdout.split()
        assert len(out) == len(rows)
        return list(map(int, out))

    return ask


def values(rng, n):
    some = [LOW, LOW + 1, -1, 0, 1, 127, 128, 255, 256, 257, 1000, TOP - 1, TOP]
    return [rng.choice(some) if rng.random() < 0.5 else rng.randint(LOW, TOP) for _ in range(n)]


def test_blocks_are_counted_up_to_the_most_there_can_be(rules):
    rng, ask = random.Random(1), []
    for _ in range(4000):
        most = rng.choice([1, 4, 1000, 2 ** 23 + 4096])
        lo, hi = values(rng, 2)
        ask.append((rng.randint(0, most), lo, hi, rng.choice([128, 256]), most))
    want = [min(n + max(0, -(-(hi - lo) // bm)), most) for n, lo, hi, bm, most in ask]
    assert rules("blocks", ask) == want


def test_a_partition_never_reaches_the_limit_early(rules):
    # most: rows / bm + experts, as the host gives it
    rng = random.Random(2)
    for _ in range(60):
        bm, experts = 256, rng.randint(1, 40)
        counts = [rng.choice([0, 1, 255, 256, 257, rng.randint(0, 3000)]) for _ in range(experts)]
        rows = sum(counts) + rng.randint(0, 5)
        most = min(rows // bm + experts, rows)
        n, lo = 0, 0
        for c in counts:
            n = rules("blocks", [(n, lo, lo + c, bm, most)])[0]
            lo += c
        assert n == sum(-(-c // bm) for c in counts)


def test_no_row_of_a_span_has_its_scales_past_the_end(rules):
    rng, ask = random.Random(3), [(8, 256, 4, 256, 3)]
    for _ in range(4000):
        rows, experts = rng.choice([1, 127, 128, 256, 5000, TOP]), rng.choice([1, 3, 40, 4096])
        lo, hi = values(rng, 2)
        if rng.random() < 0.5:
            lo, hi = rng.randint(0, 600), rng.randint(0, 1200)
        ask.append((lo, max(lo, hi), rng.choice([0, rows // 128, rows // 128 + experts - 1, rng.randint(0, 2 ** 37)]), rows, experts))
    assert rules("end", ask[:1]) == [136]  # one atom row is left
    for (lo, hi, tiles, rows, experts), end in zip(ask, rules("end", ask)):
        held = [r for r in (lo, lo + 127, lo + 128, end - 1, end, hi - 1) if lo <= r < hi]
        for r in held:
            inside = lo >= 0 and tiles + (r - lo) // 128 < rows // 128 + experts
            assert (r < end) == inside, (lo, hi, tiles, rows, experts, end, r)


def test_a_span_of_a_partition_is_whole(rules):
    rng = random.Random(4)
    for _ in range(60):
        counts = [rng.choice([0, 1, 127, 128, 129, rng.randint(0, 2000)]) for _ in range(rng.randint(1, 40))]
        rows, ask, lo, tiles = sum(counts), [], 0, 0
        for c in counts:
            ask.append((lo, lo + c, tiles, rows, len(counts)))
            lo, tiles = lo + c, tiles + -(-c // 128)
        assert rules("end", [a for a in ask if a[0] < a[1]]) == [a[1] for a in ask if a[0] < a[1]]
