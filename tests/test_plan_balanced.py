"""The views' host plan rule (csrc/plan_host.h, plan_chunk_balanced), compiled with g++: a chunk is a multiple of the
granule, covers the longest row in a bounded number of pieces, and its snake-dealt items load the busiest worker no more
than one chunk per row would."""
import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SRC = r'''
#include <cstdio>
#include <cstdlib>
#include <vector>
#include "plan_host.h"
int main(int argc, char **argv) {
    int units = atoi(argv[1]), granule = atoi(argv[2]), n = (argc - 3) / 2;
    std::vector<int> rows(n), lens(n);
    for (int b = 0; b < n; ++b) rows[b] = atoi(argv[3 + 2 * b]), lens[b] = atoi(argv[4 + 2 * b]);
    printf("%d\n", mla::plan_chunk_balanced(n, [&](int b) { return rows[b]; }, [&](int b) { return lens[b]; }, units, granule));
    return 0;
}
'''


@pytest.fixture(scope="module")
def rule(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not available")
    d = tmp_path_factory.mktemp("balanced")
    (d / "probe.cpp").write_text(SRC)
    subprocess.run([gxx, "-std=c++17", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover", "-I",
                    os.path.join(ROOT, "mla_latent_kv_24_b200", "csrc"), str(d / "probe.cpp"), "-o", str(d / "probe")], check=True)

    def run(requests, units=74, granule=128):
        flat = [str(x) for r in requests for x in r]
        return int(subprocess.run([str(d / "probe"), str(units), str(granule), *flat], check=True, capture_output=True,
                                  text=True).stdout)
    return run


def busiest(requests, chunk, units, granule, item):
    lens = [n for k, n in requests for _ in range(k)]
    full = [chunk] * sum(n // chunk for n in lens)
    last = sorted((n % chunk for n in lens if n % chunk), reverse=True)
    load = [0.0] * units
    for j, t in enumerate(full + last):
        r, p = divmod(j, units)
        load[units - 1 - p if r & 1 else p] += -(-t // granule) + item
    return max(load)


CASES = [
    [(1, 1)], [(64, 64)], [(8, 1008)], [(64, 8256)] * 8, [(0, 0), (5, 300), (0, 10)], [(0, 5)] * 3,
    [(2, n) for n in range(1024, 32768, 500)], [(1, 131072)] * 4, [(1, 1)] * 2000, [(4, 2 ** 30)], [(64, 131072)] * 600,
    [(1, 64), (13, 100000)], [(3, 128)] * 25,
]


@pytest.mark.parametrize("k", range(len(CASES)))
@pytest.mark.parametrize("units,granule", [(74, 128), (1, 128), (300, 128)])
def test_rule(rule, k, units, granule):
    requests = CASES[k]
    chunk = rule(requests, units, granule)
    assert chunk % granule == 0 and chunk >= granule
    live = [(r, n) for r, n in requests if r > 0 and n > 0]
    if not live:
        return
    items = sum(r * -(-n // chunk) for r, n in live)
    longest, total = max(n for _, n in live), sum(r * n for r, n in live)
    # pieces come from cutting the longest row in at most six, or all tokens in at most eight a worker
    assert items <= sum(r for r, _ in live) + max(6 * sum(r for r, _ in live), 8 * min(units, 256) + 8 * total // longest)
    if units <= 256 and items < 20000:
        one = -(-longest // granule) * granule
        # buckets stand for lengths within 1/64 of a chunk, and rounds of equal items for the snake's
        slack = 1.05 * busiest(live, one, units, granule, 3.7) + 0.055 * (sum(r for r, _ in live)) + 4
        assert busiest(live, chunk, units, granule, 3.7) <= slack + chunk / granule / 64 * 8


def test_random_batches_are_no_worse_than_one_chunk_per_row(rule):
    rnd = random.Random(5)
    gain = []
    for _ in range(40):
        requests = [(rnd.randint(1, 16), int(2 ** rnd.uniform(5, 15))) for _ in range(rnd.randint(1, 40))]
        chunk = rule(requests)
        one = -(-max(n for _, n in requests) // 128) * 128
        cost = lambda c: busiest(requests, c, 74, 128, 3.7) + 0.055 * sum(r * -(-n // c) for r, n in requests)  # noqa: E731
        gain.append(cost(one) / cost(chunk))
    assert min(gain) >= 0.95 and sum(gain) / len(gain) > 1.05
