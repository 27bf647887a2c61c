"""The host's choices for a tree's or window's call on the tcgen05 decode, compiled from the library's own headers with
g++: its chunk length, the chunks of each row, and which kernels absorb the queries and merge the chunks."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SMS = 148
SRC = r'''
#include <climits>
#include <cstdio>
#include <cstdlib>
#include <vector>
#include "plan_host.h"
#include "view.cuh"
using namespace mla;
// kind sinks window n_q units (L n)...
int main(int argc, char **argv) {
    const int kind = atoi(argv[1]), sinks = atoi(argv[2]), window = atoi(argv[3]), n_q = atoi(argv[4]), units = atoi(argv[5]);
    const int batch = (argc - 6) / 2;
    std::vector<int> L(batch), n(batch);
    for (int b = 0; b < batch; ++b) L[b] = atoi(argv[6 + 2 * b]), n[b] = atoi(argv[7 + 2 * b]);
    auto len = [&](int r) { return view_row_len(kind, sinks, window, L[r / n_q], n[r / n_q], n_q, n_q, r % n_q, 64, INT_MAX); };
    auto rows = [&](int b) { return kind == VIEW_TREE ? n[b] : n_q; };
    auto last = [&](int b) { return len(b * n_q + std::max(rows(b), 1) - 1); };
    const int chunk = plan_chunk_balanced(batch, rows, last, units, 128);
    const long long work = plan_count_rows(batch * n_q, len, chunk);
    printf("%d %d %d", chunk, (int)absorb_tc_pays(batch * n_q), (int)project_tc_pays(batch * n_q, work));
    for (int r = 0; r < batch * n_q; ++r) printf(" %d", (len(r) + chunk - 1) / chunk);
    printf("\n");
    return 0;
}
'''


class Choice:
    def __init__(self, chunk, absorb_tc, project_tc, chunks):
        self.chunk, self.absorb_tc, self.project_tc, self.chunks = chunk, bool(absorb_tc), bool(project_tc), chunks


def compile_choice(tmp):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not available")
    (tmp / "choice.cpp").write_text(SRC)
    subprocess.run([gxx, "-std=c++17", "-O1", "-I", os.path.join(ROOT, "mla_latent_kv_24_b200", "csrc"),
                    str(tmp / "choice.cpp"), "-o", str(tmp / "choice")], check=True)

    def run(kind, n_q, lens, nodes, sinks=0, window=1):
        flat = [str(x) for r in zip(lens, nodes) for x in r]
        o = subprocess.run([str(tmp / "choice"), str({"window": 1, "tree": 2}[kind]), str(sinks), str(window), str(n_q),
                            str(SMS // 2), *flat], check=True, capture_output=True, text=True).stdout.split()
        return Choice(int(o[0]), int(o[1]), int(o[2]), [int(x) for x in o[3:]])
    return run
