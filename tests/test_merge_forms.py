"""Which kernels absorb the queries and merge the chunks of a tree's or window's call (plan_host.h), asserted on the CPU
for each case that the GPU tests below, and those of test_gpu_tree.py, hold against the oracle.  So a change of the
plan or of the rule cannot leave a form of the merge untested: one chunk a row, two, three and more, a mixture with
empty rows inside one 128-row tile, and the clusters that take the rows where tcgen05 does not pay."""
import numpy as np
import pytest

from _merge_plan import compile_choice


@pytest.fixture(scope="module")
def choice(tmp_path_factory):
    return compile_choice(tmp_path_factory.mktemp("choice"))


# name: (T, contexts, nodes), absorption on tcgen05, merge on tcgen05, chunk counts in the first 128 rows
TREES = {
    "one chunk": ((64, (600,), (64,)), True, True, {1}),
    "two chunks": ((37, (1000,), (37,)), True, True, {2}),
    "three chunks": ((20, (2000,), (20,)), True, True, {3}),
    "five chunks": ((40, (20000,), (40,)), True, True, {5}),
    "a mixture": ((10, (1023, 2168, 351), (10, 9, 4)), True, True, {0, 1, 2, 4}),
    "one and three": ((33, (1619, 306, 651, 134), (3, 6, 17, 7)), True, True, {0, 1, 2, 5}),
    "17 rows": ((17, (90,), (17,)), True, True, {1}),
    "16 rows": ((16, (90,), (16,)), False, False, {1}),
    "16 rows, chunks": ((16, (4097, 129, 2000), (16, 9, 1)), True, True, {0, 1, 2, 4}),
}
WINDOWS = {   # s_q, lengths, sinks, window
    "window, three": ((2, (5000,) * 12, 4, 4000), True, True, {3}),
    "window, clusters": ((1, (5000,) * 18, 4, 4000), True, False, {4}),
    "window, one": ((2, tuple(100 + 37 * i for i in range(20)), 3, 90), True, True, {1}),
}


@pytest.mark.parametrize("name", TREES)
def test_tree_forms(choice, name):
    (T, ctx, nodes), absorb, project, chunks = TREES[name]
    c = choice("tree", T, [a + b for a, b in zip(ctx, nodes)], nodes)
    assert (c.absorb_tc, c.project_tc) == (absorb, project) and set(c.chunks[:128]) == chunks


@pytest.mark.parametrize("name", WINDOWS)
def test_window_forms(choice, name):
    (s_q, lens, sinks, window), absorb, project, chunks = WINDOWS[name]
    c = choice("window", s_q, lens, [0] * len(lens), sinks, window)
    assert (c.absorb_tc, c.project_tc) == (absorb, project) and set(c.chunks[:128]) == chunks


def test_forms_of_the_tree_tests_with_many_rows(choice):
    # test_gpu_tree.py::test_many_rows_with_several_chunks: all merge on tcgen05, in one chunk a row, a mixture with four,
    # and a mixture with two
    for (T, ctx, nodes), chunks in (((64, (9000, 100), (64, 64)), {1}), ((40, (700, 6000, 65, 64), (40, 17, 40, 33)), {0, 1, 4}),
                                    ((32, (130, 9000), (31, 32)), {0, 1, 2})):
        c = choice("tree", T, [a + b for a, b in zip(ctx, nodes)], nodes)
        assert c.absorb_tc and c.project_tc and set(c.chunks) == chunks


def test_rule_by_rows_and_chunks(choice):
    # 16 rows and fewer never go to tcgen05; rows of few chunks do, of many do not
    for rows in range(1, 17):
        c = choice("window", 1, [2000] * rows, [0] * rows, 0, 2000)
        assert not c.absorb_tc and not c.project_tc
    for rows in range(17, 80, 7):
        c = choice("window", 1, [2000] * rows, [0] * rows, 0, 2000)
        assert c.absorb_tc and c.project_tc == (6 * sum(c.chunks) <= rows * rows)


def held(out, c, name, visible, positions, n_of):
    import workloads as wl
    from _gpu import assert_close
    from oracle import mla as om
    got = wl.from_torch_f64(out)
    for b in range(c.B):
        n = n_of(b)
        rows = om.request_rows(c.inp.cache.f64(), c.inp.page_table, b, int(c.lens[b]))
        for g in (0, 5, 15):                                # one weight group's heads each, over every row
            hs = slice(8 * g, 8 * g + 8)
            ref = om.decode_request_masked(c.inp.q.f64()[b, :n, hs], rows, c.inp.W_uk.f64()[g:g + 1],
                                           c.inp.W_uv.f64()[g:g + 1], 8, c.w.softmax_scale, c.w.rope_base, positions(b),
                                           visible(b))
            assert_close(got[b, :n, hs], ref, "bf16", f"{name} request {b} group {g}")
        assert (got[b, n:] == 7.0).all()                    # slots without a node


@pytest.mark.gpu
@pytest.mark.parametrize("name", TREES)
def test_trees_match_oracle(name):
    import mla_latent_kv_24_b200 as mla
    from _views import TreeCase, base_workload
    T, ctx, nodes = TREES[name][0]
    c = TreeCase(base_workload("dsv2", hpw=8), T, ctx, nodes, seed=510 + T).upload()
    c.poison_stale()
    out = c.call(c.out(7.0))
    mla.mla_get_device_status()
    held(out, c, name, c.visible, c.positions, lambda b: int(c.nodes[b]))


@pytest.mark.gpu
@pytest.mark.parametrize("name", WINDOWS)
def test_windows_match_oracle(name):
    import mla_latent_kv_24_b200 as mla
    from _views import WindowCase, base_workload
    s_q, lens, sinks, window = WINDOWS[name][0]
    c = WindowCase(base_workload("dsv2", hpw=8), s_q, lens, sinks, window, seed=520)
    c.free_unseen()
    c.upload()
    out = c.call(c.out(7.0))
    mla.mla_get_device_status()
    held(out, c, name, c.visible, lambda b: int(c.lens[b]) - s_q + np.arange(s_q), lambda b: s_q)
