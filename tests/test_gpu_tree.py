"""GPU checks of the tree attention (mla_decode_tree) against the fp64 oracle with the same mask.

Tolerances: those of the other decodes (tests/_gpu.py), whose roundings these calls share (the absorbed
query, the probabilities, the merged latent and the output, half a bf16 step of 2^-8 each), and a tighter
one where the scores are all zero (test_counts_exactly_the_seen_tokens)."""
import numpy as np
import pytest
import torch

import mla_latent_kv_24_b200 as mla
import workloads as wl
from _gpu import assert_close
from _views import TreeCase, WindowCase, base_workload, tree_visible

pytestmark = pytest.mark.gpu


def check(c, what, fill=7.0):
    out = c.call(c.out(fill))
    mla.mla_get_device_status()
    got, ref = wl.from_torch_f64(out), c.reference()
    held = np.isnan(ref)
    assert (got[held] == fill).all(), "node slots without a node keep their output"
    if ref[~held].any():
        assert_close(got, ref, c.w.dtype, what)
    else:
        assert (got[~held] == 0).all()
    return out


SHAPES = [
    # (model, hpw, slots, context lengths, nodes): the first tree page starts anywhere in a step of 128 tokens
    ("dsv2", 1, 1, (0, 63, 1), (1, 1, 1)),
    ("dsv2", 1, 3, (64, 127, 5), (3, 1, 2)),
    ("dsv2", 1, 8, (1000, 0, 128, 63), (8, 8, 5, 1)),
    ("dsv2", 8, 13, (130, 700, 64), (13, 7, 12)),
    ("dsv2", 1, 33, (95, 3), (33, 32)),
    ("dsv2", 8, 64, (65, 0, 127), (64, 64, 63)),
    ("h16", 1, 5, (70, 0, 333), (5, 5, 1)),
    ("tiny", 1, 16, (0, 60, 64, 500), (16, 3, 16, 1)),
    ("tiny", 2, 64, (31, 129), (64, 40)),
]


@pytest.mark.parametrize("dense", [False, True])
@pytest.mark.parametrize("model,hpw,T,ctx,nodes", SHAPES)
def test_small_trees_match_oracle(model, hpw, T, ctx, nodes, dense):
    c = TreeCase(base_workload(model, hpw=hpw), T, ctx, nodes, seed=300 + T, dense=dense)
    c.poison_stale()
    check(c.upload(), f"tree {model} T={T} dense={dense}")


@pytest.mark.parametrize("page", [16, 32, 128])
def test_other_page_sizes(page):
    c = TreeCase(base_workload("tiny", page=page, hpw=2), 20, (15, 16, 0, 130), (20, 17, 20, 1), seed=320 + page)
    c.poison_stale()
    check(c.upload(), f"tree page {page}")


@pytest.mark.parametrize("T,ctx,nodes", [(4, (5000, 64), (4, 3)), (16, (4097, 129, 2000), (16, 9, 1)), (64, (1500,), (64,))])
def test_many_chunks_match_oracle(T, ctx, nodes):
    c = TreeCase(base_workload("dsv2", hpw=8), T, ctx, nodes, seed=330 + T)
    check(c.upload(), f"tree multi-chunk {ctx}")


def test_requests_without_nodes_take_no_part():
    c = TreeCase(base_workload("dsv2"), 6, (0, 100, 0, 70), (0, 0, 4, 6), seed=341)
    c.table_host[0] = c.table_host[1] = -5                            # nothing of theirs is read
    check(c.upload(), "idle requests")
    c = TreeCase(base_workload("dsv2"), 6, (0, 100), (0, 0), seed=342)
    check(c.upload(), "no nodes at all")


def test_nodes_that_see_nothing_give_zeros():
    c = TreeCase(base_workload("dsv2"), 5, (0, 0, 64), (5, 3, 5), seed=343)
    c.masks[0] = [0, 1 << 1, 0, 0, 1 << 63]                          # bits past the nodes count for nothing
    c.masks[1, :3] = 0
    c.masks[2] = 0
    out = check(c.upload(), "empty rows")
    assert (out[0, [0, 2, 3, 4]] == 0).all() and (out[1, :3] == 0).all() and out[0, 1].abs().sum() > 0
    t = TreeCase(base_workload("tiny"), 5, (0, 0), (5, 2), seed=344)
    t.masks[:] = 0
    out = check(t.upload(), "empty rows fp32")
    assert (out[0] == 0).all() and (out[1, :2] == 0).all()


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf"), 3.0e38])
@pytest.mark.parametrize("model", ["dsv2", "tiny"])
def test_rows_of_other_branches_may_hold_anything(model, value):
    # two branches behind a common context: what the second one's rows hold never reaches the first one
    T, ctx = 12, (100, 0, 61)
    c = TreeCase(base_workload(model), T, ctx, (T,) * 3, seed=345)
    first, second = sum(1 << i for i in range(0, T, 2)), sum(1 << i for i in range(1, T, 2))
    c.masks[:, 0::2], c.masks[:, 1::2] = np.uint64(first), np.uint64(second)
    for b in range(3):
        c.poison(b, ctx[b] + np.arange(1, T, 2), value)
    c.poison_stale()
    c.upload()
    got, ref = wl.from_torch_f64(c.call(c.out())), c.reference()
    mla.mla_get_device_status()
    assert_close(got[:, 0::2], ref[:, 0::2], c.w.dtype, f"other branch {value}")


def test_counts_exactly_the_seen_tokens():
    # Zero queries weigh every seen token alike, and a latent column that is 1 for one token and 0 for the
    # others shows that token's weight: 1 / seen.  Every probability is exactly 1 and the sums are small
    # whole numbers, so the only roundings are the merged latent's and the output's: 2 x 2^-8 of 1 / seen,
    # while one token too many or too few moves it by 1 / (seen + 1) >= 1 / 61 of it.
    T, ctx = 20, (40, 0, 24)
    c = TreeCase(base_workload("dsv2", hpw=8), T, ctx, (T, T, 17), seed=346, dense=True)
    c.q.zero_()
    c.cache.zero_()
    c.W_uv.zero_()
    c.W_uv[:, torch.arange(128), torch.arange(128)] = 1.0           # out = the first 128 latent columns
    for b in range(3):
        L = int(c.lens[b])
        pg, r = c.slots(b, np.arange(L))
        c.cache[torch.from_numpy(pg.astype(np.int64)).cuda(), torch.from_numpy(r.astype(np.int64)).cuda(),
                torch.arange(L, device="cuda")] = 1.0
    c.poison_stale()
    got = wl.from_torch_f64(c.upload().call(c.out()))
    mla.mla_get_device_status()
    for b in range(3):
        n, L = int(c.nodes[b]), int(c.lens[b])
        vis = tree_visible(L, n, c.masks[b])
        want = vis / np.maximum(vis.sum(1, keepdims=True), 1)
        for j in range(n):
            assert (got[b, j, :, L:] == 0).all()
            err = np.abs(got[b, j, :, :L] - want[j][None])
            assert (err <= 2.02 * 2 ** -8 * want[j][None]).all(), (b, j)


def test_a_chain_is_the_causal_decode():
    # nodes in a row, each seeing those before it: mla_decode_absorbed's s_q queries
    w = base_workload("dsv2")
    c = TreeCase(w, 4, (96, 700, 0), (4, 4, 4), seed=347)
    c.depths[:] = np.arange(4)
    c.masks[:] = np.asarray([1, 3, 7, 15], np.uint64)
    tree = c.upload().call(c.out())
    nb = mla.mla_decode_workspace_size(c.dims, 3, 4, c.lens)
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    out = c.out()
    mla.mla_decode_absorbed(c.dims, c.q, c.W_uk, c.W_uv, c.cache, c.d["page_table"], c.d["seq_lens"], c.lens, 3, 4,
                            c.max_pages, c.n_pages, out, ws)
    mla.mla_get_device_status()
    assert_close(wl.from_torch_f64(tree), wl.from_torch_f64(out), "bf16", "chain vs causal decode")


def test_large_scores_keep_the_running_maximum():
    # scores far apart (queries 40 times larger): the maximum moves by more than a lazy rescale forgives
    c = TreeCase(base_workload("dsv2"), 9, (900, 300), (9, 4), seed=348)
    c.q.mul_(40.0)
    c.inp.q.data = wl.f32_to_bf16_bits(wl.bf16_bits_to_f32(c.inp.q.data) * np.float32(40))
    assert torch.equal(c.q, wl.to_torch(c.inp.q))
    out = c.upload().call(c.out())
    mla.mla_get_device_status()
    got, ref = wl.from_torch_f64(out), c.reference()
    # A score is the sum of 576 products of the absorbed query, rounded by half a step of 2^-8 each, and
    # bf16 latents; scores of this size are off by whole units, which can swap which token wins, so rows are
    # compared where one token's weight is above 0.999 and no other is within 30 units of score.
    assert np.isfinite(got[~np.isnan(ref)]).all()
    from oracle import mla as om
    rows_checked = 0
    for b in range(2):
        L, n = int(c.lens[b]), int(c.nodes[b])
        rows = om.request_rows(c.inp.cache.f64(), c.inp.page_table, b, L)
        for j in range(n):
            seen = np.flatnonzero(c.visible(b)[j])
            for h in range(0, c.w.H, 16):
                q = om._q_tilde(c.inp.q.f64()[b, j, h], 128, c.positions(b)[j], c.w.rope_base)
                K = np.concatenate([rows[:, :512] @ c.inp.W_uk.f64()[h].T, rows[:, 512:]], 1)[seen]
                s = np.sort(K @ q * c.w.softmax_scale)
                q_lat = c.inp.W_uk.f64()[h].T @ q[:128]
                # the largest error the absorbed query's rounding can cause in any score
                off = 2 ** -8 * c.w.softmax_scale * (np.abs(rows[seen][:, :512]) @ np.abs(q_lat) +
                                                     np.abs(rows[seen][:, 512:]) @ np.abs(q[128:])).max()
                if s[-1] - s[-2] > 2 * off + 12:      # the others' weight is below L e^-12 in any rounding
                    rows_checked += 1
                    # what is left: the rounding of the winner's probability (its reference may lag behind the
                    # maximum), of the merged latent and of the output, and L e^-12 of other rows
                    tol = 3 * 2 ** -8 * np.abs(c.inp.W_uv.f64()[h]) @ np.abs(rows[seen][np.argmax(K @ q)][:512]) + 0.05
                    assert (np.abs(got[b, j, h] - ref[b, j, h]) <= tol).all()
    assert rows_checked > 0


def test_captured_call_replays_and_two_graphs_keep_their_workspaces():
    cases = [TreeCase(base_workload("dsv2"), 7, (300, 64), (7, 5), seed=350).upload(),
             TreeCase(base_workload("dsv2"), 7, (1000, 10), (6, 7), seed=351).upload()]
    eager = [c.call(c.out()).clone() for c in cases]
    torch.cuda.synchronize()
    outs, graphs = [c.out() for c in cases], []
    for c, o in zip(cases, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.call(o)
        graphs.append(g)
    for o in outs:
        o.zero_()
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    mla.mla_get_device_status()
    for o, e in zip(outs, eager):
        assert torch.equal(o, e)
    del graphs


def test_two_streams_at_once():
    cases = [TreeCase(base_workload("dsv2"), 16, (900, 400), (16, 11), seed=352 + i).upload() for i in range(2)]
    alone = [c.call(c.out()).clone() for c in cases]
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in cases], [c.out() for c in cases]
    torch.cuda.synchronize()
    for _ in range(5):
        for c, s, o in zip(cases, streams, outs):
            with torch.cuda.stream(s):
                c.call(o)
    torch.cuda.synchronize()
    mla.mla_get_device_status()
    for o, e in zip(outs, alone):
        assert torch.equal(o, e)


def test_counts_that_contradict_the_host_are_reported():
    c = TreeCase(base_workload("dsv2"), 6, (100, 300), (6, 3), seed=356).upload()
    good = c.d["n_nodes"].clone()
    for bad in ([6, 4], [9, 3], [-1, 3], [6, 0]):
        c.d["n_nodes"] = c.dev(np.asarray(bad, np.int32))
        out = c.call(c.out(3.0))
        with pytest.raises(mla.MlaError) as e:
            mla.mla_get_device_status()
        assert e.value.status == 1
        assert (out == 3.0).all()                                    # nothing was written
    c.d["n_nodes"] = good
    check(c, "after a refused plan")


def test_out_of_range_page_is_reported():
    c = TreeCase(base_workload("dsv2"), 6, (200, 64), (6, 3), seed=357)
    keep = c.table_host.copy()
    for bad in (-1, c.n_pages, 1 << 30):
        c.table_host = keep.copy()
        c.table_host[0, 1] = bad
        c.upload().call(c.out())
        with pytest.raises(mla.MlaError) as e:
            mla.mla_get_device_status()
        assert e.value.status == 5
    c.table_host = keep
    check(c.upload(), "after a bad page")


@pytest.mark.parametrize("T,ctx,nodes", [(64, (9000, 100), (64, 64)), (40, (700, 6000, 65, 64), (40, 17, 40, 33)),
                                         (32, (130, 9000), (31, 32))])
def test_many_rows_with_several_chunks(T, ctx, nodes):
    # more than 96 rows merge by tiles of 128 on tcgen05, and the long request's rows have several chunks; one
    # weight group's heads are held against the oracle, over every row
    c = TreeCase(base_workload("dsv2", hpw=8), T, ctx, nodes, seed=360 + T).upload()
    out = c.call(c.out(7.0))
    mla.mla_get_device_status()
    got = wl.from_torch_f64(out)
    from oracle import mla as om
    for b in range(c.B):
        n, L = int(c.nodes[b]), int(c.lens[b])
        rows = om.request_rows(c.inp.cache.f64(), c.inp.page_table, b, L)
        for g in (0, 9):
            hs = slice(8 * g, 8 * g + 8)
            ref = om.decode_request_masked(c.inp.q.f64()[b, :n, hs], rows, c.inp.W_uk.f64()[g:g + 1],
                                           c.inp.W_uv.f64()[g:g + 1], 8, c.w.softmax_scale, c.w.rope_base, c.positions(b),
                                           c.visible(b))
            assert_close(got[b, :n, hs], ref, "bf16", f"many rows T={T} request {b} group {g}")
        assert (got[b, n:] == 7.0).all()


@pytest.mark.parametrize("windowed", [False, True])
def test_large_scores_in_causal_rows(windowed):
    # the same for rows that see all before them, with and without a window: O is rescaled out of line in every step
    # whose maximum rises, and columns left out of it would keep the earlier tokens' sum
    w = base_workload("dsv2")
    c = WindowCase(w, 4, (1400, 700), 3, 900, seed=349)
    c.q.mul_(40.0)
    c.inp.q.data = wl.f32_to_bf16_bits(wl.bf16_bits_to_f32(c.inp.q.data) * np.float32(40))
    if not windowed:
        c.sinks, c.window = 0, 1 << 20
    c.upload()
    out = c.out()
    if windowed:
        c.call(out)
    else:
        ws = torch.full((mla.mla_decode_workspace_size(c.dims, 2, 4, c.lens),), 255, dtype=torch.uint8, device="cuda")
        mla.mla_decode_absorbed(c.dims, c.q, c.W_uk, c.W_uv, c.cache, c.d["page_table"], c.d["seq_lens"], c.lens, 2, 4,
                                c.max_pages, c.n_pages, out, ws)
    mla.mla_get_device_status()
    got, ref = wl.from_torch_f64(out), c.reference()
    assert np.isfinite(got).all()
    from oracle import mla as om
    rows_checked = rising = 0
    for b in range(2):
        rows = om.request_rows(c.inp.cache.f64(), c.inp.page_table, b, int(c.lens[b]))
        for j in range(4):
            seen = np.flatnonzero(c.visible(b)[j])
            for h in range(0, w.H, 16):
                q = om._q_tilde(c.inp.q.f64()[b, j, h], 128, int(c.lens[b]) - 4 + j, w.rope_base)
                K = np.concatenate([rows[:, :512] @ c.inp.W_uk.f64()[h].T, rows[:, 512:]], 1)[seen]
                s = K @ q * w.softmax_scale
                rising += s[128:].max() > s[:128].max() + 20
                top = np.sort(s)
                q_lat = c.inp.W_uk.f64()[h].T @ q[:128]
                off = 2 ** -8 * w.softmax_scale * (np.abs(rows[seen][:, :512]) @ np.abs(q_lat) +
                                                   np.abs(rows[seen][:, 512:]) @ np.abs(q[128:])).max()
                if top[-1] - top[-2] > 2 * off + 12:      # as above: the winner's weight is 1 in any rounding
                    rows_checked += 1
                    tol = 3 * 2 ** -8 * np.abs(c.inp.W_uv.f64()[h]) @ np.abs(rows[seen][np.argmax(s)][:512]) + 0.05
                    assert (np.abs(got[b, j, h] - ref[b, j, h]) <= tol).all()
    assert rows_checked > 0 and rising > 0
