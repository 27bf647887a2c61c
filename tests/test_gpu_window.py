"""GPU checks of the sliding window with sinks (mla_decode_window, gqla_decode_window) against the fp64
oracle with the same mask.  Pages that no query sees have no valid page-table entry, and every other row
that none sees holds NaN.  Tolerances: those of the other decodes (tests/_gpu.py)."""
import numpy as np
import pytest
import torch

import mla_latent_kv_24_b200 as mla
import workloads as wl
from _gpu import assert_close
from _views import WindowCase, base_workload

pytestmark = pytest.mark.gpu


def check(c, what, grouped=False):
    exp = c.expand() if grouped else None
    c.free_unseen(exp)
    out = c.upload(grouped).call(c.out(float("nan")), exp)
    mla.mla_get_device_status()
    assert_close(wl.from_torch_f64(out), c.reference(), c.w.dtype, what)
    return out


BIG = 2 ** 31 - 1
SHAPES = [
    # (s_q, lengths, sinks, window)
    (1, (1, 64, 65, 1000), 0, 1),
    (1, (1, 64, 700, 129), 4, 64),
    (2, (2, 130, 1000), 64, 65),
    (3, (3, 64, 500), 1, 2),
    (4, (4, 700, 131), 100, 127),
    (1, (500, 63), BIG, 1),
    (2, (500, 63), 0, BIG),
    (4, (900, 200), 65, 300),
]


@pytest.mark.parametrize("model,hpw", [("dsv2", 1), ("dsv2", 8), ("h16", 2), ("tiny", 1)])
@pytest.mark.parametrize("s_q,lens,sinks,window", SHAPES)
def test_absorbed_windows_match_oracle(model, hpw, s_q, lens, sinks, window):
    c = WindowCase(base_workload(model, hpw=hpw), s_q, lens, sinks, window, seed=400 + s_q)
    check(c, f"window {model} {s_q} {sinks}+{min(window, 9999)}")


@pytest.mark.parametrize("s_q,lens,sinks,window", SHAPES)
def test_grouped_windows_match_oracle(s_q, lens, sinks, window):
    c = WindowCase(base_workload("gqla"), s_q, lens, sinks, window, seed=420 + s_q)
    check(c, f"gqa window {s_q} {sinks}+{min(window, 9999)}", grouped=True)


@pytest.mark.parametrize("H,hpw,dtype", [(16, 4, "bf16"), (8, 2, "fp32")])
def test_grouped_windows_on_the_cuda_cores(H, hpw, dtype):
    w = wl.small_workload(wl.WORKLOADS["1"], H=H, hpw=hpw, dtype=dtype, shuffle_pages=True)
    for s_q, lens, sinks, window in SHAPES[1:4]:
        c = WindowCase(w, s_q, lens, sinks, window, seed=430 + s_q)
        check(c, f"gqa window {dtype} H={H} {s_q}", grouped=True)


@pytest.mark.parametrize("page", [16, 32, 128])
def test_other_page_sizes(page):
    c = WindowCase(base_workload("tiny", page=page), 2, (2, 130, 700), 20, 100, seed=440 + page)
    check(c, f"window page {page}")


@pytest.mark.parametrize("s_q,lens,sinks,window", [(1, (6000,), 64, 3000), (2, (5000, 129, 9000), 130, 4000), (4, (7000, 300), 4, 2500)])
def test_many_chunks_match_oracle(s_q, lens, sinks, window):
    c = WindowCase(base_workload("gqla"), s_q, lens, sinks, window, seed=450 + s_q)
    check(c, f"window multi-chunk {s_q}")
    c = WindowCase(base_workload("gqla"), s_q, lens, sinks, window, seed=450 + s_q)
    check(c, f"gqa window multi-chunk {s_q}", grouped=True)


def test_far_along_a_long_request():
    # position 131071 with a window of 200: three or four pages and the sinks' are all that exists
    L, S, W = 131072, 4, 200
    w = base_workload("dsv2")
    c = WindowCase(w, 1, (S + W + 64,), S, W, seed=460)              # the rows that exist
    table = np.full((1, L // 64), -1, np.int32)
    have = c.inp.page_table[0]
    first = (L - W) // 64
    table[0, 0] = have[0]
    table[0, first:] = have[1:1 + L // 64 - first]
    c.table_host, c.lens, c.max_pages = table, np.asarray([L], np.int32), table.shape[1]
    c.upload()
    out = c.call(c.out())
    mla.mla_get_device_status()
    t = np.concatenate([np.arange(S), np.arange(L - W, L)])
    rows = c.inp.cache.f64()[table[0, t // 64], t % 64]
    import oracle
    ref = oracle.decode_request_masked(c.inp.q.f64()[0], rows, c.inp.W_uk.f64(), c.inp.W_uv.f64(), 1, w.softmax_scale,
                                       w.rope_base, [L - 1], np.ones((1, S + W), bool))
    assert_close(wl.from_torch_f64(out)[0], ref, "bf16", "window at position 131071")


@pytest.mark.parametrize("s_q", [1, 2])
def test_a_window_over_everything_is_the_causal_decode(s_q):
    c = WindowCase(base_workload("gqla"), s_q, (700, 64, 130), 0, 100000, seed=470 + s_q)
    exp = c.expand()
    for grouped in (False, True):
        got = c.upload(grouped).call(c.out(), exp)
        out = c.out()
        size = mla.gqla_decode_workspace_size if grouped else mla.mla_decode_workspace_size
        ws = torch.empty(size(c.dims, 3, s_q, c.lens), dtype=torch.uint8, device="cuda")
        if grouped:
            mla.gqla_decode_grouped(c.dims, c.q, exp, c.cache, c.d["page_table"], c.d["seq_lens"], c.lens, 3, s_q,
                                    c.max_pages, c.n_pages, out, ws)
        else:
            mla.mla_decode_absorbed(c.dims, c.q, c.W_uk, c.W_uv, c.cache, c.d["page_table"], c.d["seq_lens"], c.lens, 3,
                                    s_q, c.max_pages, c.n_pages, out, ws)
        mla.mla_get_device_status()
        assert_close(wl.from_torch_f64(got), wl.from_torch_f64(out), "bf16", f"whole window grouped={grouped}")


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_tokens_only_another_query_sees_do_not_reach_a_query_on_the_absorbed_path(value):
    # every query is a plan row of its own there: the newest token of the second query may hold anything
    c = WindowCase(base_workload("dsv2"), 2, (300, 65), 4, 50, seed=480)
    for b, L in enumerate(c.lens):
        c.poison(b, np.asarray([int(L) - 1]), value)
    got, ref = wl.from_torch_f64(c.upload().call(c.out())), c.reference()
    mla.mla_get_device_status()
    assert_close(got[:, 0], ref[:, 0], "bf16", "first query")


def test_captured_call_replays():
    c = WindowCase(base_workload("gqla"), 2, (1000, 64, 300), 4, 200, seed=481)
    exp = c.expand()
    for grouped in (False, True):
        eager = c.upload(grouped).call(c.out(), exp).clone()
        torch.cuda.synchronize()
        out, g = c.out(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.call(out, exp)
        out.zero_()
        for _ in range(3):
            g.replay()
        torch.cuda.synchronize()
        mla.mla_get_device_status()
        assert torch.equal(out, eager)
        del g


def test_page_of_the_window_out_of_range_is_reported():
    c = WindowCase(base_workload("gqla"), 1, (500, 300), 4, 100, seed=482)
    exp = c.expand()
    c.table_host[0, 500 // 64] = c.n_pages
    for grouped in (False, True):
        c.upload(grouped).call(c.out(), exp)
        with pytest.raises(mla.MlaError) as e:
            mla.mla_get_device_status()
        assert e.value.status == 5


def test_lengths_that_contradict_the_host_are_reported():
    c = WindowCase(base_workload("dsv2"), 2, (500, 300), 0, 5000, seed=483).upload()
    c.d["seq_lens"] = c.dev(np.asarray([500, 1], np.int32))
    c.call(c.out())
    with pytest.raises(mla.MlaError) as e:
        mla.mla_get_device_status()
    assert e.value.status == 1


@pytest.mark.parametrize("B", [17, 24, 130])
def test_rows_of_several_chunks_under_either_merge(B):
    # a few more rows than one tile of the clusters' merge, with many chunks (17) or some (24), and more rows than one
    # tile of the other
    lens = [1400 - 7 * b for b in range(B - 1)] + [1] if B < 100 else [300 - b for b in range(B)]
    c = WindowCase(base_workload("gqla"), 1, lens, 70, 1000, seed=484 + B)
    c.free_unseen()
    out = c.upload().call(c.out())
    mla.mla_get_device_status()
    assert_close(wl.from_torch_f64(out), c.reference(), "bf16", f"window, {B} rows")
