"""Failure detection of the bounded waits in the products per head around a tree's or window's decode (head_gemm.cu),
without a GPU fault.  The hook withholds the completion signal of one block; the waits on it run out after a short
limit, MLA_ERR_TIMEOUT is recorded, the kernels stop, free their tensor memory and return, and the same context then
computes the same bits as before."""
import time

import pytest
import torch

import mla_latent_kv_24_b200 as mla
from _views import TreeCase, WindowCase, base_workload

pytestmark = pytest.mark.gpu


def tree(T, ctx, nodes):
    return TreeCase(base_workload("dsv2", hpw=8), T, ctx, nodes, seed=71).upload()


def window(lens):
    return WindowCase(base_workload("dsv2", hpw=8), 1, lens, 2, 60, seed=72).upload()


# 40 and 24 rows of one chunk each (at most two steps of 128 tokens), 130 rows in two tiles, and 64 rows of which half
# have several chunks.  Block 0 is withheld from the absorption, the decode and the projection alike; a decode of two
# steps has no step 3 or 7, and of the absorption's one block neither, so those are the projection's alone.
CASES = {
    "tree": lambda: tree(40, (126, 65), (40, 33)),
    "window": lambda: window(tuple(70 + i for i in range(24))),
    "two tiles": lambda: tree(64, (30, 0, 9), (64, 64, 2)),
    "chunks": lambda: tree(32, (9000, 100), (32, 32)),
}


@pytest.mark.parametrize("name,withhold", [("tree", 0), ("tree", 3), ("tree", 5), ("tree", 7), ("window", 0), ("window", 7),
                                           ("two tiles", 1), ("two tiles", 5), ("chunks", 0), ("chunks", 7)])
def test_withheld_block_times_out_and_the_context_recovers(name, withhold):
    c = CASES[name]()
    c.ws.zero_()            # what a stopped call leaves in the workspace is finite
    want = c.call(c.out()).clone()
    mla.mla_get_device_status()
    out = c.out(7.0)
    mla.mla_debug_decode_fault(withhold, 2000)
    try:
        t0 = time.perf_counter()
        c.call(out)
        with pytest.raises(mla.MlaError) as e:
            mla.mla_get_device_status()
        elapsed = time.perf_counter() - t0
    finally:
        mla.mla_debug_decode_fault(-1, 0)
    assert e.value.status == 6, e.value
    assert elapsed < 2.0, elapsed                                 # the short limit, in these kernels too
    if name == "tree" and withhold >= 3:                          # only the projection: no tile of it was finished
        assert (out == 7.0).all()
    for _ in range(2):
        got = c.call(c.out())
        mla.mla_get_device_status()
        assert torch.equal(got.view(torch.int16), want.view(torch.int16))


def test_the_signal_of_the_last_block_but_one_has_no_waiter():
    # the last block's signal comes after the products of all blocks before it, and no operands follow block 6's
    c = CASES["tree"]()
    want = c.call(c.out()).clone()
    mla.mla_debug_decode_fault(6, 2000)
    try:
        got = c.call(c.out())
        mla.mla_get_device_status()
    finally:
        mla.mla_debug_decode_fault(-1, 0)
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))
