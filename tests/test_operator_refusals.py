"""What the tree, window and page calls refuse before anything is enqueued, on CPU: through the C ABI with
addresses that are never followed, and the binding's own checks."""
import ctypes

import numpy as np
import pytest
import torch

import mla_latent_kv_24_b200 as mla

OK, INVALID, UNSUPPORTED = 0, 1, 2
P = 256                                    # an aligned address; refused calls never follow it


def i32(x):
    a = np.ascontiguousarray(np.asarray(x, np.int32))
    return a, a.ctypes.data_as(ctypes.c_void_p)


def tree(dims=None, batch=1, T=8, lens=(64,), nodes=(8,), max_pages=1, q=P, mask=P, depths=P, n_nodes=P, uk=P, hosts=True):
    (a, lp), (b, np_) = i32(lens), i32(nodes)
    d = dims or mla.make_dims()
    return mla.load().mla_decode_tree(ctypes.byref(d), q, uk, P, P, P, P, n_nodes, lp if hosts else None, np_, depths, mask,
                                      batch, T, max_pages, 1, P, P, 1 << 40, None)


def test_tree_arguments():
    assert tree(T=0) == INVALID and tree(T=65) == INVALID                 # 1..64 nodes
    assert tree(nodes=(9,)) == INVALID and tree(nodes=(-1,)) == INVALID   # outside the slots
    assert tree(lens=(7,)) == INVALID                                     # fewer tokens than nodes
    assert tree(lens=(65,)) == INVALID                                    # longer than the page table
    assert tree(batch=0) == INVALID and tree(max_pages=0) == INVALID
    assert tree(q=None) == INVALID and tree(uk=None) == INVALID and tree(hosts=False) == INVALID
    assert tree(mask=None) == INVALID and tree(depths=None) == INVALID and tree(n_nodes=None) == INVALID
    assert tree(mask=P + 4) == INVALID                                    # not 8-byte aligned
    assert "aligned" in mla.mla_last_error_string()
    assert tree(q=P + 8) == INVALID
    assert tree(dims=mla.make_dims(d_c=1024)) == UNSUPPORTED
    big = 1 << 15
    assert tree(batch=big, T=64, lens=[64] * big, nodes=[8] * big) == UNSUPPORTED      # batch * max_nodes
    with pytest.raises(mla.MlaError) as e:
        mla.mla_decode_tree_workspace_size(mla.make_dims(), 1, 70, [64], [8])
    assert e.value.status == INVALID
    with pytest.raises(ValueError):                                       # host copies shorter than the batch
        mla.mla_decode_tree_workspace_size(mla.make_dims(), 2, 8, [64], [8, 8])


def window(f="mla", sinks=4, win=64, s_q=1, lens=(64,), max_pages=1, batch=1, q=P):
    a, lp = i32(lens)
    d = mla.make_dims(heads_per_group=8)
    lib = mla.load()
    if f == "mla":
        return lib.mla_decode_window(ctypes.byref(d), q, P, P, P, P, P, lp, batch, s_q, sinks, win, max_pages, 1, P, P,
                                     1 << 40, None)
    return lib.gqla_decode_window(ctypes.byref(d), q, P, P, P, P, lp, batch, s_q, sinks, win, max_pages, 1, P, P, 1 << 40, None)


@pytest.mark.parametrize("f", ["mla", "gqla"])
def test_window_arguments(f):
    assert window(f, sinks=-1) == INVALID and window(f, win=0) == INVALID and window(f, win=-5) == INVALID
    assert window(f, s_q=0) == INVALID and window(f, s_q=5) == INVALID
    assert window(f, s_q=2, lens=(1,)) == INVALID and window(f, lens=(65,)) == INVALID
    assert window(f, q=None) == INVALID and window(f, batch=0) == INVALID
    size = mla.mla_decode_window_workspace_size if f == "mla" else mla.gqla_decode_window_workspace_size
    for sinks, win in ((-1, 64), (0, 0)):
        with pytest.raises(mla.MlaError) as e:
            size(mla.make_dims(heads_per_group=8), 1, 1, sinks, win, [64])
        assert e.value.status == INVALID


def test_append_slots_arguments():
    lib, d = mla.load(), mla.make_dims()
    call = lambda slots, n=4: lib.mla_cache_append_slots(ctypes.byref(d), P, 5120, P, P, P, slots, P, n, P, 1, 1, 1, P, None)  # noqa: E731
    assert call(None) == INVALID and call(P, -1) == INVALID
    assert call(None, 0) == OK                                            # nothing to append


def test_pool_arguments():
    lib = mla.load()
    d = ctypes.byref(mla.make_dims())

    def reserve(new=P, lens=P, table=P, batch=1, max_pages=1, refs=P, n=1):
        return lib.mla_cache_reserve(d, new, lens, table, batch, max_pages, refs, n, None)
    assert reserve(new=None) == INVALID and reserve(lens=None) == INVALID and reserve(refs=None) == INVALID
    assert reserve(batch=0) == INVALID and reserve(max_pages=0) == INVALID and reserve(n=0) == INVALID
    assert reserve(refs=P + 4) == INVALID
    assert reserve(batch=8193) == UNSUPPORTED and reserve(n=(1 << 30) + 1) == UNSUPPORTED
    assert reserve(max_pages=1 << 26) == UNSUPPORTED                      # tokens pass 31 bits

    def fork(src=P, dst=P, n_fork=1, lat=P, exp=None, layers=1):
        return lib.mla_cache_fork(d, src, dst, n_fork, P, P, 1, 1, P, 1, lat, exp, layers, None)
    assert fork(src=None) == INVALID and fork(dst=None) == INVALID and fork(n_fork=-1) == INVALID
    assert fork(n_fork=0) == OK and fork(src=None, dst=None, n_fork=0) == OK
    assert fork(layers=0) == INVALID and fork(lat=P + 8) == INVALID and fork(exp=P + 8) == INVALID
    assert fork(n_fork=8193) == UNSUPPORTED and fork(layers=65536) == UNSUPPORTED

    def release(req=P, first=None, last=None, n=1):
        return lib.mla_cache_release(d, req, first, last, n, P, P, 1, 1, P, 1, None)
    assert release(req=None) == INVALID and release(n=-1) == INVALID
    assert release(first=P) == INVALID and release(last=P) == INVALID     # a range has both ends
    assert release(n=0) == OK

    def accept(ctx=P, nodes=P, acc=P, n_acc=P, T=8, batch=1, layers=1):
        return lib.mla_cache_accept(d, ctx, nodes, acc, n_acc, T, P, P, batch, 1, P, 1, P, None, layers, None)
    assert accept(ctx=None) == INVALID and accept(nodes=None) == INVALID and accept(acc=None) == INVALID
    assert accept(n_acc=None) == INVALID and accept(T=0) == INVALID and accept(T=65) == INVALID
    assert accept(layers=0) == INVALID and accept(batch=8193) == UNSUPPORTED


def test_binding_refuses_host_tensors():
    x = torch.zeros(64, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        mla.mla_cache_reserve(mla.make_dims(), x, x, x, 1, 1, x, 1)


@pytest.mark.gpu
def test_binding_refuses_short_or_narrow_tensors():
    i = lambda n, dt=torch.int32: torch.zeros(n, dtype=dt, device="cuda")  # noqa: E731
    d = mla.make_dims(n_heads=4, d_c=32, d_rope=8, d_nope=16, d_v=16, dtype="fp32")
    with pytest.raises(ValueError, match="page_refs"):
        mla.mla_cache_reserve(d, i(2), i(2), i(8), 2, 4, i(3), 4)
    with pytest.raises(ValueError, match="seq_lens"):
        mla.mla_cache_reserve(d, i(2), i(2, torch.int64), i(8), 2, 4, i(4), 4)
    with pytest.raises(ValueError, match="latent_cache"):
        mla.mla_cache_fork(d, i(1), i(1), 1, i(2), i(8), 2, 4, i(4), 4, torch.zeros(10, device="cuda"), None, 1)
    with pytest.raises(ValueError, match="contiguous"):
        mla.mla_cache_reserve(d, i(4)[::2], i(2), i(8), 2, 4, i(4), 4)
    q, cache = torch.zeros(4, 4, 24, device="cuda"), torch.zeros(64, 40, device="cuda")
    W, out, ws = torch.zeros(4, 16, 32, device="cuda"), torch.zeros(4, 4, 16, device="cuda"), torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError, match="tree_mask"):
        mla.mla_decode_tree(d, q, W, W, cache, i(1), i(1), i(1), [8], [4], i(4), i(4), 1, 4, 1, 1, out, ws)
    with pytest.raises(mla.MlaError) as e:                                # more bytes claimed than the workspace has
        mla.mla_decode_tree(d, q, W, W, cache, i(1), i(1), i(1), [8], [4], i(4), i(4, torch.int64), 1, 4, 1, 1, out,
                            ws[:256], workspace_bytes=1 << 30)
    assert e.value.status == 3


def test_pool_sizes_whose_page_counts_pass_31_bits():
    # a sum over all requests' pages would wrap
    d, lib = ctypes.byref(mla.make_dims()), mla.load()
    for batch, max_pages in ((64, 1 << 25), (8192, 1 << 18)):
        assert lib.mla_cache_reserve(d, P, P, P, batch, max_pages, P, 1, None) == UNSUPPORTED
        assert lib.mla_cache_fork(d, P, P, 1, P, P, batch, max_pages, P, 1, P, None, 1, None) == UNSUPPORTED
        assert lib.mla_cache_release(d, P, None, None, 1, P, P, batch, max_pages, P, 1, None) == UNSUPPORTED
        assert lib.mla_cache_accept(d, P, P, P, P, 8, P, P, batch, max_pages, P, 1, P, None, 1, None) == UNSUPPORTED
