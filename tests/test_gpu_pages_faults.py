"""Calls on the page pool that its other tests do not make: what a fork reports, refuses and takes."""
import numpy as np
import pytest

import mla_latent_kv_24_b200 as mla
from test_gpu_pages import Pool, refused

pytestmark = pytest.mark.gpu


def fork(p, src, dst, cached=True):
    mla.mla_cache_fork(p.dims, p.i32(src), p.i32(dst), len(src), *p.tail(), p.d_lat if cached else None, None,
                       p.layers if cached else 1)


@pytest.mark.parametrize("cached", [True, False])
@pytest.mark.parametrize("bad", [8, 1 << 30])
def test_a_partial_page_outside_the_pool_is_reported_without_caches_too(cached, bad):
    p = Pool("dsv2", (100, 0), 8)
    keep = p.table[0, 1]
    p.table[0, 1] = bad
    p.upload()
    fork(p, (0,), (1,), cached)
    refused(5)
    # the fork is carried out but for the rows that it cannot copy
    p.table[1, :2] = p.table[0, 0], p.free()[0]
    p.refs[p.table[0, 0]] += 1
    p.refs[p.table[1, 1]] = 1
    p.lens[1] = 100
    p.check()
    assert p.refs[keep] == 1


def dropped_pool(free_pages):
    """Request 0 has dropped its partly filled last page, request 1 has not; `free_pages` pages are free."""
    p = Pool("dsv2", (100, 70, 0, 0, 0, 0), 3 + max(1, free_pages), layers=2, seed=free_pages)
    p.both("release", (0,), (1,), (2,))
    p.refs[p.free()[free_pages:]] = 1                       # someone else's
    p.upload()
    assert len(p.free()) == free_pages
    return p


def m_fork_dropped(p, src, dst, ids):
    for s, d in zip(src, dst):
        full, rem = divmod(int(p.lens[s]), p.page)
        p.table[d, :full] = p.table[s, :full]
        p.refs[p.table[s, :full]] += 1
        if rem and p.table[s, full] < 0:
            p.table[d, full] = -1
        elif rem:
            p.table[d, full] = pg = ids.pop(0)
            p.refs[pg] = 1
            p.lat[:, pg, :rem] = p.lat[:, p.table[s, full], :rem]
        p.lens[d] = p.lens[s]


def test_a_fork_that_needs_no_page_is_carried_out_in_a_full_pool():
    p = dropped_pool(0)
    fork(p, (0, 0), (2, 4))
    mla.mla_get_device_status()
    m_fork_dropped(p, (0, 0), (2, 4), [])
    p.check()
    fork(p, (0, 1), (3, 5))                                 # the second needs one
    refused(7)
    p.check()


@pytest.mark.parametrize("n_free", [1, 2])
def test_dropped_pages_have_no_turn_where_pages_are_few(n_free):
    p = dropped_pool(n_free)
    free = p.free()
    fork(p, (0, 1, 0), (2, 3, 4))
    mla.mla_get_device_status()
    m_fork_dropped(p, (0, 1, 0), (2, 3, 4), free[:1])
    p.check()


def test_dropped_pages_pass_their_turn_over():
    p = dropped_pool(5)
    free = p.free()
    src, dst = (0, 1, 0, 1), (2, 3, 4, 5)
    fork(p, src, dst)
    mla.mla_get_device_status()
    m_fork_dropped(p, src, dst, [free[1], free[3]])
    p.check()


def test_many_forks_of_sources_with_and_without_their_last_page():
    # more forks than the planning block has threads, and pages in several tiles of its scan
    n = 1500
    p = Pool("fp32", (20, 5) + (0,) * n, 3000, seed=8)
    p.both("release", (0,), (1,), (2,))
    src = [i % 3 % 2 for i in range(n)]
    dst = list(range(2, 2 + n))
    for few in (False, True):
        if few:
            p.both("release", tuple(dst))
            free = p.free()
            p.refs[free[sum(src) + 10:]] = 1
            p.upload()
        free = p.free()
        fork(p, src, dst)
        mla.mla_get_device_status()
        m_fork_dropped(p, src, dst, free[:] if few else [free[i] for i in range(n) if src[i]])
        p.check()


@pytest.mark.parametrize("src,dst,length", [
    ((0,), (2,), -101),                 # the mark that a carried-out fork of request 0 (100 tokens) would leave
    ((0, 1, 0), (2, 3, 4), -101),
    ((1, 0), (3, 2), -101),
    ((1,), (2,), -65),
    ((4,), (2,), -1),                   # of an empty source
    ((0,), (2,), -1),
    ((0, 4), (3, 2), -1),
    ((0,), (2,), -2 ** 31),
])
def test_a_refused_fork_leaves_any_length(src, dst, length):
    p = Pool("dsv2", (100, 64, 0, 0, 0), 12, layers=2, seed=3)
    p.lens[2] = length
    p.upload()
    for cached in (True, False):
        fork(p, src, dst, cached)
        refused(5)
        p.check()


def test_a_captured_fork_refused_in_one_replay_and_not_in_the_next():
    import torch
    p = Pool("dsv2", (100, 64, 0, 0), 12, layers=2, seed=4)
    src, dst, tail = p.i32((0,)), p.i32((2,)), p.tail()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mla.mla_cache_fork(p.dims, src, dst, 1, *tail, p.d_lat, None, p.layers)
    for rounds in range(3):
        for length in (-101, 64, -1):
            p.lens[2] = length
            p.d_lens.copy_(torch.from_numpy(p.lens))
            g.replay()
            refused(5)
            p.check()
        p.lens[2] = 0
        p.d_lens.copy_(torch.from_numpy(p.lens))
        for _ in range(2):
            g.replay()
            mla.mla_get_device_status()
            p.m_fork((0,), (2,))
            p.check()
            p.both("release", (2,))
    del g


def test_forks_of_two_pools_on_two_streams():
    # one pool's forks are carried out while the other's are refused, in no order between them
    import torch
    a, b = Pool("dsv2", (100, 0), 8, layers=2, seed=5), Pool("dsv2", (100, 64, 0), 8, layers=2, seed=6)
    b.lens[2] = -101
    b.upload()
    torch.cuda.synchronize()
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    src, dst_a, dst_b = a.i32((0,)), a.i32((1,)), a.i32((2,))
    torch.cuda.synchronize()
    for _ in range(200):
        with torch.cuda.stream(one):
            mla.mla_cache_fork(a.dims, src, dst_a, 1, *a.tail(), a.d_lat, None, a.layers)
            mla.mla_cache_release(a.dims, dst_a, None, None, 1, *a.tail())
        with torch.cuda.stream(two):
            mla.mla_cache_fork(b.dims, src, dst_b, 1, *b.tail(), b.d_lat, None, b.layers)
    with torch.cuda.stream(one):
        mla.mla_cache_fork(a.dims, src, dst_a, 1, *a.tail(), a.d_lat, None, a.layers)
    torch.cuda.synchronize()
    refused(5)
    b.check()
    # what a released page holds is the last fork's rows: the model makes one fork
    a.m_fork((0,), (1,))
    a.check()
