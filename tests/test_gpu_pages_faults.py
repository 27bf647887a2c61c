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
