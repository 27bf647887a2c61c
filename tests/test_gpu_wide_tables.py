"""Page tables whose rows hold 2^31 tokens and more: the product of pages and page size passes 31 bits, the lengths do
not.  Results have to be those of the same call with a narrow table, bit for bit."""
import numpy as np
import pytest
import torch

import mla_latent_kv_24_b200 as mla
import workloads as wl
from _gpu import Dev
from _views import TreeCase, WindowCase, base_workload

pytestmark = pytest.mark.gpu
WIDE = [1 << 25, (1 << 26) + 1]          # times 64 or more tokens: wraps below zero, and to one page


def widen(table, pages):
    t = torch.zeros(1, pages, dtype=torch.int32, device="cuda")
    t[:, :table.shape[1]] = table.clamp_min(0)
    return t


@pytest.mark.parametrize("pages", WIDE)
@pytest.mark.parametrize("op", ["tree", "window", "grouped window"])
@pytest.mark.parametrize("model", ["gqla", "tiny"])
def test_views(model, op, pages):
    w = base_workload(model)
    if op == "tree":
        c = TreeCase(w, 7, (200,), (7,), seed=81).upload()
    else:
        c = WindowCase(w, 3, (200,), 2, 80, seed=82).upload(op == "grouped window")
    extra = (c.expand(),) if op == "grouped window" else ()
    want = c.call(c.out(), *extra).clone()
    mla.mla_get_device_status()
    c.d["page_table"], c.max_pages = widen(c.d["page_table"], pages * 64 // w.page), pages * 64 // w.page
    got = c.call(c.out(7.0), *extra)
    mla.mla_get_device_status()
    assert torch.equal(got, want)


@pytest.mark.parametrize("pages", WIDE)
@pytest.mark.parametrize("model", ["gqla", "tiny"])
def test_causal_decodes_and_appends(model, pages):
    w = wl.small_workload(base_workload(model), B=1, s_q=2, lens=[200], seed=83)
    v = Dev(wl.make_inputs(w))
    exp = v.expand()
    want = v.decode_absorbed().clone(), v.decode_grouped(exp).clone()
    narrow, width = v.page_table, v.max_pages
    wide = widen(narrow, pages * 64 // w.page)
    v.page_table, v.max_pages = wide, wide.shape[1]
    got = v.decode_absorbed(), v.decode_grouped(exp)
    mla.mla_get_device_status()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    d, hidden = v.dims, 256
    h = torch.randn(2, hidden, device="cuda").to(v.tdtype)
    W1, W2 = torch.randn(d.d_c, hidden, device="cuda").to(v.tdtype), torch.randn(d.d_rope, hidden, device="cuda").to(v.tdtype)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    req, slots, pos = i32(0, 0), i32(70, 199), i32(71, 500)
    caches = []
    for table, n in ((narrow, width), (wide, wide.shape[1])):
        cache, e = v.cache.clone(), exp.clone()
        mla.mla_cache_append_slots(d, h, hidden, W1, W2, req, slots, pos, 2, table, 1, n, v.inp.n_pages, cache)
        mla.gqla_expand_tokens(d, v.W_uk, v.W_uv, cache, req, slots, 2, table, 1, n, v.inp.n_pages, e)
        mla.mla_get_device_status()
        caches.append((cache, e))
    assert torch.equal(caches[0][0], caches[1][0]) and torch.equal(caches[0][1], caches[1][1])
    assert not torch.equal(caches[0][0], v.cache) and np.isfinite(caches[0][1].float().cpu().numpy()).all()
