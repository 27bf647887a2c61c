"""The operators together, as a serving loop calls them: draft, verify, accept over several steps on both
caches; a window that frees its pages; branches of one request.  After every accepted path the cache has to
be the one that appending the accepted tokens one by one would have left."""
import numpy as np
import pytest
import torch

import mla_latent_kv_24_b200 as mla
import oracle
import workloads as wl
from _gpu import assert_close, dims_of
from _views import random_tree, tree_visible

pytestmark = pytest.mark.gpu


class Engine:
    """A batch of requests with a page pool on the device; the host keeps lengths and hidden states."""

    def __init__(self, dtype, batch, n_pages, hidden, seed, max_pages=24):
        base = wl.WORKLOADS["5_8192_1"] if dtype == "bf16" else \
            wl.small_workload(wl.WORKLOADS["1"], H=8, hpw=2, d_c=32, page=64)
        self.w = w = wl.small_workload(base, B=1, s_q=1, lens=[1], hidden=hidden, seed=seed)
        inp = wl.make_inputs(w)
        self.inp, self.dims, self.rng = inp, dims_of(w), np.random.default_rng(seed)
        self.W_uk, self.W_uv, self.W_dkv, self.W_kr = (wl.to_torch(t) for t in (inp.W_uk, inp.W_uv, inp.W_dkv, inp.W_kr))
        self.dt = torch.bfloat16 if w.dtype == "bf16" else torch.float32
        self.batch, self.n_pages, self.max_pages, self.G = batch, n_pages, max_pages, w.H // w.hpw
        self.table = torch.full((batch, max_pages), -1, dtype=torch.int32, device="cuda")
        self.lens_d = torch.zeros(batch, dtype=torch.int32, device="cuda")
        self.refs = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
        self.cache = torch.full((1, n_pages, w.page, w.d_row), float("nan"), dtype=self.dt, device="cuda")
        self.exp = torch.full((1, n_pages, self.G, w.page, w.d_n + w.d_v), float("nan"), dtype=self.dt, device="cuda")
        self.lens = np.zeros(batch, np.int64)
        self.tokens = [[] for _ in range(batch)]                     # hidden states of the tokens kept, per request

    def i32(self, a):
        return torch.tensor(np.asarray(a).astype(np.int32), device="cuda")

    def tail(self):
        return self.lens_d, self.table, self.batch, self.max_pages, self.refs, self.n_pages

    def hidden(self, n):
        x = self.rng.standard_normal((n, self.w.hidden), dtype=np.float32)
        t = wl.Tensor(wl.f32_to_bf16_bits(x) if self.w.dtype == "bf16" else x, self.w.dtype)
        return t.f64(), wl.to_torch(t)

    def queries(self, T):
        x = self.rng.standard_normal((self.batch, T, self.w.H, self.w.d_n + self.w.d_r), dtype=np.float32)
        t = wl.Tensor(wl.f32_to_bf16_bits(x) if self.w.dtype == "bf16" else x, self.w.dtype)
        return t.f64(), wl.to_torch(t)

    def append(self, req, slots, positions, h):
        a = [self.i32(x) for x in (req, slots, positions)]
        mla.mla_cache_append_slots(self.dims, h, self.w.hidden, self.W_dkv, self.W_kr, *a, len(req), self.table,
                                   self.batch, self.max_pages, self.n_pages, self.cache[0])
        mla.gqla_expand_tokens(self.dims, self.W_uk, self.W_uv, self.cache[0], a[0], a[1], len(req), self.table,
                               self.batch, self.max_pages, self.n_pages, self.exp[0])

    def grow(self, counts):
        """Appends counts[b] new tokens to every request."""
        new = self.lens + np.asarray(counts)
        mla.mla_cache_reserve(self.dims, self.i32(new), *self.tail())
        req = np.repeat(np.arange(self.batch), counts)
        slots = np.concatenate([np.arange(a, b) for a, b in zip(self.lens, new)]) if len(req) else np.zeros(0)
        h64, h = self.hidden(len(req))
        self.append(req, slots, slots, h)
        for i, b in enumerate(req):
            self.tokens[b].append(h64[i])
        self.lens = new

    def rows(self, b):
        """Cache rows of the tokens kept, in 64 bits from the hidden states."""
        h = np.stack(self.tokens[b])
        return oracle.down_project(h, self.inp.W_dkv.f64(), self.inp.W_kr.f64(), np.arange(len(h)), self.w.rope_base,
                                   self.w.d_c)

    def on_device(self, cache, b):
        t = np.arange(self.lens[b])
        table = self.table.cpu().numpy()
        return cache[0][torch.from_numpy(table[b, t // 64].astype(np.int64)).cuda(), ...], t % 64

    def check_cache(self):
        """The device's rows are the tokens' rows: rounded once (half a step of the type, plus the float32
        accumulation), and the expanded rows are what expanding the latent pages gives, bit for bit."""
        u = 2 ** -8 if self.w.dtype == "bf16" else 2 ** -24
        table = self.table.cpu().numpy()
        full = torch.empty_like(self.exp[0])
        clean = torch.nan_to_num(self.cache[0])
        mla.gqla_expand_cache(self.dims, self.W_uk, self.W_uv, clean, None, 0, self.n_pages, full)
        for b in range(self.batch):
            if not self.lens[b]:
                continue
            t = np.arange(self.lens[b])
            pg, r = table[b, t // 64], t % 64
            held = pg >= 0
            pg, r = torch.from_numpy(pg[held].astype(np.int64)).cuda(), torch.from_numpy(r[held]).cuda()
            got, ref = wl.from_torch_f64(self.cache[0][pg, r]), self.rows(b)[held]
            # |sum| error in float32 over `hidden` products of |h| |W|: below hidden 2^-24 sum |h_i W_i|; a
            # rotation mixes two columns and adds two more roundings
            h = np.abs(np.stack(self.tokens[b])[held])
            mass = np.concatenate([h @ np.abs(self.inp.W_dkv.f64()).T, h @ np.abs(self.inp.W_kr.f64()).T], 1)
            mass[:, self.w.d_c:] = np.repeat(mass[:, self.w.d_c::2] + mass[:, self.w.d_c + 1::2], 2, axis=1)
            tol = u * np.abs(ref) + (self.w.hidden + 8) * 2 ** -24 * mass
            assert (np.abs(got - ref) <= tol).all(), (b, np.abs(got - ref).max())
            assert torch.equal(self.exp[0][pg, :, r], full[pg, :, r])

    def cached(self, b, n):
        """The first n rows that request b's page table holds on the device, in 64 bits (what an attention
        over the cache has to be held against); zeros for dropped pages."""
        table = self.table.cpu().numpy()
        t = np.arange(n)
        pg = table[b, t // 64]
        x = wl.from_torch_f64(self.cache[0][torch.from_numpy(np.maximum(pg, 0).astype(np.int64)).cuda(),
                                            torch.from_numpy(t % 64).cuda()])
        x[pg < 0] = 0
        return x

    def attend(self, b, q64, n_rows, positions, visible):
        return oracle.decode_request_masked(q64, self.cached(b, n_rows), self.inp.W_uk.f64(), self.inp.W_uv.f64(),
                                            self.w.hpw, self.w.softmax_scale, self.w.rope_base, positions, visible)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_draft_verify_accept(dtype):
    T, batch = 12, 3
    e = Engine(dtype, batch, n_pages=24, hidden=256 if dtype == "bf16" else 64, seed=500)
    e.grow([60, 130, 1])
    mla.mla_get_device_status()
    for step in range(4):
        nodes = np.asarray([T, T - step, 0 if step == 2 else 5])
        ctx = e.lens.copy()
        depths, masks = np.zeros((batch, T), np.int32), np.zeros((batch, T), np.uint64)
        for b in range(batch):
            depths[b, :nodes[b]], masks[b, :nodes[b]] = random_tree(e.rng, int(nodes[b]))
        total = ctx + nodes
        mla.mla_cache_reserve(e.dims, e.i32(total), *e.tail())
        req = np.repeat(np.arange(batch), nodes)
        slots = np.concatenate([np.arange(a, b) for a, b in zip(ctx, total)])
        pos = np.concatenate([ctx[b] + depths[b, :nodes[b]] for b in range(batch)])
        h64, h = e.hidden(len(req))
        e.append(req, slots, pos, h)
        q64, q = e.queries(T)
        lens32, nodes32 = total.astype(np.int32), nodes.astype(np.int32)
        ws = torch.empty(mla.mla_decode_tree_workspace_size(e.dims, batch, T, lens32, nodes32), dtype=torch.uint8,
                         device="cuda")
        out = torch.zeros((batch, T, e.w.H, e.w.d_v), dtype=e.dt, device="cuda")
        mla.mla_decode_tree(e.dims, q, e.W_uk, e.W_uv, e.cache[0], e.table, e.lens_d, e.i32(nodes), lens32, nodes32,
                            e.i32(depths), torch.from_numpy(masks.view(np.int64)).cuda(), batch, T, e.max_pages,
                            e.n_pages, out, ws)
        mla.mla_get_device_status()
        got = wl.from_torch_f64(out)
        for b in range(batch):
            n = int(nodes[b])
            if n:
                ref = e.attend(b, q64[b, :n], int(total[b]), ctx[b] + depths[b, :n],
                               tree_visible(int(total[b]), n, masks[b]))
                assert_close(got[b, :n], ref, dtype, f"step {step} request {b}")
        # the deepest node's path is accepted (request 1 accepts nothing in one step)
        acc, n_acc = np.zeros((batch, T), np.int32), np.zeros(batch, np.int32)
        first = np.concatenate([[0], np.cumsum(nodes)])
        for b in range(batch):
            n = int(nodes[b])
            if n == 0 or (b == 1 and step == 1):
                continue
            j = int(np.argmax(depths[b, :n]))
            path = [i for i in range(n) if (int(masks[b, j]) >> i) & 1]
            assert [int(depths[b, i]) for i in path] == list(range(len(path)))
            acc[b, :len(path)], n_acc[b] = path, len(path)
            for i in path:
                e.tokens[b].append(h64[first[b] + i])
        mla.mla_cache_accept(e.dims, e.i32(ctx), e.i32(nodes), e.i32(acc), e.i32(n_acc), T, *e.tail(), e.cache, e.exp, 1)
        mla.mla_get_device_status()
        e.lens = ctx + n_acc
        assert np.array_equal(e.lens_d.cpu().numpy(), e.lens)
        assert int(e.refs.sum()) == sum(-(-int(L) // 64) for L in e.lens)
        e.check_cache()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_branches_grow_apart(dtype):
    # one prompt, three branches; one is dropped and another forked into its place, each growing by itself
    e = Engine(dtype, 4, n_pages=14, hidden=256 if dtype == "bf16" else 64, seed=501)
    e.grow([150, 0, 0, 0])
    mla.mla_cache_fork(e.dims, e.i32([0, 0]), e.i32([1, 3]), 2, *e.tail(), e.cache, e.exp, 1)
    for b in (1, 3):
        e.tokens[b], e.lens[b] = list(e.tokens[0]), 150
    e.grow([1, 5, 0, 60])
    e.check_cache()
    mla.mla_cache_release(e.dims, e.i32([1]), None, None, 1, *e.tail())
    mla.mla_cache_fork(e.dims, e.i32([3]), e.i32([1]), 1, *e.tail(), e.cache, e.exp, 1)
    e.tokens[1], e.lens[1] = list(e.tokens[3]), e.lens[3]
    e.grow([0, 2, 3, 1])
    mla.mla_get_device_status()
    e.check_cache()
    refs = e.refs.cpu().numpy()
    assert refs.max() == 3 and (refs > 0).sum() == len(set(e.table.cpu().numpy()[e.table.cpu().numpy() >= 0]))
    # pages: two shared by all, one more shared by 1 and 3, and everybody's own
    mla.mla_cache_release(e.dims, e.i32([0, 1, 2, 3]), None, None, 4, *e.tail())
    mla.mla_get_device_status()
    assert int(e.refs.abs().sum()) == 0 and int(e.lens_d.sum()) == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_a_window_lives_on_its_own_pages(dtype):
    # 16 pages serve two requests of up to 700 tokens: the pages behind the window go back to the pool
    S, W, batch = 4, 130, 2
    e = Engine(dtype, batch, n_pages=16, hidden=256 if dtype == "bf16" else 64, seed=502)
    e.grow([100, 3])
    for step in range(12):
        s_q = 1 + step % 2
        e.grow([50, 25])
        # behind the first query's window, the sinks' page stays
        last = np.maximum(1, (e.lens - s_q - W + 1) // 64)
        mla.mla_cache_release(e.dims, e.i32([0, 1]), e.i32([1, 1]), e.i32(last), 2, *e.tail())
        lens32 = e.lens.astype(np.int32)
        q64, q = e.queries(s_q)
        for grouped in (False, True):
            out = torch.zeros((batch, s_q, e.w.H, e.w.d_v), dtype=e.dt, device="cuda")
            if grouped:
                nb = mla.gqla_decode_window_workspace_size(e.dims, batch, s_q, S, W, lens32)
                ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
                mla.gqla_decode_window(e.dims, q, e.exp[0], e.cache[0], e.table, e.lens_d, lens32, batch, s_q, S, W,
                                       e.max_pages, e.n_pages, out, ws)
            else:
                nb = mla.mla_decode_window_workspace_size(e.dims, batch, s_q, S, W, lens32)
                ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
                mla.mla_decode_window(e.dims, q, e.W_uk, e.W_uv, e.cache[0], e.table, e.lens_d, lens32, batch, s_q, S, W,
                                      e.max_pages, e.n_pages, out, ws)
            mla.mla_get_device_status()
            got = wl.from_torch_f64(out)
            for b in range(batch):
                L = int(e.lens[b])
                p = L - s_q + np.arange(s_q)
                t = np.arange(L)[None]
                vis = (t <= p[:, None]) & ((t < S) | (t > p[:, None] - W))
                assert_close(got[b], e.attend(b, q64[b], L, p, vis), dtype, f"window step {step} grouped={grouped}")
    e.check_cache()
    assert e.lens.max() == 700
