"""GPU checks of the page pool: reserving, forking, releasing pages, and moving accepted rows together.
Everything is whole numbers and copied bytes, so each call is held exactly against a plain Python model
of the pool."""
import numpy as np
import pytest
import torch

import mla_latent_kv_24_b200 as mla

pytestmark = pytest.mark.gpu

SHAPES = {
    "dsv2": dict(n_heads=128, heads_per_group=8),
    "fp32": dict(n_heads=4, d_c=32, d_rope=8, d_nope=16, d_v=16, dtype="fp32", page_size=16),
    # rows of the expanded cache of 29 values: 58 bytes in bf16, 116 in fp32
    "odd bf16": dict(n_heads=4, heads_per_group=2, d_c=32, d_rope=8, d_nope=16, d_v=13, page_size=32),
    "odd fp32": dict(n_heads=4, heads_per_group=2, d_c=32, d_rope=8, d_nope=16, d_v=13, page_size=128, dtype="fp32"),
}


class Pool:
    """The pool on the device and a plain model of it."""

    def __init__(self, shape, lens, n_pages, layers=1, slack=3, seed=0, expanded=False):
        self.kw = SHAPES[shape]
        self.dims = d = mla.make_dims(**self.kw)
        self.page, self.layers, self.n_pages, self.batch = d.page_size, layers, n_pages, len(lens)
        rng = np.random.default_rng(seed)
        need = [-(-L // self.page) for L in lens]
        self.max_pages = max(need) + slack
        ids = rng.permutation(n_pages)[:sum(need)]
        self.lens, self.refs = np.asarray(lens, np.int32), np.zeros(n_pages, np.int32)
        self.table = np.full((self.batch, self.max_pages), -1, np.int32)
        at = 0
        for b, k in enumerate(need):
            self.table[b, :k] = ids[at:at + k]
            self.refs[ids[at:at + k]] = 1
            at += k
        dt = torch.float32 if d.dtype else torch.bfloat16
        g = torch.Generator().manual_seed(seed)
        shape_l = (layers, n_pages, self.page, d.d_c + d.d_rope)
        G = d.n_heads // d.heads_per_group
        shape_e = (layers, n_pages, G, self.page, d.d_nope + d.d_v)
        self.lat = torch.randn(shape_l, generator=g).to(dt)
        self.exp = torch.randn(shape_e, generator=g).to(dt) if expanded else None
        self.upload()

    def upload(self):
        c = lambda a: torch.from_numpy(a.copy()).cuda()  # noqa: E731
        self.d_lens, self.d_table, self.d_refs = c(self.lens), c(self.table), c(self.refs)
        self.d_lat = self.lat.cuda()
        self.d_exp = None if self.exp is None else self.exp.cuda()

    def check(self):
        assert np.array_equal(self.d_lens.cpu().numpy(), self.lens)
        assert np.array_equal(self.d_table.cpu().numpy(), self.table)
        assert np.array_equal(self.d_refs.cpu().numpy(), self.refs)
        assert torch.equal(self.d_lat.cpu(), self.lat)
        if self.exp is not None:
            assert torch.equal(self.d_exp.cpu(), self.exp)

    def pages(self, L):
        return -(-int(L) // self.page)

    def i32(self, x):
        return torch.tensor(list(x), dtype=torch.int32, device="cuda")

    def tail(self):
        return self.d_lens, self.d_table, self.batch, self.max_pages, self.d_refs, self.n_pages

    def free(self):
        return list(np.flatnonzero(self.refs == 0))

    # device calls
    def reserve(self, new):
        mla.mla_cache_reserve(self.dims, self.i32(new), *self.tail())

    def fork(self, src, dst):
        mla.mla_cache_fork(self.dims, self.i32(src), self.i32(dst), len(src), *self.tail(), self.d_lat, self.d_exp,
                           self.layers)

    def release(self, req, first=None, last=None):
        mla.mla_cache_release(self.dims, self.i32(req), None if first is None else self.i32(first),
                              None if last is None else self.i32(last), len(req), *self.tail())

    def accept(self, ctx, nodes, accepted, max_nodes, refs=True):
        acc = np.zeros((self.batch, max_nodes), np.int32)
        for b, a in enumerate(accepted):
            acc[b, :len(a)] = a
        mla.mla_cache_accept(self.dims, self.i32(ctx), self.i32(nodes), torch.from_numpy(acc).cuda(),
                             self.i32(len(a) for a in accepted), max_nodes, self.d_lens, self.d_table, self.batch,
                             self.max_pages, self.d_refs if refs else None, self.n_pages, self.d_lat, self.d_exp,
                             self.layers)

    # the model
    def m_reserve(self, new):
        free = self.free()
        for b, n in enumerate(new):
            for k in range(self.pages(self.lens[b]), self.pages(n)):
                self.table[b, k] = pg = free.pop(0)
                self.refs[pg] = 1
            self.lens[b] = n

    def m_fork(self, src, dst):
        free, before = self.free(), self.lens.copy()
        for s, d in zip(src, dst):
            L = int(before[s])                        # a source is what it was before the call
            full, rem = divmod(L, self.page)
            for k in range(full):
                self.table[d, k] = self.table[s, k]
                if self.table[s, k] >= 0:
                    self.refs[self.table[s, k]] += 1
            if rem:
                self.table[d, full] = pg = free.pop(0)
                self.refs[pg] = 1
                a = int(self.table[s, full])
                self.lat[:, pg, :rem] = self.lat[:, a, :rem]
                if self.exp is not None:
                    self.exp[:, pg, :, :rem] = self.exp[:, a, :, :rem]
            self.lens[d] = L

    def m_drop(self, b, k0, k1):
        for k in range(k0, k1):
            if self.table[b, k] >= 0:
                self.refs[self.table[b, k]] -= 1
                self.table[b, k] = -1

    def m_release(self, req, first=None, last=None):
        for i, b in enumerate(req):
            have = self.pages(self.lens[b])
            self.m_drop(b, 0 if first is None else max(0, first[i]), have if first is None else min(have, last[i]))
        if first is None:
            self.lens[list(req)] = 0

    def m_accept(self, ctx, nodes, accepted, refs=True):
        for b, a in enumerate(accepted):
            old_l, old_e = self.lat.clone(), None if self.exp is None else self.exp.clone()
            for k, i in enumerate(a):
                f, t = ctx[b] + i, ctx[b] + k
                fp, tp = int(self.table[b, f // self.page]), int(self.table[b, t // self.page])
                self.lat[:, tp, t % self.page] = old_l[:, fp, f % self.page]
                if self.exp is not None:
                    self.exp[:, tp, :, t % self.page] = old_e[:, fp, :, f % self.page]
            self.lens[b] = ctx[b] + len(a)
            if refs:
                self.m_drop(b, self.pages(self.lens[b]), self.pages(ctx[b] + nodes[b]))

    def both(self, name, *a, **kw):
        getattr(self, name)(*a, **kw)
        getattr(self, "m_" + name)(*[x for i, x in enumerate(a) if not (name == "accept" and i == 3)], **kw)
        mla.mla_get_device_status()
        self.check()


def refused(status):
    with pytest.raises(mla.MlaError) as e:
        mla.mla_get_device_status()
    assert e.value.status == status


@pytest.mark.parametrize("n_pages", [40, 1023, 16384 + 5, 50000])
def test_reserve_takes_the_lowest_free_pages(n_pages):
    p = Pool("fp32", (0, 1, 15, 16, 17, 130, 0), n_pages, slack=40 if n_pages > 100 else 3, seed=n_pages)
    p.both("reserve", (0, 1, 16, 17, 48, 130, 5))
    p.both("reserve", p.lens + 1)
    if n_pages > 100:
        p.both("reserve", p.lens + 300)


def test_reserve_when_only_the_last_pages_are_free():
    p = Pool("fp32", (16, 0), 16384 * 2 + 37, slack=30)
    p.refs[:] = 1
    p.refs[[7, 16390, -3, -2, -1]] = 0                # the last tile is a ragged one
    p.upload()
    p.both("reserve", (48, 48))
    p.reserve((48, 49))
    refused(7)
    p.check()


@pytest.mark.parametrize("batch", [1, 1024, 1025, 8192])
def test_reserve_for_many_requests(batch):
    rng = np.random.default_rng(batch)
    lens = rng.integers(0, 40, size=batch)
    p = Pool("fp32", tuple(lens), int(sum(-(-lens // 16))) + 3 * batch, slack=4, seed=batch)
    p.both("reserve", p.lens + rng.integers(0, 30, size=batch).astype(np.int32))


def test_a_refused_reserve_changes_nothing():
    p = Pool("dsv2", (100, 64, 0), 5, slack=4)
    p.reserve((300, 64, 1))                           # two pages free, four asked
    refused(7)
    p.check()
    for new in ((99, 64, 1), (100, 64, -1), (100, 64, p.max_pages * 64 + 1), (100, 64, 2 ** 31 - 1)):
        p.reserve(new)
        refused(5)
        p.check()
    p.lens[1] = -7                                    # a length that cannot be
    p.upload()
    p.reserve((100, 64, 1))
    refused(5)
    p.check()


@pytest.mark.parametrize("shape", list(SHAPES))
@pytest.mark.parametrize("layers,expanded", [(1, False), (3, True)])
def test_fork_shares_full_pages_and_copies_the_partial_one(shape, layers, expanded):
    page = mla.make_dims(**SHAPES[shape]).page_size
    lens = (page, 0, 2 * page + 5, 0, 1, 0, 0, 0, 0, 3 * page - 1, 0)
    p = Pool(shape, lens, 30, layers=layers, expanded=expanded, seed=layers)
    p.both("fork", (2, 2, 0, 4, 1), (3, 1, 7, 8, 6))  # request 1 is an empty source, and becomes a copy of 2
    p.both("fork", (3, 9), (10, 5))                   # a copy of a copy
    p.both("reserve", p.lens + 1)                     # every holder of a copied page grows by itself
    p.both("release", (2, 3, 9))
    p.both("fork", (1, 10, 1), (2, 3, 9))


@pytest.mark.parametrize("n", [1, 1023, 1025, 8000])
def test_many_forks_of_one_request(n):
    p = Pool("fp32", (37,) + (0,) * n, n + 10, seed=n)
    p.both("fork", (0,) * n, tuple(range(n, 0, -1)))
    p.both("release", tuple(range(0, n + 1, 2)))


def test_fork_of_a_request_with_dropped_pages():
    p = Pool("dsv2", (500, 0), 20)
    p.both("release", (0,), (1,), (5,))
    p.both("fork", (0,), (1,))
    p.both("release", (1,))
    p.both("release", (0,))
    assert (p.refs == 0).all()


def test_a_refused_fork_changes_nothing():
    p = Pool("dsv2", (100, 64, 30, 0, 0, 0), 8, layers=2)
    for src, dst in [((0, 0), (3, 3)),                # one destination twice
                     ((0, 0), (3, 1)),                # one that is in use
                     ((0, 1), (1, 3)), ((0,), (0,)),
                     ((0, 6), (3, 4)), ((0, -1), (3, 4)), ((0, 0), (3, 6)), ((0, 0), (-1, 3))]:
        p.fork(src, dst)
        refused(5)
        p.check()
    p = Pool("dsv2", (100, 64, 30, 0, 0, 0), 6)       # two pages free
    p.fork((0, 2, 2), (3, 4, 5))
    refused(7)
    p.check()
    p.both("fork", (0, 2, 1), (3, 4, 5))
    p.lens[1] = p.max_pages * 64 + 1
    p.lens[5] = 0
    p.upload()
    p.fork((1,), (5,))
    refused(5)
    p.check()


def test_fork_reports_a_page_outside_the_pool():
    p = Pool("dsv2", (100, 0), 6)
    p.table[0, 1] = 6
    p.upload()
    before = p.lat.clone()
    p.fork((0,), (1,))
    refused(5)
    assert torch.equal(p.d_lat.cpu(), before)


def test_release_of_ranges_and_twice():
    p = Pool("fp32", (160, 33, 16, 0), 20)
    p.both("release", (0, 1, 2, 3), (2, -5, 0, 0), (4, 1, 99, 7))
    p.both("release", (0, 0, 0), (1, 3, 9), (5, 8, 1))                   # ranges that overlap, an empty one
    p.both("release", (0, 1, 0, 1))                                       # the same request twice
    p.both("release", (0, 1, 2, 3))
    assert (p.refs == 0).all()


def test_release_reports_what_cannot_be():
    p = Pool("fp32", (40, 40), 8)
    for req in ((2,), (-1,)):
        p.release(req)
        refused(5)
        p.check()
    held = int(p.table[0, 1])
    p.refs[held] = 0                                                      # nobody holds it: no count below 0
    p.table[0, 2] = 8                                                     # outside the pool
    p.upload()
    p.release((0,))
    refused(5)
    p.refs[p.table[0, 0]] -= 1
    p.table[0, :3] = -1
    p.lens[0] = 0
    p.check()


@pytest.mark.parametrize("shape", list(SHAPES))
@pytest.mark.parametrize("layers,expanded", [(1, False), (2, True)])
def test_accepted_rows_move_together(shape, layers, expanded):
    page = mla.make_dims(**SHAPES[shape]).page_size
    ctx = (page - 2, 0, 3 * page, 17, 5, page - 1, 2 * page)
    nodes = (64, 64, 30, 0, 7, 64, 40)
    acc = (list(range(0, 64, 3)), [63], list(range(30)), [], [], list(range(64)), [0, 1, 2, 9, 10, 39])
    p = Pool(shape, ctx, 60, layers=layers, expanded=expanded, slack=6, seed=5)
    p.both("reserve", np.asarray(ctx) + np.asarray(nodes))
    p.both("accept", ctx, nodes, acc, 64)


def test_accept_without_counts_keeps_the_pages():
    p = Pool("dsv2", (60, 64), 20, slack=3)
    p.both("reserve", (120, 130))
    p.both("accept", (60, 64), (60, 64), ([1, 40, 59], []), 64, refs=False)


def test_accept_leaves_bad_requests_as_they_were():
    good, ctx, nodes = [0, 2, 5], (60, 100, 10), (8, 8, 8)
    bad = [[0, 0], [2, 1], [8], [-1], [0, 1, 9], [-100000, -90000, 3], [2 ** 31 - 1, -2 ** 31]]
    for acc in bad:
        p = Pool("dsv2", ctx, 30, slack=3, seed=9)
        p.both("reserve", np.asarray(ctx) + 8)
        p.accept(ctx, nodes, (good, acc, good), 8)
        refused(5)
        keep = p.lens.copy()
        p.m_accept((60, 0, 10), (8, 0, 8), (good, [], good))
        p.lens[1] = keep[1]
        p.check()
    for c, n in (((60, -1, 10), nodes), ((60, 1 << 30, 10), nodes), (ctx, (8, 9, 8)), (ctx, (8, -1, 8)), (ctx, (8, 2, 8))):
        p = Pool("dsv2", ctx, 30, slack=3, seed=9)
        p.both("reserve", np.asarray(ctx) + 8)
        p.accept(c, n, (good, good, good), 8)
        refused(5)
        keep = p.lens.copy()
        p.m_accept((60, 0, 10), (8, 0, 8), (good, [], good))
        p.lens[1] = keep[1]
        p.check()


def test_pages_outside_the_pool_stop_an_accept():
    p = Pool("dsv2", (60,), 8)
    p.both("reserve", (80,))
    p.table[0, 1] = 8
    p.upload()
    before = p.lat.clone()
    p.accept((60,), (20,), ([0, 10],), 20)
    refused(5)
    assert torch.equal(p.d_lat.cpu(), before) and int(p.d_lens[0]) == 80


def test_a_captured_round_replays():
    # reserve, accept, release, fork in one graph: each replay starts from the lengths the last one left
    p = Pool("dsv2", (100, 60, 0), 30, slack=4, layers=2)
    ctx, nodes, acc = (100, 60, 0), (20, 20, 0), ([3, 7], [0, 1, 19], [])
    a = np.zeros((3, 20), np.int32)
    for b, x in enumerate(acc):
        a[b, :len(x)] = x
    args = [p.i32(np.asarray(ctx) + np.asarray(nodes)), p.i32(ctx), p.i32(nodes), torch.from_numpy(a).cuda(),
            p.i32(len(x) for x in acc), p.i32([2]), p.i32([1])]

    def step():
        mla.mla_cache_reserve(p.dims, args[0], *p.tail())
        mla.mla_cache_accept(p.dims, args[1], args[2], args[3], args[4], 20, *p.tail(), p.d_lat, None, 2)
        mla.mla_cache_fork(p.dims, args[6], args[5], 1, *p.tail(), p.d_lat, None, 2)
        mla.mla_cache_release(p.dims, args[5], None, None, 1, *p.tail())

    def model():
        p.m_reserve(np.asarray(ctx) + np.asarray(nodes))
        p.m_accept(ctx, nodes, acc)
        p.m_fork((1,), (2,))
        p.m_release((2,))
    step()
    model()
    torch.cuda.synchronize()
    p.check()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(3):
        g.replay()
        model()
    torch.cuda.synchronize()
    mla.mla_get_device_status()
    p.check()
    del g


def test_accept_takes_no_nodes_that_a_request_does_not_have():
    # a context too long would drop pages that the request never had; what lies behind the nodes goes with its pages
    for ctx in ((60, 101, 10), (60, 300, 10), (60, 2 ** 31 - 1, 10)):
        p = Pool("dsv2", (60, 100, 10), 30, slack=3, seed=9)
        p.both("reserve", (68, 108, 18))
        p.accept(ctx, (8, 8, 8), ([0, 2, 5],) * 3, 8)
        refused(5)
        p.m_accept((60, 0, 10), (8, 0, 8), ([0, 2, 5], [], [0, 2, 5]))
        p.lens[1] = 108
        p.check()
    p = Pool("dsv2", (60, 100, 10), 30, slack=3, seed=9)
    p.both("reserve", (68, 260, 18))
    p.accept((60, 20, 10), (8, 8, 8), ([0, 2, 5],) * 3, 8)
    mla.mla_get_device_status()
    p.m_accept((60, 20, 10), (8, 8, 8), ([0, 2, 5],) * 3)
    p.m_drop(1, 1, 5)
    p.check()
    p = Pool("dsv2", (60, 100, 10), 30, slack=3, seed=9)
    p.both("reserve", (68, 100, 18))
    p.accept((60, 0, 10), (8, 0, 8), ([0, 2, 5], [], [0, 2, 5]), 8)    # without nodes: takes no part, whatever ctx is
    mla.mla_get_device_status()
    p.m_accept((60, 100, 10), (8, 0, 8), ([0, 2, 5], [], [0, 2, 5]))
    p.check()


def test_a_fork_refused_for_a_length_that_cannot_be_leaves_it():
    p = Pool("dsv2", (100, 64, 0, 0), 8)
    p.lens[2] = -101                                                    # what a carried-out fork of request 0 notes
    p.upload()
    p.fork((1, 1), (2, 3))
    refused(5)
    p.check()


@pytest.mark.parametrize("B", [2, 40])
@pytest.mark.parametrize("op", ["causal", "window", "tree", "grouped", "append"])
def test_a_call_right_behind_one_that_changes_lengths(op, B):
    # reserve -> accept (trims) -> the call, with no host or other kernel between; held against the same calls with
    # the host waiting after each.  The calls' first kernels read lengths before their predecessor has ended.
    ctx, n = 130 + 5 * np.arange(B), 8
    p = Pool("dsv2", (0,) * B, 6 * B + 3, slack=6 + 5 * B // 64, seed=11, expanded=op == "grouped")
    d, T = p.dims, 2
    g = torch.Generator().manual_seed(4)
    rnd = lambda *s: torch.randn(s, generator=g).mul_(0.2).to(torch.bfloat16).cuda()  # noqa: E731
    q, W_uk, W_uv = rnd(B, T, 128, 192), rnd(16, 128, 512), rnd(16, 128, 512)
    lens = (ctx + T).astype(np.int32)
    full, d_ctx, nodes, n_acc = p.i32(ctx + n), p.i32(ctx), p.i32([n] * B), p.i32([T] * B)
    acc = torch.arange(n, dtype=torch.int32, device="cuda").repeat(B, 1)
    every, t_nodes, depths = p.i32(range(B)), p.i32([T] * B), p.i32([0, 1] * B)
    mask = torch.tensor([1, 3] * B, dtype=torch.int64, device="cuda")
    out = torch.empty(B, T, 128, 128, dtype=torch.bfloat16, device="cuda")
    size = {"causal": lambda: mla.mla_decode_workspace_size(d, B, T, lens),
            "window": lambda: mla.mla_decode_window_workspace_size(d, B, T, 4, 100, lens),
            "tree": lambda: mla.mla_decode_tree_workspace_size(d, B, T, lens, [T] * B),
            "grouped": lambda: mla.gqla_decode_window_workspace_size(d, B, T, 4, 100, lens),
            "append": lambda: 256}[op]()
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    h, W = rnd(B, 512), rnd(576, 512)
    where = (p.d_table, p.d_lens, lens, B, T)
    cache = p.d_lat[0]

    def step(wait):
        mla.mla_cache_reserve(d, full, *p.tail())
        wait()
        if op != "append":
            mla.mla_cache_accept(d, d_ctx, nodes, acc, n_acc, n, *p.tail(), p.d_lat, None, 1)
            wait()
        if op == "causal":
            mla.mla_decode_absorbed(d, q, W_uk, W_uv, cache, *where, p.max_pages, p.n_pages, out, ws)
        elif op == "window":
            mla.mla_decode_window(d, q, W_uk, W_uv, cache, *where, 4, 100, p.max_pages, p.n_pages, out, ws)
        elif op == "tree":
            mla.mla_decode_tree(d, q, W_uk, W_uv, cache, p.d_table, p.d_lens, t_nodes, lens, [T] * B, depths, mask, B, T,
                                p.max_pages, p.n_pages, out, ws)
        elif op == "grouped":
            mla.gqla_decode_window(d, q, p.d_exp[0], cache, *where, 4, 100, p.max_pages, p.n_pages, out, ws)
        else:
            mla.mla_cache_append(d, h, 512, W[:512], W[512:], every, d_ctx, B, p.d_table, B, p.max_pages, p.n_pages, cache)
        wait()
        mla.mla_cache_release(d, every, None, None, B, *p.tail())
        wait()

    result = cache if op == "append" else out
    step(torch.cuda.synchronize)
    mla.mla_get_device_status()
    want = result.clone()
    assert op == "append" or want.float().abs().sum() > 0
    for _ in range(20):
        if op != "append":
            out.zero_()
        step(lambda: None)
        step(lambda: None)
        mla.mla_get_device_status()
        assert torch.equal(result, want)
    assert (p.d_refs == 0).all() and (p.d_lens == 0).all()


@pytest.mark.parametrize("cached", [True, False])
def test_fork_of_a_request_whose_last_page_was_dropped(cached):
    p = Pool("dsv2", (100, 70, 0, 0, 0), 10, layers=2)
    p.both("release", (0,), (1,), (2,))
    lat = (p.d_lat, p.layers) if cached else (None, 1)
    mla.mla_cache_fork(p.dims, p.i32((0, 1, 0)), p.i32((2, 3, 4)), 3, *p.tail(), lat[0], None, lat[1])
    mla.mla_get_device_status()
    free = p.free()
    p.refs[p.table[0, 0]] += 2
    p.refs[p.table[1, 0]] += 1
    p.table[2, 0] = p.table[4, 0] = p.table[0, 0]
    p.table[3, :2] = p.table[1, 0], free[1]                 # the second of three pages taken; the others are free again
    p.refs[free[1]] = 1
    p.lens[2:] = 100, 70, 100
    if cached:
        p.lat[:, free[1], :6] = p.lat[:, p.table[1, 1], :6]
    else:
        p.lat = p.d_lat.cpu()
    p.check()


def status():
    try:
        mla.mla_get_device_status()
    except mla.MlaError as e:
        return e.status
    return 0


@pytest.mark.parametrize("seed", range(24))
def test_random_sequences(seed):
    rs = np.random.RandomState(seed)
    shape, nb = list(SHAPES)[seed % 4], int(rs.choice([1, 3, 8, 40]))
    page = mla.make_dims(**SHAPES[shape]).page_size
    lens = tuple(int(x) for x in rs.choice([0, 0, 1, page - 1, page, page + 1, 3 * page + 5], size=nb))
    n_pages = max(1, sum(-(-x // page) for x in lens) + int(rs.randint(0, 6 * nb + 1)))
    p = Pool(shape, lens, n_pages, layers=1 + seed % 2, slack=5, seed=seed, expanded=seed % 3 == 0)

    def some(lo, hi, n):
        return [int(x) for x in rs.randint(lo, hi, size=n)]

    for op in rs.choice(["reserve", "fork", "release", "range", "accept", "accept"], size=12):
        if op == "reserve":
            new = np.minimum(p.lens + rs.choice([0, 0, 1, page, 2 * page - 1], size=nb), p.max_pages * page).astype(np.int32)
            need, args = sum(p.pages(new[b]) - p.pages(p.lens[b]) for b in range(nb)), (new,)
        elif op == "fork":
            dst = [int(x) for x in rs.permutation(np.flatnonzero(p.lens == 0))][:rs.randint(1, nb + 1)]
            if not dst:
                continue
            src = some(0, nb, len(dst))
            need, args = sum(int(p.lens[s]) % page > 0 for s in src), (src, dst)
        elif op == "release":
            need, args = 0, (sorted(set(some(0, nb, 3))),)
        elif op == "range":                                    # full pages, ranges that overlap or are empty
            req = some(0, nb, 3)
            first = some(-2, 5, 3)
            last = [min(int(p.lens[b]) // page, a + int(rs.randint(-1, 3))) for b, a in zip(req, first)]
            op, need, args = "release", 0, (req, first, last)
        else:                                                  # trees in pages that their request holds alone
            max_nodes = int(rs.choice([1, 8, 64]))
            nodes, acc = [], []
            for b in range(nb):
                L, n = int(p.lens[b]), 0
                while n < min(max_nodes, L) and p.table[b, (L - n - 1) // page] >= 0 and \
                        p.refs[p.table[b, (L - n - 1) // page]] == 1:
                    n += 1
                nodes.append(int(rs.randint(0, n + 1)))
                acc.append(sorted(int(x) for x in rs.permutation(nodes[-1])[:rs.randint(0, nodes[-1] + 1)]))
            need, args = 0, (p.lens - np.asarray(nodes, np.int32), nodes, acc, max_nodes)
        getattr(p, op)(*args)
        if need > len(p.free()):
            assert status() == 7
        else:
            assert status() == 0
            getattr(p, "m_" + op)(*(args[:3] if op == "accept" else args))
        p.check()
