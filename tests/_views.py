"""Helpers of the tree and window tests: inputs, the oracle with a mask, and the library's calls."""
import numpy as np
import torch

import mla_latent_kv_24_b200 as mla
import oracle
import workloads as wl
from _gpu import dims_of


def base_workload(model="dsv2", **kw):
    """The DeepSeek-V2 shape in bf16 (tensor-core kernels), or one of the shapes of the CUDA-core kernels."""
    if model == "dsv2":
        return wl.small_workload(wl.WORKLOADS["4"], lens_loguniform=None, shuffle_pages=True, **kw)
    if model == "gqla":
        return wl.small_workload(wl.WORKLOADS["5_8192_1"], shuffle_pages=True, **kw)
    if model == "tiny":                                              # fp32
        return wl.small_workload(wl.WORKLOADS["1"], shuffle_pages=True, **kw)
    if model == "h16":                                               # bf16, fewer heads: CUDA cores, tensor-core merge
        return wl.small_workload(wl.WORKLOADS["4"], lens_loguniform=None, shuffle_pages=True, H=16, **kw)
    raise KeyError(model)


class Case:
    """Device copies of seeded inputs whose requests have `lens` cached tokens and T queries each.  Lengths of
    zero get a page of their own that nothing names."""

    def __init__(self, w, T, lens, seed):
        self.w, self.T = w, T
        self.lens = np.asarray(lens, np.int32)
        self.inp = inp = wl.make_inputs(wl.small_workload(w, B=len(lens), s_q=T, lens=[max(1, int(x)) for x in lens], seed=seed))
        self.dims = dims_of(w)
        self.cache = wl.to_torch(inp.cache)
        self.q, self.W_uk, self.W_uv = (wl.to_torch(t) for t in (inp.q, inp.W_uk, inp.W_uv))
        self.table_host = inp.page_table.copy()
        for b, L in enumerate(self.lens):                            # entries past the request: never read
            self.table_host[b, (int(L) + w.page - 1) // w.page:] = -1
        self.tdtype = torch.bfloat16 if w.dtype == "bf16" else torch.float32
        self.B, self.max_pages, self.n_pages = len(lens), self.table_host.shape[1], inp.n_pages

    def dev(self, a):
        return torch.from_numpy(np.ascontiguousarray(a)).cuda()

    def slots(self, b, tokens):
        t = np.asarray(tokens)
        return self.inp.page_table[b, t // self.w.page], t % self.w.page

    def poison(self, b, tokens, value=float("nan"), expanded=None):
        """Writes `value` into the cache rows of these tokens on the device (the oracle keeps the inputs')."""
        if len(tokens):
            pg, r = self.slots(b, tokens)
            pg, r = torch.from_numpy(pg.astype(np.int64)).cuda(), torch.from_numpy(r.astype(np.int64)).cuda()
            self.cache[pg, r] = value
            if expanded is not None:
                expanded[pg, :, r] = value

    def poison_stale(self, expanded=None):
        for b, L in enumerate(self.lens):
            page = self.w.page
            end = max(1, (int(L) + page - 1) // page) * page
            self.poison(b, np.arange(int(L), end), expanded=expanded)

    def oracle(self, b, n, positions, visible):
        inp, w = self.inp, self.w
        rows = oracle.request_rows(inp.cache.f64(), inp.page_table, b, int(self.lens[b])) if self.lens[b] else \
            np.zeros((0, w.d_row))
        return oracle.decode_request_masked(inp.q.f64()[b, :n], rows, inp.W_uk.f64(), inp.W_uv.f64(), w.hpw,
                                            w.softmax_scale, w.rope_base, positions, visible)

    def out(self, fill=0.0):
        return torch.full((self.B, self.T, self.w.H, self.w.d_v), fill, dtype=self.tdtype, device="cuda")


def random_tree(rng, n, dense=False):
    """(depths, masks) of n nodes, parents first; dense: any bits at all, a node's own included or not."""
    depth, mask = np.zeros(n, np.int32), np.zeros(n, np.uint64)
    for i in range(n):
        if dense:
            depth[i] = rng.integers(0, n)
            mask[i] = np.uint64(int(rng.integers(0, 1 << 32)) << 32 | int(rng.integers(0, 1 << 32)))
        else:
            p = int(rng.integers(-1, i)) if i else -1
            depth[i] = 0 if p < 0 else depth[p] + 1
            mask[i] = (np.uint64(0) if p < 0 else mask[p]) | np.uint64(1 << i)
    return depth, mask


def tree_visible(L, n, masks):
    vis = np.zeros((n, L), bool)
    vis[:, :L - n] = True
    for j in range(n):
        for i in range(n):
            vis[j, L - n + i] = bool((int(masks[j]) >> i) & 1)
    return vis


class TreeCase(Case):
    def __init__(self, w, T, ctx, nodes, seed, dense=False):
        super().__init__(w, T, np.asarray(ctx) + np.asarray(nodes), seed)
        self.ctx, self.nodes = np.asarray(ctx, np.int32), np.asarray(nodes, np.int32)
        rng = np.random.default_rng(seed + 1)
        self.depths = rng.integers(-1000, 1000, size=(self.B, T)).astype(np.int32)      # of slots without a node too
        self.masks = rng.integers(0, 1 << 63, size=(self.B, T)).astype(np.uint64)
        for b in range(self.B):
            n = int(self.nodes[b])
            self.depths[b, :n], self.masks[b, :n] = random_tree(rng, n, dense)

    def positions(self, b):
        return self.ctx[b] + self.depths[b, :self.nodes[b]]

    def visible(self, b):
        return tree_visible(int(self.lens[b]), int(self.nodes[b]), self.masks[b])

    def upload(self):
        self.d = dict(page_table=self.dev(self.table_host), seq_lens=self.dev(self.lens), n_nodes=self.dev(self.nodes),
                      depths=self.dev(self.depths), tree_mask=self.dev(self.masks.view(np.int64)))
        nb = mla.mla_decode_tree_workspace_size(self.dims, self.B, self.T, self.lens, self.nodes)
        self.ws = torch.full((max(nb, 256),), 255, dtype=torch.uint8, device="cuda")     # scratch: any bytes, NaN here
        return self

    def call(self, out, ws=None, stream=None):
        d = self.d
        mla.mla_decode_tree(self.dims, self.q, self.W_uk, self.W_uv, self.cache, d["page_table"], d["seq_lens"],
                            d["n_nodes"], self.lens, self.nodes, d["depths"], d["tree_mask"], self.B, self.T,
                            self.max_pages, self.n_pages, out, self.ws if ws is None else ws, stream=stream)
        return out

    def reference(self):
        """The oracle's output, NaN where nothing is written."""
        ref = np.full((self.B, self.T, self.w.H, self.w.d_v), np.nan)
        for b in range(self.B):
            n = int(self.nodes[b])
            if n:
                ref[b, :n] = self.oracle(b, n, self.positions(b), self.visible(b))
        return ref


class WindowCase(Case):
    def __init__(self, w, s_q, lens, sinks, window, seed):
        super().__init__(w, s_q, lens, seed)
        self.sinks, self.window = sinks, window

    def visible(self, b):
        L, T = int(self.lens[b]), self.T
        t, p = np.arange(L)[None], (L - T + np.arange(T))[:, None]
        return (t <= p) & ((t < self.sinks) | (t > p - self.window))

    def free_unseen(self, expanded=None):
        """Pages that no query sees lose their entry; other rows that none sees hold NaN."""
        for b, L in enumerate(self.lens):
            seen = self.visible(b).any(0)
            self.poison(b, np.flatnonzero(~seen), expanded=expanded)
            for k in range((int(L) + self.w.page - 1) // self.w.page):
                if not seen[k * self.w.page:(k + 1) * self.w.page].any():
                    self.table_host[b, k] = -1 if k % 2 else 1 << 30
        self.poison_stale(expanded)

    def upload(self, grouped=False):
        self.grouped = grouped
        self.d = dict(page_table=self.dev(self.table_host), seq_lens=self.dev(self.lens))
        size = mla.gqla_decode_window_workspace_size if grouped else mla.mla_decode_window_workspace_size
        nb = size(self.dims, self.B, self.T, self.sinks, self.window, self.lens)
        self.ws = torch.full((max(nb, 256),), 255, dtype=torch.uint8, device="cuda")
        return self

    def expand(self):
        w = self.w
        exp = torch.empty((self.n_pages, w.H // w.hpw, w.page, w.d_n + w.d_v), dtype=self.tdtype, device="cuda")
        mla.gqla_expand_cache(self.dims, self.W_uk, self.W_uv, self.cache, None, 0, self.n_pages, exp)
        return exp

    def call(self, out, expanded=None, ws=None):
        d, ws = self.d, self.ws if ws is None else ws
        if self.grouped:
            mla.gqla_decode_window(self.dims, self.q, expanded, self.cache, d["page_table"], d["seq_lens"], self.lens,
                                   self.B, self.T, self.sinks, self.window, self.max_pages, self.n_pages, out, ws)
        else:
            mla.mla_decode_window(self.dims, self.q, self.W_uk, self.W_uv, self.cache, d["page_table"], d["seq_lens"],
                                  self.lens, self.B, self.T, self.sinks, self.window, self.max_pages, self.n_pages,
                                  out, ws)
        return out

    def reference(self):
        ref = np.zeros((self.B, self.T, self.w.H, self.w.d_v))
        for b, L in enumerate(self.lens):
            ref[b] = self.oracle(b, self.T, int(L) - self.T + np.arange(self.T), self.visible(b))
        return ref
