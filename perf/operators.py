"""Speculative and long-context serving over the paged latent cache: the operators, in plain form and
through the library's entry points.

  tree     attention of a tree of drafted tokens over the latent cache (mla_decode_tree)
  window   decode with a sliding window and a few first tokens that stay visible, on the absorbed
           path (mla_decode_window)
  gwindow  the same on the GQA path over the per-group expanded cache (gqla_decode_window)
  fork     dropping branches and forking others into their place: shared full pages, a copied partial
           page (mla_cache_release, mla_cache_fork)
  accept   the cache side of a drafting step: pages for the drafted rows, then the accepted path moved
           together and the pages behind it freed (mla_cache_reserve, mla_cache_accept)

`own` False computes them with elementary torch operations in float32; True calls the library.
"""
import math
import random

import numpy as np
import torch

own = False

PAGE = 64
#: Attention shapes: the DeepSeek-V2 shape of the benchmark and the tiny float32 one of the tests.
MODELS = {
    "dsv2": dict(H=128, d_c=512, d_r=64, d_n=128, d_v=128, dtype="bf16"),
    "tiny": dict(H=4, d_c=32, d_r=8, d_n=16, d_v=16, dtype="fp32"),
}
ROPE_BASE = 10000.0


# ------------------------------------------------------------------------------------- the cases
def listed():
    return [
        # one user, a small tree: the latency of a drafting step
        dict(name="tree one user", op="tree", model="dsv2", hpw=1, B=1, nodes=8, ragged_nodes=False, lo=1000, hi=1000, n=1),
        # a ragged batch on GQLA weights, every request with its own length and number of nodes
        dict(name="tree ragged gqla", op="tree", model="dsv2", hpw=8, B=24, nodes=13, ragged_nodes=True, lo=1024, hi=32768, n=2),
        # the most nodes a call takes, uniform lengths: bound by the tensor cores
        dict(name="tree wide", op="tree", model="dsv2", hpw=1, B=8, nodes=64, ragged_nodes=False, lo=8192, hi=8192, n=3),
        # float32 storage at the tiny shape (the CUDA-core kernels)
        dict(name="tree fp32", op="tree", model="tiny", hpw=1, B=4, nodes=16, ragged_nodes=True, lo=60, hi=1030, n=4),
        # one user far beyond the window
        dict(name="window one user", op="window", model="dsv2", hpw=1, B=1, s_q=1, sinks=4, window=1024, lo=131072, hi=131072, n=5),
        # a ragged batch with two-token drafts; some requests are shorter than the window
        dict(name="window ragged", op="window", model="dsv2", hpw=1, B=64, s_q=2, sinks=64, window=4096, lo=1024, hi=32768, n=6),
        # the GQA path, a small batch
        dict(name="gqa window small", op="gwindow", model="dsv2", hpw=8, B=4, s_q=1, sinks=4, window=1000, lo=8192, hi=8192, n=7),
        # the GQA path at the benchmark's batch: bound by memory
        dict(name="gqa window batch", op="gwindow", model="dsv2", hpw=8, B=32, s_q=2, sinks=16, window=8192, lo=16384, hi=65536, n=8),
        # a few parallel samples of one prompt, one layer
        dict(name="fork few", op="fork", model="dsv2", src=1, fan=4, lo=1000, hi=1000, layers=1, n=9),
        # beam search over a batch: a copy in every layer
        dict(name="fork beams", op="fork", model="dsv2", src=16, fan=4, lo=64, hi=4096, layers=32, n=10),
        # one layer, small batch
        dict(name="accept few", op="accept", model="dsv2", B=4, nodes=16, lo=1000, hi=4096, layers=1, n=11),
        # every layer of a model, a large batch of wide trees
        dict(name="accept batch", op="accept", model="dsv2", B=64, nodes=64, lo=64, hi=2048, layers=32, n=12),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "tree", "window", "gwindow", "fork", "accept"])
    n = rng.randrange(1 << 30)
    if op == "tree":
        model = rng.choice(["dsv2", "dsv2", "dsv2", "tiny"])
        B = _log_int(rng, 1, 32)
        nodes = _log_int(rng, 1, 64)
        most = 8 * 64 * 8192 // (B * nodes) if model == "dsv2" else 1030     # the work of the largest listed case
        hi = _log_int(rng, 64, max(65, min(32768, most)))
        lo = hi if rng.random() < 0.3 else max(1, hi // rng.choice([2, 8, 32]))
        return dict(op=op, model=model, hpw=rng.choice([1, 8]) if model == "dsv2" else rng.choice([1, 2]), B=B,
                    nodes=nodes, ragged_nodes=rng.random() < 0.7, lo=lo, hi=hi, n=n)
    if op in ("window", "gwindow"):
        s_q = rng.randint(1, 4)
        window = _log_int(rng, 1, 8192)
        B = _log_int(rng, 1, 64 if op == "window" else 32)
        if op == "window" and B * s_q * window > 64 * 2 * 4096:
            B = max(1, 64 * 2 * 4096 // (s_q * window))
        hi = _log_int(rng, 16, 65536)
        return dict(op=op, model="dsv2", hpw=8 if op == "gwindow" else rng.choice([1, 8]), B=B, s_q=s_q,
                    sinks=rng.choice([0, 1, 4, 16, 64, 100]), window=window, lo=max(4, hi // rng.choice([1, 2, 16])), hi=hi, n=n)
    layers = _log_int(rng, 1, 32)
    hi = _log_int(rng, 64, 4096 if op == "fork" else 2048)
    lo = max(1, hi // rng.choice([1, 4, 64]))
    model = rng.choice(["dsv2", "dsv2", "tiny"])
    if op == "fork":
        return dict(op=op, model=model, src=_log_int(rng, 1, 16), fan=rng.randint(1, 4), lo=lo, hi=hi, layers=layers, n=n)
    return dict(op=op, model=model, B=_log_int(rng, 1, 64), nodes=_log_int(rng, 1, 64), lo=lo, hi=hi, layers=layers, n=n)


def _lens(case, count):
    """Request lengths, log-uniform in [lo, hi]: a property of the case."""
    r = random.Random(case["n"])
    return [min(case["hi"], max(case["lo"], _log_int(r, case["lo"], case["hi"]))) for _ in range(count)]


def _node_counts(case):
    r = random.Random(case["n"] + 1)
    return [r.randint(max(1, case["nodes"] // 2), case["nodes"]) if case.get("ragged_nodes") else case["nodes"]
            for _ in range(case["B"])]


def _accepted_counts(case):
    r = random.Random(case["n"] + 2)
    return [r.randint(0, min(case["nodes"], 1 + case["nodes"] // 4, 8)) for _ in range(case["B"])]


def _pages_of(length):
    return (length + PAGE - 1) // PAGE


# ------------------------------------------------------------------------------------- the work
def work(case):
    m = MODELS[case["model"]]
    e = 2 if m["dtype"] == "bf16" else 4
    row, op = m["d_c"] + m["d_r"], case["op"]
    if op in ("tree", "window", "gwindow"):
        groups = m["H"] // case["hpw"]
        tokens = pairs = rows = 0
        if op == "tree":
            for ctx, n in zip(_lens(case, case["B"]), _node_counts(case)):
                tokens += ctx + n
                pairs += n * (ctx + 1)          # every node sees the context and at least itself
                rows += n
        else:
            S, W, s_q = case["sinks"], case["window"], case["s_q"]
            for L in _lens(case, case["B"]):
                lo = max(0, L - s_q - W + 1)
                tokens += L - lo + min(S, lo)
                rows += s_q
                for j in range(s_q):
                    p = L - s_q + j
                    w0 = max(0, p - W + 1)
                    pairs += p + 1 - w0 + min(S, w0)
        io = rows * m["H"] * (m["d_n"] + m["d_r"] + m["d_v"]) * e
        if op == "gwindow":
            return dict(bytes=tokens * (groups * (m["d_n"] + m["d_v"]) + m["d_r"]) * e + io,
                        flops=pairs * 2 * m["H"] * (m["d_n"] + m["d_r"] + m["d_v"]))
        weights = groups * (m["d_n"] + m["d_v"]) * m["d_c"] * e
        return dict(bytes=tokens * row * e + weights + io,
                    flops=pairs * 2 * m["H"] * (row + m["d_c"]) + rows * m["H"] * 2 * m["d_c"] * (m["d_n"] + m["d_v"]))
    if op == "fork":
        b = 0
        for L in _lens(case, case["src"]):
            b += case["fan"] * (2 * (L % PAGE) * row * e * case["layers"] + 8 * _pages_of(L))
        return dict(bytes=b + 64, flops=0)
    b = sum(2 * a * row * e * case["layers"] + 64 for a in _accepted_counts(case))
    return dict(bytes=b, flops=0)


# ------------------------------------------------------------------------------------- the inputs
def _tree(rs, n):
    """A random tree of n nodes, parents before children: (depth of each node, mask of each node's
    ancestors and itself as 64 bits)."""
    depth, mask = np.zeros(n, np.int32), np.zeros(n, np.uint64)
    for i in range(n):
        p = rs.randint(max(-1, i - 8), i)     # a parent among the last nodes, or a root
        depth[i] = 0 if p < 0 else depth[p] + 1
        mask[i] = (np.uint64(0) if p < 0 else mask[p]) | (np.uint64(1) << np.uint64(i))
    return depth, mask


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    rs = np.random.RandomState(int(seed) % (1 << 31))
    m = MODELS[case["model"]]
    dt = torch.bfloat16 if m["dtype"] == "bf16" else torch.float32
    row = m["d_c"] + m["d_r"]
    s = dict(case=case, m=m, dt=dt, op=case["op"])

    def normal(*shape, std=1.0):
        x = torch.empty(shape, dtype=dt, device="cuda")
        x.normal_(0.0, std, generator=g)
        return x

    def dev(a):
        return torch.from_numpy(np.ascontiguousarray(a)).cuda()

    if case["op"] in ("tree", "window", "gwindow"):
        B, H = case["B"], m["H"]
        groups = H // case["hpw"]
        ctx = np.asarray(_lens(case, B), np.int32)
        if case["op"] == "tree":
            T = case["nodes"]
            counts = np.asarray(_node_counts(case), np.int32)
            lens = ctx + counts
            depth, mask = np.zeros((B, T), np.int32), np.zeros((B, T), np.uint64)
            for b in range(B):
                depth[b, :counts[b]], mask[b, :counts[b]] = _tree(rs, int(counts[b]))
            s.update(T=T, n_nodes_host=counts, n_nodes=dev(counts), depths=dev(depth), tree_mask=dev(mask.view(np.int64)))
        else:
            T = case["s_q"]
            lens = np.maximum(ctx, T).astype(np.int32)
        # Pages that no query sees have been freed: their entries are -1 and the pool holds the others.
        need = []
        for b in range(B):
            k = np.arange(_pages_of(int(lens[b])))
            if case["op"] != "tree":
                lo = max(0, int(lens[b]) - T - case["window"] + 1)
                k = k[(k * PAGE < case["sinks"]) | ((k + 1) * PAGE > lo)]
            need.append(k)
        total = sum(len(k) for k in need)
        ids = rs.permutation(total).astype(np.int32)
        table = np.full((B, max(_pages_of(int(x)) for x in lens)), -1, np.int32)
        at = 0
        for b, k in enumerate(need):
            table[b, k] = ids[at:at + len(k)]
            at += len(k)
        std_w = 0.02 if m["dtype"] == "bf16" else 1 / math.sqrt(m["d_c"])
        s.update(B=B, H=H, hpw=case["hpw"], groups=groups, lens_host=lens, lens=dev(lens), page_table=dev(table),
                 max_pages=table.shape[1], n_pages=total, q=normal(B, T, H, m["d_n"] + m["d_r"]),
                 cache=normal(total, PAGE, row), out=torch.zeros((B, T, H, m["d_v"]), dtype=dt, device="cuda"))
        if case["op"] == "gwindow":
            s["expanded"] = normal(total, groups, PAGE, m["d_n"] + m["d_v"], std=0.45)
        else:
            s.update(W_uk=normal(groups, m["d_n"], m["d_c"], std=std_w), W_uv=normal(groups, m["d_v"], m["d_c"], std=std_w))
        return s

    L = case["layers"]
    if case["op"] == "fork":
        src = _lens(case, case["src"])
        n_dst = case["src"] * case["fan"]
        batch = case["src"] + n_dst
        lens = np.asarray(src + [0] * n_dst, np.int32)
        spare = n_dst + 3
        order = rs.permutation(batch).astype(np.int32)          # which slot of the batch holds which request
        src_req = np.repeat(order[:case["src"]], case["fan"]).astype(np.int32)
        s.update(n_fork=n_dst, src_req=dev(src_req), dst_req=dev(order[case["src"]:]))
    else:
        B = batch = case["B"]
        ctx = np.asarray(_lens(case, B), np.int32)
        counts = np.full(B, case["nodes"], np.int32)
        n_acc = np.asarray(_accepted_counts(case), np.int32)
        accepted = np.zeros((B, case["nodes"]), np.int32)
        for b in range(B):
            k, n = int(n_acc[b]), int(counts[b])
            # The accepted path: node 0, then later nodes; a row that moves comes from behind the path.
            stay = 0 if k == 0 else 1 if n - k >= k - 1 else k
            tail = np.sort(rs.choice(np.arange(k, n), size=k - stay, replace=False)) if k > stay else np.zeros(0, np.int64)
            accepted[b, :k] = np.concatenate([np.arange(stay), tail])
        lens = ctx
        spare = sum(_pages_of(int(c) + case["nodes"]) - _pages_of(int(c)) for c in ctx) + 3
        order = np.arange(batch)
        s.update(B=B, nodes=case["nodes"], ctx=dev(ctx), new_lens=dev(ctx + counts), n_nodes=dev(counts),
                 n_accepted=dev(n_acc), accepted=dev(accepted))
    per = [_pages_of(int(x)) for x in lens]
    total = sum(per) + spare
    ids = rs.permutation(total).astype(np.int32)
    max_pages = max(per) + 2
    table = np.full((batch, max_pages), -1, np.int32)
    refs = np.zeros(total, np.int32)
    at, all_lens = 0, np.zeros(batch, np.int32)
    for i, k in enumerate(per):
        b = int(order[i])
        table[b, :k] = ids[at:at + k]
        refs[ids[at:at + k]] = 1
        all_lens[b] = lens[i]
        at += k
    s.update(batch=batch, max_pages=max_pages, n_pages=total, layers=L, lens=dev(all_lens), page_table=dev(table),
             refs=dev(refs), cache=normal(L, total, PAGE, row))
    return s


# ------------------------------------------------------------------------------------- plain forms
def _rope(x, pos, base=ROPE_BASE):
    """Interleaved pairs of x[..., d] turned by pos * base^(-2i/d); angles in float64."""
    d = x.shape[-1]
    ang = pos.double()[..., None] * base ** (-2.0 * torch.arange(d // 2, device=x.device, dtype=torch.float64) / d)
    c, sn = ang.cos().to(x.dtype), ang.sin().to(x.dtype)
    x0, x1 = x[..., 0::2], x[..., 1::2]
    return torch.stack([x0 * c - x1 * sn, x0 * sn + x1 * c], dim=-1).flatten(-2)


def _weights(scores, visible):
    """Softmax over the visible entries of the last dimension; a row that sees nothing has no weights."""
    scores = scores.masked_fill(~visible, float("-inf"))
    top = scores.amax(-1, keepdim=True)
    e = torch.exp(scores - torch.where(torch.isfinite(top), top, torch.zeros_like(top)))
    total = e.sum(-1, keepdim=True)
    return e / torch.where(total > 0, total, torch.ones_like(total))


def _gather(table, pages, tokens, held):
    """Rows of a paged tensor at `tokens` [B, n]; those not `held` read as zeros."""
    page = torch.gather(table, 1, (tokens // PAGE).long())
    held = held & (page >= 0)
    at = torch.where(held, page * PAGE + tokens % PAGE, torch.zeros_like(page)).long()
    return pages[at].float().masked_fill(~held.reshape(held.shape + (1,) * (pages.dim() - 1)), 0.0)


def _absorbed(s, pos, tokens, held, visible):
    """Absorbed attention of s["q"] at positions pos [B, T] over the cache rows `tokens` [B, n], of
    which query (b, j) sees visible[b, j]."""
    m, q = s["m"], s["q"].float()
    rep = lambda w: w.float().repeat_interleave(s["hpw"], 0)  # noqa: E731
    rows = _gather(s["page_table"], s["cache"].reshape(-1, m["d_c"] + m["d_r"]), tokens, held)
    q_lat = torch.einsum("bthn,hnc->bthc", q[..., :m["d_n"]], rep(s["W_uk"]))
    q_cat = torch.cat([q_lat, _rope(q[..., m["d_n"]:], pos[..., None])], -1)
    B, T, H, _ = q_cat.shape
    scores = torch.matmul(q_cat.reshape(B, T * H, -1), rows.transpose(1, 2)).reshape(B, T, H, -1)
    w = _weights(scores / math.sqrt(m["d_n"] + m["d_r"]), visible[:, :, None])
    o = torch.matmul(w.reshape(B, T * H, -1), rows[..., :m["d_c"]]).reshape(B, T, H, -1)
    return torch.einsum("bthc,hvc->bthv", o, rep(s["W_uv"])).to(s["dt"])


def _tree_view(s):
    """Positions [B, T], tokens [B, n], which of them exist, and which a node sees."""
    n = int(s["lens_host"].max())
    t = torch.arange(n, device="cuda")[None]
    ctx = (s["lens"] - s["n_nodes"])[:, None]
    held = t < s["lens"][:, None]
    node = (t - ctx).clamp(0, 63)
    bit = (s["tree_mask"][:, :, None] >> node[:, None]) & 1
    visible = held[:, None] & ((t < ctx)[:, None] | (bit == 1))
    return ctx + s["depths"], t.expand(s["B"], n), held, visible


def _window_view(s):
    """As _tree_view: the sinks, then the tokens from the first query's window on."""
    c = s["case"]
    S, W, T = c["sinks"], c["window"], c["s_q"]
    L = s["lens"][:, None]
    lo = (L - T - W + 1).clamp(min=0)
    near = lo + torch.arange(min(int(s["lens_host"].max()), W + T - 1), device="cuda")[None]
    far = torch.arange(S, device="cuda")[None].expand(s["B"], S)
    tokens = torch.cat([far, near], 1)
    held = torch.cat([far < torch.minimum(lo, L), near < L], 1)       # a sink inside the window counts once
    pos = L - T + torch.arange(T, device="cuda")[None]
    p = pos[..., None]
    t = tokens[:, None]
    visible = held[:, None] & (t <= p) & ((t < S) | (t > p - W))
    return pos, tokens.clamp(max=s["max_pages"] * PAGE - 1), held, visible


def _grouped(s, pos, tokens, held, visible):
    m, q = s["m"], s["q"].float()
    B, T, H, _ = q.shape
    G, hpw = s["groups"], s["hpw"]
    ex = s["expanded"].permute(0, 2, 1, 3).reshape(-1, G, m["d_n"] + m["d_v"])
    kv = _gather(s["page_table"], ex, tokens, held)                                       # [B, n, G, 256]
    kr = _gather(s["page_table"], s["cache"].reshape(-1, m["d_c"] + m["d_r"])[:, m["d_c"]:], tokens, held)
    qg = q.reshape(B, T, G, hpw, -1)
    scores = torch.einsum("btgid,bngd->btgin", qg[..., :m["d_n"]], kv[..., :m["d_n"]])
    scores += torch.einsum("btgid,bnd->btgin", _rope(qg[..., m["d_n"]:], pos[..., None, None]), kr)
    w = _weights(scores / math.sqrt(m["d_n"] + m["d_r"]), visible[:, :, None, None])
    return torch.einsum("btgin,bngd->btgid", w, kv[..., m["d_n"]:]).reshape(B, T, H, -1).to(s["dt"])


def _lowest_free(refs, ranks, wanted):
    """The ranks-th lowest page that nobody holds (rank 0 is the lowest), where `wanted`."""
    upto = torch.cumsum((refs == 0).int(), 0)
    return torch.searchsorted(upto, (ranks + 1).int().contiguous()).int().masked_fill(~wanted, 0)


def _plain_fork(s):
    table, refs, lens, cache = s["page_table"], s["refs"], s["lens"], s["cache"]
    k = torch.arange(s["max_pages"], device="cuda")[None]
    src, dst = s["src_req"].long(), s["dst_req"].long()
    # drop what the destinations hold
    old = table[dst]
    drop = (k < (lens[dst][:, None] + PAGE - 1) // PAGE) & (old >= 0)
    refs.index_add_(0, old.clamp(min=0).flatten().long(), -drop.flatten().int())
    table[dst] = torch.where(drop, torch.full_like(old, -1), old)
    # share the full pages, copy the partial one
    L = lens[src]
    full, rem = L // PAGE, L % PAGE
    part = rem > 0
    new = _lowest_free(refs, torch.cumsum(part.int(), 0) - 1, part)
    mine = table[src]
    share = k < full[:, None]
    refs.index_add_(0, mine.clamp(min=0).flatten().long(), (share & (mine >= 0)).flatten().int())
    refs.index_add_(0, new.long(), part.int())
    entry = torch.where(share, mine, table[dst])
    table[dst] = torch.where((k == full[:, None]) & part[:, None], new[:, None], entry)
    lens[dst] = L
    last = torch.gather(mine, 1, torch.where(part, full, torch.zeros_like(full))[:, None].long())
    r = torch.arange(PAGE, device="cuda")[None]
    at_src = last * PAGE + r                                                        # [n, PAGE]
    at_dst = torch.where(r < rem[:, None], new[:, None] * PAGE + r, at_src)         # the others stay where they are
    flat = cache.reshape(s["layers"], -1, cache.shape[-1])
    flat[:, at_dst.flatten().long()] = flat[:, at_src.flatten().long()]
    return dict(page_table=table, refs=refs, lens=lens, cache=cache)


def _plain_accept(s):
    table, refs, lens, cache = s["page_table"], s["refs"], s["lens"], s["cache"]
    k = torch.arange(s["max_pages"], device="cuda")[None]
    # pages for the drafted rows
    have, want = (lens + PAGE - 1) // PAGE, (s["new_lens"] + PAGE - 1) // PAGE
    fresh = (k >= have[:, None]) & (k < want[:, None])
    ranks = (torch.cumsum(fresh.flatten().int(), 0) - 1).reshape(fresh.shape)
    new = _lowest_free(refs, ranks.flatten(), fresh.flatten()).reshape(fresh.shape)
    refs.index_add_(0, new.flatten().long(), fresh.flatten().int())
    table.copy_(torch.where(fresh, new, table))
    # the accepted rows move together behind the context
    i = torch.arange(s["nodes"], device="cuda")[None]
    moved = i < s["n_accepted"][:, None]
    slot = lambda t: (torch.gather(table, 1, (t // PAGE).long()) * PAGE + t % PAGE).long()  # noqa: E731
    ctx = s["ctx"][:, None]
    at_src = slot(torch.where(moved, ctx + s["accepted"], ctx - 1))                  # a row that stays, for the others
    at_dst = slot(torch.where(moved, ctx + i, ctx - 1))
    flat = cache.reshape(s["layers"], -1, cache.shape[-1])
    flat[:, at_dst.flatten()] = flat[:, at_src.flatten()]
    # the pages behind them are freed
    lens.copy_(s["ctx"] + s["n_accepted"])
    keep = (lens + PAGE - 1) // PAGE
    drop = (k >= keep[:, None]) & (k < want[:, None])
    refs.index_add_(0, table.clamp(min=0).flatten().long(), -(drop & (table >= 0)).flatten().int())
    table.masked_fill_(drop, -1)
    return dict(page_table=table, refs=refs, lens=lens, cache=cache)


def _plain(s):
    if s["op"] == "tree":
        out = _absorbed(s, *_tree_view(s))
        node = torch.arange(s["T"], device="cuda")[None]
        return torch.where((node < s["n_nodes"][:, None])[..., None, None], out, s["out"])   # others keep theirs
    if s["op"] == "window":
        return _absorbed(s, *_window_view(s))
    if s["op"] == "gwindow":
        return _grouped(s, *_window_view(s))
    return _plain_fork(s) if s["op"] == "fork" else _plain_accept(s)


# ------------------------------------------------------------------------------------- the library
def _own(s):
    import mla_latent_kv_24_b200 as mla
    m, op = s["m"], s["op"]
    if "dims" not in s:
        s["dims"] = mla.make_dims(n_heads=m["H"], heads_per_group=s.get("hpw", 1), d_c=m["d_c"], d_rope=m["d_r"],
                                  d_nope=m["d_n"], d_v=m["d_v"], page_size=PAGE, rope_base=ROPE_BASE, dtype=m["dtype"])
        size = 0
        if op == "tree":
            size = mla.mla_decode_tree_workspace_size(s["dims"], s["B"], s["T"], s["lens_host"], s["n_nodes_host"])
        elif op == "window":
            size = mla.mla_decode_window_workspace_size(s["dims"], s["B"], s["case"]["s_q"], s["case"]["sinks"],
                                                        s["case"]["window"], s["lens_host"])
        elif op == "gwindow":
            size = mla.gqla_decode_window_workspace_size(s["dims"], s["B"], s["case"]["s_q"], s["case"]["sinks"],
                                                         s["case"]["window"], s["lens_host"])
        s["ws"] = torch.empty(max(size, 256), dtype=torch.uint8, device="cuda")
    d = s["dims"]
    if op == "tree":
        mla.mla_decode_tree(d, s["q"], s["W_uk"], s["W_uv"], s["cache"], s["page_table"], s["lens"], s["n_nodes"],
                            s["lens_host"], s["n_nodes_host"], s["depths"], s["tree_mask"], s["B"], s["T"],
                            s["max_pages"], s["n_pages"], s["out"], s["ws"])
        return s["out"]
    if op == "window":
        c = s["case"]
        mla.mla_decode_window(d, s["q"], s["W_uk"], s["W_uv"], s["cache"], s["page_table"], s["lens"], s["lens_host"],
                              s["B"], c["s_q"], c["sinks"], c["window"], s["max_pages"], s["n_pages"], s["out"], s["ws"])
        return s["out"]
    if op == "gwindow":
        c = s["case"]
        mla.gqla_decode_window(d, s["q"], s["expanded"], s["cache"], s["page_table"], s["lens"], s["lens_host"],
                               s["B"], c["s_q"], c["sinks"], c["window"], s["max_pages"], s["n_pages"], s["out"], s["ws"])
        return s["out"]
    table, refs, lens, cache = s["page_table"], s["refs"], s["lens"], s["cache"]
    if op == "fork":
        mla.mla_cache_release(d, s["dst_req"], None, None, s["n_fork"], lens, table, s["batch"], s["max_pages"], refs, s["n_pages"])
        mla.mla_cache_fork(d, s["src_req"], s["dst_req"], s["n_fork"], lens, table, s["batch"], s["max_pages"], refs,
                           s["n_pages"], cache, None, s["layers"])
    else:
        mla.mla_cache_reserve(d, s["new_lens"], lens, table, s["batch"], s["max_pages"], refs, s["n_pages"])
        mla.mla_cache_accept(d, s["ctx"], s["n_nodes"], s["accepted"], s["n_accepted"], s["nodes"], lens, table,
                             s["batch"], s["max_pages"], refs, s["n_pages"], cache, None, s["layers"])
    return dict(page_table=table, refs=refs, lens=lens, cache=cache)


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    """Attention by its definition in float64: per request and head, keys and values up-projected from
    the latent (or taken from the expanded cache), softmax over the tokens a query sees."""
    if case["op"] in ("fork", "accept"):
        return None                       # rows are copied, not computed
    s = prepare(case, seed)
    m, T = s["m"], (s["T"] if case["op"] == "tree" else case["s_q"])
    d_n, d_c, H = m["d_n"], m["d_c"], m["H"]
    out = s["out"].double()
    table = s["page_table"].cpu().numpy()
    theta = ROPE_BASE ** (-2.0 * torch.arange(m["d_r"] // 2, device="cuda", dtype=torch.float64) / m["d_r"])
    depths = s["depths"].cpu().numpy() if case["op"] == "tree" else None
    masks = s["tree_mask"].cpu().numpy().view(np.uint64) if case["op"] == "tree" else None
    for b in range(s["B"]):
        L = int(s["lens_host"][b])
        n = int(s["n_nodes_host"][b]) if case["op"] == "tree" else T
        t = np.arange(L)
        sees, pos = np.zeros((n, L), bool), np.zeros(n)
        for j in range(n):
            if case["op"] == "tree":
                ctx = L - n
                sees[j, :ctx] = True
                for i in range(n):
                    sees[j, ctx + i] = bool((int(masks[b, j]) >> i) & 1)
                pos[j] = ctx + depths[b, j]
            else:
                pos[j] = L - n + j
                sees[j] = (t <= pos[j]) & ((t < case["sinks"]) | (t > pos[j] - case["window"]))
        t = t[sees.any(0)]
        sees = torch.from_numpy(sees[:, t]).cuda()
        page, r = torch.from_numpy(table[b, t // PAGE].astype(np.int64)).cuda(), torch.from_numpy(t % PAGE).cuda()
        rows = s["cache"][page, r].double()
        ang = torch.from_numpy(pos).cuda()[:, None] * theta                           # [n, d_r / 2]
        q = s["q"][b, :n].double()
        z = torch.view_as_complex(q[..., d_n:].reshape(n, H, -1, 2).contiguous()) * torch.polar(torch.ones_like(ang), ang)[:, None]
        q_r = torch.view_as_real(z).reshape(n, H, -1)
        for h in range(H):
            w = h // s["hpw"]
            if case["op"] == "gwindow":
                K, V = s["expanded"][page, w, r].double().split([d_n, m["d_v"]], -1)
            else:
                K, V = rows[:, :d_c] @ s["W_uk"][w].double().T, rows[:, :d_c] @ s["W_uv"][w].double().T
            x = (q[:, h, :d_n] @ K.T + q_r[:, h] @ rows[:, d_c:].T) / math.sqrt(d_n + m["d_r"])
            x = torch.where(sees, x, torch.full_like(x, -math.inf))
            out[b, :n, h] = torch.nan_to_num(torch.softmax(x, -1)) @ V
    return out
