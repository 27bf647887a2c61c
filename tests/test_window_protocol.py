"""Model check of the grouped (GQA-path) decode's stages where a window leaves pages partly seen (decode_grouped.cu),
on CPU.

With a window any page may be partly seen, not only the chunk's last one: each warp then zeroes its rows that no query
sees with ordinary stores, and the stage is later refilled by a tensor copy.  Ordinary stores and tensor copies go
through different proxies, which an mbarrier alone does not order: a store may still be under way when the copy has
written the same bytes, and then undoes them.  A proxy fence by the storing lanes, before their warp arrives on the
stage's `empty` barrier, ends that.  In the model a store is under way until it is fenced or until it happens to land;
stores, copies and warps run in random order.  Whether the kernel has the fence is read from its source."""
import os
import random
import re

import pytest

STAGES, WARPS = 2, 4
SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mla_latent_kv_24_b200", "csrc")


def zeroing_branch():
    """The source of the kernel's branch that zeroes the rows that no query of a window sees."""
    text = open(os.path.join(SRC, "decode_grouped.cu")).read()
    m = re.search(r"if constexpr \(WIN\) \{(.*?)\n        \} else if", text, re.S)
    assert m and "make_uint4(0u, 0u, 0u, 0u)" in m.group(1)
    return m.group(1)


def simulate(partly, seed, fence):
    """partly[i][w]: warp w zeroes its rows of page i.  Raises AssertionError where a warp reads other bytes than its
    page's copy wrote, as it zeroed them."""
    rnd = random.Random(seed)
    n = len(partly)
    full, empty = [0] * STAGES, [0] * STAGES            # completed phases of `full`; arrivals on `empty` so far
    rows = [[None] * WARPS for _ in range(STAGES)]       # what a warp's rows of a stage hold: (page, zeroed)
    copies, stores = [], []                             # under way: (stage, page); (stage, warp, value)

    def land_store(k):
        st, w, value = stores.pop(k)
        rows[st][w] = value

    def copy_engine():
        while True:
            yield lambda: copies
            st, page = copies.pop(rnd.randrange(len(copies)))
            rows[st] = [(page, False)] * WARPS
            full[st] += 1

    def store_engine():
        while True:
            yield lambda: stores
            land_store(rnd.randrange(len(stores)))

    def warp(w):
        if w == 0:
            copies.extend((i, i) for i in range(min(STAGES, n)))
        for i in range(n):
            st = i % STAGES
            yield lambda: full[st] > i // STAGES
            mine = [k for k, s in enumerate(stores) if s[:2] == (st, w)]
            assert rows[st][w] == (i, False), ("page", i, "warp", w, "holds", rows[st][w], "stores under way", len(mine))
            if partly[i][w]:
                stores.append((st, w, (i, True)))
                yield lambda: True
                if fence:
                    for k in [k for k, s in enumerate(stores) if s[:2] == (st, w)][::-1]:
                        land_store(k)
            yield lambda: True                          # products on the stage (a warp sees its own stores)
            empty[st] += 1
            if w == 0 and i + STAGES < n:
                yield lambda: empty[st] == WARPS * (i // STAGES + 1)
                copies.append((st, i + STAGES))

    roles = [warp(w) for w in range(WARPS)] + [copy_engine(), store_engine()]
    waits = {r: next(co) for r, co in enumerate(roles)}
    while any(r < WARPS for r in waits):
        ready = [r for r, cond in waits.items() if cond()]
        assert ready, "deadlock"
        r = rnd.choice(ready)
        try:
            waits[r] = next(roles[r])
        except StopIteration:
            del waits[r]


def cases():
    rnd = random.Random(17)
    for seed in range(300):
        n = rnd.randint(1, 9)
        # a sinks' page and a window's first page at the front, the last page, or any pages at all
        some = [i in (0, 1, n - 1) or seed % 3 == 0 and rnd.random() < 0.5 for i in range(n)]
        yield [[s and rnd.random() < 0.7 for _ in range(WARPS)] for s in some], seed


def test_zeroed_rows_are_refilled_in_order():
    fence = "fence_proxy_async_smem" in zeroing_branch()
    for partly, seed in cases():
        simulate(partly, seed, fence)


def test_the_model_sees_a_missing_fence():
    with pytest.raises(AssertionError):
        for partly, seed in cases():
            simulate(partly, seed, False)


def test_the_fence_is_before_the_warp_goes_on():
    # by every storing lane, behind its stores and before the warp meets (and so before it arrives on `empty`)
    b = zeroing_branch()
    assert b.index("make_uint4") < b.index("fence_proxy_async_smem") < b.index("__syncwarp")
