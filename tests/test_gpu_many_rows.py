"""Calls with as many query rows as the library takes (2^20): more row tiles than one dimension of a grid holds.
One head, so that the rows are what is large; held against 64 bits on the GPU, 4,096 rows at a time."""
import pytest
import torch

import mla_latent_kv_24_b200 as mla
from _gpu import BF16_REL, FP32_REL

pytestmark = pytest.mark.gpu

# n_heads, d_c, d_rope, d_nope, d_v, page: CUDA cores throughout in float32; in bf16 the absorption and the merge of
# the tensor cores around the CUDA-core decode
SHAPES = {"fp32": dict(n_heads=1, d_c=8, d_rope=8, d_nope=8, d_v=5, page_size=64, dtype="fp32"),
          "bf16 small": dict(n_heads=1, d_c=16, d_rope=8, d_nope=8, d_v=16, page_size=64),
          "bf16": dict(n_heads=1, d_c=512, d_rope=64, d_nope=128, d_v=128, page_size=64)}


def rope(x, pos, base=10000.0):
    d = x.shape[-1]
    ang = pos[..., None].double() * base ** (-torch.arange(0, d, 2, device=x.device, dtype=torch.float64) / d)
    c, s, a, b = ang.cos(), ang.sin(), x[..., 0::2], x[..., 1::2]
    return torch.stack((a * c - b * s, a * s + b * c), -1).flatten(-2)


class Many:
    """B requests of one page each, T queries a request, `L` tokens."""

    def __init__(self, shape, B, T, L):
        self.d = d = mla.make_dims(**SHAPES[shape])
        self.B, self.T, self.L = B, T, L
        self.dt = torch.float32 if d.dtype else torch.bfloat16
        g = torch.Generator(device="cuda").manual_seed(B + T)
        rnd = lambda *s: torch.randn(s, generator=g, device="cuda").to(self.dt)  # noqa: E731
        self.q = rnd(B, T, 1, d.d_nope + d.d_rope)
        self.uk, self.uv = rnd(1, d.d_nope, d.d_c) * d.d_nope ** -0.5, rnd(1, d.d_v, d.d_c) * d.d_c ** -0.5
        self.cache = rnd(B, 64, d.d_c + d.d_rope)
        self.table = torch.randperm(B, generator=g, device="cuda").to(torch.int32).reshape(B, 1)
        self.lens = torch.full((B,), L, dtype=torch.int32, device="cuda")
        self.lens_host = self.lens.cpu().numpy()
        self.out = torch.full((B, T, 1, d.d_v), float("nan"), dtype=self.dt, device="cuda")
        self.depths = torch.randint(0, 9, (B, T), generator=g, device="cuda", dtype=torch.int32)
        self.mask = torch.randint(-2 ** 62, 2 ** 62, (B, T), generator=g, device="cuda") | 1

    def call(self, op):
        d, B, T = self.d, self.B, self.T
        host = (self.lens_host, [T] * B)
        size = {"tree": lambda: mla.mla_decode_tree_workspace_size(d, B, T, *host),
                "window": lambda: mla.mla_decode_window_workspace_size(d, B, T, 1, 3, self.lens_host),
                "causal": lambda: mla.mla_decode_workspace_size(d, B, T, self.lens_host)}[op]()
        ws = torch.empty(size, dtype=torch.uint8, device="cuda")
        a = (d, self.q, self.uk, self.uv, self.cache, self.table, self.lens)
        if op == "tree":
            n = torch.full((B,), T, dtype=torch.int32, device="cuda")
            mla.mla_decode_tree(*a, n, *host, self.depths, self.mask, B, T, 1, B, self.out, ws)
        elif op == "window":
            mla.mla_decode_window(*a, self.lens_host, B, T, 1, 3, 1, B, self.out, ws)
        else:
            mla.mla_decode_absorbed(*a, self.lens_host, B, T, 1, B, self.out, ws)
        mla.mla_get_device_status()

    def check(self, op):
        d, T, L = self.d, self.T, self.L
        step = 4096 // T
        t = torch.arange(L, device="cuda")
        p0 = (L - T + torch.arange(T, device="cuda"))[:, None]
        causal = t <= p0
        for b in range(0, self.B, step):
            e = slice(b, b + step)
            q, rows = self.q[e, :, 0].double(), self.cache[self.table[e, 0].long(), :L].double()
            if op == "tree":                                # no context: L = T nodes
                vis = (self.mask[e][..., None] >> t) & 1 == 1
                pos = self.depths[e]
            else:
                vis = (causal & ((t < 1) | (t > p0 - 3)) if op == "window" else causal).expand(q.shape[0], T, L)
                pos = p0[:, 0].expand(q.shape[0], T)
            k = torch.cat((q[..., :d.d_nope] @ self.uk[0].double(), rope(q[..., d.d_nope:], pos)), -1)
            s = (k @ rows.transpose(1, 2)) * (d.d_nope + d.d_rope) ** -0.5
            ref = s.masked_fill(~vis, float("-inf")).softmax(-1) @ rows[..., :d.d_c] @ self.uv[0].double().T
            got = self.out[e, :, 0].double()
            assert torch.isfinite(got).all(), b
            rel = ((got - ref).norm() / ref.norm()).item()
            assert rel <= (BF16_REL if self.dt == torch.bfloat16 else FP32_REL), (b, rel)


@pytest.mark.parametrize("shape,op,B,T,L", [
    ("fp32", "tree", 1 << 14, 64, 64), ("fp32", "tree", 8320, 64, 64), ("fp32", "window", 1 << 18, 4, 6),
    ("fp32", "causal", 1 << 18, 4, 6), ("bf16 small", "tree", 1 << 14, 64, 64), ("bf16 small", "causal", 131080, 4, 5),
    ("bf16", "tree", 1 << 14, 64, 64), ("bf16", "window", 1 << 18, 4, 6)])
def test_the_largest_number_of_rows(shape, op, B, T, L):
    c = Many(shape, B, T, L)
    c.call(op)
    c.check(op)


@pytest.mark.parametrize("op", ["tree", "window", "causal"])
def test_more_rows_are_refused_before_anything_is_enqueued(op):
    B, T = ((1 << 14) + 1, 64) if op == "tree" else ((1 << 18) + 1, 4)
    d = mla.make_dims(**SHAPES["fp32"])
    lens = [64] * B
    z = torch.zeros(B * T * 16, device="cuda")
    i = torch.zeros(B * T * 2, dtype=torch.int32, device="cuda")
    with pytest.raises(mla.MlaError) as e:
        if op == "tree":
            mla.mla_decode_tree(d, z, z, z, z, i, i, i, lens, [T] * B, i, i.view(torch.int64), B, T, 1, 1, z, z)
        elif op == "window":
            mla.mla_decode_window(d, z, z, z, z, i, i, lens, B, T, 1, 3, 1, 1, z, z)
        else:
            mla.mla_decode_absorbed(d, z, z, z, z, i, i, lens, B, T, 1, 1, z, z)
    assert e.value.status == 2
