"""Calls right behind a kernel that lets its dependents launch before it has written their inputs.

The library's kernels are launched with programmatic stream serialisation, so such a producer (a matrix product
with an early trigger, for instance) is still running when a call's first kernel starts.  Every input of every entry
point, weights and the pool's state included, is written here by a producer that triggers at once and stores 200 us
later; until then the inputs hold other values of the same kind.  The results have to be those of a call on settled
inputs, bit for bit.
"""
import ctypes
import subprocess

import numpy as np
import pytest
import torch

import mla_latent_kv_24_b200 as mla
import workloads as wl
from _gpu import Dev
from _views import TreeCase, WindowCase, base_workload
from mla_latent_kv_24_b200 import build

pytestmark = pytest.mark.gpu

MAX_JOBS = 16
PRODUCER = r"""
#include <cuda_runtime.h>
struct Jobs { char *dst[%(n)d]; const char *src[%(n)d]; long long bytes[%(n)d]; int n; };
__device__ unsigned long long now() {
    unsigned long long t;
    asm volatile("mov.u64 %%0, %%globaltimer;" : "=l"(t));
    return t;
}
__global__ void __launch_bounds__(1024) produce_kernel(Jobs j, unsigned long long delay_ns) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const unsigned long long t0 = now();
    for (int i = 0; i < (1 << 16) && now() - t0 < delay_ns; ++i) __nanosleep(500);
    for (int k = 0; k < j.n; ++k) {
        const long long words = j.bytes[k] / 4;
        for (long long i = threadIdx.x; i < words; i += 1024)
            reinterpret_cast<int *>(j.dst[k])[i] = reinterpret_cast<const int *>(j.src[k])[i];
        for (long long i = 4 * words + threadIdx.x; i < j.bytes[k]; i += 1024) j.dst[k][i] = j.src[k][i];
    }
}
extern "C" int produce(const Jobs *j, unsigned long long delay_ns, cudaStream_t st) {
    produce_kernel<<<1, 1024, 0, st>>>(*j, delay_ns);
    return (int)cudaGetLastError();
}
""" % dict(n=MAX_JOBS)


class Jobs(ctypes.Structure):
    _fields_ = [("dst", ctypes.c_void_p * MAX_JOBS), ("src", ctypes.c_void_p * MAX_JOBS),
                ("bytes", ctypes.c_longlong * MAX_JOBS), ("n", ctypes.c_int)]


@pytest.fixture(scope="module")
def produce(tmp_path_factory):
    d = tmp_path_factory.mktemp("producer")
    (d / "p.cu").write_text(PRODUCER)
    subprocess.run([build.nvcc(), *build.ARCH, "-O1", "-shared", "-Xcompiler", "-fPIC", "-cudart", "static",
                    "-o", str(d / "p.so"), str(d / "p.cu")], check=True)
    lib = ctypes.CDLL(str(d / "p.so"))
    lib.produce.argtypes = [ctypes.POINTER(Jobs), ctypes.c_ulonglong, ctypes.c_void_p]

    def run(pairs, delay_ns=200_000):
        assert len(pairs) <= MAX_JOBS
        j = Jobs()
        for k, (dst, src) in enumerate(pairs):
            assert dst.is_contiguous() and src.is_contiguous() and dst.nbytes == src.nbytes
            j.dst[k], j.src[k], j.bytes[k] = dst.data_ptr(), src.data_ptr(), dst.nbytes
        j.n = len(pairs)
        assert lib.produce(ctypes.byref(j), delay_ns, torch.cuda.current_stream().cuda_stream) == 0

    return run


def other(t):
    """Values of the same kind as t's in other places."""
    return torch.roll(t.reshape(-1), 1).reshape(t.shape).contiguous()


class Op:
    """A call, its inputs as (tensor, stale values) and what it writes."""

    def __init__(self, call, inputs, outputs):
        self.call, self.outputs = call, outputs
        self.inputs = [(t, t.clone(), s) for t, s in inputs]

    def settle(self, fresh):
        for t, f, s in self.inputs:
            t.copy_(f if fresh else s)
        for o in self.outputs:
            if not any(o is t for t, _, _ in self.inputs):
                o.zero_()
        torch.cuda.synchronize()

    def result(self):
        torch.cuda.synchronize()
        mla.mla_get_device_status()
        return [o.clone() for o in self.outputs]


def _tree(model, T, ctx, nodes):
    c = TreeCase(base_workload(model), T, ctx, nodes, seed=41).upload()
    d, out = c.d, c.out()
    inputs = [(c.q, other(c.q)), (c.W_uk, other(c.W_uk)), (c.W_uv, other(c.W_uv)), (c.cache, other(c.cache)),
              (d["page_table"], d["page_table"].flip(1).clamp_min(0).contiguous()), (d["seq_lens"], d["seq_lens"] - 1),
              (d["n_nodes"], d["n_nodes"] - 1), (d["depths"], d["depths"] + 3), (d["tree_mask"], other(d["tree_mask"]))]
    return Op(lambda: c.call(out), inputs, [out])


def _window(model, s_q, lens, grouped=False):
    c = WindowCase(base_workload(model), s_q, lens, 3, 90, seed=42).upload(grouped)
    d, out, exp = c.d, c.out(), c.expand() if grouped else None
    inputs = [(c.q, other(c.q)), (c.cache, other(c.cache)), (d["seq_lens"], d["seq_lens"] - 1),
              (d["page_table"], d["page_table"].flip(1).clamp_min(0).contiguous())]
    inputs += [(exp, other(exp))] if grouped else [(c.W_uk, other(c.W_uk)), (c.W_uv, other(c.W_uv))]
    return Op(lambda: c.call(out, exp), inputs, [out])


def _dev(model, s_q, lens):
    w = wl.small_workload(base_workload(model), B=len(lens), s_q=s_q, lens=list(lens), seed=43)
    return Dev(wl.make_inputs(w))


def _common(v):
    return [(v.q, other(v.q)), (v.cache, other(v.cache)), (v.seq_lens, v.seq_lens - 1),
            (v.page_table, v.page_table.flip(1).contiguous())]


def _weights(v):
    return [(v.W_uk, other(v.W_uk)), (v.W_uv, other(v.W_uv))]


def _causal(model, s_q, lens, noalloc=False):
    v = _dev(model, s_q, lens)
    w = v.inp.w
    out = torch.zeros((w.B, s_q, w.H, w.d_v), dtype=v.tdtype, device="cuda")
    nb = mla.mla_decode_workspace_size(v.dims, w.B, s_q, v.inp.seq_lens)
    ws = torch.full((max(nb, 256),), 255, dtype=torch.uint8, device="cuda")
    args = (v.dims, v.q, v.W_uk, v.W_uv, v.cache, v.page_table, v.seq_lens, v.inp.seq_lens, w.B, s_q, v.max_pages,
            v.inp.n_pages, out)
    call = (lambda: mla.mla_decode_absorbed_noalloc(*args)) if noalloc else (lambda: mla.mla_decode_absorbed(*args, ws))
    return Op(call, _common(v) + _weights(v), [out])


def _grouped(model, s_q, lens, prefill=False):
    v = _dev(model, s_q, lens)
    w = v.inp.w
    exp = v.expand()
    out = torch.zeros((w.B, s_q, w.H, w.d_v), dtype=v.tdtype, device="cuda")
    size, fn = (mla.mla_prefill_workspace_size, mla.mla_prefill_expanded) if prefill else \
        (mla.gqla_decode_workspace_size, mla.gqla_decode_grouped)
    ws = torch.full((max(size(v.dims, w.B, s_q, v.inp.seq_lens), 256),), 255, dtype=torch.uint8, device="cuda")
    return Op(lambda: fn(v.dims, v.q, exp, v.cache, v.page_table, v.seq_lens, v.inp.seq_lens, w.B, s_q, v.max_pages,
                         v.inp.n_pages, out, ws), _common(v) + [(exp, other(exp))], [out])


def _append(model, hidden, slots=False, projected=True):
    v = _dev(model, 1, (130, 70, 300, 65))
    d, n = v.dims, 4
    g = torch.Generator().manual_seed(44)
    rnd = lambda *s: torch.randn(s, generator=g).to(v.tdtype).cuda()  # noqa: E731
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    h = rnd(n, hidden)
    W = [rnd(d.d_c, hidden), rnd(d.d_rope, hidden)] if projected else []
    req, slot, pos = i32(3, 1, 0, 2), i32(64, 33, 129, 250), i32(7, 3000, 129, 251)
    tail = (n, v.page_table, 4, v.max_pages, v.inp.n_pages, v.cache)
    Wk = W if projected else [None, None]
    if slots:
        call = lambda: mla.mla_cache_append_slots(d, h, hidden, *Wk, req, slot, pos, *tail)  # noqa: E731
    else:
        call = lambda: mla.mla_cache_append(d, h, hidden, *Wk, req, slot, *tail)  # noqa: E731
    inputs = [(h, other(h)), (req, other(req)), (slot, i32(0, 1, 2, 3)), (pos, pos + 1), (v.cache, other(v.cache)),
              (v.page_table, v.page_table.flip(1).contiguous())] + [(x, other(x)) for x in W]
    return Op(call, inputs, [v.cache])


def _expand(model, tokens):
    v = _dev(model, 1, (130, 70, 300, 65))
    w = v.inp.w
    exp = torch.zeros((v.inp.n_pages, w.H // w.hpw, w.page, w.d_n + w.d_v), dtype=v.tdtype, device="cuda")
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    inputs = [(v.cache, other(v.cache))] + _weights(v)
    if not tokens:
        ids = i32(*range(v.inp.n_pages - 1))
        return Op(lambda: mla.gqla_expand_cache(v.dims, v.W_uk, v.W_uv, v.cache, ids, len(ids), v.inp.n_pages, exp),
                  inputs + [(ids, ids + 1)], [exp])
    req, pos = i32(3, 1, 0, 2), i32(64, 33, 129, 250)
    return Op(lambda: mla.gqla_expand_tokens(v.dims, v.W_uk, v.W_uv, v.cache, req, pos, 4, v.page_table, 4, v.max_pages,
                                             v.inp.n_pages, exp),
              inputs + [(req, other(req)), (pos, i32(1, 2, 3, 4)), (v.page_table, v.page_table.flip(1).contiguous())], [exp])


def _pool(name):
    from test_gpu_pages import Pool
    p = Pool("dsv2", (100, 150, 0, 70, 0), 20, layers=2, seed=5)
    p.both("reserve", (100, 150, 0, 78, 0))
    torch.cuda.synchronize()
    i32, tail = p.i32, p.tail()
    stale_lens = i32((64, 64, 1, 64, 1))
    state = [(p.d_lens, stale_lens), (p.d_table, p.d_table.flip(1).contiguous()), (p.d_refs, torch.ones_like(p.d_refs))]
    rows = [(p.d_lat, other(p.d_lat))]
    if name == "reserve":
        new = i32((200, 150, 90, 78, 0))
        args = [(new, i32((100, 150, 1, 78, 1)))]
        call = lambda: mla.mla_cache_reserve(p.dims, new, *tail)  # noqa: E731
    elif name == "fork":
        src, dst = i32((0, 3)), i32((2, 4))
        args = [(src, i32((1, 1))), (dst, i32((4, 2)))]
        call = lambda: mla.mla_cache_fork(p.dims, src, dst, 2, *tail, p.d_lat, None, 2)  # noqa: E731
    elif name == "release":
        req, a, b = i32((1, 3)), i32((1, 0)), i32((3, 1))
        args = [(req, i32((0, 2))), (a, i32((0, 0))), (b, i32((1, 9)))]
        call = lambda: mla.mla_cache_release(p.dims, req, a, b, 2, *tail)  # noqa: E731
    else:
        ctx, n, acc, n_acc = i32((100, 150, 0, 70, 0)), i32((0, 0, 0, 8, 0)), i32(range(40)) % 8, i32((0, 0, 0, 3, 0))
        acc[24:27] = i32((1, 4, 6))
        args = [(ctx, ctx + 1), (n, n + 1), (acc, torch.zeros_like(acc)), (n_acc, n_acc + 2)]
        call = lambda: mla.mla_cache_accept(p.dims, ctx, n, acc, n_acc, 8, *tail, p.d_lat, None, 2)  # noqa: E731
    return Op(call, state + rows + args, [p.d_lens, p.d_table, p.d_refs, p.d_lat])


FEW, MANY = (130, 70, 300, 65), tuple(66 + 7 * i for i in range(40))
OPS = {
    "append": lambda: _append("dsv2", 512),
    "append slots": lambda: _append("dsv2", 512, slots=True),
    "append general": lambda: _append("tiny", 40),
    "append projected": lambda: _append("dsv2", 576, projected=False),
    "causal": lambda: _causal("dsv2", 1, FEW),
    "causal many": lambda: _causal("dsv2", 2, MANY),
    "causal fp32": lambda: _causal("tiny", 2, FEW),
    "causal 16 heads": lambda: _causal("h16", 1, FEW),
    "no allocation": lambda: _causal("dsv2", 1, FEW, noalloc=True),
    "window": lambda: _window("dsv2", 2, FEW),
    "window many": lambda: _window("dsv2", 2, MANY),
    "window fp32": lambda: _window("tiny", 2, FEW),
    "tree": lambda: _tree("dsv2", 4, (126, 65), (4, 3)),
    "tree many": lambda: _tree("dsv2", 40, (126, 65), (40, 33)),
    "tree fp32": lambda: _tree("tiny", 9, (126, 65), (9, 5)),
    "grouped": lambda: _grouped("gqla", 2, FEW),
    "grouped fp32": lambda: _grouped("tiny", 2, FEW),
    "grouped window": lambda: _window("gqla", 2, FEW, grouped=True),
    "prefill": lambda: _grouped("gqla", 30, (130, 70), prefill=True),
    "expand": lambda: _expand("gqla", False),
    "expand fp32": lambda: _expand("tiny", False),
    "expand tokens": lambda: _expand("gqla", True),
    "reserve": lambda: _pool("reserve"),
    "fork": lambda: _pool("fork"),
    "release": lambda: _pool("release"),
    "accept": lambda: _pool("accept"),
}


@pytest.mark.parametrize("name", OPS)
def test_inputs_of_a_producer_that_triggers_early(produce, name):
    op = OPS[name]()
    op.settle(True)
    op.call()
    want = op.result()
    assert any((x != 0).any() for x in want)
    for _ in range(3):
        op.settle(False)
        produce([(t, f) for t, f, _ in op.inputs])
        op.call()
        got = op.result()
        for x, y in zip(got, want):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_the_producer_writes_late(produce):
    # a copy that is not behind the producer sees the old values, one behind it the new ones
    a = torch.zeros(1 << 10, dtype=torch.int32, device="cuda")
    b, early, late, side = torch.ones_like(a), torch.empty_like(a), torch.empty_like(a), torch.cuda.Stream()
    with torch.cuda.stream(side):
        early.copy_(a)
    torch.cuda.synchronize()
    produce([(a, b)], 5_000_000)
    with torch.cuda.stream(side):
        early.copy_(a)
    late.copy_(a)
    torch.cuda.synchronize()
    assert early.sum() == 0 and late.sum() == a.numel()
