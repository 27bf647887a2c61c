#!/usr/bin/env python3
"""Throughput of one MLA decode step on B200: cache tokens/s, achieved HBM TB/s and TFLOP/s
against the measured roofline.

A step is one pass of the decode hot path over one batch: the new tokens' cache append
(down-projection + RoPE + paged scatter), then the absorbed decode (query absorption through
W_UK, split-KV flash decode over the latent cache, split combine + W_UV) -- or, with
``--path grouped``, the append, the expansion of the touched pages and the GQA-path decode.
Inputs are seeded synthetic tensors shaped like the workload; they are resident in HBM before
the timed region (``value``), or copied from pinned host memory inside it (``e2e``).

    python bench.py [--gpus N] [--steps K] [--warmup W] [--workload 3] [--path absorbed]
    python bench.py --impl reference ...     # the CPU oracle, timed on a bounded sample

Under torchrun every rank decodes its own batch (weak scaling, no collective on the data
path); the time is the max over ranks.
"""
from __future__ import annotations

import argparse
import datetime
import hashlib
import json
import os
import statistics
import subprocess
import sys
import time

import numpy as np

ROOT = os.path.dirname(os.path.abspath(__file__))
sys.path.insert(0, ROOT)

import workloads as wl  # noqa: E402

METRIC = "MLA decode: cache tokens/s, achieved HBM TB/s & TFLOPS vs B200 roofline"
UNIT = "cache tokens/s"
L2_BYTES = 126 * 1024 * 1024
FALLBACK_PEAKS = {"hbm_gbs": 6650.0, "bf16_tflops": 1590.0, "bf16_tflops_sustained": 1400.0}
MAIN_KERNEL_SOURCES = {"absorbed": ["decode_tc.cu", "decode_simt.cu", "tc_ptx.cuh", "common.cuh"],
                       "grouped": ["decode_grouped.cu", "decode_simt.cu", "warp_mma.cuh", "tc_ptx.cuh", "common.cuh"]}


def parse():
    ap = argparse.ArgumentParser()
    ap.add_argument("--gpus", type=int, default=1)
    ap.add_argument("--steps", type=int, default=200)
    ap.add_argument("--warmup", type=int, default=5)
    ap.add_argument("--workload", default="3", choices=sorted(wl.WORKLOADS))
    ap.add_argument("--path", default=None, choices=["absorbed", "grouped"])
    ap.add_argument("--impl", default="ours", choices=["ours", "reference"])
    ap.add_argument("--cpu-seconds", type=float, default=12.0, help="CPU work budget of the oracle sample")
    ap.add_argument("--no-cpu-baseline", action="store_true")
    ap.add_argument("--no-e2e", action="store_true")
    ap.add_argument("--no-secondary", action="store_true",
                    help="skip the other workloads' kernel and step timings (reported under `secondary`)")
    ap.add_argument("--secondary-steps", type=int, default=20)
    a = ap.parse_args()
    if a.warmup < 3:
        a.warmup = 3
    if a.path is None:
        a.path = "grouped" if a.workload.startswith("5_") else "absorbed"
    return a


# --------------------------------------------------------------------------- accounting
def algorithmic(w: wl.Workload, lens: np.ndarray, path: str):
    """Algorithmic bytes/flops of the main attention kernel (per launch) and of the step.

    Absorbed: each request's cache rows are read once (d_c + d_r bf16 = 1152 B/token) plus the
    absorbed queries; flops = per visible token 2 * H * ((d_c + d_r) + d_c).  Grouped: per token
    the expanded K|V of every group plus the shared RoPE key (8320 B/token); flops per visible
    token 2 * H * ((d_n + d_r) + d_v).  Split partials are implementation overhead, not counted.
    """
    e = 2 if w.dtype == "bf16" else 4
    rows = w.B * w.s_q
    visible = int(sum(int(L) - w.s_q + j + 1 for L in lens for j in range(w.s_q)))
    tokens = int(lens.sum())
    if path == "absorbed":
        k_bytes = tokens * w.d_row * e + rows * w.H * w.d_row * e
        k_flops = visible * 2 * w.H * (w.d_row + w.d_c)
        step_bytes = (k_bytes + w.n_w * w.d_c * (w.d_n + w.d_v) * e + rows * w.H * (w.d_qk + w.d_v) * e
                      + w.d_row * w.hidden * e + rows * w.hidden * e)
        step_flops = k_flops + rows * w.H * 2 * w.d_c * (w.d_n + w.d_v) + rows * 2 * w.d_row * w.hidden
    else:
        G = w.n_w
        k_bytes = tokens * (G * (w.d_n + w.d_v) + w.d_r) * e + rows * w.H * w.d_qk * e
        k_flops = visible * 2 * w.H * (w.d_qk + w.d_v)
        # + the new tokens' expansion: W_UK and W_UV read, their latent rows read, [K_g | V_g] written
        expand_bytes = (G * w.d_c * (w.d_n + w.d_v) + rows * w.d_row + rows * G * (w.d_n + w.d_v)) * e
        step_bytes = (k_bytes + rows * w.H * w.d_v * e + w.d_row * w.hidden * e + rows * w.hidden * e
                      + expand_bytes)
        step_flops = k_flops + rows * 2 * w.d_row * w.hidden + rows * G * 2 * w.d_c * (w.d_n + w.d_v)
    return dict(kernel_bytes=k_bytes, kernel_flops=k_flops, step_bytes=step_bytes, step_flops=step_flops,
                tokens=tokens)


def load_peaks():
    p = os.path.join(ROOT, "MEASURED_PEAKS.json")
    if os.path.exists(p):
        with open(p) as f:
            d = json.load(f)
        return d, "measured"
    return dict(FALLBACK_PEAKS), "fallback"


def source_hash(names):
    h = hashlib.sha256()
    for n in names:
        p = os.path.join(ROOT, "mla_latent_kv_24_b200", "csrc", n)
        if os.path.exists(p):
            h.update(open(p, "rb").read())
    return h.hexdigest()[:16]


def recorded_traffic(path: str, workload: str):
    """Per-launch DRAM bytes of the main kernel from a committed ncu summary, if the kernel's
    source is unchanged since it was captured (the summary records the source hash)."""
    fn = os.path.join(ROOT, "profiles", f"traffic_{path}_{workload}.txt")
    if not os.path.exists(fn):
        return None
    vals = {}
    for line in open(fn):
        if ":" in line and not line.startswith("#"):
            k, v = line.split(":", 1)
            vals[k.strip()] = v.strip()
    if vals.get("source_sha256_16") != source_hash(MAIN_KERNEL_SOURCES[path]):
        return None
    try:
        return float(vals["dram_bytes_per_launch"])
    except (KeyError, ValueError):
        return None


# --------------------------------------------------------------------------- clocks
class Clocks:
    Q = ("index,clocks.sm,clocks.max.sm,power.draw,clocks_event_reasons.active,clocks_event_reasons.hw_slowdown,"
         "clocks_event_reasons.hw_thermal_slowdown,clocks_event_reasons.sw_thermal_slowdown,"
         "clocks_event_reasons.sw_power_cap")

    def __init__(self, index: int):
        self.index = index
        self.proc = None
        self.t0 = self.t1 = None

    def start(self):
        try:
            self.proc = subprocess.Popen(["nvidia-smi", "-i", str(self.index), f"--query-gpu={self.Q}",
                                          "--format=csv,noheader,nounits", "-lms", "50"],
                                         stdout=subprocess.PIPE, stderr=subprocess.DEVNULL, text=True)
        except OSError:
            self.proc = None
        time.sleep(0.15)

    def mark(self, which):
        setattr(self, which, time.time())

    def stop(self):
        if self.proc is None:
            return {"sm_mhz": None, "sm_max_mhz": None, "reasons": ["nvidia-smi unavailable"], "samples": 0}
        time.sleep(0.1)
        self.proc.terminate()
        out, _ = self.proc.communicate(timeout=10)
        rows = [r.split(",") for r in out.strip().splitlines() if r.count(",") >= 8]
        sm, mx, reasons = [], [], set()
        names = ["hw_slowdown", "hw_thermal_slowdown", "sw_thermal_slowdown", "sw_power_cap"]
        for r in rows:
            try:
                sm.append(float(r[1]))
                mx.append(float(r[2]))
            except ValueError:
                continue
            for n, v in zip(names, r[5:9]):
                if v.strip().lower() == "active":
                    reasons.add(n)
        return {"sm_mhz": statistics.median(sm) if sm else None, "sm_max_mhz": max(mx) if mx else None,
                "reasons": sorted(reasons), "samples": len(sm)}


# --------------------------------------------------------------------------- reference arm
def blas_threads():
    try:
        from threadpoolctl import threadpool_info
        n = [i.get("num_threads", 1) for i in threadpool_info() if i.get("user_api") == "blas"]
        return max(n) if n else 1
    except Exception:
        return len(os.sched_getaffinity(0))


def oracle_sample(inp: wl.DecodeInputs, budget_s: float):
    """Times the fp64 oracle on whole (request, weight group) units of the workload: all heads of
    the group and all queries of the request over the request's full cache.  Returns
    (estimated seconds for the whole workload, units timed, seconds spent, description)."""
    import oracle
    w = inp.w
    q, W_uk, W_uv = inp.q.f64(), inp.W_uk.f64(), inp.W_uv.f64()
    b = int(np.argmax(inp.seq_lens))
    L = int(inp.seq_lens[b])
    n = (L + w.page - 1) // w.page
    bits = inp.cache.data[inp.page_table[b, :n]].reshape(n * w.page, w.d_row)[:L]
    rows = wl.bf16_bits_to_f64(bits) if w.dtype == "bf16" else bits.astype(np.float64)
    spent, units = 0.0, 0
    while units == 0 or (spent < budget_s and units < w.n_w):
        g = units
        heads = list(range(g * w.hpw, (g + 1) * w.hpw))
        t0 = time.perf_counter()
        oracle.decode_request_expanded(q[b], rows, W_uk, W_uv, w.hpw, w.softmax_scale, w.rope_base, heads=heads)
        spent += time.perf_counter() - t0
        units += 1
    per_unit = spent / units
    # Units of other requests scale with their length.
    est = per_unit * w.n_w * float(inp.seq_lens.sum()) / L
    desc = (f"{units} of {w.B * w.n_w} (request, weight-group) units: request {b} (L={L}), "
            f"{units * w.hpw} heads x {w.s_q} queries over the full cache; scaled by length to the workload")
    return est, units, spent, desc


# --------------------------------------------------------------------------- ranks
def reduce_over_ranks(dist, device, times_ms, tokens):
    """Whole-job figures of a weak-scaling run: the max over ranks of each device time (every rank
    decodes its own batch; the job ends with the slowest) and the sum of the ranks' cache tokens
    (ragged workloads draw different lengths per rank).  With dist None the run has one rank."""
    import torch
    t = torch.tensor(list(times_ms), dtype=torch.float64, device=device)
    n = torch.tensor([float(tokens)], dtype=torch.float64, device=device)
    if dist is not None:
        dist.all_reduce(t, op=dist.ReduceOp.MAX)
        dist.all_reduce(n, op=dist.ReduceOp.SUM)
    return t.tolist(), n.item()


# --------------------------------------------------------------------------- secondary workloads
# Workloads timed beside the headline one, each on its own path: the absorbed path on the short
# uniform and the ragged MTP batches, the grouped (GQA) path on the GQLA batches at 8K (s_q 1, 2)
# and 64K (s_q 2) tokens.
SECONDARY = [("2", "absorbed"), ("4", "absorbed"), ("5_8192_1", "grouped"), ("5_8192_2", "grouped"),
             ("5_65536_2", "grouped")]


def device_inputs(w, seed, dev):
    """Seeded inputs of workload `w` drawn on the device (torch Philox), with the recipe's shapes and
    distributions (std 0.02 weights, std 1 latents / queries / hidden states, bf16), and the
    recipe's host-side lengths and page table.  Used for the secondary timings, whose multi-GB
    caches would take a minute to draw on the host; parity is tested on the host-drawn inputs."""
    import torch
    rng = np.random.default_rng(seed)
    lens = wl.seq_lens(w, rng)
    pt, n_pages = wl.page_table(w, lens, rng)
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    def normal(shape, std):
        return (torch.randn(shape, generator=g, device=dev, dtype=torch.float32) * std).to(torch.bfloat16)
    t = {"W_uk": normal((w.n_w, w.d_n, w.d_c), 0.02), "W_uv": normal((w.n_w, w.d_v, w.d_c), 0.02),
         "W_dkv": normal((w.d_c, w.hidden), 0.02), "W_kr": normal((w.d_r, w.hidden), 0.02),
         "q": normal((w.B, w.s_q, w.H, w.d_qk), 1.0), "h": normal((w.B * w.s_q, w.hidden), 1.0)}
    cache = torch.empty((n_pages, w.page, w.d_row), dtype=torch.bfloat16, device=dev)
    for p0 in range(0, n_pages, 4096):
        p1 = min(n_pages, p0 + 4096)
        cache[p0:p1] = normal((p1 - p0, w.page, w.d_row), 1.0)
    t["cache"] = cache
    return lens, pt, n_pages, t


def time_secondary(key, path, steps, warmup, dev, peaks):
    """Kernel and step time of one secondary workload (inputs resident in HBM, L2 flushed between
    steps when the step's bytes fit in twice the L2), with the clocks seen meanwhile."""
    import torch
    import mla_latent_kv_24_b200 as mla
    w = wl.WORKLOADS[key]
    lens, pt_np, n_pages, t = device_inputs(w, w.seed + 7919, dev)
    dims = mla.make_dims(n_heads=w.H, heads_per_group=w.hpw, d_c=w.d_c, d_rope=w.d_r, d_nope=w.d_n, d_v=w.d_v,
                         page_size=w.page, softmax_scale=w.softmax_scale, rope_base=w.rope_base, dtype=w.dtype)
    page_table = torch.from_numpy(pt_np).to(dev)
    seq_lens = torch.from_numpy(lens).to(dev)
    req_np, pos_np = wl.new_token_positions(lens, w.s_q)
    req, pos = torch.from_numpy(req_np).to(dev), torch.from_numpy(pos_np).to(dev)
    max_pages = pt_np.shape[1]
    out = torch.empty((w.B, w.s_q, w.H, w.d_v), dtype=torch.bfloat16, device=dev)
    grouped = path == "grouped"
    if grouped:
        expanded = torch.empty((n_pages, w.n_w, w.page, w.d_n + w.d_v), dtype=torch.bfloat16, device=dev)
        mla.gqla_expand_cache(dims, t["W_uk"], t["W_uv"], t["cache"], None, 0, n_pages, expanded)
        nb = mla.gqla_decode_workspace_size(dims, w.B, w.s_q, lens)
    else:
        nb = mla.mla_decode_workspace_size(dims, w.B, w.s_q, lens)
    ws = torch.empty(max(nb, 256), dtype=torch.uint8, device=dev)
    acct = algorithmic(w, lens, path)
    flush = torch.empty(256 * 1024 * 1024, dtype=torch.uint8, device=dev) if acct["step_bytes"] < 2 * L2_BYTES else None

    def step():
        mla.mla_cache_append(dims, t["h"], w.hidden, t["W_dkv"], t["W_kr"], req, pos, len(req_np), page_table, w.B,
                             max_pages, n_pages, t["cache"])
        if grouped:
            mla.gqla_expand_tokens(dims, t["W_uk"], t["W_uv"], t["cache"], req, pos, len(req_np), page_table, w.B,
                                   max_pages, n_pages, expanded)
            mla.gqla_decode_grouped(dims, t["q"], expanded, t["cache"], page_table, seq_lens, lens, w.B, w.s_q,
                                    max_pages, n_pages, out, ws)
        else:
            mla.mla_decode_absorbed(dims, t["q"], t["W_uk"], t["W_uv"], t["cache"], page_table, seq_lens, lens, w.B,
                                    w.s_q, max_pages, n_pages, out, ws)

    time.sleep(1.0)   # each secondary workload starts from an idle GPU, as the headline does
    for _ in range(warmup):
        step()
    mla.mla_get_device_status()
    # enough steps for the clock sampler (50 ms period) to see the timed region several times
    c0, c1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    c0.record()
    for _ in range(3):
        step()
    c1.record()
    torch.cuda.synchronize()
    per_step_s = max(c0.elapsed_time(c1) / 3e3, 1e-6)
    steps = int(min(4000, max(steps, 0.4 / per_step_s)))
    ev = [tuple(torch.cuda.Event(enable_timing=True) for _ in range(4)) for _ in range(steps)]
    for e in ev:
        for x in e:
            x.record()
    torch.cuda.synchronize()
    clocks = Clocks(dev.index or 0)
    clocks.start()
    # whole steps: back to back between two events unless a flush separates them
    if flush is None:
        ev[0][0].record()
        for _ in range(steps):
            step()
        ev[0][1].record()
        torch.cuda.synchronize()
        step_us = ev[0][0].elapsed_time(ev[0][1]) * 1e3 / steps
    else:
        for i in range(steps):
            flush.zero_()
            ev[i][0].record()
            step()
            ev[i][1].record()
        torch.cuda.synchronize()
        step_us = statistics.mean(s0.elapsed_time(s1) for s0, s1, _, _ in ev) * 1e3
    # the main kernel alone, bracketed by the library's profiling events
    for i in range(steps):
        if flush is not None:
            flush.zero_()
        mla.mla_set_profile_events(ev[i][2], ev[i][3])
        step()
    mla.mla_set_profile_events(None, None)
    torch.cuda.synchronize()
    clk = clocks.stop()
    mla.mla_get_device_status()
    kern_us = statistics.mean(k0.elapsed_time(k1) for _, _, k0, k1 in ev) * 1e3
    kb, kf = acct["kernel_bytes"], acct["kernel_flops"]
    t_hbm = kb / (peaks["hbm_gbs"] * 1e9)
    t_tc = kf / (peaks["bf16_tflops"] * 1e12)
    bound = "hbm" if (t_hbm >= t_tc or grouped) else "tensor"
    ks = kern_us / 1e6
    achieved = kb / ks / 1e9 if bound == "hbm" else kf / ks / 1e12
    peak = peaks["hbm_gbs"] if bound == "hbm" else peaks["bf16_tflops"]
    res = {"workload": w.name, "path": path, "kernel_us": kern_us, "step_us": step_us, "bound": bound,
           "achieved": achieved, "unit": "GB/s" if bound == "hbm" else "TFLOP/s", "frac": achieved / peak,
           "kernel_tbs": kb / ks / 1e12, "kernel_tflops": kf / ks / 1e12,
           "cache_tokens_per_s": acct["tokens"] / (step_us / 1e6), "steps": steps, "clocks": clk,
           "inputs": "device-drawn (seeded)", "start": "after 1 s idle"}
    del t, ws, out
    if grouped:
        del expanded
    torch.cuda.empty_cache()
    return res


# --------------------------------------------------------------------------- GPU arm
def run_ours(a, rank, world, local_rank):
    import torch
    import mla_latent_kv_24_b200 as mla
    dist = None
    if world > 1:
        import torch.distributed as dist
        dist.init_process_group("nccl", timeout=datetime.timedelta(seconds=300))
    torch.cuda.set_device(local_rank)
    dev = torch.device("cuda", local_rank)
    w = wl.WORKLOADS[a.workload]
    inp = wl.make_inputs(w, seed=w.seed + 1009 * rank)
    dims = mla.make_dims(n_heads=w.H, heads_per_group=w.hpw, d_c=w.d_c, d_rope=w.d_r, d_nope=w.d_n, d_v=w.d_v,
                         page_size=w.page, softmax_scale=w.softmax_scale, rope_base=w.rope_base, dtype=w.dtype)
    tdt = torch.bfloat16 if w.dtype == "bf16" else torch.float32
    T = lambda t: wl.to_torch(t, dev)  # noqa: E731
    q0, W_uk, W_uv, W_dkv, W_kr, cache, h0 = (T(inp.q), T(inp.W_uk), T(inp.W_uv), T(inp.W_dkv), T(inp.W_kr),
                                               T(inp.cache), T(inp.h))
    # A step's inputs (hidden states and queries) live in one device buffer, so the end-to-end loop
    # brings them in with one host-to-device copy.
    assert h0.dtype == q0.dtype and (h0.numel() * h0.element_size()) % 16 == 0
    hq = torch.empty(h0.numel() + q0.numel(), dtype=h0.dtype, device=dev)
    h = hq[:h0.numel()].view(h0.shape)
    q = hq[h0.numel():].view(q0.shape)
    h.copy_(h0)
    q.copy_(q0)
    del h0, q0
    page_table = torch.from_numpy(inp.page_table).to(dev)
    seq_lens = torch.from_numpy(inp.seq_lens).to(dev)
    req_np, pos_np = wl.new_token_positions(inp.seq_lens, w.s_q)
    req, pos = torch.from_numpy(req_np).to(dev), torch.from_numpy(pos_np).to(dev)
    max_pages = inp.page_table.shape[1]
    out = torch.empty((w.B, w.s_q, w.H, w.d_v), dtype=tdt, device=dev)
    grouped = a.path == "grouped"
    if grouped:
        G = w.n_w
        expanded = torch.empty((inp.n_pages, G, w.page, w.d_n + w.d_v), dtype=tdt, device=dev)
        mla.gqla_expand_cache(dims, W_uk, W_uv, cache, None, 0, inp.n_pages, expanded)
        nb = mla.gqla_decode_workspace_size(dims, w.B, w.s_q, inp.seq_lens)
    else:
        nb = mla.mla_decode_workspace_size(dims, w.B, w.s_q, inp.seq_lens)
    ws = torch.empty(max(nb, 256), dtype=torch.uint8, device=dev)
    torch.cuda.synchronize()
    acct = algorithmic(w, inp.seq_lens, a.path)
    working = acct["step_bytes"]
    flush = torch.empty(256 * 1024 * 1024, dtype=torch.uint8, device=dev) if working < 2 * L2_BYTES else None
    stream = torch.cuda.current_stream()

    def step():
        mla.mla_cache_append(dims, h, w.hidden, W_dkv, W_kr, req, pos, len(req_np), page_table, w.B, max_pages,
                             inp.n_pages, cache)
        if grouped:
            mla.gqla_expand_tokens(dims, W_uk, W_uv, cache, req, pos, len(req_np), page_table, w.B, max_pages,
                                   inp.n_pages, expanded)
            mla.gqla_decode_grouped(dims, q, expanded, cache, page_table, seq_lens, inp.seq_lens, w.B, w.s_q,
                                    max_pages, inp.n_pages, out, ws)
        else:
            mla.mla_decode_absorbed(dims, q, W_uk, W_uv, cache, page_table, seq_lens, inp.seq_lens, w.B, w.s_q,
                                    max_pages, inp.n_pages, out, ws)

    def timed_loop(K, e2e_bufs=None, profile=False):
        """K steps on the device clock.  Without a flush the steps run back to back between two
        events, so each step's kernels chain as they do in a serving loop (programmatic launches
        overlap a kernel's launch and set-up with its predecessor); with a flush, or with `profile` (the
        library's events around the main attention kernel, which break that chaining), each step
        is bracketed by its own events.  Returns (total step ms, mean kernel ms or None, wall s)."""
        per_step = flush is not None or profile
        n_ev = K if per_step else 1
        ev = [(torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True),
               torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)) for _ in range(n_ev)]
        for e in ev:           # create the events before handing them to the library
            for x in e:
                x.record()
        torch.cuda.synchronize()
        if dist:
            dist.barrier()
        torch.cuda.synchronize()
        wall0 = time.perf_counter()
        if not per_step:
            ev[0][0].record()
        for i in range(K):
            if flush is not None:
                flush.zero_()
            if per_step:
                s0, s1, k0, k1 = ev[i]
                if profile:
                    mla.mla_set_profile_events(k0, k1)
                s0.record()
            if e2e_bufs is not None:
                hq_host, out_host = e2e_bufs
                hq.copy_(hq_host, non_blocking=True)
                step()
                out_host.copy_(out, non_blocking=True)
            else:
                step()
            if per_step:
                s1.record()
        if not per_step:
            ev[0][1].record()
        mla.mla_set_profile_events(None, None)
        torch.cuda.synchronize()
        wall = time.perf_counter() - wall0
        if dist:
            dist.barrier()
        torch.cuda.synchronize()
        step_ms = sum(s0.elapsed_time(s1) for s0, s1, _, _ in ev)
        kern_ms = statistics.mean(k0.elapsed_time(k1) for _, _, k0, k1 in ev) if profile else None
        return step_ms, kern_ms, wall

    for _ in range(a.warmup):
        step()
    mla.mla_get_device_status()
    clocks = Clocks(local_rank)
    clocks.start()
    total_ms, _, wall = timed_loop(a.steps)                       # the headline: whole steps
    _, kern_ms, _ = timed_loop(a.steps, profile=True)             # the main kernel, for the roofline
    clk = clocks.stop()
    mla.mla_get_device_status()

    e2e = None
    if not a.no_e2e:
        hq_host = hq.cpu().pin_memory()
        out_host = torch.empty(out.shape, dtype=out.dtype).pin_memory()
        for _ in range(a.warmup):
            hq.copy_(hq_host, non_blocking=True)
            step()
            out_host.copy_(out, non_blocking=True)
        e2e_ms, _, _ = timed_loop(a.steps, (hq_host, out_host))
        mla.mla_get_device_status()
        e2e = (e2e_ms, hq_host.numel() * hq_host.element_size(), out_host.numel() * out_host.element_size())

    (total_ms, kern_ms, e2e_ms), tokens_all = reduce_over_ranks(dist, dev, [total_ms, kern_ms, e2e[0] if e2e else 0.0],
                                                                acct["tokens"])

    if rank == 0:
        peaks, peak_src = load_peaks()
        ms = total_ms / a.steps
        value = tokens_all * a.steps / (total_ms / 1e3)
        kb, kf = acct["kernel_bytes"], acct["kernel_flops"]
        t_hbm = kb / (peaks["hbm_gbs"] * 1e9)
        t_tc = kf / (peaks["bf16_tflops"] * 1e12)
        bound = "hbm" if (t_hbm >= t_tc or a.path == "grouped") else "tensor"
        ks = kern_ms / 1e3
        achieved = kb / ks / 1e9 if bound == "hbm" else kf / ks / 1e12
        peak = peaks["hbm_gbs"] if bound == "hbm" else peaks["bf16_tflops"]
        traffic = recorded_traffic(a.path, a.workload)
        # append, (expand,) q absorb or q RoPE carrying the plan, decode, combine; shapes without the
        # tensor-core q absorption launch the plan as a kernel of its own
        mma_absorb = w.dtype == "bf16" and (w.d_n, w.d_c, w.d_r) == (128, 512, 64)
        launches_per_step = 5 if grouped or not mma_absorb else 4
        line = {
            "metric": METRIC, "value": value, "unit": UNIT, "n_gpus": world, "steps": a.steps,
            "warmup": a.warmup, "ms_per_step": ms, "higher_is_better": True, "scaling": "weak",
            "vs_baseline": None, "dtype": w.dtype,
            "data": "synthetic: seeded normal latents/queries, N(0,0.02) weights, rounded to bf16",
            "config": {"workload": w.name, "path": a.path, "batch_per_gpu": w.B, "s_q": w.s_q,
                       "cache_len": "ragged" if w.lens is None else int(w.lens[0]),
                       "tokens_per_gpu": acct["tokens"], "heads": w.H, "heads_per_group": w.hpw,
                       "d_c": w.d_c, "d_rope": w.d_r, "page": w.page,
                       "l2": ("flushed between steps (256 MB write, outside the step events)" if flush is not None
                              else f"not flushed: {acct['step_bytes'] / 2**20:.0f} MiB per step > 2x L2")},
            "roofline": {"bound": bound, "achieved": achieved, "peak": peak,
                         "unit": "GB/s" if bound == "hbm" else "TFLOP/s", "frac": achieved / peak,
                         "traffic": traffic, "peak_source": f"{peak_src} (burst)",
                         "kernel": "main attention kernel", "kernel_ms": kern_ms,
                         "kernel_bytes": kb, "kernel_flops": kf,
                         "kernel_tbs": kb / ks / 1e12, "kernel_tflops": kf / ks / 1e12,
                         "roofline_frac": max(t_hbm, t_tc) / ks},
            "step_tbs": acct["step_bytes"] / (ms / 1e3) / 1e12, "step_tflops": acct["step_flops"] / (ms / 1e3) / 1e12,
            "gpu_launches": launches_per_step * a.steps,
            "clocks": clk,
            "impl": "ours",
        }
        if e2e is not None:
            line["e2e"] = {"value": tokens_all * a.steps / (e2e_ms / 1e3), "unit": UNIT,
                           "h2d_bytes_per_step": e2e[1], "d2h_bytes_per_step": e2e[2]}
        if world == 1 and not a.no_secondary:
            line["secondary"] = [time_secondary(k, pth, a.secondary_steps, a.warmup, dev, peaks)
                                 for k, pth in SECONDARY if k != a.workload]
        if world == 1 and not a.no_cpu_baseline:
            est, units, spent, desc = oracle_sample(inp, a.cpu_seconds)
            line["cpu_baseline"] = {"value": acct["tokens"] / est, "unit": UNIT, "cores": blas_threads(),
                                    "kind": "oracle", "sample": desc, "seconds": spent,
                                    "estimated": True}
        print(json.dumps(line), flush=True)
    if dist:
        dist.barrier()
        dist.destroy_process_group()


def run_reference(a, rank, world):
    """The CPU oracle as the reference arm: each step times one bounded sample of the workload."""
    if rank != 0:
        return
    w = wl.WORKLOADS[a.workload]
    inp = wl.make_inputs(w)
    acct = algorithmic(w, inp.seq_lens, a.path)
    per_step_budget = max(0.5, 60.0 / max(1, a.steps + a.warmup))
    for _ in range(a.warmup):
        oracle_sample(inp, 0.0)
    ests = []
    for _ in range(a.steps):
        est, units, spent, desc = oracle_sample(inp, per_step_budget)
        ests.append(est)
    est = statistics.mean(ests)
    value = acct["tokens"] / est
    line = {"metric": METRIC, "value": value, "unit": UNIT, "n_gpus": world, "steps": a.steps, "warmup": a.warmup,
            "ms_per_step": est * 1e3, "ms_per_step_kind": "estimated: the oracle timed on a sample of "
            "(request, weight-group) units, scaled by length to the whole workload",
            "higher_is_better": True, "scaling": "weak", "vs_baseline": None,
            "dtype": "f64", "data": "synthetic: seeded normal latents/queries, N(0,0.02) weights, rounded to bf16",
            "config": {"workload": w.name, "path": a.path, "batch_per_gpu": w.B, "s_q": w.s_q,
                       "cache_len": "ragged" if w.lens is None else int(w.lens[0]), "tokens_per_gpu": acct["tokens"]},
            "impl": "reference",
            "cpu_baseline": {"value": value, "unit": UNIT, "cores": blas_threads(), "kind": "oracle", "sample": desc,
                             "estimated": True},
            "e2e": {"value": value, "unit": UNIT, "h2d_bytes_per_step": 0, "d2h_bytes_per_step": 0}}
    print(json.dumps(line), flush=True)


def main():
    a = parse()
    rank = int(os.environ.get("RANK", "0"))
    world = int(os.environ.get("WORLD_SIZE", "1"))
    local_rank = int(os.environ.get("LOCAL_RANK", "0"))
    if a.impl == "reference":
        run_reference(a, rank, world)
    else:
        run_ours(a, rank, world, local_rank)


if __name__ == "__main__":
    main()
