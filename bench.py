#!/usr/bin/env python
"""Benchmark of paged FP8-KV decode attention on GB300: one JSON line on rank 0.

Metric: achieved HBM GB/s (algorithmic bytes / time; fraction of the measured peak) and
query rows/s.  Headline workload: long-context decode at 128K -- batch 8, one KV head,
16 query heads per KV head, head_dim 128, pages of 128 tokens, every context 131072,
q_len 1, per-token e4m3 K/V scales.  A step is one pa_decode call over the whole batch.
The timed region replays a CUDA graph of K back-to-back calls that cycle through several
copies of the KV cache whose total exceeds 3x the L2, so that every call reads its KV
from HBM.  The same run times the other decode workloads (dense 8K, 128K with a scalar
scale, the BF16-KV control, ragged speculative decode, sparse selected pages and the
per-token-as-decode prefill) and reports them under "workloads".

--impl reference times the fp64 CPU oracle (the reference implementation of this
build) on the host cores, on bounded samples of the same workload.
Multi-GPU: the path is replicated (independent batches per GPU, no collective); value
is the sum over ranks divided by the slowest rank's time.
"""
from __future__ import annotations

import argparse
import dataclasses
import json
import math
import os
import subprocess
import sys
import threading
import time

ROOT = os.path.dirname(os.path.abspath(__file__))
sys.path.insert(0, ROOT)

import numpy as np  # noqa: E402

METRIC = "FP8-KV paged decode: achieved HBM GB/s (% of GB300 peak), query rows/s"
FALLBACK_HBM_GBS = 6800.0


def parse():
    ap = argparse.ArgumentParser()
    ap.add_argument("--gpus", type=int, default=1)
    ap.add_argument("--steps", type=int, default=40000)
    ap.add_argument("--warmup", type=int, default=50)
    ap.add_argument("--impl", default="ours", choices=["ours", "reference"])
    ap.add_argument("--workload", default="long128k",
                    choices=["dense8k", "bf16ctl", "long128k_scalar", "long128k", "ragged",
                             "sparse", "kv_write", "prefill", "indexer"])
    ap.add_argument("--partition", type=int, default=0, help="split-K partition tokens (0 = balanced)")
    ap.add_argument("--no-e2e", action="store_true")
    ap.add_argument("--no-cpu", action="store_true")
    ap.add_argument("--tcgen05", action="store_true",
                    help="FP8 plans with one query token: run the tcgen05 kernel (PA_PLAN_TCGEN05)")
    ap.add_argument("--profile", type=int, default=0,
                    help="only run --warmup + this many direct pa_decode calls (for ncu)")
    ap.add_argument("--pools", type=int, default=0,
                    help="with --profile: this many KV copies instead of the rotation's "
                         "(ncu flushes L2 before each captured launch, so one copy keeps a "
                         "capture's device memory small)")
    ap.add_argument("--trace", action="store_true",
                    help="diagnostic: with the traced library, the per-CTA launch trace of "
                         "back-to-back calls of the decode workload (no timing line)")
    ap.add_argument("--only", action="store_true",
                    help="time the selected workload only (no 'workloads' key)")
    ap.add_argument("--extra-steps", type=int, default=200,
                    help="timed calls of each workload under 'workloads'")
    return ap.parse_args()


# DRAM bytes per launch (dram__bytes_read.sum + dram__bytes_write.sum) of the decode kernel
# from one ncu capture per workload, valid only for the kernel sources they were taken on
# (sha256 over the code, comments stripped, of the C header and the decode kernels'
# translation unit); any other code gives traffic null.
MEASURED_TRAFFIC = {
    "long128k": {"bytes": 279870976, "csrc_sha256": "f4da2999452d327622423c1087d51a776dc0a44675b57a16e000e16613a13438"},
    "long128k_scalar": {"bytes": 271453440, "csrc_sha256": "f4da2999452d327622423c1087d51a776dc0a44675b57a16e000e16613a13438"},
    "dense8k": {"bytes": 69881856, "csrc_sha256": "f4da2999452d327622423c1087d51a776dc0a44675b57a16e000e16613a13438"},
    "bf16ctl": {"bytes": 136912128, "csrc_sha256": "f4da2999452d327622423c1087d51a776dc0a44675b57a16e000e16613a13438"},
    "ragged": {"bytes": 144009728, "csrc_sha256": "f4da2999452d327622423c1087d51a776dc0a44675b57a16e000e16613a13438"},
    "sparse": {"bytes": 70716672, "csrc_sha256": "f4da2999452d327622423c1087d51a776dc0a44675b57a16e000e16613a13438"},
    "prefill": {"bytes": 11238400, "csrc_sha256": "f4da2999452d327622423c1087d51a776dc0a44675b57a16e000e16613a13438"},
}


def _code_text(path):
    """A source file without its comments and blank space, so that a comment edit keeps
    the hash of the code it was measured on."""
    import re
    with open(path, "r", encoding="utf-8") as fh:
        text = fh.read()
    text = re.sub(r"/\*.*?\*/", " ", text, flags=re.S)
    text = re.sub(r"//[^\n]*", " ", text)
    return " ".join(text.split()).encode()


def csrc_sha256():
    import hashlib
    h = hashlib.sha256()
    files = [os.path.join(ROOT, "include", "pa.h")]
    cdir = os.path.join(ROOT, "paged_fp8_kv_04_gb300", "csrc")
    # the decode kernels' translation unit (pa_api.cu and the headers it includes)
    files += [os.path.join(cdir, f) for f in sorted(os.listdir(cdir))
              if f.endswith(".cuh") or f == "pa_api.cu"]
    for f in files:
        h.update(os.path.basename(f).encode())
        h.update(_code_text(f))
    return h.hexdigest()


# The same for the quantise-and-write kernel (sha256 over the C header and pa_kv_write.cu).
# The indexer's two launches of one call (score + select), from the same kind of capture.
MEASURED_TRAFFIC_INDEXER = {"bytes": 557066496, "src_sha256": "e43c835aab743bf9b2028a35aee6fb760934dbea886c2bfbf66f29bf234743af"}
MEASURED_TRAFFIC_KV_WRITE = {"bytes": 171430144, "src_sha256": "15f09cf1b01e5aeec14716226a2a040b4e213762b700073086ae1cbe49d9a9a3"}


def index_sha256():
    import hashlib
    h = hashlib.sha256()
    for f in (os.path.join(ROOT, "include", "pa.h"),
              os.path.join(ROOT, "paged_fp8_kv_04_gb300", "csrc", "pa_index.cu")):
        h.update(os.path.basename(f).encode())
        h.update(_code_text(f))
    return h.hexdigest()


def kv_write_sha256():
    import hashlib
    h = hashlib.sha256()
    for f in (os.path.join(ROOT, "include", "pa.h"),
              os.path.join(ROOT, "paged_fp8_kv_04_gb300", "csrc", "pa_kv_write.cu")):
        h.update(os.path.basename(f).encode())
        h.update(_code_text(f))
    return h.hexdigest()


def measured_traffic(workload, sha=None):
    t = MEASURED_TRAFFIC.get(workload)
    if not t or t["bytes"] is None or t["csrc_sha256"] != (sha or csrc_sha256()):
        return None
    return t["bytes"]


def peak_hbm():
    path = os.path.join(ROOT, "MEASURED_PEAKS.json")
    try:
        with open(path) as f:
            return float(json.load(f)["hbm_gbs"]), "measured"
    except Exception:
        return FALLBACK_HBM_GBS, "fallback"


def tensor_peak():
    try:
        with open(os.path.join(ROOT, "MEASURED_PEAKS.json")) as f:
            return float(json.load(f)["bf16_tflops"])
    except Exception:
        return 1900.0


def make_workload(name):
    from paged_fp8_kv_04_gb300 import synth
    if name == "dense8k":
        p = synth.dense_8k(1)
        desc = ("dense decode 8K: batch 32, Hkv 1, group 16, head_dim 128, page 128, "
                "context 8192, q_len 1, per-token e4m3 K/V")
    elif name == "bf16ctl":
        p = synth.dense_8k(1, kv_dtype="bf16")
        desc = "dense decode 8K BF16-KV control (same shapes, dequantised values in bf16)"
    elif name == "long128k_scalar":
        p = synth.long_128k(2, scale_mode="scalar")
        desc = "long-context decode 128K: batch 8, context 131072, q_len 1, scalar e4m3 scales"
    elif name == "long128k":
        p = synth.long_128k(2, scale_mode="per_token")
        desc = "long-context decode 128K: batch 8, context 131072, q_len 1, per-token e4m3 scales"
    elif name == "prefill":
        p = synth.prefill_as_decode(6, 2048, 6144)
        desc = ("per-token-as-decode prefill: a 2048-token chunk after 6144 prompt tokens of one "
                "sequence, 2048 requests of q_len 1 sharing its block table, page 128, per-token "
                "e4m3 K/V")
    elif name == "ragged":
        p = synth.ragged_spec(3, "A")
        desc = "ragged speculative decode: 31 requests (30 x q_len 4 + 1 x q_len 1, 121 rows)"
    else:
        p = synth.sparse_selected(4)
        desc = ("sparse selected-page decode: batch 32, context 131072, 64 selected pages, "
                "q_len 1/4 (80 rows)")
    return p, desc


def algorithmic_bytes(p):
    """KV bytes of every attended (token, KV head) + Q + out + page indices."""
    from paged_fp8_kv_04_gb300 import synth
    per_tok = synth.kv_bytes_per_token(p)
    ps = p.page_size
    tokens = 0
    pages = 0
    for r in range(p.num_seqs):
        L = int(p.context_lens[r])
        if p.selected is None:
            tokens += L
            pages += (L + ps - 1) // ps
        else:
            sel = [int(x) for x in p.selected[r, :p.num_selected[r]] if x >= 0]
            tokens += sum(min(ps, L - s * ps) for s in sel if s * ps < L)
            pages += len(sel) * 2  # selected entry + block-table entry
    kv = tokens * p.num_kv_heads * per_tok
    qo = 2 * p.num_rows * p.num_kv_heads * p.group_size * p.head_dim * 2
    return kv + qo + 4 * pages * p.num_kv_heads, kv


class ClockSampler:
    """nvidia-smi samples of SM clock and throttle reasons while the timed region runs."""

    FIELDS = ("clocks.sm,clocks.max.sm,power.draw,clocks_event_reasons.active,"
              "clocks_event_reasons.hw_slowdown,clocks_event_reasons.hw_thermal_slowdown,"
              "clocks_event_reasons.sw_thermal_slowdown,clocks_event_reasons.sw_power_cap")

    def __init__(self, gpu_index):
        self.idx = gpu_index
        self.proc = None
        self.lines = []

    def start(self):
        try:
            self.proc = subprocess.Popen(
                ["nvidia-smi", "-i", str(self.idx), f"--query-gpu={self.FIELDS}",
                 "--format=csv,noheader,nounits", "-lms", "100"],
                stdout=subprocess.PIPE, stderr=subprocess.DEVNULL, text=True)
            self.thread = threading.Thread(target=self._read, daemon=True)
            self.thread.start()
        except Exception:
            self.proc = None

    def _read(self):
        for line in self.proc.stdout:
            self.lines.append(line.strip())

    def stop(self):
        if self.proc is None:
            return {"sm_mhz": None, "sm_max_mhz": None, "reasons": ["nvidia-smi unavailable"]}
        self.proc.terminate()
        try:
            self.proc.wait(timeout=5)
        except Exception:
            self.proc.kill()
        self.thread.join(timeout=2)
        sm, mx, reasons = [], [], set()
        names = ["hw_slowdown", "hw_thermal_slowdown", "sw_thermal_slowdown", "sw_power_cap"]
        for ln in self.lines:
            parts = [x.strip() for x in ln.split(",")]
            if len(parts) < 8:
                continue
            try:
                sm.append(float(parts[0]))
                mx.append(float(parts[1]))
            except ValueError:
                continue
            for n, v in zip(names, parts[4:8]):
                if v.lower() == "active":
                    reasons.add(n)
        return {"sm_mhz": float(np.median(sm)) if sm else None,
                "sm_max_mhz": max(mx) if mx else None, "reasons": sorted(reasons),
                "samples": len(sm)}


def pre_queue(stream, cycles=2_000_000):
    """A short device-side sleep (about a millisecond) ahead of the timed region's start
    event, so that the host's launch of the CUDA graph after it is over before the device
    reaches the event: the timed region holds device time only."""
    import torch
    with torch.cuda.stream(stream):
        torch.cuda._sleep(cycles)


def max_over_ranks(ms, world, dev):
    """The slowest rank's timed region (ms): every rank gets the maximum."""
    if world <= 1:
        return ms
    import torch
    import torch.distributed as dist
    t = torch.tensor([ms], dtype=torch.float64, device=dev)
    dist.all_reduce(t, op=dist.ReduceOp.MAX)
    return float(t.item())


def whole_job_rates(bytes_per_step, rows_per_step, steps, world, t_max_ms):
    """GB/s and rows/s of the whole job: every rank's steps over the slowest rank's time
    (replicas: each rank runs the same workload)."""
    sec = t_max_ms / 1e3
    return world * bytes_per_step * steps / sec / 1e9, world * rows_per_step * steps / sec


def dist_setup(args):
    world = int(os.environ.get("WORLD_SIZE", "1"))
    rank = int(os.environ.get("RANK", "0"))
    local = int(os.environ.get("LOCAL_RANK", "0"))
    return world, rank, local


def time_oracle(p, target_s=10.0):
    """The oracle, as it stands, on all host cores: whole batches of p repeated until about
    target_s of wall time.  Returns (GB/s, rows/s, seconds, cores, passes)."""
    from oracle import oracle as O
    # the oracle threads over (request, KV head) pairs: no more threads than pairs do work
    cores = max(1, min(os.cpu_count() or 1, p.num_seqs * p.num_kv_heads))
    passes = 0
    t0 = time.perf_counter()
    while True:
        O.decode(p, threads=cores)
        passes += 1
        dt = time.perf_counter() - t0
        if dt >= target_s or passes >= 200:
            break
    total, kv = algorithmic_bytes(p)
    return total * passes / dt / 1e9, p.num_rows * passes / dt, dt, cores, passes


def bench_reference_kv_write(args):
    from oracle import oracle as O
    from paged_fp8_kv_04_gb300 import synth
    c = synth.kv_write_prefill_8k(5)
    n = 16384
    sub = dataclasses.replace(c, k_new=c.k_new[:n], v_new=c.v_new[:n], slot_mapping=c.slot_mapping[:n])
    bufs = (c.k_cache.copy(), c.v_cache.copy(), c.k_scale.copy(), c.v_scale.copy())
    for _ in range(args.warmup):
        O.kv_quantize_write(sub.k_new, sub.v_new, sub.slot_mapping, *bufs)
    t0 = time.perf_counter()
    for _ in range(args.steps):
        O.kv_quantize_write(sub.k_new, sub.v_new, sub.slot_mapping, *bufs)
    dt = time.perf_counter() - t0
    value = kv_write_bytes(sub) * args.steps / dt / 1e9
    line = {
        "impl": "reference", "metric": KV_WRITE_METRIC, "value": value, "unit": "GB/s",
        "n_gpus": args.gpus, "steps": args.steps, "warmup": args.warmup,
        "ms_per_step": dt / args.steps * 1e3, "higher_is_better": True, "scaling": "weak",
        "vs_baseline": None, "dtype": "fp32 decisions, exact e4m3 rounding", "data": "synthetic",
        "config": {"workload": c.name, "sample": f"the first {n} tokens per step"},
        "cpu_baseline": {"value": value, "unit": "GB/s", "cores": 1, "kind": "oracle",
                         "sample": f"the first {n} tokens of the workload"},
        "e2e": {"value": value, "unit": "GB/s", "h2d_bytes_per_step": 0, "d2h_bytes_per_step": 0},
    }
    print(json.dumps(line), flush=True)


def bench_reference_indexer(args):
    from oracle import oracle as O
    from paged_fp8_kv_04_gb300 import synth
    ip = synth.index_decode_128k(8)
    one = dataclasses.replace(ip, q=ip.q[:1], block_table=ip.block_table[:1],
                              context_lens=ip.context_lens[:1],
                              cu_seqlens_q=np.array([0, 1], dtype=np.int32))
    for _ in range(args.warmup):
        O.index_topk(one)
    t0 = time.perf_counter()
    for _ in range(args.steps):
        O.index_topk(one)
    dt = time.perf_counter() - t0
    value = indexer_bytes(one) * args.steps / dt / 1e9
    line = {
        "impl": "reference", "metric": INDEXER_METRIC, "value": value, "unit": "GB/s",
        "n_gpus": args.gpus, "steps": args.steps, "warmup": args.warmup,
        "ms_per_step": dt / args.steps * 1e3, "higher_is_better": True, "scaling": "weak",
        "vs_baseline": None, "dtype": "f64", "data": "synthetic",
        "config": {"workload": ip.name, "sample": "request 0 (one row, 131072 positions) per step"},
        "cpu_baseline": {"value": value, "unit": "GB/s", "cores": 1, "kind": "oracle",
                         "sample": "request 0 of the workload (one row)"},
        "e2e": {"value": value, "unit": "GB/s", "h2d_bytes_per_step": 0, "d2h_bytes_per_step": 0},
    }
    print(json.dumps(line), flush=True)


def bench_reference(args):
    world, rank, _ = dist_setup(args)
    if rank != 0:
        return
    if args.workload == "kv_write":
        return bench_reference_kv_write(args)
    if args.workload == "indexer":
        return bench_reference_indexer(args)
    p, desc = make_workload(args.workload)
    # Each step: up to one request per host core (the oracle threads over (request, KV
    # head) pairs), each truncated to n leading tokens, so that the whole --steps/--warmup
    # run stays within about two minutes.
    idx = list(range(min(os.cpu_count() or 1, p.num_seqs)))
    cores = max(1, len(idx) * p.num_kv_heads)
    from oracle import oracle as O
    from paged_fp8_kv_04_gb300.synth import subset

    def sample(n):
        q = subset(p, idx)
        L = np.minimum(q.context_lens, n).astype(np.int32)
        if q.selected is not None:
            return dataclasses.replace(q, context_lens=np.maximum(L, q.q_lens))
        return dataclasses.replace(q, context_lens=np.maximum(L, q.q_lens))

    probe = sample(256)
    t0 = time.perf_counter()
    O.decode(probe, threads=cores)
    per_tok = (time.perf_counter() - t0) / 256
    budget = 120.0 / max(args.steps + args.warmup, 1)
    n = int(max(16, min(int(p.context_lens.max()), budget / max(per_tok, 1e-9))))
    q = sample(n)
    for _ in range(args.warmup):
        O.decode(q, threads=cores)
    t0 = time.perf_counter()
    for _ in range(args.steps):
        O.decode(q, threads=cores)
    dt = time.perf_counter() - t0
    total, _ = algorithmic_bytes(q)
    value = total * args.steps / dt / 1e9
    line = {
        "impl": "reference", "metric": METRIC, "value": value, "unit": "GB/s",
        "n_gpus": args.gpus, "steps": args.steps, "warmup": args.warmup,
        "ms_per_step": dt / args.steps * 1e3, "higher_is_better": True, "scaling": "weak",
        "vs_baseline": None, "dtype": "f64", "data": "synthetic",
        "config": {"workload": desc, "sample": f"{len(idx)} requests x first {n} tokens per step"},
        "rows_per_s": q.num_rows * args.steps / dt,
        "cpu_baseline": {"value": value, "unit": "GB/s", "cores": cores, "kind": "oracle",
                         "sample": f"{len(idx)} requests of the workload, each cut to its first {n} tokens"},
        "e2e": {"value": value, "unit": "GB/s", "h2d_bytes_per_step": 0, "d2h_bytes_per_step": 0},
    }
    print(json.dumps(line), flush=True)


def _decode_setup(name, dev, tcgen05=False, partition=0, pools=0):
    """Problem, plan and rotating KV copies of a decode workload on the device."""
    import torch
    from paged_fp8_kv_04_gb300 import device as dv
    p, desc = make_workload(name)
    d = dv.to_device(p, dev)
    plan = dv.plan_for(p, device=dev, partition_tokens=partition, tcgen05=tcgen05)
    total_bytes, kv_bytes = algorithmic_bytes(p)
    # Rotating copies of the KV cache (and scales) so that no call finds its KV in L2.
    l2 = torch.cuda.get_device_properties(dev).L2_cache_size
    pool_bytes = sum(d[k].numel() * d[k].element_size() for k in
                     ("k_cache", "v_cache", "k_scale", "v_scale") if d.get(k) is not None)
    touched = max(kv_bytes, 1)
    npools = max(3, int(math.ceil(3 * l2 / touched)) + 1)
    npools = min(npools, max(3, int(40e9 // max(pool_bytes, 1))))
    if pools > 0:
        npools = pools
    pools = [d] + [dict(d, **{k: d[k].clone() for k in ("k_cache", "v_cache", "k_scale", "v_scale")
                              if d.get(k) is not None}) for _ in range(npools - 1)]
    out = torch.empty(d["q"].shape, dtype=torch.bfloat16, device=dev)
    keep = []
    args_list = []
    for pd in pools:
        kw = dv.call_kwargs(p, pd)
        args_list.append(plan.args(pd["q"], pd["k_cache"], pd["v_cache"], pd["block_table"],
                                   pd["context_lens"], out=out, keep=keep, **kw))
    # the copies were made on torch's stream; the decodes run on another one
    torch.cuda.synchronize(dev)
    # the pools stay referenced for as long as the argument blocks that point into them
    return dict(p=p, desc=desc, d=d, plan=plan, total=total_bytes, kv=kv_bytes, npools=npools,
                pool_bytes=pool_bytes, l2=l2, out=out, keep=keep, args_list=args_list,
                pools=pools)


def _graph_time(w, stream, dev, K, warmup, local, world=1):
    """W direct calls, then a CUDA graph of back-to-back calls replayed until exactly K calls
    ran inside the timed region (CUDA events on the launching stream, clocks sampled)."""
    import torch
    plan, args_list, npools = w["plan"], w["args_list"], w["npools"]
    with torch.cuda.stream(stream):
        for i in range(max(warmup, 3)):
            plan.decode_args(args_list[i % npools], stream=stream)
    torch.cuda.synchronize(dev)
    assert plan.device_status() == 0
    chunk = max(c for c in range(1, min(K, 1000) + 1) if K % c == 0)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream):
        for i in range(chunk):
            plan.decode_args(args_list[i % npools], stream=stream)
    with torch.cuda.stream(stream):
        g.replay()
    torch.cuda.synchronize(dev)
    clocks = ClockSampler(local)
    clocks.start()
    time.sleep(0.3)
    if world > 1:
        import torch.distributed as dist
        dist.barrier()
    torch.cuda.synchronize(dev)
    e0 = torch.cuda.Event(enable_timing=True)
    e1 = torch.cuda.Event(enable_timing=True)
    pre_queue(stream)
    with torch.cuda.stream(stream):  # CUDAGraph.replay launches on the current stream
        e0.record(stream)
        for _ in range(K // chunk):
            g.replay()
        e1.record(stream)
    torch.cuda.synchronize(dev)
    if world > 1:
        import torch.distributed as dist
        dist.barrier()
    ms = e0.elapsed_time(e1)
    clk = clocks.stop()
    flags = plan.device_status()
    del g
    return ms, clk, flags


def _prefill_roofline(p, us_per_call):
    """The prefill rows share one sequence's pages, so the attended bytes come from L2
    many times over: the bound is the contraction, 4 * D * g flops per attended token."""
    flops = 4 * p.head_dim * p.group_size * p.num_kv_heads * int(p.context_lens.astype(np.int64).sum())
    tf = flops / (us_per_call * 1e-6) / 1e12
    tpeak = tensor_peak()
    return {"bound": "tensor", "achieved": tf, "peak": tpeak, "unit": "TFLOP/s",
            "frac": tf / tpeak, "traffic": measured_traffic("prefill"),
            "peak_kind": "measured bf16_tflops (cuBLAS burst); f16 mma.sync runs below it"}


def _extra_workloads(args, dev, stream, local, skip):
    """Every other decode workload, timed the same way, for the 'workloads' key."""
    import torch
    peak, _ = peak_hbm()
    sha = csrc_sha256()
    res = {}
    for name in ("dense8k", "long128k", "long128k_scalar", "bf16ctl", "ragged", "sparse", "prefill"):
        if name == skip:
            continue
        w = _decode_setup(name, dev)
        K = args.extra_steps
        ms, clk, flags = _graph_time(w, stream, dev, K, args.warmup, local)
        us = ms / K * 1e3
        gbs = w["total"] / (us * 1e-6) / 1e9
        info = w["plan"].info()
        entry = {"workload": w["desc"], "us_per_call": us, "gbs": gbs, "frac": gbs / peak,
                 "rows_per_s": w["p"].num_rows / (us * 1e-6), "steps": K,
                 "algorithmic_bytes_per_call": int(w["total"]),
                 "traffic": measured_traffic(name, sha), "grid_ctas": info["grid_ctas"],
                 "stages": info["stages"], "clocks": clk, "device_flags": flags}
        if name == "prefill":
            entry["roofline"] = _prefill_roofline(w["p"], us)
            entry["tokens_per_s"] = entry["rows_per_s"]
        res[name] = entry
        del w
        torch.cuda.synchronize(dev)
        torch.cuda.empty_cache()
    return res


TRACE_MARKS = ["entry", "prologue", "producer_wait", "consumer_wait", "first_tile",
                "last_tile", "partial_stored", "arrived", "merge_start", "merge_end", "exit"]


def trace_decode(args, dev, calls=16):
    """Launch trace of `calls` back-to-back decode calls (one CUDA graph, replayed after a
    warm replay) with the traced library: for each mark, the median over calls of the
    median and of the latest CTA, in us after the previous call's last CTA exited."""
    import ctypes
    import torch
    from paged_fp8_kv_04_gb300 import binding, build as libbuild
    binding._lib = binding.lib(libbuild.build(trace=True))
    w = _decode_setup(args.workload, dev, tcgen05=False, partition=args.partition)
    plan, args_list, npools = w["plan"], w["args_list"], w["npools"]
    stream = torch.cuda.Stream(device=dev)
    with torch.cuda.stream(stream):
        for i in range(max(args.warmup, 3)):
            plan.decode_args(args_list[i % npools], stream=stream)
    torch.cuda.synchronize(dev)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream):
        for i in range(calls):
            plan.decode_args(args_list[i % npools], stream=stream)
    for _ in range(2):
        pre_queue(stream)
        with torch.cuda.stream(stream):
            g.replay()
        torch.cuda.synchronize(dev)
    assert plan.device_status() == 0
    buf = np.zeros((16, 1024, 16), dtype=np.uint64)
    st = binding.lib().pa_debug_trace(ctypes.c_void_p(buf.ctypes.data), buf.nbytes)
    if st != 0:
        raise RuntimeError(f"pa_debug_trace: status {st}")
    grid = plan.info()["grid_ctas"]
    t = buf[:, :grid, :].astype(np.int64)
    t = t[np.argsort(t[:, 0, 11])]                 # slots in launch order
    busy = t[-1, :, 13] > t[-1, :, 12]
    ends = t[:, :, 10].max(axis=1)
    stats = {m: ([], []) for m in TRACE_MARKS}
    for c in range(1, t.shape[0]):                 # calls that follow another back to back
        rel = (t[c] - ends[c - 1]) / 1e3
        for k, m in enumerate(TRACE_MARKS):
            v = rel[busy, k]
            v = v[t[c, busy, k] >= t[c, busy, 0]]     # marks this call reached
            if v.size:
                stats[m][0].append(float(np.median(v)))
                stats[m][1].append(float(np.max(v)))
    line = {"trace": args.workload, "grid_ctas": int(grid), "busy_ctas": int(busy.sum()),
            "calls": int(t.shape[0] - 1),
            "us_per_call": round(float(np.median(np.diff(ends[1:]))) / 1e3, 2),
            "after_previous_call_us": {m: [round(float(np.median(a)), 2), round(float(np.median(b)), 2)]
                                       for m, (a, b) in stats.items() if a},
            "cols": "median CTA, latest CTA (medians over calls)"}
    print(json.dumps(line), flush=True)


def bench_ours(args):
    import torch
    world, rank, local = dist_setup(args)
    if world > 1:
        import torch.distributed as dist
        dist.init_process_group("nccl")
    torch.cuda.set_device(local)
    dev = torch.device("cuda", local)

    import __graft_entry__
    if rank == 0 or world == 1:
        __graft_entry__.build()
    if world > 1:
        import torch.distributed as dist
        dist.barrier()
        __graft_entry__.build()
    from paged_fp8_kv_04_gb300 import device as dv

    if args.workload == "kv_write":
        return bench_kv_write(args, dev, rank, world, local)
    if args.workload == "indexer":
        return bench_indexer(args, dev, rank, world, local)
    if args.trace:
        return trace_decode(args, dev)
    w = _decode_setup(args.workload, dev, tcgen05=args.tcgen05, partition=args.partition,
                      pools=args.pools if args.profile else 0)
    p, desc, plan, d, out, keep = w["p"], w["desc"], w["plan"], w["d"], w["out"], w["keep"]
    total_bytes, npools, args_list = w["total"], w["npools"], w["args_list"]
    pool_bytes, l2 = w["pool_bytes"], w["l2"]
    stream = torch.cuda.Stream(device=dev)

    if args.profile:
        with torch.cuda.stream(stream):
            for i in range(args.warmup + args.profile):
                plan.decode_args(args_list[i % npools], stream=stream)
        torch.cuda.synchronize(dev)
        print(json.dumps({"profile_calls": args.warmup + args.profile,
                          "device_flags": plan.device_status()}), flush=True)
        return

    K = args.steps
    ms, clk, flags = _graph_time(w, stream, dev, K, args.warmup, local, world)

    # per-launch time of direct (non-graph) calls, for reference
    e2 = torch.cuda.Event(enable_timing=True)
    e3 = torch.cuda.Event(enable_timing=True)
    nd = min(max(K, 20), 2000)
    with torch.cuda.stream(stream):
        e2.record(stream)
        for i in range(nd):
            plan.decode_args(args_list[i % npools], stream=stream)
        e3.record(stream)
    torch.cuda.synchronize(dev)
    direct_us = e2.elapsed_time(e3) / nd * 1e3

    t_max = max_over_ranks(ms, world, dev)
    value, rows_s = whole_job_rates(total_bytes, p.num_rows, K, world, t_max)
    us_per_call = ms / K * 1e3

    # end to end through the C ABI: pinned host inputs -> device, decode, output -> host
    e2e = None
    if not args.no_e2e:
        host = {k: v.cpu().pin_memory() for k, v in d.items()}
        dbuf = {k: torch.empty_like(v) for k, v in d.items()}
        hout = torch.empty(out.shape, dtype=out.dtype).pin_memory()
        kw = dv.call_kwargs(p, dbuf)
        a_e2e = plan.args(dbuf["q"], dbuf["k_cache"], dbuf["v_cache"], dbuf["block_table"],
                          dbuf["context_lens"], out=out, keep=keep, **kw)
        h2d = sum(v.numel() * v.element_size() for v in host.values())
        d2h = out.numel() * out.element_size()
        steps_e2e = 30
        with torch.cuda.stream(stream):
            for it in range(steps_e2e + 3):
                if it == 3:
                    torch.cuda.synchronize(dev)
                    t0 = time.perf_counter()
                for k in host:
                    dbuf[k].copy_(host[k], non_blocking=True)
                plan.decode_args(a_e2e, stream=stream)
                hout.copy_(out, non_blocking=True)
            torch.cuda.synchronize(dev)
        dt = (time.perf_counter() - t0) / steps_e2e
        e2e = {"value": world * total_bytes / dt / 1e9, "unit": "GB/s",
               "h2d_bytes_per_step": int(h2d), "d2h_bytes_per_step": int(d2h),
               "ms_per_step": dt * 1e3}
        del host, dbuf, hout

    info = plan.info()
    extra = None
    if not args.only and args.partition == 0 and not args.tcgen05:
        del w, d, out, keep, args_list, plan
        torch.cuda.empty_cache()
        extra = _extra_workloads(args, dev, stream, local, args.workload)

    if rank != 0:
        return
    peak, peak_kind = peak_hbm()
    achieved = total_bytes / (us_per_call * 1e-6) / 1e9
    cpu = None
    if not args.no_cpu:
        gbs, rps, dt, cores, passes = time_oracle(p)
        cpu = {"value": gbs, "unit": "GB/s", "cores": cores, "kind": "oracle",
               "sample": f"the full batch ({p.num_rows} rows) {passes} times, {dt:.1f} s wall",
               "rows_per_s": rps}
    line = {
        "metric": METRIC, "value": value, "unit": "GB/s", "n_gpus": world, "steps": K,
        "warmup": args.warmup, "ms_per_step": t_max / K, "higher_is_better": True,
        "scaling": "weak", "vs_baseline": None, "dtype": "e4m3 KV, f16 mma, f32 accumulate"
        if p.kv_dtype == "fp8" else "bf16 mma, f32 accumulate", "data": "synthetic",
        "config": {"workload": desc, "l2": f"{npools} rotating KV copies ({npools * pool_bytes / 1e6:.0f} MB vs L2 {l2 / 1e6:.0f} MB)",
                   "timed": "CUDA graph replay of back-to-back pa_decode calls",
                   "kernel": "tcgen05" if info["kernel"] == 1 else "mma.sync",
                   "grid_ctas": info["grid_ctas"], "stages": info["stages"],
                   "partition_tokens": args.partition},
        "pct_of_peak": 100.0 * achieved / peak,
        "rows_per_s": rows_s,
        "us_per_call_graph": us_per_call, "us_per_call_direct": direct_us,
        "algorithmic_bytes_per_call": int(total_bytes),
        "roofline": {"bound": "hbm", "achieved": achieved, "peak": peak, "unit": "GB/s",
                     "frac": achieved / peak, "traffic": measured_traffic(args.workload),
                     "peak_kind": f"{peak_kind} hbm_gbs (copy)"},
        "cpu_baseline": cpu, "e2e": e2e, "gpu_launches": K, "clocks": clk,
        "device_flags": flags,
    }
    if args.workload == "prefill":
        line["roofline"] = _prefill_roofline(p, us_per_call)
        line["attended_bytes_per_s_note"] = "value counts attended KV bytes, most served from L2"
        line["tokens_per_s"] = rows_s
    if extra is not None:
        line["workloads"] = extra
    print(json.dumps(line), flush=True)


KV_WRITE_METRIC = "FP8 KV quantise-and-write: achieved HBM GB/s (% of GB300 peak)"
INDEXER_METRIC = "Indexer block score + top-k: achieved HBM GB/s (% of GB300 peak)"


def indexer_bytes(ip):
    """Index keys (128 B) and scales (4 B) of every position of every request, read once
    per request; queries, page scores, selections and the block table."""
    ps = ip.k_cache.shape[1]
    pos = int(ip.context_lens.astype(np.int64).sum())
    pages = int(((ip.context_lens.astype(np.int64) + ps - 1) // ps).sum())
    per = 128 + (4 if ip.k_scale is not None else 0)
    R, H = ip.q.shape[:2]
    out = R * ip.block_table.shape[1] * 4 + R * ip.topk * 4 + R * 4
    return pos * per + R * H * 128 * 2 + out + pages * 4


def bench_indexer(args, dev, rank, world, local):
    """pa_index_topk on the sparse decode's indexer step (batch 32, context 131072)."""
    import torch
    from paged_fp8_kv_04_gb300 import binding as B, synth
    ip = synth.index_decode_128k(8)
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)
    q, kc = t(ip.q.view(np.int16)), t(ip.k_cache)
    ks = None if ip.k_scale is None else t(ip.k_scale)
    bt, L, cu = t(ip.block_table), t(ip.context_lens), t(ip.cu_seqlens_q)
    R, stride = ip.num_rows, ip.block_table.shape[1]
    sel = torch.empty((R, ip.topk), dtype=torch.int32, device=dev)
    nsel = torch.empty((R,), dtype=torch.int32, device=dev)
    scores = torch.empty((R, stride), dtype=torch.float32, device=dev)
    maxq = int(np.diff(ip.cu_seqlens_q).max())
    a = B.index_args(q, kc, ks, bt, L, cu, sel, nsel, scores, topk=ip.topk, max_q_len=maxq,
                     sm_scale=ip.sm_scale)
    total = indexer_bytes(ip)
    stream = torch.cuda.Stream(device=dev)
    with torch.cuda.stream(stream):
        for _ in range(max(args.warmup, 3) + args.profile):
            B.index_topk(a, stream=stream)
    torch.cuda.synchronize(dev)
    if args.profile:
        print(json.dumps({"profile_calls": max(args.warmup, 3) + args.profile}), flush=True)
        return
    K = args.steps
    chunk = max(c_ for c_ in range(1, min(K, 100) + 1) if K % c_ == 0)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream):
        for _ in range(chunk):
            B.index_topk(a, stream=stream)
    with torch.cuda.stream(stream):
        g.replay()
    torch.cuda.synchronize(dev)
    clocks = ClockSampler(local)
    clocks.start()
    time.sleep(0.3)
    e0 = torch.cuda.Event(enable_timing=True)
    e1 = torch.cuda.Event(enable_timing=True)
    pre_queue(stream)
    with torch.cuda.stream(stream):
        e0.record(stream)
        for _ in range(K // chunk):
            g.replay()
        e1.record(stream)
    torch.cuda.synchronize(dev)
    ms = e0.elapsed_time(e1)
    clk = clocks.stop()
    us = ms / K * 1e3
    achieved = total / (us * 1e-6) / 1e9
    if rank != 0:
        return
    cpu = None
    if not args.no_cpu:
        from oracle import oracle as O
        one = dataclasses.replace(ip, q=ip.q[:1], block_table=ip.block_table[:1],
                                  context_lens=ip.context_lens[:1],
                                  cu_seqlens_q=np.array([0, 1], dtype=np.int32))
        t0 = time.perf_counter()
        passes = 0
        while time.perf_counter() - t0 < 5.0:
            O.index_topk(one)
            passes += 1
        dt = time.perf_counter() - t0
        cpu = {"value": indexer_bytes(one) * passes / dt / 1e9, "unit": "GB/s", "cores": 1,
               "kind": "oracle", "sample": f"request 0 (one row, 131072 positions), {passes} times, {dt:.1f} s"}
    peak, peak_kind = peak_hbm()
    line = {
        "metric": INDEXER_METRIC, "value": achieved, "unit": "GB/s", "n_gpus": world,
        "steps": K, "warmup": args.warmup, "ms_per_step": ms / K, "higher_is_better": True,
        "scaling": "weak", "vs_baseline": None, "dtype": "e4m3 keys, f32 dot products",
        "data": "synthetic",
        "config": {"workload": ip.name, "l2": "one 554 MB index cache (> 3 x L2)",
                   "timed": "CUDA graph replay of back-to-back pa_index_topk calls (two launches each)"},
        "us_per_call_graph": us, "rows_per_s": R / (us * 1e-6),
        "algorithmic_bytes_per_call": int(total),
        "roofline": {"bound": "hbm", "achieved": achieved, "peak": peak, "unit": "GB/s",
                     "frac": achieved / peak,
                     "traffic": (MEASURED_TRAFFIC_INDEXER["bytes"]
                                 if MEASURED_TRAFFIC_INDEXER["src_sha256"] == index_sha256() else None),
                     "peak_kind": f"{peak_kind} hbm_gbs (copy)"},
        "cpu_baseline": cpu, "e2e": None, "gpu_launches": 2 * K, "clocks": clk,
    }
    print(json.dumps(line), flush=True)


def kv_write_bytes(c):
    """bf16 K and V in, e4m3 codes and fp32 scales out, one int64 slot per token."""
    T, Hkv, D = c.k_new.shape
    live = int((c.slot_mapping >= 0).sum())
    return live * Hkv * (2 * 2 * D + 2 * (D + 4)) + T * 8


def bench_kv_write(args, dev, rank, world, local):
    """pa_kv_quantize_write over the dense-8K batch written at once (262144 tokens)."""
    import torch
    from paged_fp8_kv_04_gb300 import binding as B, synth
    c = synth.kv_write_prefill_8k(5)
    desc = c.name
    to = lambda a: (torch.from_numpy(a).view(torch.int16) if a.dtype == np.uint16
                    else torch.from_numpy(a)).to(dev)
    k0, v0 = to(c.k_new), to(c.v_new)
    ins = [(k0, v0), (k0.clone(), v0.clone())]   # two 134-MB input sets alternate (> L2)
    slots = to(c.slot_mapping)
    kc, vc, ks, vs = to(c.k_cache), to(c.v_cache), to(c.k_scale), to(c.v_scale)
    total_bytes = kv_write_bytes(c)
    alist = [B.kv_write_args(k, v, slots, kc, vc, ks, vs) for k, v in ins]
    stream = torch.cuda.Stream(device=dev)
    if args.profile:
        with torch.cuda.stream(stream):
            for i in range(args.warmup + args.profile):
                B.kv_quantize_write(None, None, None, kc, None, None, None, stream=stream,
                                    args=alist[i % 2])
        torch.cuda.synchronize(dev)
        print(json.dumps({"profile_calls": args.warmup + args.profile}), flush=True)
        return
    with torch.cuda.stream(stream):
        for i in range(max(args.warmup, 3)):
            B.kv_quantize_write(None, None, None, kc, None, None, None, stream=stream,
                                args=alist[i % 2])
    torch.cuda.synchronize(dev)
    K = args.steps
    chunk = max(c_ for c_ in range(1, min(K, 200) + 1) if K % c_ == 0)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream):
        for i in range(chunk):
            B.kv_quantize_write(None, None, None, kc, None, None, None, stream=stream,
                                args=alist[i % 2])
    with torch.cuda.stream(stream):
        g.replay()
    torch.cuda.synchronize(dev)
    clocks = ClockSampler(local)
    clocks.start()
    time.sleep(0.3)
    e0 = torch.cuda.Event(enable_timing=True)
    e1 = torch.cuda.Event(enable_timing=True)
    pre_queue(stream)
    with torch.cuda.stream(stream):
        e0.record(stream)
        for _ in range(K // chunk):
            g.replay()
        e1.record(stream)
    torch.cuda.synchronize(dev)
    ms = e0.elapsed_time(e1)
    clk = clocks.stop()
    us = ms / K * 1e3
    achieved = total_bytes / (us * 1e-6) / 1e9
    e2e = None
    if not args.no_e2e:
        hk, hv, hs = (x.cpu().pin_memory() for x in (k0, v0, slots))
        hkc = torch.empty(kc.shape, dtype=kc.dtype).pin_memory()
        hks = torch.empty(ks.shape, dtype=ks.dtype).pin_memory()
        dk, dv_, ds = torch.empty_like(k0), torch.empty_like(v0), torch.empty_like(slots)
        a = B.kv_write_args(dk, dv_, ds, kc, vc, ks, vs)
        steps = 10
        with torch.cuda.stream(stream):
            for it in range(steps + 2):
                if it == 2:
                    torch.cuda.synchronize(dev)
                    t0 = time.perf_counter()
                dk.copy_(hk, non_blocking=True)
                dv_.copy_(hv, non_blocking=True)
                ds.copy_(hs, non_blocking=True)
                B.kv_quantize_write(None, None, None, kc, None, None, None, stream=stream, args=a)
                hkc.copy_(kc, non_blocking=True)
                hks.copy_(ks, non_blocking=True)
            torch.cuda.synchronize(dev)
        dt = (time.perf_counter() - t0) / steps
        e2e = {"value": total_bytes / dt / 1e9, "unit": "GB/s",
               "h2d_bytes_per_step": int(sum(x.numel() * x.element_size() for x in (hk, hv, hs))),
               "d2h_bytes_per_step": int(hkc.numel() + hks.numel() * 4),
               "ms_per_step": dt * 1e3,
               "note": "K codes and K scales read back; V stays on the device"}
    if rank != 0:
        return
    cpu = None
    if not args.no_cpu:
        from oracle import oracle as O
        n = 16384
        sub = dataclasses.replace(c, k_new=c.k_new[:n], v_new=c.v_new[:n],
                                  slot_mapping=c.slot_mapping[:n])
        kcc, vcc, kss, vss = c.k_cache.copy(), c.v_cache.copy(), c.k_scale.copy(), c.v_scale.copy()
        t0 = time.perf_counter()
        passes = 0
        while time.perf_counter() - t0 < 5.0:
            O.kv_quantize_write(sub.k_new, sub.v_new, sub.slot_mapping, kcc, vcc, kss, vss)
            passes += 1
        dt = time.perf_counter() - t0
        cpu = {"value": kv_write_bytes(sub) * passes / dt / 1e9, "unit": "GB/s", "cores": 1,
               "kind": "oracle", "sample": f"the first {n} tokens, {passes} times, {dt:.1f} s"}
    peak, peak_kind = peak_hbm()
    line = {
        "metric": KV_WRITE_METRIC, "value": achieved, "unit": "GB/s", "n_gpus": world,
        "steps": K, "warmup": args.warmup, "ms_per_step": ms / K, "higher_is_better": True,
        "scaling": "weak", "vs_baseline": None, "dtype": "bf16 in, fp32 scale, e4m3 out",
        "data": "synthetic",
        "config": {"workload": desc, "l2": "two 134 MB input sets alternate (> L2)",
                   "timed": "CUDA graph replay of back-to-back pa_kv_quantize_write calls"},
        "us_per_call_graph": us, "algorithmic_bytes_per_call": int(total_bytes),
        "roofline": {"bound": "hbm", "achieved": achieved, "peak": peak, "unit": "GB/s",
                     "frac": achieved / peak,
                     "traffic": (MEASURED_TRAFFIC_KV_WRITE["bytes"]
                                 if MEASURED_TRAFFIC_KV_WRITE["bytes"] is not None and
                                 MEASURED_TRAFFIC_KV_WRITE["src_sha256"] == kv_write_sha256()
                                 else None),
                     "peak_kind": f"{peak_kind} hbm_gbs (copy)"},
        "cpu_baseline": cpu, "e2e": e2e, "gpu_launches": K, "clocks": clk,
    }
    print(json.dumps(line), flush=True)


def main():
    args = parse()
    if args.impl == "reference":
        bench_reference(args)
    else:
        bench_ours(args)


if __name__ == "__main__":
    main()
