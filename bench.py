#!/usr/bin/env python3
"""Benchmark of the two-stage draft LM head on one GB300 (or N replicas).

Workload: the Llama-3-8B-shaped head (n=128256, d=4096, r=256) with rows
shuffled by a seeded permutation and the fused local Top-k (tile=256,
k_tile=2 -> 1002 candidates per hidden vector), M hidden vectors per call.
A step is one lmhead_two_stage call: projection, fused score + tile top-k,
gather of W[ids], exact logits, softmax. Inputs are synthetic and seeded
(see synth/), resident in HBM before timing; 4 rotating copies of every
input (> 2x the 129 MB L2) keep each step's reads cold.

  python bench.py [--gpus N] [--steps K] [--warmup W] [--M 64] [--impl ours|reference]

Prints one JSON line on stdout (and the tables beside it - the sweep over M, every
configuration, the steps after q, the other routes - as one on stderr). Under torchrun (N > 1) every rank runs an independent
replica on its own hidden vectors (no collective on the data path) and rank
0 prints the aggregate over ranks with the max time over ranks.
"""
from __future__ import annotations

import argparse
import json
import os
import statistics
import subprocess
import sys
import time

import numpy as np

ROOT = os.path.dirname(os.path.abspath(__file__))
sys.path.insert(0, ROOT)

import synth  # noqa: E402

METRIC = "two-stage LM-head hidden vecs/s (n=128256,d=4096,r=256); % of HBM roofline"
WORKLOAD = synth.workload(2)
NROT = 4


def parse():
    p = argparse.ArgumentParser()
    p.add_argument("--gpus", type=int, default=1)
    p.add_argument("--steps", type=int, default=400)
    p.add_argument("--warmup", type=int, default=20)
    p.add_argument("--M", type=int, default=64)
    p.add_argument("--impl", choices=("ours", "reference"), default="ours")
    p.add_argument("--no-sweep", action="store_true")
    p.add_argument("--no-configs", action="store_true",
                   help="skip the per-configuration table (configs 1-4, all modes and heads)")
    p.add_argument("--no-cpu", action="store_true")
    p.add_argument("--cpu-sample", type=int, default=-1, help=argparse.SUPPRESS)
    p.add_argument("--rotations", type=int, default=NROT,
                   help="input copies cycled through (>= 4 keeps every read cold in L2)")
    return p.parse_args()


# ---------------------------------------------------------------- inputs
def head_inputs(wl=WORKLOAD):
    """Seeded head + its Freq-aware SVD factors (offline prep, cached on disk),
    with the factor rows shuffled by the workload's permutation."""
    from draft_lm_head_gb300 import prep

    def builder():
        W = synth.make_head(wl.n, wl.d, wl.head_seed_index)
        counts = synth.zipf_counts(wl.n, wl.zipf_s, wl.head_seed_index)
        fac = prep.freq_aware_factors(W, counts, wl.r)
        return {"W": W, "counts": counts, "A": fac["A"], "B": fac["B"]}

    key = f"head:{wl.head_seed_index}:{wl.n}:{wl.d}:{wl.r}:{wl.zipf_s}"
    head = dict(synth.head_cache(key, builder))
    tok = synth.shuffle_perm(wl.n, wl.index) if wl.shuffle else np.arange(wl.n, dtype=np.int32)
    head["A"] = np.ascontiguousarray(head["A"][tok])
    head["tok"] = tok
    return head


def workload_config(M, world, nrot):
    """The workload both arms report: the headline head at M hidden vectors."""
    wl = WORKLOAD
    K = (wl.n // wl.T) * wl.k_tile + min(wl.k_tile, wl.n % wl.T)
    return {"workload": "llama3-8b-shaped head n=128256 d=4096 r=256, shuffled rows, "
                        "fused local top-k tile=256 k_tile=2",
            "n": wl.n, "d": wl.d, "r": wl.r, "M": M, "mode": "local", "tile": wl.T,
            "k_tile": wl.k_tile, "candidates": K,
            "l2": f"{nrot} rotating copies of every input" + (" (> 2x L2)" if nrot >= 4 else ""),
            "launch": "CUDA graph replay of library calls",
            "parallelism": f"replicas x{world} (independent hidden vectors)"}


def hidden(W, M, rank):
    h, _ = synth.make_hidden(W, M, WORKLOAD.index, stream_offset=rank)
    return h


def ncu_traffic(kernel, M):
    """DRAM bytes per launch of `kernel` from the committed ncu capture, or None
    when the capture was taken at another M or the kernel's source changed."""
    import hashlib
    path = os.path.join(ROOT, "profiles", "ncu_traffic.json")
    if not os.path.exists(path):
        return None
    with open(path) as fh:
        rec = json.load(fh).get(kernel)
    if not rec or rec.get("M") != M:
        return None
    src = os.path.join(ROOT, rec["source"])
    if not os.path.exists(src):
        return None
    with open(src, "rb") as fh:
        if hashlib.sha1(fh.read()).hexdigest() != rec["source_sha1"]:
            return None
    return int(rec["dram_bytes"])


def peaks():
    path = os.path.join(ROOT, "MEASURED_PEAKS.json")
    if os.path.exists(path):
        with open(path) as fh:
            pk = json.load(fh)
        return float(pk["hbm_gbs"]), "measured"
    return 6800.0, "fallback"


def pstats(xs):
    """median, p10 and p90 of a list of per-call times (us)."""
    xs = sorted(xs)
    n = len(xs)

    def q(p):
        return xs[min(n - 1, int(round(p * (n - 1))))]
    return {"median": round(statistics.median(xs), 2), "p10": round(q(0.1), 2),
            "p90": round(q(0.9), 2), "calls": n}


def per_call_us(torch, fns, reps=100, warm=20, graph=False):
    """Device time of each of `reps` calls, with events around each call on
    the current stream; call i runs fns[i % len(fns)] (one per input copy, so
    consecutive calls read different copies: cold L2). graph=True replays a
    CUDA graph of the same call instead of launching it from the host."""
    run = [g.replay for g in (make_graph(torch, f) for f in fns)] if graph else fns
    n = len(run)
    for i in range(max(warm, n)):
        run[i % n]()
    torch.cuda.synchronize()
    ev = [(torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True))
          for _ in range(reps)]
    for i, (a, b) in enumerate(ev):
        a.record()
        run[i % n]()
        b.record()
    torch.cuda.synchronize()
    return [a.elapsed_time(b) * 1e3 for a, b in ev]


# ---------------------------------------------------------------- clocks
class ClockSampler:
    FIELDS = ("clocks.sm,clocks.max.sm,clocks_event_reasons.active,"
              "clocks_event_reasons.hw_slowdown,clocks_event_reasons.hw_thermal_slowdown,"
              "clocks_event_reasons.sw_thermal_slowdown,clocks_event_reasons.sw_power_cap")

    def __init__(self, index):
        self.index = index
        self.proc = None

    def start(self):
        try:
            self.proc = subprocess.Popen(
                ["nvidia-smi", "-i", str(self.index), f"--query-gpu={self.FIELDS}",
                 "--format=csv,noheader,nounits", "-lms", "100"],
                stdout=subprocess.PIPE, stderr=subprocess.DEVNULL, text=True)
        except OSError:
            self.proc = None

    def stop(self):
        if self.proc is None:
            return None
        self.proc.terminate()
        try:
            out, _ = self.proc.communicate(timeout=5)
        except subprocess.TimeoutExpired:
            self.proc.kill()
            out, _ = self.proc.communicate()
        sm, mx, reasons = [], [], set()
        names = ("hw_slowdown", "hw_thermal_slowdown", "sw_thermal_slowdown", "sw_power_cap")
        for line in out.strip().splitlines():
            parts = [x.strip() for x in line.split(",")]
            if len(parts) < 7:
                continue
            try:
                sm.append(float(parts[0]))
                mx.append(float(parts[1]))
            except ValueError:
                continue
            for nm, v in zip(names, parts[3:7]):
                if v.lower() == "active":
                    reasons.add(nm)
        if not sm:
            return {"sm_mhz": None, "sm_max_mhz": None, "reasons": [], "samples": 0}
        return {"sm_mhz": statistics.median(sm), "sm_max_mhz": max(mx),
                "reasons": sorted(reasons), "samples": len(sm)}


# ---------------------------------------------------------------- CPU oracle timing
def oracle_sample_rate(head, h_bits, budget_s=12.0, rows=4):
    """Time the oracle as it stands on `rows` hidden vectors of the workload,
    repeated for about `budget_s`; returns (vecs/s, cores, sample text)."""
    import oracle as O
    wl = WORKLOAD
    A64 = O.bf16_bits_to_f64(head["A"])
    B64 = O.bf16_bits_to_f64(head["B"])
    tok = head["tok"]
    h64 = O.bf16_bits_to_f64(h_bits[:rows])

    def one_pass():
        u = O.project_u(B64, h64)
        S = O.lowrank_scores(A64, u)
        for m in range(rows):
            ids, _ = O.local_topk(S[m], tok, wl.T, wl.k_tile)
            Wr = O.bf16_bits_to_f64(head["W"][ids])
            L = O.candidate_logits(Wr, h64[m], np.arange(ids.size))
            O.candidate_softmax(L)

    done, t0 = 0, time.perf_counter()
    while True:
        one_pass()
        done += rows
        if time.perf_counter() - t0 >= budget_s:
            break
    dt = time.perf_counter() - t0
    cores = len(os.sched_getaffinity(0))
    return done / dt, cores, f"{done} hidden vectors ({rows} per pass) of the M={rows} slice, {dt:.1f} s"


# ---------------------------------------------------------------- GPU arm
def make_graph(torch, fn):
    """Capture fn() (a sequence of library calls on the current stream)."""
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        fn()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fn()
    torch.cuda.synchronize()
    return g


def max_over_ranks(x, world, device):
    """The largest of every rank's x (a timing in ms); x itself when alone."""
    if world <= 1:
        return float(x)
    import torch
    import torch.distributed as dist
    t = torch.tensor([float(x)], dtype=torch.float64, device=device)
    dist.all_reduce(t, op=dist.ReduceOp.MAX)
    return float(t.item())


def aggregate_rate(world, rows_per_rank, steps, ms):
    """Whole-job hidden vectors/s: every rank's rows of every step over the
    slowest rank's time."""
    return world * rows_per_rank * steps / (ms / 1e3)


def time_after_q(torch, L, out, hbm, reps=50):
    """Graph-replayed timings of the steps that consume q: EAGLE-2 draft
    selection (top-8 per row with path values and a Gumbel-max draw) on the
    headline call's q, and chain verification of 8 chains of 4 drafts against
    synthetic dense target rows of the full vocabulary (seeded; the residual is
    drawn wherever a draft is rejected)."""
    ids, _, q = out
    M, K = q.shape
    g = torch.Generator(device="cuda")
    g.manual_seed(1234)
    U = torch.rand((M, K), generator=g, device="cuda").clamp_(1e-7, 1 - 1e-7)
    parent = torch.rand(M, generator=g, device="cuda")
    res = {}

    def timed(fn, inner=20):
        # `inner` calls per graph: one replay of a single short kernel is bound
        # by the host's graph-launch rate, not by the kernel
        gr = make_graph(torch, lambda: [fn() for _ in range(inner)])
        gr.replay()
        torch.cuda.synchronize()
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        for _ in range(reps):
            gr.replay()
        b.record()
        torch.cuda.synchronize()
        return a.elapsed_time(b) * 1e3 / (reps * inner)

    us = timed(lambda: L.draft_select(q, ids, 8, parent, U))
    by = M * K * 12 + M * 4
    res["draft_select"] = {"M": M, "K": K, "k_sel": 8, "us": round(us, 2), "bytes": by,
                           "hbm_frac": round(by / (us * 1e-6) / 1e9 / hbm, 4)}
    n, Bc, Kd, Kc = WORKLOAD.n, 8, 4, K
    p = torch.softmax(torch.randn((Bc, Kd + 1, n), generator=g, device="cuda") * 2.5, dim=-1)
    cid = ids[:Bc * Kd].reshape(Bc, Kd, Kc).contiguous()
    cq = q[:Bc * Kd].reshape(Bc, Kd, Kc).contiguous()
    # chains 0-3 draft each row's most likely candidate (q(x) >> p(x): rejected at
    # once, the residual path with the candidate hash); chains 4-7 its first
    # candidate (p(x) >= q(x): accepted, then the bonus draw)
    x = cid[:, :, 0].clone()
    best = cid.gather(2, cq.argmax(dim=2, keepdim=True)).squeeze(2)
    x[:Bc // 2] = best[:Bc // 2]
    x = x.contiguous()
    r = torch.rand((Bc, Kd), generator=g, device="cuda")
    u = torch.rand((Bc, Kd + 1), generator=g, device="cuda")
    tok, cnt = L.verify_chain(p, x, cid, cq, r, u)
    acc = int(cnt.sum().item())
    us = timed(lambda: L.verify_chain(p, x, cid, cq, r, u))
    res["verify_chain"] = {"chains": Bc, "drafts": Kd, "n": n, "K": Kc, "us": round(us, 2),
                           "accepted_total": acc,
                           "note": "one full-vocabulary pass of p per chain at its stop position; "
                                   "half the chains rejected at once, half accepted to the bonus"}
    return res


def time_noalloc(torch, L, head, rot_h, hbm, reps=40):
    """Graph-replayed timings of the no-allocation entry point
    (lmhead_two_stage_local_noalloc: CUDA-core scoring at every M, softmax
    inside the gather, scratch in a fixed device array) on the headline head
    at M = 1 and 64, beside the workspace call's numbers in the sweep."""
    import ctypes
    n, d = head["W"].shape
    r = head["B"].shape[0]
    lib = L.load()

    def dev(bits):
        return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).cuda().view(torch.bfloat16)

    res = []
    for Mx in (1, 64):
        hs = [dev(hidden(head["W"], Mx, 0)) for _ in rot_h]
        K = L.candidate_count(L.LOCAL, n, WORKLOAD.T, WORKLOAD.k_tile)
        outs = [(torch.empty((Mx, K), dtype=torch.int32, device="cuda"),
                 torch.empty((Mx, K), dtype=torch.float32, device="cuda"),
                 torch.empty((Mx, K), dtype=torch.float32, device="cuda")) for _ in rot_h]
        status = []

        def calls():
            st = torch.cuda.current_stream().cuda_stream
            for j, rt in enumerate(rot_h):
                Wt, At, Bt, tk = rt[0], rt[1], rt[2], rt[3]
                ids, lg, q = outs[j]
                status.append(lib.lmhead_two_stage_local_noalloc(
                    Wt.data_ptr(), At.data_ptr(), Bt.data_ptr(), hs[j].data_ptr(), tk.data_ptr(),
                    n, d, r, Mx, WORKLOAD.T, WORKLOAD.k_tile, ctypes.c_float(1.0),
                    ids.data_ptr(), lg.data_ptr(), q.data_ptr(), st))

        gr = make_graph(torch, calls)
        if any(x != 0 for x in status):
            raise RuntimeError(f"lmhead_two_stage_local_noalloc returned {status}")
        gr.replay()
        torch.cuda.synchronize()
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        for _ in range(reps // len(rot_h)):
            gr.replay()
        b.record()
        torch.cuda.synchronize()
        us = a.elapsed_time(b) * 1e3 / (reps // len(rot_h) * len(rot_h))
        res.append({"M": Mx, "us": round(us, 2), "vecs_per_s": round(Mx / us * 1e6, 1)})
        del gr
    return res


def time_shards(torch, L, head, hbm, M=64, shard_counts=(2, 4), reps=40):
    """The vocabulary-sharded local head on one GPU: for G shards of whole
    tiles (the headline head, M hidden vectors), each shard's call (selection
    and gather over its own rows, then the softmax from all shards' row stats)
    replayed alone in a graph. The slowest shard is what every GPU of a G-GPU
    call would spend, before the 8-byte-per-row all-gather of the stats."""
    from draft_lm_head_gb300 import shard as SH
    n, d = head["W"].shape
    r = head["B"].shape[0]
    T, k = WORKLOAD.T, WORKLOAD.k_tile

    def dev(bits):
        return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).cuda().view(torch.bfloat16)

    B = dev(head["B"])
    h = dev(hidden(head["W"], M, 0))
    res = []
    for G in shard_counts:
        per = []
        for (p0, p1) in SH.shard_ranges(n, T, G):
            Ws, As, toks, rowmap = SH.shard_inputs(head["W"], head["A"], head["tok"], p0, p1)
            Ws, As = dev(Ws), dev(As)
            toks = torch.from_numpy(toks).cuda()
            rowmap = torch.from_numpy(rowmap).cuda()
            K = L.candidate_count(L.LOCAL, p1 - p0, T, k)
            out = (torch.empty((M, K), dtype=torch.int32, device="cuda"),
                   torch.empty((M, K), dtype=torch.float32, device="cuda"),
                   torch.empty((M, 2), dtype=torch.float32, device="cuda"))
            q = torch.empty((M, K), dtype=torch.float32, device="cuda")
            all_stats = torch.ones((G, M, 2), dtype=torch.float32, device="cuda")
            ws = L.Workspace()

            def call():
                L.shard_two_stage(Ws, As, B, h, toks, rowmap, T, k, workspace=ws, out=out)
                L.shard_softmax(all_stats, out[1], out=q)

            gr = make_graph(torch, call)
            gr.replay()
            torch.cuda.synchronize()
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            for _ in range(reps):
                gr.replay()
            b.record()
            torch.cuda.synchronize()
            per.append(round(a.elapsed_time(b) * 1e3 / reps, 2))
            del gr, Ws, As
        res.append({"shards": G, "M": M, "shard_us": per, "slowest_us": max(per),
                    "note": "each shard alone on one GPU, its W rows resident (one copy)"})
        torch.cuda.empty_cache()
    return res


def time_cluster(torch, L, head, rot_h, hbm, group=128, G=8, reps=40):
    """Graph-replayed timings of the cluster-level route on the same head (A
    in vocabulary order, groups of `group` consecutive rows, the G best groups
    per hidden vector, G*group = 1024 candidates like the global route's C)
    at M = 1 and 64, with the algorithmic bytes: A, B, h once, each distinct
    selected group's W block once, outputs."""
    n, d = head["W"].shape
    r = head["B"].shape[0]
    A_voc = np.empty_like(head["A"])
    A_voc[head["tok"]] = head["A"]

    def dev(bits):
        return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).cuda().view(torch.bfloat16)

    copies = [(rt[0], dev(A_voc), rt[2]) for rt in rot_h]  # the headline's W and B copies
    ws = L.Workspace()
    res = []
    for Mx in (1, 64):
        hs = [dev(hidden(head["W"], Mx, 0)) for _ in copies]
        K = G * group
        outs = [(torch.empty((Mx, G), dtype=torch.int32, device="cuda"),
                 torch.empty((Mx, K), dtype=torch.int32, device="cuda"),
                 torch.empty((Mx, K), dtype=torch.float32, device="cuda"),
                 torch.empty((Mx, K), dtype=torch.float32, device="cuda")) for _ in copies]

        def calls():
            for j, (Wt, At, Bt) in enumerate(copies):
                L.cluster_two_stage(Wt, At, Bt, hs[j], group, G, workspace=ws, out=outs[j])

        gr = make_graph(torch, calls)
        gr.replay()
        torch.cuda.synchronize()
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        for _ in range(reps // len(copies)):
            gr.replay()
        b.record()
        torch.cuda.synchronize()
        us = a.elapsed_time(b) * 1e3 / (reps // len(copies) * len(copies))
        Ug = int(np.unique(outs[0][0].cpu().numpy()).size)
        by = 2 * n * r + 2 * r * d + 2 * Mx * d + 2 * d * group * Ug + Mx * (4 * G + 12 * K)
        res.append({"M": Mx, "group": group, "G": G, "candidates": K, "us": round(us, 2),
                    "vecs_per_s": round(Mx / us * 1e6, 1), "unique_groups": Ug, "bytes": by,
                    "hbm_frac": round(by / (us * 1e-6) / 1e9 / hbm, 4)})
        del gr
    return res


# ---------------------------------------------------------------- every configuration
# (workload, kind, mode, C_or_tile, k_tile, M values): configuration 1 is the
# global path on the unshuffled head, 2 the headline head (local, and global
# at the local candidate count and at 1024), 3 the draft-tree head, 4 the wide
# head; the dense full-vocabulary head beside each, and the 32000-row
# frequency-pruned head on the wide one.
CONFIG_PLAN = (
    (1, "two_stage", "global", 1024, 0, (1, 4, 8)),
    (2, "two_stage", "local", 256, 2, (1, 8, 16, 32, 64)),
    (2, "two_stage", "global", 1002, 0, (1, 8, 16, 32, 64)),
    (2, "two_stage", "global", 1024, 0, (1, 8, 16, 32, 64)),
    (2, "dense", None, 0, 0, (1, 4, 8, 16, 32, 64)),
    (3, "two_stage", "local", 256, 2, (80,)),
    (3, "two_stage", "global", 1024, 0, (80,)),
    (3, "dense", None, 0, 0, (80,)),
    (4, "two_stage", "local", 256, 4, (1, 8, 32, 128, 512)),
    (4, "dense", None, 0, 0, (1, 8, 32, 128, 512)),
    (4, "pruned", None, 32000, 0, (1, 8, 32, 128, 512)),
)


def config_hidden(wl, W, M):
    if wl.tree:
        h, _ = synth.make_tree_hidden(W, M // len(synth.TREE_PARENT), wl.index)
    else:
        h, _ = synth.make_hidden(W, M, wl.index)
    return h


def time_configs(torch, L, hbm, reps=100):
    """Per-call latency of every configuration: stream-launched and CUDA-graph
    replayed (median, p10, p90 over `reps` calls rotating over NROT copies of
    every input), hidden vecs/s and the whole call's HBM fraction from the
    graph median, with the algorithmic bytes (2nr + 2rd + 2Md + 2dU + 12MK for
    the two-stage head, U the distinct candidate rows; 2nd + 2Md + 12Mn for the
    dense head, softmax included; the same over the kept rows for the pruned
    head)."""
    from draft_lm_head_gb300 import prep

    def dev(bits):
        return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).cuda().view(torch.bfloat16)

    rows = []
    for idx in sorted({p[0] for p in CONFIG_PLAN}):
        wl = synth.workload(idx)
        head = head_inputs(wl)
        n, d, r = wl.n, wl.d, wl.r
        W0, A0, B0 = dev(head["W"]), dev(head["A"]), dev(head["B"])
        tok0 = torch.from_numpy(np.ascontiguousarray(head["tok"], dtype=np.int32)).cuda()
        rot = [(W0, A0, B0, tok0)] + [(W0.clone(), A0.clone(), B0.clone(), tok0.clone())
                                      for _ in range(NROT - 1)]
        pruned = None
        ws = L.Workspace()
        for (ci, kind, mode, C, k, Ms) in CONFIG_PLAN:
            if ci != idx:
                continue
            if kind == "pruned" and pruned is None:
                Wp, _ = prep.pruned_rows(head["W"], head["counts"], C)
                pruned = [dev(Wp) for _ in range(NROT)]
            for M in Ms:
                hb = config_hidden(wl, head["W"], M)
                hs = [dev(hb) for _ in range(NROT)]
                ent = {"config": idx, "head": kind, "M": M}
                if kind == "two_stage":
                    md = L.LOCAL if mode == "local" else L.GLOBAL
                    K = L.candidate_count(md, n, C, k)
                    outs = [(torch.empty((M, K), dtype=torch.int32, device="cuda"),
                             torch.empty((M, K), dtype=torch.float32, device="cuda"),
                             torch.empty((M, K), dtype=torch.float32, device="cuda"))
                            for _ in range(NROT)]
                    fns = [lambda j=j: L.two_stage(md, rot[j][0], rot[j][1], rot[j][2], hs[j],
                                                   rot[j][3], C, k, workspace=ws, out=outs[j])
                           for j in range(NROT)]
                    ent.update({"mode": mode, "candidates": K})
                    ent.update({"tile": C, "k_tile": k} if mode == "local" else {"C": C})
                elif kind == "dense":
                    lg = torch.empty((M, n), dtype=torch.float32, device="cuda")
                    q = torch.empty((M, n), dtype=torch.float32, device="cuda")
                    fns = [lambda j=j: L.dense_head(rot[j][0], hs[j], out=(lg, q))
                           for j in range(NROT)]
                else:
                    lg = torch.empty((M, C), dtype=torch.float32, device="cuda")
                    q = torch.empty((M, C), dtype=torch.float32, device="cuda")
                    fns = [lambda j=j: L.pruned_head(pruned[j], hs[j], out=(lg, q))
                           for j in range(NROT)]
                    ent["kept_rows"] = C
                st = pstats(per_call_us(torch, fns, reps))
                gr = pstats(per_call_us(torch, fns, reps, graph=True))
                if kind == "two_stage":
                    U = int(np.unique(outs[0][0].cpu().numpy()).size)
                    by = 2 * n * r + 2 * r * d + 2 * M * d + 2 * d * U + 12 * M * K
                    ent["unique_rows"] = U
                elif kind == "dense":
                    by = 2 * n * d + 2 * M * d + 12 * M * n
                else:
                    by = 2 * C * d + 2 * M * d + 12 * M * C
                us = gr["median"]
                ent.update({"stream_us": st, "graph_us": gr, "us": us,
                            "vecs_per_s": round(M / us * 1e6, 1), "bytes": by,
                            "hbm_frac": round(by / (us * 1e-6) / 1e9 / hbm, 4)})
                rows.append(ent)
                del fns, hs
        del rot, pruned
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
    return rows


def dense_speedups(rows):
    """Two-stage vs dense latency (graph medians) per configuration and M."""
    dense = {(e["config"] if e["config"] != 1 else 2, e["M"]): e["us"]
             for e in rows if e["head"] == "dense"}
    out = []
    for e in rows:
        if e["head"] != "two_stage":
            continue
        key = (e["config"] if e["config"] != 1 else 2, e["M"])
        if key in dense:
            out.append({"config": e["config"], "mode": e["mode"], "M": e["M"],
                        "two_stage_us": e["us"], "dense_us": dense[key],
                        "speedup": round(dense[key] / e["us"], 2)})
    return out


# ---------------------------------------------------------------- CPU oracle legs
CPU_MODES = {0: ("local", 128, 4), 1: ("global", 1024, 0), 2: ("local", 256, 2),
             3: ("local", 256, 2), 4: ("local", 256, 4)}


def oracle_config_rate(idx, budget_s=2.5):
    """The oracle as it stands on configuration idx: steps u -> scores ->
    Top-k -> logits -> q for one hidden vector at a time (the configuration's
    first M rows in turn), repeated for about budget_s. Returns a record."""
    import oracle as O
    wl = synth.workload(idx)
    mode, C, k = CPU_MODES[idx]
    head = head_inputs(wl)
    A64 = O.bf16_bits_to_f64(head["A"])
    B64 = O.bf16_bits_to_f64(head["B"])
    tok = head["tok"]
    h64 = O.bf16_bits_to_f64(config_hidden(wl, head["W"], max(wl.Ms)))
    done, t0 = 0, time.perf_counter()
    while True:
        hm = h64[done % h64.shape[0]][None]
        u = O.project_u(B64, hm)
        S = O.lowrank_scores(A64, u)[0]
        ids = O.local_topk(S, tok, C, k)[0] if mode == "local" else O.global_topk(S, tok, C)[0]
        Lg = O.candidate_logits(O.bf16_bits_to_f64(head["W"][ids]), hm[0], np.arange(ids.size))
        O.candidate_softmax(Lg)
        done += 1
        if time.perf_counter() - t0 >= budget_s:
            break
    dt = time.perf_counter() - t0
    return {"config": idx, "mode": mode, "vecs_per_s": round(done / dt, 3),
            "us_per_vec": round(dt / done * 1e6, 1), "vectors": done}


def cpu_configs():
    """Oracle rates per configuration: all host cores for configurations 0-4,
    one thread (BLAS pinned to one thread in a child process) for 0-2."""
    cores = len(os.sched_getaffinity(0))
    out = []
    for idx in range(5):
        rec = oracle_config_rate(idx)
        rec["threads"] = cores
        out.append(rec)
    env = dict(os.environ, OPENBLAS_NUM_THREADS="1", OMP_NUM_THREADS="1", MKL_NUM_THREADS="1")
    for idx in range(3):
        p = subprocess.run([sys.executable, os.path.abspath(__file__), "--cpu-sample", str(idx)],
                           capture_output=True, text=True, env=env, timeout=300)
        if p.returncode == 0 and p.stdout.strip():
            rec = json.loads(p.stdout.strip().splitlines()[-1])
            rec["threads"] = 1
            out.append(rec)
    return out


def parity_sample(head, hb, out, rows=(0, 31, 63)):
    """Parity of the timed call on a few of its rows against the oracle
    (the boundary rule of the candidate ids, the logits and q tolerances):
    counts of excused ids inside the 1e-3 band and needing the u-rounding
    slack, and the largest logit and q errors."""
    sys.path.insert(0, os.path.join(ROOT, "tests"))
    import oracle as O
    import parity as P
    wl = WORKLOAD
    ids, lg, q = (t.cpu().numpy() for t in out)
    M = ids.shape[0]
    rows = [m for m in rows if m < M]
    A64 = O.bf16_bits_to_f64(head["A"])
    B64 = O.bf16_bits_to_f64(head["B"])
    h64 = O.bf16_bits_to_f64(hb[rows])
    S = O.lowrank_scores(A64, O.project_u(B64, h64))
    SL = P.u_slack(A64, B64, h64, M_call=M)
    counts = P.check_ids("local", ids[rows], S, head["tok"], wl.T, wl.k_tile, slack_pos=SL)
    ex = P.exact_logits(head["W"], h64, ids[rows])
    P.check_logits(lg[rows], ex)
    P.check_q(q[rows], ex)
    rel = np.abs(lg[rows] - ex) / np.maximum(np.abs(ex), 1.0)
    qerr = max(float(np.abs(q[m] - O.candidate_softmax(ex[i])).max()) for i, m in enumerate(rows))
    return {"rows": rows, "ids_compared": counts["compared"], "excused_band": counts["band"],
            "excused_slack": counts["slack"], "logit_max_rel_err": float(rel.max()),
            "q_max_abs_err": qerr, "passed": True}


def run_ours(args):
    import ctypes
    global NROT
    NROT = max(1, args.rotations)

    import torch
    import torch.distributed as dist

    rank = int(os.environ.get("RANK", 0))
    world = int(os.environ.get("WORLD_SIZE", 1))
    local = int(os.environ.get("LOCAL_RANK", 0))
    torch.cuda.set_device(local)
    if world > 1:
        dist.init_process_group("nccl", device_id=torch.device("cuda", local))
    from draft_lm_head_gb300 import build
    if rank == 0:
        build.build()
    if world > 1:
        dist.barrier()
    import draft_lm_head_gb300 as L
    lib = L.load()

    wl = WORKLOAD
    n, d, r, M = wl.n, wl.d, wl.r, args.M
    head = head_inputs()
    hb = hidden(head["W"], M, rank)

    def dev(bits):
        return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).cuda().view(torch.bfloat16)

    W0, A0, B0 = dev(head["W"]), dev(head["A"]), dev(head["B"])
    tok0 = torch.from_numpy(head["tok"]).cuda()
    h0 = dev(hb)
    rot = [(W0, A0, B0, tok0, h0)] + [(W0.clone(), A0.clone(), B0.clone(), tok0.clone(), h0.clone())
                                      for _ in range(NROT - 1)]
    K = L.candidate_count(L.LOCAL, n, wl.T, wl.k_tile)
    nl = lib.lmhead_two_stage_launches(L.LOCAL, wl.k_tile)
    ws = L.Workspace()

    def outputs(Mx):
        return [(torch.empty((Mx, K), dtype=torch.int32, device="cuda"),
                 torch.empty((Mx, K), dtype=torch.float32, device="cuda"),
                 torch.empty((Mx, K), dtype=torch.float32, device="cuda")) for _ in range(NROT)]

    outs = outputs(M)

    def step(j, hx=None, out=None):
        Wt, At, Bt, tk, ht = rot[j % NROT]
        return L.two_stage(L.LOCAL, Wt, At, Bt, ht if hx is None else hx[j % NROT], tk, wl.T,
                           wl.k_tile, workspace=ws, out=(out or outs)[j % NROT])

    # one graph holding NROT consecutive steps (one per input copy), plus singles
    g_all = make_graph(torch, lambda: [step(j) for j in range(NROT)])
    g_one = [make_graph(torch, lambda j=j: step(j)) for j in range(NROT)]

    def run_steps(k):
        for _ in range(k // NROT):
            g_all.replay()
        for j in range(k % NROT):
            g_one[j].replay()

    sampler = ClockSampler(local)
    run_steps(max(args.warmup, 3))
    torch.cuda.synchronize()
    sampler.start()
    time.sleep(0.3)
    if world > 1:
        dist.barrier()
    torch.cuda.synchronize()
    e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    e0.record()
    run_steps(args.steps)
    e1.record()
    torch.cuda.synchronize()
    if world > 1:
        dist.barrier()
    ms = max_over_ranks(e0.elapsed_time(e1), world, "cuda")
    value = aggregate_rate(world, M, args.steps, ms)
    launches = nl * args.steps

    # per-kernel durations: the profiled entry point records an event after every launch
    evs = [[torch.cuda.Event(enable_timing=True) for _ in range(nl + 1)] for _ in range(NROT)]
    for row in evs:
        for e in row:
            e.record()
    torch.cuda.synchronize()
    wsb = ws.get(L.workspace_size(L.LOCAL, n, d, r, M, wl.T, wl.k_tile), h0.device)

    def prof_step(j):
        Wt, At, Bt, tk, ht = rot[j]
        ids, lg, q = outs[j]
        handles = (ctypes.c_void_p * (nl + 1))(*[e.cuda_event for e in evs[j]])
        L.check(lib.lmhead_two_stage_profiled(
            L.LOCAL, Wt.data_ptr(), At.data_ptr(), Bt.data_ptr(), ht.data_ptr(), tk.data_ptr(),
            n, d, r, M, wl.T, wl.k_tile, 1.0, ids.data_ptr(), lg.data_ptr(), q.data_ptr(),
            wsb.data_ptr(), wsb.numel(), handles, nl + 1,
            torch.cuda.current_stream().cuda_stream), "two_stage_profiled")

    names = ["project_u", "score_local_topk", "gather_logits", "candidate_softmax"][:nl]
    samples = {k: [] for k in names}
    prof_mode = "stream, events between the launches of one call"
    for i in range(args.steps):
        j = i % NROT
        prof_step(j)
        torch.cuda.synchronize()
        for k, nm in enumerate(names):
            samples[nm].append(evs[j][k].elapsed_time(evs[j][k + 1]))
    kern_us = {k: 1e3 * statistics.fmean(v) for k, v in samples.items()}

    ids_h = outs[0][0].cpu().numpy()
    U = int(np.unique(ids_h).size)
    bytes_kernel = {
        "project_u": 2 * r * d + 2 * M * d + 2 * M * r,
        "score_local_topk": 2 * n * r + 2 * M * r + 4 * M * K,
        "gather_logits": 2 * d * U + 2 * M * d + 4 * M * K + 4 * M * K,
        "candidate_softmax": 4 * M * K + 4 * M * K,
    }
    step_bytes = 2 * n * r + 2 * r * d + 2 * M * d + 2 * d * U + 12 * M * K
    hbm, peak_kind = peaks()
    dom = max(kern_us, key=kern_us.get)
    achieved = bytes_kernel[dom] / (kern_us[dom] * 1e-6) / 1e9
    roof = {"bound": "hbm", "kernel": dom, "achieved": round(achieved, 1), "peak": hbm,
            "unit": "GB/s", "frac": round(achieved / hbm, 4), "peak_kind": peak_kind,
            "bytes_per_launch": bytes_kernel[dom], "traffic": ncu_traffic(dom, M),
            "timing": prof_mode}

    # end to end through the public API: host buffers, copies inside the timed region
    h_host = [torch.from_numpy(np.ascontiguousarray(hb).view(np.int16)).view(torch.bfloat16).pin_memory()
              for _ in range(NROT)]
    host_out = [tuple(torch.empty(t.shape, dtype=t.dtype).pin_memory() for t in outs[0])
                for _ in range(NROT)]
    h_dev = [torch.empty_like(h0) for _ in range(NROT)]

    # h goes in on one copy stream, the call runs on the compute stream and the
    # outputs come back on another, so each step's copies overlap the
    # neighbouring steps' compute (steps are independent batches of hidden
    # vectors); events keep every buffer's reuse ordered
    cs = torch.cuda.current_stream()
    hs, ds = torch.cuda.Stream(), torch.cuda.Stream()
    ev_h = [torch.cuda.Event() for _ in range(NROT)]
    ev_c = [torch.cuda.Event() for _ in range(NROT)]
    ev_d = [torch.cuda.Event() for _ in range(NROT)]
    used = [False] * NROT

    def e2e_step(i):
        j = i % NROT
        with torch.cuda.stream(hs):
            if used[j]:
                hs.wait_event(ev_c[j])  # the call that last read h_dev[j] has finished
            h_dev[j].copy_(h_host[j], non_blocking=True)
            ev_h[j].record(hs)
        cs.wait_event(ev_h[j])
        if used[j]:
            cs.wait_event(ev_d[j])  # outs[j] has been copied out
        Wt, At, Bt, tk, _ = rot[j]
        res = L.two_stage(L.LOCAL, Wt, At, Bt, h_dev[j], tk, wl.T, wl.k_tile, workspace=ws,
                          out=outs[j])
        ev_c[j].record(cs)
        with torch.cuda.stream(ds):
            ds.wait_event(ev_c[j])
            for dst, src in zip(host_out[j], res):
                dst.copy_(src, non_blocking=True)
            ev_d[j].record(ds)
        used[j] = True

    for i in range(3):
        e2e_step(i)
    torch.cuda.synchronize()
    e0.record()
    for i in range(args.steps):
        e2e_step(i)
    cs.wait_stream(ds)
    e1.record()
    torch.cuda.synchronize()
    ms_e2e = max_over_ranks(e0.elapsed_time(e1), world, "cuda")
    e2e = {"value": round(aggregate_rate(world, M, args.steps, ms_e2e), 1), "unit": "hidden vecs/s",
           "h2d_bytes_per_step": int(hb.nbytes),
           "d2h_bytes_per_step": int(sum(t.numel() * t.element_size() for t in outs[0])),
           "copies": "pinned host buffers; h in and ids/logits/q out on their own streams, "
                     "overlapping the neighbouring steps' compute; stream-launched calls"}

    # sweep over M (graph replay) with the dense head beside it, for context
    sweep = []
    if not args.no_sweep and rank == 0:
        reps = 40
        for Mx in (1, 8, 16, 32, 64):
            hxs = [dev(hidden(head["W"], Mx, rank)) for _ in range(NROT)]
            ox = outputs(Mx)
            g = make_graph(torch, lambda: [step(j, hxs, ox) for j in range(NROT)])
            g.replay()
            torch.cuda.synchronize()
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            for _ in range(reps // NROT):
                g.replay()
            b.record()
            torch.cuda.synchronize()
            us = a.elapsed_time(b) * 1e3 / (reps // NROT * NROT)
            Ux = int(np.unique(ox[0][0].cpu().numpy()).size)
            by = 2 * n * r + 2 * r * d + 2 * Mx * d + 2 * d * Ux + 12 * Mx * K
            dl = torch.empty((Mx, n), dtype=torch.float32, device="cuda")
            dq = torch.empty((Mx, n), dtype=torch.float32, device="cuda")
            gd = make_graph(torch, lambda: [L.dense_head(rot[j][0], hxs[j], out=(dl, dq))
                                            for j in range(2)])
            a.record()
            for _ in range(4):
                gd.replay()
            b.record()
            torch.cuda.synchronize()
            dus = a.elapsed_time(b) * 1e3 / 8
            sweep.append({"M": Mx, "us": round(us, 2), "vecs_per_s": round(Mx / us * 1e6, 1),
                          "unique_rows": Ux, "bytes": by,
                          "hbm_frac": round(by / (us * 1e-6) / 1e9 / hbm, 4),
                          "dense_us": round(dus, 2)})
            del g, gd
    # per-call latency of the headline call: stream-launched and graph-replayed
    lat = {"stream": pstats(per_call_us(torch, [lambda j=j: step(j) for j in range(NROT)], 200)),
           "graph": pstats(per_call_us(torch, [lambda j=j: step(j) for j in range(NROT)], 200,
                                       graph=True))}
    # the steps after q (draft selection, chain verification), for context
    after_q = {}
    cluster = []
    noalloc = []
    shards = []
    if not args.no_sweep and rank == 0:
        after_q = time_after_q(torch, L, outs[0], hbm)
        cluster = time_cluster(torch, L, head, rot, hbm)
        noalloc = time_noalloc(torch, L, head, rot, hbm)
        try:
            shards = time_shards(torch, L, head, hbm)
        except Exception as exc:  # a side measurement: report it, keep the line
            shards = [{"error": f"{type(exc).__name__}: {exc}"}]
    configs = []
    if not args.no_configs and rank == 0:
        configs = time_configs(torch, L, hbm)
    clocks = sampler.stop()

    cpu = cpu_rates = None
    parity = None
    if rank == 0 and not args.no_cpu:
        rate, cores, sample = oracle_sample_rate(head, hb)
        cpu = {"value": round(rate, 3), "unit": "hidden vecs/s", "cores": cores, "kind": "oracle",
               "sample": sample}
        parity = parity_sample(head, hb, outs[0])
        if not args.no_configs:
            cpu_rates = cpu_configs()

    if rank == 0:
        line = {
            "metric": METRIC, "value": round(value, 1), "unit": "hidden vecs/s", "n_gpus": world,
            "steps": args.steps, "warmup": args.warmup, "ms_per_step": round(ms / args.steps, 5),
            "higher_is_better": True, "scaling": "weak", "vs_baseline": None, "dtype": "bf16",
            "data": "synthetic: seeded rank-64+noise bf16 head, Zipf(1.1) counts, recipe hidden states",
            "config": workload_config(M, world, NROT),
            "roofline": roof, "cpu_baseline": cpu, "e2e": e2e, "gpu_launches": launches,
            "clocks": clocks, "kernel_us": {k: round(v, 3) for k, v in kern_us.items()},
            "step_bytes": step_bytes,
            "step_hbm_frac": round(step_bytes / (ms / args.steps * 1e-3) / 1e9 / hbm, 4),
            "unique_rows": U, "latency_us": lat, "parity_counts": parity,
        }
        # the tables beside the headline would make its line too long to be read
        # back whole: they are a line of their own on stderr
        tables = {
            "sweep": sweep, "configs": configs, "vs_dense": dense_speedups(configs),
            "after_q": after_q, "cluster_route": cluster, "noalloc": noalloc, "sharded": shards,
            "cpu_per_config": cpu_rates,
        }
        print(json.dumps(tables), file=sys.stderr, flush=True)
        print(json.dumps(line), flush=True)
    if world > 1:
        dist.barrier()
        dist.destroy_process_group()


# ---------------------------------------------------------------- reference arm
def run_reference(args):
    rank = int(os.environ.get("RANK", 0))
    world = int(os.environ.get("WORLD_SIZE", 1))
    if rank != 0:
        return
    import oracle as O
    wl = WORKLOAD
    rows = 8  # hidden vectors of the workload's batch per timed step (bounded CPU time)
    head = head_inputs()
    hb = hidden(head["W"], args.M, 0)[:rows]
    A64 = O.bf16_bits_to_f64(head["A"])
    B64 = O.bf16_bits_to_f64(head["B"])
    h64 = O.bf16_bits_to_f64(hb)

    def step():
        u = O.project_u(B64, h64)
        S = O.lowrank_scores(A64, u)
        for m in range(rows):
            ids, _ = O.local_topk(S[m], head["tok"], wl.T, wl.k_tile)
            Lg = O.candidate_logits(O.bf16_bits_to_f64(head["W"][ids]), h64[m], np.arange(ids.size))
            O.candidate_softmax(Lg)

    for _ in range(max(args.warmup, 0)):
        step()
    t0 = time.perf_counter()
    for _ in range(args.steps):
        step()
    dt = time.perf_counter() - t0
    value = rows * args.steps / dt
    cores = len(os.sched_getaffinity(0))
    line = {
        "impl": "reference", "metric": METRIC, "value": round(value, 3), "unit": "hidden vecs/s",
        "n_gpus": world, "steps": args.steps, "warmup": args.warmup,
        "ms_per_step": round(dt / args.steps * 1e3, 3), "higher_is_better": True,
        "scaling": "weak", "vs_baseline": None, "dtype": "f64",
        "data": "synthetic: seeded rank-64+noise bf16 head, Zipf(1.1) counts, recipe hidden states",
        "config": workload_config(args.M, world, max(1, args.rotations)),
        "cpu_baseline": {"value": round(value, 3), "unit": "hidden vecs/s", "cores": cores,
                         "kind": "oracle",
                         "sample": f"{rows} of the workload's {args.M} hidden vectors per step "
                                   "(the whole path for each), fp64 NumPy oracle on the host cores"},
        "e2e": {"value": round(value, 3), "unit": "hidden vecs/s", "h2d_bytes_per_step": 0,
                "d2h_bytes_per_step": 0},
    }
    print(json.dumps(line), flush=True)


def main():
    args = parse()
    if args.cpu_sample >= 0:  # child of cpu_configs: one oracle rate, one JSON line
        print(json.dumps(oracle_config_rate(args.cpu_sample)), flush=True)
        return
    if args.impl == "reference":
        run_reference(args)
    else:
        run_ours(args)


if __name__ == "__main__":
    main()
