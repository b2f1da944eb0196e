"""Benchmark of the batched speculative-sampling verify step on one MI355X.

    python bench.py [--gpus 1] [--steps K] [--warmup W] [--no-cpu-baseline]
                    [--calibrate]

Workload: B=64 rows, K=5 drafted tokens, V=128256 (Llama-3 vocabulary),
bfloat16 logits, temperature 0.7, top-p off -- the batched workload of the
seeded generator.  Three distinct input sets (3 x 180.6 MB, more than the
256 MB Infinity Cache) are resident in HBM and rotated call by call, so no
call finds its inputs in the cache.  A step is one spec_verify call: the
statistics pass over every needed logit row (k_stats), then the row pass
(k_rows): acceptance decision, residual or bonus masses, inverse-CDF draw.

Prints one JSON line.  `value` is verified draft positions per second; the
roofline object prices the dominant kernel (the statistics pass) against
MI355X's 8 TB/s HBM peak using the logical bytes it must read, sum_b
(2 L_b + 1) V e; the cpu_baseline object times the float64 oracle on the
host cores on a bounded sample of the same workload.
"""

import argparse
import hashlib
import json
import multiprocessing as mp
import os
import sys
import time

ROOT = os.path.dirname(os.path.abspath(__file__))
sys.path.insert(0, ROOT)

HBM_PEAK_GBS = 8000.0
WORKLOAD_CFG = 2
N_SETS = 3
TRAFFIC_FILE = os.path.join(ROOT, "profiles", "traffic_stats_batched.json")
KERNEL_SOURCES = [os.path.join(ROOT, "rejection_sampling_verifier_amd", "csrc", f)
                  for f in ("sv_kernels.hip", "sv_device.h", "sv_internal.h")]


def kernel_source_sha():
    h = hashlib.sha256()
    for f in KERNEL_SOURCES:
        with open(f, "rb") as fh:
            h.update(fh.read())
    return h.hexdigest()[:16]


def stored_traffic(workload_name):
    """HBM bytes per statistics-pass launch from the committed counter runs,
    or None when they were taken on another workload or the kernel sources
    changed since."""
    try:
        with open(TRAFFIC_FILE) as f:
            t = json.load(f)
    except (OSError, ValueError):
        return None
    if t.get("kernel_source_sha") != kernel_source_sha() or t.get("workload") != workload_name:
        return None
    return t.get("hbm_bytes_per_launch")


# ---------------------------------------------------------------------------
# CPU baseline: the oracle, unchanged, on a bounded sample
# ---------------------------------------------------------------------------
_SAMPLE = None


def _oracle_rows(args):
    import oracle

    si, rows = args
    inp = _SAMPLE[si]
    # the task's rows only (the oracle widens every row it is handed); the
    # Philox row index restarts at 0, which changes no amount of work
    r0, r1 = rows[0], rows[-1] + 1
    oracle.verify(inp.target[r0:r1], inp.draft[r0:r1], inp.draft_tokens[r0:r1],
                  None if inp.draft_len is None else inp.draft_len[r0:r1], inp.temperature, inp.top_p, inp.seed)
    return sum(int(inp.lengths()[r]) for r in range(r0, r1))


def _oracle_smc(args):
    import numpy as np

    import oracle

    si, i0, i1 = args
    inp = _SAMPLE[si]
    oracle.smc_step(inp.target[i0:i1], inp.draft[i0:i1], inp.draft_tokens[i0:i1], np.zeros(i1 - i0),
                    inp.temperature, SMC_ESS_FRACTION, inp.seed)
    return (i1 - i0) * inp.K


def cpu_baseline_smc(sets, budget_particles, workload_name):
    """The SMC oracle on sub-batches of 4 particles (each a valid step)."""
    global _SAMPLE
    _SAMPLE = sets
    cores = max(1, min(POOL, os.cpu_count() or 1))
    work, n = [], 0
    for si, inp in enumerate(sets):
        for i0 in range(0, inp.B, 4):
            if n >= budget_particles:
                break
            work.append((si, i0, min(i0 + 4, inp.B)))
            n += min(i0 + 4, inp.B) - i0
    positions, dt, passes = _timed_passes(_oracle_smc, work, cores)
    return {
        "value": positions / dt,
        "unit": "scored positions/s",
        "cores": cores,
        "kind": "oracle",
        "sample": f"{n} particles of the {workload_name} workload as SMC particles, {passes} passes ({positions} "
                  f"drafted positions), float64 NumPy oracle, 4 particles per task over {cores} processes, "
                  f"{dt:.1f} s wall",
    }


def host_cpu():
    """The host's CPU model and logical CPU count."""
    model = "unknown"
    try:
        with open("/proc/cpuinfo") as f:
            for line in f:
                if line.startswith("model name"):
                    model = line.split(":", 1)[1].strip()
                    break
    except OSError:
        pass
    return model, os.cpu_count() or 1


# worker processes of the oracle pool: the GPU machine's CPU share is 16
POOL = 16


def cpu_baseline(sets, budget_rows, workload_name):
    global _SAMPLE
    _SAMPLE = sets
    model, logical = host_cpu()
    cores = max(1, min(POOL, logical))
    work = []
    n = 0
    for si, inp in enumerate(sets):
        for b in range(inp.B):
            if n >= budget_rows:
                break
            work.append((si, [b]))
            n += 1
    positions, dt, passes = _timed_passes(_oracle_rows, work, cores)
    # one worker on a sixteenth of the sample: the single-core rate
    p1, dt1, passes1 = _timed_passes(_oracle_rows, work[: max(1, len(work) // 16)], 1, wall=CPU_WALL_S)
    return {
        "value": positions / dt,
        "unit": "positions/s",
        "cores": cores,
        "kind": "oracle",
        "value_1_worker": p1 / dt1,
        "host_cpu": model,
        "host_logical_cpus": logical,
        "sample": f"{len(work)} batch rows of the {workload_name} workload, {passes} passes ({positions} draft "
                  f"positions), float64 NumPy oracle, one row per task over {cores} processes, {dt:.1f} s wall; "
                  f"one process: {len(work[: max(1, len(work) // 16)])} rows, {passes1} passes ({p1} positions), "
                  f"{dt1:.1f} s",
    }


CPU_WALL_S = 1.5  # about 10-30 s of CPU work over the pool


def _timed_passes(fn, work, cores, wall=None):
    """Passes over the sample until CPU_WALL_S of wall time (at most 20)."""
    wall = CPU_WALL_S if wall is None else wall
    ctx = mp.get_context("fork")
    positions, passes = 0, 0
    with ctx.Pool(cores) as pool:
        t0 = time.perf_counter()
        while passes < 20 and (passes == 0 or time.perf_counter() - t0 < wall):
            positions += sum(pool.map(fn, work, chunksize=1))
            passes += 1
        dt = time.perf_counter() - t0
    return positions, dt, passes


# ---------------------------------------------------------------------------
# GPU clocks and the per-call distribution
# ---------------------------------------------------------------------------
WARMUP_SPIN_S = 0.3


def device_warmup(binding, torch, dev, dsets):
    """Streams the input sets with the streaming-read kernel for about
    WARMUP_SPIN_S so that the clocks reach their steady state before the
    warmup steps (an idle GPU runs its first tens of milliseconds slower);
    no verify call is made."""
    sink = torch.empty(1024, dtype=torch.int32, device=dev)
    bufs = [t for ds in dsets for t in ds[:2]]
    t0 = time.perf_counter()
    n = 0
    while time.perf_counter() - t0 < WARMUP_SPIN_S:
        for b in bufs:
            binding.stream_read(b, sink, unroll=8)
            n += 1
        torch.cuda.synchronize()
    print(f"[bench] device warm-up: {n} streaming reads in {time.perf_counter() - t0:.2f} s", file=sys.stderr,
          flush=True)


def per_call_distribution(torch, stream, step, n):
    """Each of n more calls between its own pair of events on the launch
    stream: median, p10 and p90 of the per-call times (the events sit between
    calls, not inside them)."""
    import numpy as np

    evs = [(torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)) for _ in range(n)]
    torch.cuda.synchronize()
    for i in range(n):
        evs[i][0].record(stream)
        step(i)
        evs[i][1].record(stream)
    torch.cuda.synchronize()
    us = np.array([a.elapsed_time(b) * 1e3 for a, b in evs])
    return {"median_us": round(float(np.median(us)), 3), "p10_us": round(float(np.percentile(us, 10)), 3),
            "p90_us": round(float(np.percentile(us, 90)), 3), "calls": n}


# ---------------------------------------------------------------------------
# Counter calibration: kernels of known traffic
# ---------------------------------------------------------------------------
CALIB_BYTES = 512 << 20


def calibrate(binding, torch, dev, logical):
    """A device-to-device copy (reads and writes CALIB_BYTES) and the
    streaming-read kernel (reads CALIB_BYTES), 3 launches each: the
    references that scale byte counters.  Then the streaming-read ceiling
    for the statistics pass's own byte count: the streaming-read kernel with
    its access pattern (8 vectors per lane) over three rotated buffers of
    `logical` bytes, timed with events."""
    src = torch.empty(CALIB_BYTES, dtype=torch.uint8, device=dev)
    src.fill_(7)
    dst = torch.empty_like(src)
    sink = torch.zeros(1024, dtype=torch.int32, device=dev)
    torch.cuda.synchronize()
    for _ in range(3):
        dst.copy_(src)
    for _ in range(3):
        binding.stream_read(src, sink, 4)
    torch.cuda.synchronize()
    print(f"[bench] calibration: 3 copies and 3 streaming reads of {CALIB_BYTES} bytes", file=sys.stderr, flush=True)
    del src, dst
    # the streaming-read ceiling over 1 GiB, and the device's own figures
    big = torch.full((1 << 30,), 5, dtype=torch.uint8, device=dev)
    for _ in range(5):
        binding.stream_read(big, sink, 8)
    e0 = torch.cuda.Event(enable_timing=True)
    e1 = torch.cuda.Event(enable_timing=True)
    e0.record()
    for _ in range(20):
        binding.stream_read(big, sink, 8)
    e1.record()
    torch.cuda.synchronize()
    big_GBps = (1 << 30) / (e0.elapsed_time(e1) / 20 * 1e-3) / 1e9
    del big
    props = torch.cuda.get_device_properties(dev)
    device = {"name": props.name, "arch": getattr(props, "gcnArchName", ""), "compute_units": props.multi_processor_count,
              "memory_GiB": round(props.total_memory / 2 ** 30, 1),
              "l2_MiB": round(getattr(props, "L2_cache_size", 0) / 2 ** 20, 1)}
    print(f"[bench] streaming read of 1 GiB: {big_GBps:.0f} GB/s; device {device}", file=sys.stderr, flush=True)
    nbytes = int(logical) // 16 * 16
    bufs = [torch.full((nbytes,), 3, dtype=torch.uint8, device=dev) for _ in range(N_SETS)]
    stream = torch.cuda.current_stream(dev)
    for i in range(300):
        binding.stream_read(bufs[i % N_SETS], sink, 8, stream=stream)
    e0 = torch.cuda.Event(enable_timing=True)
    e1 = torch.cuda.Event(enable_timing=True)
    reps = 600
    e0.record(stream)
    for i in range(reps):
        binding.stream_read(bufs[i % N_SETS], sink, 8, stream=stream)
    e1.record(stream)
    torch.cuda.synchronize()
    us = e0.elapsed_time(e1) / reps * 1e3
    print(f"[bench] streaming read of {nbytes} bytes: {us:.2f} us", file=sys.stderr, flush=True)
    return {"stream_read_bytes": nbytes, "stream_read_us": round(us, 3),
            "stream_read_GBps": round(nbytes / (us * 1e-6) / 1e9, 1),
            "stream_read_1GiB_GBps": round(big_GBps, 1), "device": device}


# ---------------------------------------------------------------------------
# SMC-SD step timing (--smc): the same inputs scored as N = B particles
# ---------------------------------------------------------------------------
SMC_ESS_FRACTION = 0.5


def smc_bench(args, binding, torch, dev, sets, dsets, logical, stream):
    import numpy as np

    N, K = sets[0].B, sets[0].K
    lw = torch.zeros((N,), dtype=torch.float64, device=dev)
    outs = [(torch.empty((N,), dtype=torch.int32, device=dev), torch.empty((N,), dtype=torch.float64, device=dev),
             torch.empty((N,), dtype=torch.int32, device=dev)) for _ in range(N_SETS)]

    def step(i):
        t, d, x, _, T, _, seed = dsets[i % N_SETS]
        o = outs[i % N_SETS]
        binding.smc_step(t, d, x, lw, T, SMC_ESS_FRACTION, seed, stream=stream, out_bonus=o[0], out_logw=o[1],
                         out_ancestor=o[2])

    for i in range(args.warmup):
        step(i)
    torch.cuda.synchronize()
    ev0 = torch.cuda.Event(enable_timing=True)
    ev1 = torch.cuda.Event(enable_timing=True)
    ev0.record(stream)
    for i in range(args.steps):
        step(i)
    ev1.record(stream)
    torch.cuda.synchronize()
    ms_step = ev0.elapsed_time(ev1) / args.steps
    binding.profile_read()
    binding.profile_enable(True)
    for i in range(args.steps):
        step(i)
    torch.cuda.synchronize()
    binding.profile_enable(False)
    prof = binding.profile_read()
    us = {k: prof[k][0] / prof[k][1] * 1e3 for k in ("stats", "rows", "smc") if prof[k][1]}
    print(f"[bench] smc {args.steps} steps: {ms_step * 1e3:.2f} us/step; kernels {us}", file=sys.stderr, flush=True)
    positions = N * K
    stats_s = us["stats"] * 1e-6
    cpu = None
    if not args.no_cpu_baseline:
        cpu = cpu_baseline_smc(sets, args.cpu_rows, sets[0].workload.name)
    dist = per_call_distribution(torch, stream, step, args.steps)
    line = {
        "metric": "SMC-SD step: scored particle positions/sec + logits HBM GB/s (% of peak) at N=64,K=5,V=128256",
        "value": round(positions / (ms_step / 1e3), 1),
        "unit": "scored positions/s",
        "n_gpus": 1,
        "steps": args.steps,
        "warmup": args.warmup,
        "ms_per_step": round(ms_step, 6),
        "higher_is_better": True,
        "scaling": "weak",
        "vs_baseline": None,
        "dtype": "f32+f64",
        "data": "synthetic",
        "config": {"workload": f"SMC-SD step over the {sets[0].workload.name} inputs as {N} particles",
                   "N": N, "K": K, "V": sets[0].V, "ess_fraction": SMC_ESS_FRACTION,
                   "logical_bytes_per_step": logical,
                   "logits_GBps": round(logical / (ms_step / 1e3) / 1e9, 1)},
        "roofline": {"bound": "hbm", "achieved": round(logical / stats_s / 1e9, 1), "peak": HBM_PEAK_GBS,
                     "unit": "GB/s", "frac": round(logical / stats_s / 1e9 / HBM_PEAK_GBS, 4), "traffic": None,
                     "kernel": "k_stats (statistics pass)", "kernel_us": round(us["stats"], 3),
                     "other_kernels_us": {"k_smc_rows": round(us["rows"], 3),
                                          "k_smc_resample": round(us["smc"], 3)}},
        "per_call": dist,
        "cpu_baseline": cpu,
    }
    print(json.dumps(line), flush=True)


# ---------------------------------------------------------------------------
# Greedy verify timing (--greedy): the batched workload's target logits, drafts
# that agree with the target's argmax at 70 % of positions, top-60
# ---------------------------------------------------------------------------
GREEDY_TOPK = 60


def _greedy_drafts(inp, s):
    import numpy as np

    from rejection_sampling_verifier_amd import workloads

    rng = np.random.default_rng(0x6EED + s)
    t = workloads.bf16_bits_to_f32(inp.target[:, : inp.K])
    am = np.argmax(t, axis=-1)
    return np.where(rng.random(am.shape) < 0.7, am, rng.integers(0, inp.V, size=am.shape)).astype(np.int32)


def _oracle_greedy(args):
    import oracle

    si, r0, r1 = args
    inp, x = _SAMPLE[si]
    oracle.greedy_verify(inp.target[r0:r1], x[r0:r1], None, GREEDY_TOPK)
    return (r1 - r0) * inp.K


def greedy_bench(args, binding, torch, dev, sets):
    import numpy as np

    B, K, V = sets[0].B, sets[0].K, sets[0].V
    xs = [_greedy_drafts(inp, s) for s, inp in enumerate(sets)]

    def put(a):
        return torch.from_numpy(a.view(np.int16)).to(dev).view(torch.bfloat16)

    ds = [(put(inp.target), torch.from_numpy(x).to(dev)) for inp, x in zip(sets, xs)]
    outs = [(torch.empty((B, K + 1), dtype=torch.int32, device=dev), torch.empty((B,), dtype=torch.int32, device=dev),
             torch.empty((B, GREEDY_TOPK), dtype=torch.int32, device=dev)) for _ in range(N_SETS)]
    stream = torch.cuda.current_stream(dev)

    def step(i):
        t, x = ds[i % N_SETS]
        o = outs[i % N_SETS]
        binding.greedy_verify(t, x, None, GREEDY_TOPK, stream=stream, out_tokens=o[0], out_n_accepted=o[1],
                              out_topk=o[2])

    for i in range(args.warmup):
        step(i)
    torch.cuda.synchronize()
    ev0 = torch.cuda.Event(enable_timing=True)
    ev1 = torch.cuda.Event(enable_timing=True)
    ev0.record(stream)
    for i in range(args.steps):
        step(i)
    ev1.record(stream)
    torch.cuda.synchronize()
    ms_step = ev0.elapsed_time(ev1) / args.steps
    binding.profile_read()
    binding.profile_enable(True)
    for i in range(args.steps):
        step(i)
    torch.cuda.synchronize()
    binding.profile_enable(False)
    prof = binding.profile_read()
    us = {k: prof[k][0] / prof[k][1] * 1e3 for k in ("stats", "rows") if prof[k][1]}
    logical = B * (K + 1) * V * 2  # target rows only
    print(f"[bench] greedy {args.steps} steps: {ms_step * 1e3:.2f} us/step; kernels {us}", file=sys.stderr,
          flush=True)
    cpu = None
    if not args.no_cpu_baseline:
        global _SAMPLE
        _SAMPLE = list(zip(sets, xs))
        cores = max(1, min(16, os.cpu_count() or 1))
        work = [(s, r, r + 1) for s in range(N_SETS) for r in range(B)]
        positions, dt, passes = _timed_passes(_oracle_greedy, work, cores)
        cpu = {"value": positions / dt, "unit": "positions/s", "cores": cores, "kind": "oracle",
               "sample": f"{len(work)} rows of the batched workload, {passes} passes ({positions} draft positions), "
                         f"float64 NumPy oracle, one row per task over {cores} processes, {dt:.1f} s wall"}
    stats_s = us["stats"] * 1e-6
    dist = per_call_distribution(torch, stream, step, args.steps)
    line = {
        "metric": "greedy verify + top-60: draft positions/sec + logits HBM GB/s (% of peak) at B=64,K=5,V=128256",
        "value": round(B * K / (ms_step / 1e3), 1),
        "unit": "positions/s",
        "n_gpus": 1,
        "steps": args.steps,
        "warmup": args.warmup,
        "ms_per_step": round(ms_step, 6),
        "higher_is_better": True,
        "scaling": "weak",
        "vs_baseline": None,
        "dtype": "f32",
        "data": "synthetic",
        "config": {"workload": "greedy verify, batched B=64 K=5 V=128256 bf16 target logits, top-60",
                   "B": B, "K": K, "V": V, "k": GREEDY_TOPK, "logical_bytes_per_step": logical,
                   "logits_GBps": round(logical / (ms_step / 1e3) / 1e9, 1)},
        "roofline": {"bound": "hbm", "achieved": round(logical / stats_s / 1e9, 1), "peak": HBM_PEAK_GBS,
                     "unit": "GB/s", "frac": round(logical / stats_s / 1e9 / HBM_PEAK_GBS, 4), "traffic": None,
                     "kernel": "k_stats<…, true> over the target rows", "kernel_us": round(us["stats"], 3),
                     "other_kernels_us": {"k_greedy_rows": round(us["rows"], 3)}},
        "per_call": dist,
        "cpu_baseline": cpu,
    }
    print(json.dumps(line), flush=True)


# ---------------------------------------------------------------------------
# Two-batch schedule (--overlap): batch X is verified on one stream while the
# synthetic draft producer drafts batch Y on a second stream; the roles swap
# every step.  Timed alone, one after the other on one stream, and overlapped.
# ---------------------------------------------------------------------------
def _oracle_overlap(args):
    import oracle

    si, r0, r1 = args
    inp = _SAMPLE[si]
    d, x = oracle.produce_drafts(inp.target[r0:r1], inp.K, 1000 + si)
    oracle.verify(inp.target[r0:r1], d, x, None, inp.temperature, 1.0, inp.seed)
    return (r1 - r0) * inp.K


def overlap_bench(args, binding, torch, dev, sets):
    import numpy as np

    B, K, V = sets[0].B, sets[0].K, sets[0].V
    T = float(sets[0].temperature)

    def put(a):
        return torch.from_numpy(a.view(np.int16)).to(dev).view(torch.bfloat16)

    tgt = [put(sets[i].target) for i in range(2)]
    drafts = [torch.empty((B, K, V), dtype=torch.bfloat16, device=dev) for _ in range(2)]
    toks = [torch.empty((B, K), dtype=torch.int32, device=dev) for _ in range(2)]
    outs = [(torch.empty((B, K + 1), dtype=torch.int32, device=dev), torch.empty((B,), dtype=torch.int32, device=dev))
            for _ in range(2)]
    s0 = torch.cuda.Stream(dev)
    s1 = torch.cuda.Stream(dev)
    produced = [None, None]
    verified = [None, None]

    def produce(y, i, st):
        binding.draft_produce(tgt[y], K, 1000 + i, stream=st, out=drafts[y], out_tokens=toks[y])

    def verify(x, i, st):
        binding.verify(tgt[x], drafts[x], toks[x], None, T, 1.0, 5000 + i, stream=st, out_tokens=outs[x][0],
                       out_n_accepted=outs[x][1])

    def run(mode, n, base, ev=None):
        """Issue n steps.  In the overlapped mode, step i verifies batch i % 2
        on s0 after its drafts exist and drafts batch (i + 1) % 2 on s1 after
        its previous verify; `ev` holds the (produced, verified) events."""
        produced_, verified_ = ev if ev is not None else (produced, verified)
        for i in range(base, base + n):
            x, y = i % 2, (i + 1) % 2
            if mode == "verify":
                verify(x, i, s0)
            elif mode == "produce":
                produce(y, i, s0)
            elif mode == "serial":
                produce(y, i, s0)
                verify(x, i, s0)
            else:
                if produced_[x] is not None:
                    s0.wait_event(produced_[x])
                verify(x, i, s0)
                verified_[x] = torch.cuda.Event()
                verified_[x].record(s0)
                if verified_[y] is not None:
                    s1.wait_event(verified_[y])
                produce(y, i, s1)
                produced_[y] = torch.cuda.Event()
                produced_[y].record(s1)

    # The host needs tens of microseconds to issue one step through the
    # Python binding, so each mode is captured as a HIP graph of GSTEPS steps
    # (the second stream forked from and joined back to the first) and the
    # graph is replayed: the GPU then sees every launch as soon as its
    # dependencies allow.
    GSTEPS = 10

    def graph(mode):
        torch.cuda.synchronize()
        produce(0, 0, s0)
        produce(1, 0, s0)
        run(mode, 2, 0, ([None, None], [None, None]))  # scratch sized on both streams
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s0):
            fork = torch.cuda.Event()
            fork.record(s0)
            s1.wait_event(fork)
            run(mode, GSTEPS, 0, ([None, None], [None, None]))
            join = torch.cuda.Event()
            join.record(s1)
            s0.wait_event(join)
        torch.cuda.synchronize()
        return g

    def timed(mode):
        g = graph(mode)
        reps = max(1, args.steps // GSTEPS)
        for _ in range(max(1, args.warmup // GSTEPS)):
            g.replay()
        torch.cuda.synchronize()
        e0 = torch.cuda.Event(enable_timing=True)
        e1 = torch.cuda.Event(enable_timing=True)
        e0.record(s0)
        for _ in range(reps):
            g.replay()
        e1.record(s0)
        torch.cuda.synchronize()
        return e0.elapsed_time(e1) / (reps * GSTEPS) * 1e3

    with torch.cuda.stream(s0):
        us = {m: timed(m) for m in ("verify", "produce", "serial", "overlap")}
        # the overlapped graph's last verify (step GSTEPS - 1, batch 1) against
        # the same call issued eagerly
        last = GSTEPS - 1
        got = (outs[last % 2][0].clone(), outs[last % 2][1].clone())
        ref = binding.verify(tgt[last % 2], drafts[last % 2], toks[last % 2], None, T, 1.0, 5000 + last, stream=s0)
        torch.cuda.synchronize()
        replay_ok = bool(torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1]))
    # kernel durations inside the overlapped schedule, issued eagerly
    binding.profile_read()
    binding.profile_enable(True)
    run("overlap", args.steps, 1, ([None, None], [None, None]))
    torch.cuda.synchronize()
    binding.profile_enable(False)
    prof = binding.profile_read()
    kus = {k: round(prof[k][0] / prof[k][1] * 1e3, 3) for k in ("stats", "rows", "produce") if prof[k][1]}
    print(f"[bench] two-batch schedule, {args.steps} steps each: {us}; kernels in the overlapped run {kus}",
          file=sys.stderr, flush=True)
    hidden = us["serial"] - us["overlap"]
    prod_bytes = 2 * B * K * V * 2  # the producer reads K target rows and writes K draft rows
    cpu = None
    if not args.no_cpu_baseline:
        global _SAMPLE
        _SAMPLE = sets[:2]
        cores = max(1, min(16, os.cpu_count() or 1))
        work = [(s, r, r + 1) for s in range(2) for r in range(B)]
        positions, dt, passes = _timed_passes(_oracle_overlap, work, cores)
        cpu = {"value": positions / dt, "unit": "positions/s", "cores": cores, "kind": "oracle",
               "sample": f"{len(work)} rows of two batches, {passes} passes ({positions} draft positions), "
                         f"float oracle of the producer then the verify step, one row per task over {cores} "
                         f"processes, {dt:.1f} s wall"}
    line = {
        "metric": "two-batch schedule (verify one batch while drafting the other): draft positions verified/sec "
                  "at B=64,K=5,V=128256",
        "value": round(B * K / (us["overlap"] * 1e-6), 1),
        "unit": "positions/s",
        "n_gpus": 1,
        "steps": args.steps,
        "warmup": args.warmup,
        "ms_per_step": round(us["overlap"] / 1e3, 6),
        "higher_is_better": True,
        "scaling": "weak",
        "vs_baseline": None,
        "dtype": "f32+f64",
        "data": "synthetic",
        "config": {"workload": "two batches of B=64 K=5 V=128256 bf16 T=0.7; verify on stream 0, the synthetic "
                               "draft producer on stream 1, roles swapped every step",
                   "B": B, "K": K, "V": V},
        "overlap": {"verify_alone_us": round(us["verify"], 3), "produce_alone_us": round(us["produce"], 3),
                    "serial_us": round(us["serial"], 3), "overlapped_us": round(us["overlap"], 3),
                    "hidden_us": round(hidden, 3),
                    "hidden_frac_of_shorter": round(hidden / min(us["verify"], us["produce"]), 4)},
        "kernels_us": kus,
        "graph_replay_matches_eager": replay_ok,
        "producer_GBps_alone": round(prod_bytes / (us["produce"] * 1e-6) / 1e9, 1),
        "per_call": None,  # graph replays of whole schedules: no per-call events
        "cpu_baseline": cpu,
    }
    print(json.dumps(line), flush=True)


# ---------------------------------------------------------------------------
# Two-stage verify timing (--hispec): three exit layers of one synthetic
# early-exit model, B=64, K=5, V=128256, bf16, T=0.7
# ---------------------------------------------------------------------------
def _oracle_hispec(args):
    import oracle

    si, r0, r1 = args
    h = _SAMPLE[si]
    oracle.hispec_verify(h.final[r0:r1], h.inter[r0:r1], h.draft[r0:r1], h.draft_tokens[r0:r1], None,
                         h.temperature, h.top_p, h.seed)
    return (r1 - r0) * h.draft.shape[1]


def hispec_bench(args, binding, torch, dev):
    import numpy as np

    from rejection_sampling_verifier_amd import workloads

    B, K, V = 64, 5, workloads.V_LLAMA3
    print(f"[bench] generating {N_SETS} three-layer input sets", file=sys.stderr, flush=True)
    hs = [workloads.make_hispec_inputs(B, K, V, dtype="bf16", step=s, temperature=0.7) for s in range(N_SETS)]

    def put(a):
        return torch.from_numpy(a.view(np.int16)).to(dev).view(torch.bfloat16)

    ds = [(put(h.final), put(h.inter), put(h.draft), torch.from_numpy(h.draft_tokens).to(dev), float(h.temperature),
           h.seed) for h in hs]
    outs = [(torch.empty((B, K + 2), dtype=torch.int32, device=dev), torch.empty((B,), dtype=torch.int32, device=dev),
             torch.empty((B,), dtype=torch.int32, device=dev)) for _ in range(N_SETS)]
    stream = torch.cuda.current_stream(dev)

    def step(i):
        f, it, d, x, T, seed = ds[i % N_SETS]
        o = outs[i % N_SETS]
        binding.hispec_verify(f, it, d, x, None, T, 1.0, seed, stream=stream, out_tokens=o[0], out_n_accepted=o[1],
                              out_n_stage1=o[2])

    for i in range(args.warmup):
        step(i)
    torch.cuda.synchronize()
    # logical bytes: stage 1 reads 2K + 1 rows per batch row, stage 2
    # 2 (n1 + 1) + 1 rows (n1 from each set's own result)
    rows = []
    for s in range(N_SETS):
        n1 = outs[s][2].cpu().numpy()
        rows.append(B * (2 * K + 1) + int(np.sum(2 * (n1 + 1) + 1)))
    logical = sum(rows) / N_SETS * V * 2
    ev0 = torch.cuda.Event(enable_timing=True)
    ev1 = torch.cuda.Event(enable_timing=True)
    ev0.record(stream)
    for i in range(args.steps):
        step(i)
    ev1.record(stream)
    torch.cuda.synchronize()
    ms_step = ev0.elapsed_time(ev1) / args.steps
    binding.profile_read()
    binding.profile_enable(True)
    for i in range(args.steps):
        step(i)
    torch.cuda.synchronize()
    binding.profile_enable(False)
    prof = binding.profile_read()
    us = {k: prof[k][0] / prof[k][1] * 1e3 for k in ("stats", "rows") if prof[k][1]}
    print(f"[bench] hispec {args.steps} steps: {ms_step * 1e3:.2f} us/step; per-kernel averages over both stages "
          f"{us}", file=sys.stderr, flush=True)
    cpu = None
    if not args.no_cpu_baseline:
        global _SAMPLE
        _SAMPLE = hs
        cores = max(1, min(16, os.cpu_count() or 1))
        work = [(s, r, r + 1) for s in range(N_SETS) for r in range(B)]
        positions, dt, passes = _timed_passes(_oracle_hispec, work, cores)
        cpu = {"value": positions / dt, "unit": "positions/s", "cores": cores, "kind": "oracle",
               "sample": f"{len(work)} rows of the three-layer workload, {passes} passes ({positions} draft "
                         f"positions), float64 NumPy oracle, one row per task over {cores} processes, "
                         f"{dt:.1f} s wall"}
    dist = per_call_distribution(torch, stream, step, args.steps)
    line = {
        "metric": "two-stage verify: draft positions/sec + logits HBM GB/s (% of peak) at B=64,K=5,V=128256",
        "value": round(B * K / (ms_step / 1e3), 1),
        "unit": "positions/s",
        "n_gpus": 1,
        "steps": args.steps,
        "warmup": args.warmup,
        "ms_per_step": round(ms_step, 6),
        "higher_is_better": True,
        "scaling": "weak",
        "vs_baseline": None,
        "dtype": "f32+f64",
        "data": "synthetic",
        "config": {"workload": "two-stage verify B=64 K=5 V=128256 bf16 T=0.7 (final, intermediate, draft layers)",
                   "B": B, "K": K, "V": V, "logical_bytes_per_step": logical,
                   "logits_GBps": round(logical / (ms_step / 1e3) / 1e9, 1),
                   "logits_frac_of_peak": round(logical / (ms_step / 1e3) / 1e9 / HBM_PEAK_GBS, 4)},
        "kernels_us": {"k_stats (per stage)": round(us["stats"], 3), "k_rows (per stage)": round(us["rows"], 3)},
        "per_call": dist,
        "cpu_baseline": cpu,
    }
    print(json.dumps(line), flush=True)


# ---------------------------------------------------------------------------
# --tree: a round of a drafted tree over a paged cache
# ---------------------------------------------------------------------------
TREE = dict(B=64, N=16, branch=3, layers=2, heads=32, kv_heads=8, dim=128, page=64, length=4096)


def _oracle_tree(args):
    """One sequence: the attention of one key head's queries (times key heads
    and layers that is the sequence's attention) and the verification."""
    import numpy as np

    from oracle import tree

    q, k, v, kt, vt, par, p, qd, tok, ua, uf = _SAMPLE[args]
    # the sequence's rows as one page
    tree.tree_attention(q[None], k[None, :, None], v[None, :, None], np.zeros((1, 1), np.int32), np.array([len(k)]),
                        kt[None], vt[None], par[None])
    tree.verify_tree(p[None], qd[None], tok[None], par[None], ua[None], uf[None])
    return 1


def tree_bench(args, binding, torch, dev):
    """A step: the attention of every layer, the verification and the commit of
    the accepted rows (written behind the same lengths each time), and beside
    it the fork of a set of particles."""
    import numpy as np

    from rejection_sampling_verifier_amd import workloads

    c = TREE
    B, N, L, H, Hkv, D, ps, V = (c["B"], c["N"], c["layers"], c["heads"], c["kv_heads"], c["dim"], c["page"],
                                 workloads.V_LLAMA3)
    rng = np.random.default_rng(11)
    gen = torch.Generator(device=dev).manual_seed(11)
    print(f"[bench] generating the tree round: {B} sequences, {N} nodes, {L} layers", file=sys.stderr, flush=True)
    lens_h = rng.integers(c["length"] // 2, c["length"] + 1, B).astype(np.int32)
    blocks = -(-lens_h // ps)
    width = int(blocks.max()) + 2
    pages = int(blocks.sum()) + 2 * B
    perm, at = rng.permutation(pages), 0
    table_h = np.full((B, width), -1, np.int32)
    for b in range(B):
        table_h[b, :blocks[b]] = perm[at:at + blocks[b]]
        at += blocks[b]
    par_h = np.full((B, N), -1, np.int32)
    par_h[:, 1:] = (np.arange(1, N) - 1) // c["branch"]
    P = int(par_h.max()) + 1

    def rows(*s):
        return torch.randn(s, generator=gen, device=dev, dtype=torch.float32).to(torch.bfloat16)

    k, v = rows(L, pages, ps, Hkv, D), rows(L, pages, ps, Hkv, D)
    kt, vt, q = rows(L, B, N, Hkv, D), rows(L, B, N, Hkv, D), rows(L, B, N, H, D)
    table, lens, par = (torch.from_numpy(a).to(dev) for a in (table_h, lens_h, par_h))
    logits = torch.randn((B, N, V), generator=gen, device=dev) * 2
    qd = torch.softmax(logits[:, :P] + 0.7 * torch.randn((B, P, V), generator=gen, device=dev), -1)
    p = torch.softmax(logits, -1)
    del logits
    tok = torch.zeros((B, N), dtype=torch.int32, device=dev)
    for i in range(1, N):
        tok[:, i] = torch.multinomial(qd[:, int(par_h[0, i])], 1, generator=gen)[:, 0].int()
    ua = torch.from_numpy(rng.random((B, N), np.float32)).to(dev)
    uf = torch.from_numpy(rng.random(B, np.float32)).to(dev)
    anc = torch.from_numpy((np.arange(B) // 2 * 2).astype(np.int32)).to(dev)
    outs = [torch.empty_like(q[i]) for i in range(L)]
    stream = torch.cuda.current_stream(dev)
    last = {}

    def step(i):
        for j in range(L):
            binding.tree_attention(q[j], k[j], v[j], table, lens, kt[j], vt[j], par, out=outs[j])
        _, nodes, last["n"] = binding.verify_tree(p, qd, tok, par, ua, uf)
        last["status"] = binding.cache_commit(k, v, table, lens, kt, vt, nodes, last["n"])[2]

    def fork(i):
        last["status"] = binding.cache_fork(k, v, table, lens, anc)[2]

    def timed(fn):
        for i in range(args.warmup):
            fn(i)
        torch.cuda.synchronize()
        assert int(last["status"]) == 0
        e0, e1 = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        e0.record(stream)
        for i in range(args.steps):
            fn(i)
        e1.record(stream)
        torch.cuda.synchronize()
        ms = e0.elapsed_time(e1) / args.steps
        binding.profile_read()
        binding.profile_enable(True)
        for i in range(args.steps):
            fn(i)
        torch.cuda.synchronize()
        binding.profile_enable(False)
        return ms, {kind: round(x[0] / x[1] * 1e3, 3) for kind, x in binding.profile_read().items() if x[1]}

    ms_step, us = timed(step)
    fork_ms, fork_us = timed(fork)
    n = last["n"].cpu().numpy()
    kv_bytes = 2 * int(lens_h.sum()) * Hkv * D * 2
    print(f"[bench] tree round {args.steps} steps: {ms_step * 1e3:.2f} us/step, fork {fork_ms * 1e3:.2f} us; kernels {us}",
          file=sys.stderr, flush=True)
    dist = per_call_distribution(torch, stream, step, args.steps)
    cpu = None
    if not args.no_cpu_baseline:
        global _SAMPLE
        h = lambda t: t.double().cpu().numpy()  # noqa: E731
        _SAMPLE = []
        for b in range(8):
            pg = torch.from_numpy(table_h[b, :blocks[b]].astype(np.int64)).to(dev)
            kk, vv = (h(x[0, pg, :, 0].reshape(-1, D)[:lens_h[b]]) for x in (k, v))
            _SAMPLE.append((h(q[0, b, :, :H // Hkv]), kk, vv, h(kt[0, b, :, :1]), h(vt[0, b, :, :1]), par_h[b], h(p[b]),
                            h(qd[b]), tok[b].cpu().numpy(), ua[b].cpu().numpy(), uf[b:b + 1].cpu().numpy()[0]))
        cores = max(1, min(8, os.cpu_count() or 1))
        done, dt, passes = _timed_passes(_oracle_tree, list(range(8)), cores)
        cpu = {"value": done * N / dt, "unit": "nodes/s", "cores": cores, "kind": "oracle",
               "sample": f"8 sequences of the tree round, one key head of one layer and the verification each, {passes} "
                         f"passes, float64 NumPy oracle over {cores} processes, {dt:.1f} s wall"}
    line = {
        "metric": "tree round: nodes attended and verified/sec + cache HBM GB/s (% of peak) at B=64,N=16,V=128256",
        "value": round(B * N / (ms_step / 1e3), 1),
        "unit": "nodes/s",
        "n_gpus": 1,
        "steps": args.steps,
        "warmup": args.warmup,
        "ms_per_step": round(ms_step, 6),
        "higher_is_better": True,
        "scaling": "weak",
        "vs_baseline": None,
        "dtype": "bf16 attention, f64 verification",
        "data": "synthetic",
        "config": {"workload": f"tree round B={B} N={N} (branches of {c['branch']}) {L} layers {H}/{Hkv} heads of {D}, "
                               f"{int(lens_h.min())}..{int(lens_h.max())} cached rows, V={V} fp32 probabilities",
                   "accepted_per_sequence": round(float(n.mean()), 3), "cache_bytes_per_layer": kv_bytes,
                   "attention_GBps": round(kv_bytes / (us["tree_attention"] / 1e6) / 1e9, 1),
                   "attention_frac_of_peak": round(kv_bytes / (us["tree_attention"] / 1e6) / 1e9 / HBM_PEAK_GBS, 4)},
        "kernels_us": us,
        "fork": {"us_per_call": round(fork_ms * 1e3, 3), "kernels_us": fork_us},
        "per_call": dist,
        "cpu_baseline": cpu,
    }
    print(json.dumps(line), flush=True)


# ---------------------------------------------------------------------------
# --beams: a step of beam decoding with latent attention
# ---------------------------------------------------------------------------
BEAMS = dict(B=8, W=4, layers=2, heads=128, dim_k=128, dim_p=64, dim_v=128, latent=512, page=64, length=4096, prompt=1024)


def beam_bench(args, binding, torch, dev):
    """A step: rows reserved for every beam's token; in every layer queries into
    the latent space, attention on the rows, results out of it, the new rows
    written; then the selection, the fork of the pages and the histories.  Every
    step starts from the same tables and lengths.  Beside it the attention of a
    batch of prompts in one layer."""
    import numpy as np

    from rejection_sampling_verifier_amd import workloads

    c = BEAMS
    B, W, L, H, R, DP, DK, DV, ps, V = (c["B"], c["W"], c["layers"], c["heads"], c["latent"], c["dim_p"], c["dim_k"],
                                        c["dim_v"], c["page"], workloads.V_LLAMA3)
    n, C = B * W, R + DP
    rng = np.random.default_rng(12)
    gen = torch.Generator(device=dev).manual_seed(12)
    print(f"[bench] generating the beam step: {B} requests of {W} beams, {L} layers", file=sys.stderr, flush=True)
    lens_h = np.repeat(rng.integers(c["length"] // 2, c["length"] + 1, B), W).astype(np.int32)
    blocks = -(-lens_h // ps)
    width, pages = int(blocks.max()) + 2, int(blocks.sum()) + 3 * n
    perm, at = rng.permutation(pages), 0
    table_h = np.full((n, width), -1, np.int32)
    for b in range(n):
        table_h[b, :blocks[b]] = perm[at:at + blocks[b]]
        at += blocks[b]

    def rows(*s, by=1.0):
        return (torch.randn(s, generator=gen, device=dev) * by).to(torch.bfloat16)

    cache = rows(L, pages, ps, C)
    q, latent, turned = rows(L, n, H, DK + DP), rows(L, n, R), rows(L, n, DP)
    w_k, w_v = rows(L, H, DK, R, by=R ** -0.5), rows(L, H, DV, R, by=R ** -0.5)
    w_in = w_k.transpose(2, 3).contiguous()
    table, lens = (torch.from_numpy(a).to(dev) for a in (table_h, lens_h))
    ones = torch.ones((n,), dtype=torch.int32, device=dev)
    logits = rows(B, W, V, by=2.0)
    scores = -torch.rand((B, W), generator=gen, device=dev).sort(-1)[0]
    history = torch.zeros((n, c["length"]), dtype=torch.int32, device=dev)
    # the fork takes a row's halves, as it would keys and values
    k, v = cache[..., None, :C // 2], cache[..., None, C // 2:]
    absorbed = torch.cat((rows(L, n, H, R), q[..., DK:]), -1)[:, :, None]
    own = torch.cat((latent, turned), -1)[:, :, None]
    scale = (DK + DP) ** -0.5
    stream = torch.cuda.current_stream(dev)
    last = {}

    def step(i):
        t, m, _, slots, _, last["reserved"] = binding.cache_reserve(table, lens, ones, pages=pages, page_size=ps, rows=n)
        for j in range(L):
            binding.head_product(q[j][..., :DK], w_in[j], out=absorbed[j, :, 0, :, :R])
            mid = binding.latent_attention(absorbed[j], cache[j], table, lens, own[j], dim_v=R, scale=scale)
            last["out"] = binding.head_product(mid[:, 0], w_v[j])
            binding.cache_write(cache[j], slots, latent[j], turned[j])
        anc = binding.beam_select(logits, scores)[1]
        last["status"] = binding.cache_fork(k, v, t, m, anc)[2]
        binding.beam_reorder(history, anc)

    T = 4 * c["prompt"]
    start = torch.arange(0, T + 1, c["prompt"], dtype=torch.int32, device=dev)
    first, four = torch.full((4,), c["prompt"], dtype=torch.int32, device=dev), table[::W][:4].contiguous()
    pq = rows(T, H, DK + DP)

    def prompt(i):
        last["out"] = binding.latent_prompt(pq, cache[0], four, first, start, w_k[0], w_v[0], rows=T)

    def timed(fn, steps):
        for i in range(min(args.warmup, steps)):
            fn(i)
        torch.cuda.synchronize()
        e0, e1 = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        e0.record(stream)
        for i in range(steps):
            fn(i)
        e1.record(stream)
        torch.cuda.synchronize()
        ms = e0.elapsed_time(e1) / steps
        binding.profile_read()
        binding.profile_enable(True)
        for i in range(steps):
            fn(i)
        torch.cuda.synchronize()
        binding.profile_enable(False)
        return ms, {kind: round(x[0] / x[1] * 1e3, 3) for kind, x in binding.profile_read().items() if x[1]}

    ms_step, us = timed(step, args.steps)
    assert int(last["reserved"]) == 0 and int(last["status"]) == 0
    prompt_ms, prompt_us = timed(prompt, max(1, args.steps // 10))
    cache_bytes = 2 * int(lens_h.sum()) * C
    print(f"[bench] beam step {args.steps} steps: {ms_step * 1e3:.2f} us/step, prompts {prompt_ms * 1e3:.2f} us; kernels "
          f"{us}", file=sys.stderr, flush=True)
    line = {
        "metric": "beam step: beams' tokens attended and selected/sec at B=8,W=4,V=128256",
        "value": round(n / (ms_step / 1e3), 1),
        "unit": "tokens/s",
        "n_gpus": 1,
        "steps": args.steps,
        "warmup": args.warmup,
        "ms_per_step": round(ms_step, 6),
        "higher_is_better": True,
        "scaling": "weak",
        "vs_baseline": None,
        "dtype": "bf16",
        "data": "synthetic",
        "config": {"workload": f"beam step B={B} W={W} {L} layers {H} heads on rows of {R} + {DP}, "
                               f"{int(lens_h.min())}..{int(lens_h.max())} cached rows, V={V} bf16 logits",
                   "cache_bytes_per_layer": cache_bytes,
                   "attention_GBps": round(cache_bytes / (us["latent_attention"] / 1e6) / 1e9, 1),
                   "attention_TFLOPs": round(2 * int(lens_h.sum()) * H * (C + R) / us["latent_attention"] / 1e6, 1)},
        "kernels_us": us,
        "prompts": {"tokens": T, "us_per_call": round(prompt_ms * 1e3, 3), "kernels_us": prompt_us},
        "per_call": per_call_distribution(torch, stream, step, args.steps),
    }
    print(json.dumps(line), flush=True)


# ---------------------------------------------------------------------------
# GPU timing
# ---------------------------------------------------------------------------
def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--gpus", type=int, default=1)
    ap.add_argument("--steps", type=int, default=1000)
    ap.add_argument("--warmup", type=int, default=500)
    ap.add_argument("--no-cpu-baseline", action="store_true")
    ap.add_argument("--cpu-rows", type=int, default=192)
    ap.add_argument("--workload", type=int, default=WORKLOAD_CFG,
                    help="seeded workload to time (default: the batched B=64 K=5 V=128256 bf16 one)")
    ap.add_argument("--greedy", action="store_true",
                    help="time greedy verify with the top-60 (spec_greedy_verify) on the batched target logits")
    ap.add_argument("--two-batches", action="store_true",
                    help="also time the batched calls with two independent batches in flight on two streams")
    ap.add_argument("--overlap", action="store_true",
                    help="time the two-batch schedule: verify on one stream, the synthetic draft producer on another")
    ap.add_argument("--hispec", action="store_true",
                    help="time the two-stage verify (spec_hispec_verify) on three synthetic exit layers")
    ap.add_argument("--tree", action="store_true",
                    help="time a round of drafted trees over a paged cache: spec_tree_attention per layer, "
                         "spec_verify_tree, spec_cache_commit; and spec_cache_fork")
    ap.add_argument("--beams", action="store_true",
                    help="time a step of beam decoding on a cache of latent rows: spec_cache_reserve, per layer "
                         "spec_head_product, spec_latent_attention and spec_cache_write, then spec_beam_select, "
                         "spec_cache_fork and spec_beam_reorder; and spec_latent_prompt")
    ap.add_argument("--smc", action="store_true",
                    help="time the SMC-SD step (spec_smc_step) on the same inputs instead of the verify step")
    ap.add_argument("--calibrate", action="store_true",
                    help="after timing, run a plain device copy and a streaming read of known sizes, the "
                         "references that scale hardware byte counters to bytes")
    args = ap.parse_args()
    if args.gpus != 1 or int(os.environ.get("WORLD_SIZE", "1")) != 1:
        print("bench.py measures one GPU only: the verify step is built and timed on a single MI355X "
              "(batch rows shard across GPUs with no exchange: each GPU runs this step on its own rows).",
              file=sys.stderr)
        sys.exit(2)

    import numpy as np
    import torch

    from rejection_sampling_verifier_amd import binding, workloads

    assert torch.cuda.is_available(), "bench.py needs a GPU"
    binding.load()
    dev = torch.device("cuda:0")
    torch.cuda.set_device(dev)

    if args.hispec:
        hispec_bench(args, binding, torch, dev)
        return
    if args.tree:
        tree_bench(args, binding, torch, dev)
        return
    if args.beams:
        beam_bench(args, binding, torch, dev)
        return

    print(f"[bench] generating {N_SETS} input sets of workload {args.workload}", file=sys.stderr, flush=True)
    sets = [workloads.make_inputs(args.workload, s) for s in range(N_SETS)]
    w = sets[0].workload

    def put(a):
        if a.dtype == np.uint16:
            return torch.from_numpy(a.view(np.int16)).to(dev).view(torch.bfloat16)
        return torch.from_numpy(a).to(dev)

    dsets = []
    for inp in sets:
        dsets.append((put(inp.target), put(inp.draft), torch.from_numpy(inp.draft_tokens).to(dev),
                      None if inp.draft_len is None else torch.from_numpy(inp.draft_len).to(dev),
                      float(inp.temperature), float(inp.top_p), inp.seed))
    B, K = sets[0].B, sets[0].K
    outs = [(torch.empty((B, K + 1), dtype=torch.int32, device=dev), torch.empty((B,), dtype=torch.int32, device=dev))
            for _ in range(N_SETS)]
    # per-call averages over the rotated sets (ragged workloads differ by set)
    logical = sum(s.logical_bytes() for s in sets) / N_SETS
    positions = sum(s.positions() for s in sets) / N_SETS
    stream = torch.cuda.current_stream(dev)

    if args.smc:
        smc_bench(args, binding, torch, dev, sets, dsets, logical, stream)
        return
    if args.greedy:
        greedy_bench(args, binding, torch, dev, sets)
        return
    if args.overlap:
        overlap_bench(args, binding, torch, dev, sets)
        return

    def step(i):
        t, d, x, dl, T, tp, seed = dsets[i % N_SETS]
        o = outs[i % N_SETS]
        binding.verify(t, d, x, dl, T, tp, seed, stream=stream, out_tokens=o[0],
                       out_n_accepted=o[1])

    device_warmup(binding, torch, dev, dsets)
    print(f"[bench] warmup {args.warmup}", file=sys.stderr, flush=True)
    for i in range(args.warmup):
        step(i)
    torch.cuda.synchronize()

    # timed region 1: whole calls
    ev0 = torch.cuda.Event(enable_timing=True)
    ev1 = torch.cuda.Event(enable_timing=True)
    torch.cuda.synchronize()
    ev0.record(stream)
    for i in range(args.steps):
        step(i)
    ev1.record(stream)
    torch.cuda.synchronize()
    ms_total = ev0.elapsed_time(ev1)
    ms_step = ms_total / args.steps
    print(f"[bench] {args.steps} steps: {ms_step * 1e3:.2f} us/step", file=sys.stderr, flush=True)
    dist = per_call_distribution(torch, stream, step, args.steps)
    print(f"[bench] per call: median {dist['median_us']} us, p10 {dist['p10_us']}, p90 {dist['p90_us']}",
          file=sys.stderr, flush=True)

    # timed region 2: per-kernel HIP events recorded by the library on the
    # launch stream around every kernel
    binding.profile_read()
    binding.profile_enable(True)
    torch.cuda.synchronize()
    for i in range(args.steps):
        step(i)
    torch.cuda.synchronize()
    binding.profile_enable(False)
    prof = binding.profile_read()
    stats_ms, stats_n = prof["stats"]
    res_ms, res_n = prof["rows"]
    stats_avg_s = stats_ms / 1e3 / max(stats_n, 1)
    achieved = logical / stats_avg_s / 1e9
    print(f"[bench] statistics kernel {stats_ms / max(stats_n, 1) * 1e3:.2f} us, row kernel "
          f"{res_ms / max(res_n, 1) * 1e3:.2f} us ({stats_n} launches)", file=sys.stderr, flush=True)
    kernels_sum_us = (stats_ms + res_ms + prof["topp"][0]) / max(stats_n, 1) * 1e3

    # timed region 3 (--two-batches): the same calls with two independent
    # batches in flight (calls alternate between two streams, nothing orders
    # them), as a serving loop that keeps two batches (MineDraft's
    # batch-parallel schedule) would issue them.  Reported beside the
    # sequential figure; off by default so that a kernel trace of the default
    # run holds sequential calls only.
    two = None
    if args.two_batches:
        stream_b = torch.cuda.Stream(dev)
        outs2 = [(torch.empty((B, K + 1), dtype=torch.int32, device=dev),
                  torch.empty((B,), dtype=torch.int32, device=dev)) for _ in range(2 * N_SETS)]

        def step2(i):
            t, d, x, dl, T, tp, seed = dsets[i % N_SETS]
            o = outs2[i % (2 * N_SETS)]
            binding.verify(t, d, x, dl, T, tp, seed, stream=stream if i % 2 == 0 else stream_b, out_tokens=o[0],
                           out_n_accepted=o[1])

        for i in range(min(args.warmup, 200)):
            step2(i)
        torch.cuda.synchronize()
        e0 = torch.cuda.Event(enable_timing=True)
        e1 = torch.cuda.Event(enable_timing=True)
        e0.record(stream)
        stream_b.wait_event(e0)
        for i in range(args.steps):
            step2(i)
        joined = torch.cuda.Event()
        joined.record(stream_b)
        stream.wait_event(joined)
        e1.record(stream)
        torch.cuda.synchronize()
        ms_step2 = e0.elapsed_time(e1) / args.steps
        print(f"[bench] two batches in flight: {ms_step2 * 1e3:.2f} us per call", file=sys.stderr, flush=True)
        two = {"us_per_call": round(ms_step2 * 1e3, 3),
               "positions_per_s": round(positions / (ms_step2 / 1e3), 1),
               "logits_GBps": round(logical / (ms_step2 / 1e3) / 1e9, 1),
               "logits_frac_of_peak": round(logical / (ms_step2 / 1e3) / 1e9 / HBM_PEAK_GBS, 4)}

    traffic = stored_traffic(w.name)
    roofline = {
        "bound": "hbm",
        "achieved": round(achieved, 1),
        "peak": HBM_PEAK_GBS,
        "unit": "GB/s",
        "frac": round(achieved / HBM_PEAK_GBS, 4),
        "traffic": traffic,
        "kernel": "k_stats (statistics pass: every needed logit row read once)",
        "kernel_us": round(stats_avg_s * 1e6, 3),
        "kernels_sum_us": round(kernels_sum_us, 3),
        "timing": "per-dispatch HIP events on the launch stream over a second region of the same calls",
        "other_kernels_us": dict({"k_rows": round(res_ms / max(res_n, 1) * 1e3, 3)},
                                 **({"k_topp": round(prof["topp"][0] / prof["topp"][1] * 1e3, 3)}
                                    if prof["topp"][1] else {})),
        "algorithmic_bytes_per_launch": logical,
    }

    calib = None
    if args.calibrate:
        calib = calibrate(binding, torch, dev, logical)
        roofline["frac_of_stream_read"] = round(calib["stream_read_us"] / (stats_avg_s * 1e6), 4)

    cpu = None
    if not args.no_cpu_baseline:
        print("[bench] cpu baseline (oracle)", file=sys.stderr, flush=True)
        cpu = cpu_baseline(sets, args.cpu_rows, w.name)

    value = positions / (ms_step / 1e3)
    line = {
        "metric": "verified draft positions/sec + logits HBM GB/s (% of peak) at B=64,K=5,V=128256",
        "value": round(value, 1),
        "unit": "positions/s",
        "n_gpus": 1,
        "steps": args.steps,
        "warmup": args.warmup,
        "ms_per_step": round(ms_step, 6),
        "higher_is_better": True,
        "scaling": "weak",
        "vs_baseline": None,
        "dtype": "f32+f64",
        "data": "synthetic",
        "config": {
            "workload": w.name,
            "B": B, "K": K, "V": sets[0].V, "temperature": float(sets[0].temperature),
            "top_p": float(sets[0].top_p), "logits_dtype": w.dtype,
            "arithmetic": "statistics pass: fp32 exp2 and lane/wave sums, fp64 merges; decisions fp64; the draw "
                          "fp64 throughout (exponentials, normalisers, masses)",
            "logical_bytes_per_step": logical,
            "positions_per_step": positions,
            "logits_GBps": round(logical / (ms_step / 1e3) / 1e9, 1),
            "logits_frac_of_peak": round(logical / (ms_step / 1e3) / 1e9 / HBM_PEAK_GBS, 4),
            "input_sets_rotated": N_SETS,
            "parallelism": "single GPU",
        },
        "roofline": roofline,
        "per_call": dist,
        "cpu_baseline": cpu,
        **({"two_batches_in_flight": two} if two else {}),
        **({"calibration": calib} if calib else {}),
    }
    print(json.dumps(line), flush=True)


if __name__ == "__main__":
    main()
