"""Time one operation of the serving iteration alone, through the C ABI.

    python -m intra_device_overlapped_b200.opbench --op decode_attention --workload llama3_8b_layer \
        --requests 64 --sm 16 --reps 5

Ops: ``decode_attention`` (requests [0, --requests) of the workload's decode batch, KV read from the
paged pool), ``prefill_attention`` (the workload's prefill chunk), ``gemm`` (--m x --n x --k bf16,
random operands), ``iteration`` (whole serving iterations of the workload with a plan forced by
--nano / --template / --sm-attn, the sequential one by default; one iteration of the Llama-3-8B
layer launches the QKV, O, gate/up and down GEMMs in that order; --persistent runs each layer as
one persistent kernel instead), and on the workload's decode batch, over a 4-bit KV cache of one layer,
``kv4_decode_attention`` and the operations that feed it: ``page_map``, ``rope``, ``kv4_append`` and
``kv4_read`` (the last two on --rows rows in place of the batch's, if given). ``--sm`` is the persistent grid (0 = every SM). The printed line holds the mean
launch time over --reps launches (CUDA events on the launching stream, after --warmup launches) and
the algorithmic bytes or FLOPs of one launch, so that a profiler can target a small, known case.
--power-s S adds the op's steady state under load: S seconds of back-to-back launches after 1 s,
with the median SM clock and board power that nvidia-smi samples meanwhile.
"""
from __future__ import annotations

import argparse
import json

import numpy as np
import torch

from . import (NF_DTYPE_BF16, NF_DTYPE_F32, check, nf_kv4_page_bytes, nf_kv4_workspace_bytes, nf_op_decode_attention,
               nf_op_gemm_bf16, nf_op_kv4_append, nf_op_kv4_decode_attention, nf_op_kv4_read, nf_op_page_map,
               nf_op_prefill_attention, nf_op_rope, nf_rope_config, nf_rope_frequencies)

KV4_OPS = ("kv4_decode_attention", "kv4_append", "kv4_read", "rope", "page_map")


def _power(launch, seconds: float, stream) -> dict:
    """Steady state of `launch` run back to back: 1 s of warm-up, then `seconds` of launches while
    nvidia-smi samples the SM clock and the board power every 50 ms (medians reported)."""
    import statistics
    import subprocess
    import threading
    import time
    smi = subprocess.Popen(["nvidia-smi", "--id=0", "--query-gpu=clocks.sm,power.draw,clocks_event_reasons.active",
                            "--format=csv,noheader,nounits", "-lms", "50"], stdout=subprocess.PIPE, text=True)
    lines = []
    reader = threading.Thread(target=lambda: [lines.append(x.strip()) for x in smi.stdout], daemon=True)
    reader.start()
    try:
        t0 = time.time()
        while time.time() - t0 < 1.0:
            for _ in range(8):
                launch()
            torch.cuda.synchronize()
        mark = len(lines)
        e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        n = 0
        e0.record(stream)
        t0 = time.time()
        while time.time() - t0 < seconds:
            for _ in range(8):
                launch()
            n += 8
            torch.cuda.synchronize()
        e1.record(stream)
        torch.cuda.synchronize()
        rows = [x.split(",") for x in lines[mark:] if x.count(",") == 2]
    finally:
        smi.terminate()
    sm = [float(r[0]) for r in rows if r[0].strip()]
    pw = [float(r[1]) for r in rows if r[1].strip()]
    return {"steady_us": round(e0.elapsed_time(e1) * 1000.0 / max(n, 1), 2),
            "sm_mhz": statistics.median(sm) if sm else None, "power_w": statistics.median(pw) if pw else None,
            "samples": len(sm), "reasons": sorted({r[2].strip() for r in rows})}


def _time(launch, reps: int, warmup: int, stream) -> float:
    for _ in range(warmup):
        launch()
    torch.cuda.synchronize()
    e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    e0.record(stream)
    for _ in range(reps):
        launch()
    e1.record(stream)
    torch.cuda.synchronize()
    return e0.elapsed_time(e1) * 1000.0 / reps


def _kv4(args, w, dev, stream):
    """One operation over a 4-bit cache of one layer of workload `w`: (launch, figures, bytes of one launch, status word)."""
    from synth.workloads import make_batch
    s, b = w.shape, make_batch(w)
    R = args.requests or b.num_decode
    nq, nkv, d = s.n_q_heads, s.n_kv_heads, s.head_dim
    g = torch.Generator(device=dev).manual_seed(0)
    i32 = lambda a: torch.as_tensor(np.ascontiguousarray(a, dtype=np.int32), device=dev)  # noqa: E731
    randn = lambda *n: torch.randn(n, device=dev, generator=g)  # noqa: E731
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    ctx, st = np.asarray(b.ctx_lens[:R]), stream.cuda_stream
    pages = -(-(ctx + 1) // s.page_size)
    num_pages = int(b.num_pages)
    if args.op == "page_map":
        held = -(-ctx // s.page_size)
        width = int(pages.max())
        table = np.zeros((R, width))
        for r in range(R):
            table[r, :held[r]] = b.page_indices[b.page_indptr[r]:b.page_indptr[r] + held[r]]
        spare = i32(np.concatenate([b.page_indices[b.page_indptr[r] + held[r]:b.page_indptr[r + 1]] for r in range(R)] +
                                   [np.zeros(1)]))
        lens, table, count, left = i32(ctx), i32(table), i32([spare.numel()]), i32([0])
        out = [torch.empty(n, dtype=torch.int32, device=dev) for n in (R, R + 1, int(pages.sum()), R, R)]
        launch = lambda: check(nf_op_page_map(  # noqa: E731
            lens.data_ptr(), 0, R, table.data_ptr(), width, spare.data_ptr(), spare.numel(), count.data_ptr(), num_pages,
            out[0].data_ptr(), out[1].data_ptr(), out[2].data_ptr(), out[2].numel(), out[3].data_ptr(), out[4].data_ptr(),
            R, left.data_ptr(), status.data_ptr(), st), "page_map")
        return launch, {"requests": R, "pages": int(pages.sum())}, 8 * int(pages.sum()) + 24 * R, status
    if args.op == "rope":
        T = args.rows or R
        rows, pos = randn(T, (nq + 2 * nkv) * d), i32(np.resize(ctx, T))
        code, freq, scale = nf_rope_frequencies(nf_rope_config(theta=s.rope_theta, rot_dim=d))
        check(code, "rope frequencies")
        freq = torch.tensor(freq, dtype=torch.float64, device=dev)
        q, k = (torch.empty((T, n, d), dtype=torch.bfloat16, device=dev) for n in (nq, nkv))
        launch = lambda: check(nf_op_rope(  # noqa: E731
            rows.data_ptr(), rows.stride(0), q.data_ptr(), nq * d, nq, rows.data_ptr() + 4 * nq * d, rows.stride(0),
            k.data_ptr(), nkv * d, nkv, NF_DTYPE_F32, NF_DTYPE_BF16, pos.data_ptr(), T, d, d, 0, freq.data_ptr(), scale,
            st), "rope")
        return launch, {"rows": T}, T * (nq + nkv) * d * 6, status
    pool = torch.randint(0, 256, (num_pages, nkv, 2, 9 * d), dtype=torch.uint8, device=dev, generator=g)
    pool[..., 8 * d:].view(torch.bfloat16).fill_(0.1)
    assert pool[0].numel() == nf_kv4_page_bytes(nkv, d)
    if args.op == "kv4_decode_attention":
        size = nf_kv4_workspace_bytes(nq, nkv, d)
        ws = torch.zeros(size, dtype=torch.uint8, device=dev)
        q = randn(R, nq, d).to(torch.bfloat16)
        o, lens, indptr, indices = torch.empty_like(q), i32(ctx + 1), i32(b.page_indptr[:R + 1]), i32(b.page_indices)
        launch = lambda: check(nf_op_kv4_decode_attention(  # noqa: E731
            q.data_ptr(), nq * d, o.data_ptr(), nq * d, pool.data_ptr(), num_pages, lens.data_ptr(), indptr.data_ptr(),
            indices.data_ptr(), R, nq, nkv, d, 0.0, ws.data_ptr(), size, status.data_ptr(), args.sm, st), "kv4 attention")
        return launch, {"requests": R}, int((ctx + 1).sum()) * nkv * d * 9 // 8 + 4 * R * nq * d, status
    T = args.rows or R
    slots = torch.randperm(num_pages * s.page_size, device=dev, generator=g)[:T].to(torch.int32)
    T = slots.numel()
    k, v = (randn(T, nkv, d).to(torch.bfloat16) for _ in range(2))
    if args.op == "kv4_append":
        launch = lambda: check(nf_op_kv4_append(  # noqa: E731
            k.data_ptr(), nkv * d, NF_DTYPE_BF16, v.data_ptr(), nkv * d, NF_DTYPE_BF16, slots.data_ptr(), T,
            pool.data_ptr(), num_pages, nkv, d, status.data_ptr(), st), "kv4 append")
    else:
        launch = lambda: check(nf_op_kv4_read(  # noqa: E731
            pool.data_ptr(), num_pages, slots.data_ptr(), T, nkv, d, k.data_ptr(), nkv * d, v.data_ptr(), nkv * d,
            NF_DTYPE_BF16, status.data_ptr(), st), "kv4 read")
    return launch, {"rows": T}, T * nkv * d * (4 + 9 / 8), status


def main(argv=None) -> dict:
    ap = argparse.ArgumentParser()
    ap.add_argument("--op", choices=["decode_attention", "prefill_attention", "gemm", "iteration", *KV4_OPS],
                    required=True)
    ap.add_argument("--nano", type=int, default=1)
    ap.add_argument("--template", type=int, default=0)
    ap.add_argument("--sm-attn", type=int, default=0)
    ap.add_argument("--persistent", action="store_true",
                    help="iteration: one persistent kernel per layer (nf_forward_iteration_persistent)")
    ap.add_argument("--workload", default="llama3_8b_layer")
    ap.add_argument("--layers", type=int, default=0, help="build only this many layers of the workload (0: all)")
    ap.add_argument("--requests", type=int, default=0, help="decode requests (0 = all)")
    ap.add_argument("--rows", type=int, default=0, help="rope, kv4_append, kv4_read: this many rows (0 = --requests)")
    ap.add_argument("--sm", type=int, default=0)
    ap.add_argument("--reps", type=int, default=5)
    ap.add_argument("--warmup", type=int, default=2)
    ap.add_argument("--m", type=int, default=1536)
    ap.add_argument("--n", type=int, default=4096)
    ap.add_argument("--k", type=int, default=4096)
    ap.add_argument("--power-s", type=float, default=0.0,
                    help="also run the op back to back for this many seconds (after 1 s) and report the median "
                         "SM clock and board power sampled by nvidia-smi")
    args = ap.parse_args(argv)
    dev = "cuda:0"
    torch.cuda.set_device(dev)
    stream = torch.cuda.current_stream(dev)
    out = {"op": args.op, "sm": args.sm}

    if args.op == "gemm":
        M, N, K = args.m, args.n, args.k
        g = torch.Generator(device=dev).manual_seed(0)
        a = torch.randn((M, K), device=dev, generator=g).to(torch.bfloat16)
        b = (torch.randn((N, K), device=dev, generator=g) * 0.02).to(torch.bfloat16)
        c = torch.empty((M, N), dtype=torch.float32, device=dev)
        launch = lambda: check(nf_op_gemm_bf16(a.data_ptr(), b.data_ptr(), c.data_ptr(), M, N, K, args.sm,
                                               stream.cuda_stream), "gemm")
        us = _time(launch, args.reps, args.warmup, stream)
        out.update({"shape": [M, N, K], "us": round(us, 2), "tflops": round(2.0 * M * N * K / us / 1e6, 1)})
        if args.power_s > 0:
            out["power"] = _power(launch, args.power_s, stream)
    elif args.op in KV4_OPS:
        from synth.workloads import WORKLOADS
        launch, figures, nbytes, status = _kv4(args, WORKLOADS[args.workload], dev, stream)
        us = _time(launch, args.reps, args.warmup, stream)
        out.update({"workload": args.workload, **figures, "bytes": int(nbytes), "us": round(us, 2),
                    "gbs": round(nbytes / us / 1e3, 1)})
        if args.power_s > 0:
            out["power"] = _power(launch, args.power_s, stream)
        check(int(status.item()), "status")
    else:
        from synth.workloads import WORKLOADS
        from .harness import DeviceWorkload
        w = WORKLOADS[args.workload]
        if args.layers > 0:
            from dataclasses import replace
            w = replace(w, shape=replace(w.shape, n_layers=min(args.layers, w.shape.n_layers)))
        dw = DeviceWorkload(w, dev, keep_logits=False)
        s, bt = w.shape, dw.batch
        q = torch.zeros((dw.T, s.n_q_heads, s.head_dim), dtype=torch.bfloat16, device=dev)
        o = torch.zeros_like(q)
        if args.op == "iteration":
            plan = dw.plan(nano=args.nano, template=args.template, sm_attn=args.sm_attn)
            launch = lambda: dw.forward(plan, stream, persistent=args.persistent)
            us = _time(launch, args.reps, args.warmup, stream)
            out.update({"workload": args.workload, "plan": plan.describe(), "persistent": args.persistent,
                        "us": round(us, 2)})
        elif args.op == "decode_attention":
            R = args.requests or bt.num_decode
            pages = sum(-(-(int(c) + 1) // s.page_size) for c in bt.ctx_lens[:R])
            nbytes = pages * 2 * s.n_kv_heads * s.page_size * s.head_dim * 2
            launch = lambda: check(nf_op_decode_attention(dw.model, q.data_ptr(), o.data_ptr(), dw.io, 0, 0, R,
                                                          args.sm, stream.cuda_stream), "decode")
            us = _time(launch, args.reps, args.warmup, stream)
            out.update({"workload": args.workload, "requests": R, "kv_bytes": nbytes, "us": round(us, 2),
                        "gbs": round(nbytes / us / 1e3, 1)})
        else:
            R, C = bt.num_decode, bt.prefill_len
            flops = 4.0 * s.n_q_heads * s.head_dim * C * (C + 1) / 2
            launch = lambda: check(nf_op_prefill_attention(dw.model, q.data_ptr(), o.data_ptr(), dw.io, 0, R, C,
                                                           args.sm, stream.cuda_stream), "prefill")
            us = _time(launch, args.reps, args.warmup, stream)
            out.update({"workload": args.workload, "chunk": C, "flops": flops, "us": round(us, 2),
                        "tflops": round(flops / us / 1e6, 2)})
        if args.power_s > 0:
            out["power"] = _power(launch, args.power_s, stream)
        check(dw.sync(), "status")
        dw.close()
    print(json.dumps(out), flush=True)
    return out


if __name__ == "__main__":
    main()
