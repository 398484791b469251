"""Cases of the operators around a 4-bit paged KV cache: page tables and slot maps built on the GPU, rotary
positions, rows written to and read from the cache, and decode attention over it.

``run`` computes an operator either in its plain form (elementary torch operations) or, with ``own`` set,
through the library's entry points. A page of the cache holds 16 slots; per KV head it is a K tile followed
by a V tile of 9 d bytes each: 8 d bytes of codes (two 4-bit codes to a byte, value = (code - 8) * scale),
then one bf16 scale for each slot and group of 32 columns. Where a code stands in its tile:

    K: slot s, column 32 j + 8 t + 2 p + h:            byte s d/2 + t d/8 + 4 j + 2 h + p // 2
    V: slot 8 e + 2 t + h, column 32 j + 4 g + p:      byte e 4 d + t d + g d/8 + 4 j + 2 h + p // 2

p % 2 chooses the low or the high half of the byte (p in 0..3, h in 0..1, t in 0..3, g in 0..7).
"""
import math
import random

import torch

own = False

PAGE = 16
GROUP = 32
LARGEST, SMALLEST = 2.0 ** 60, 2.0 ** -60  # magnitudes that the cache holds
DTYPES = {"bf16": (torch.bfloat16, 0), "f32": (torch.float32, 1)}


def listed():
    return [
        # one decode step of the benchmark batch: 512 running requests, one new token each
        {"name": "map_decode_512", "op": "map", "requests": 512, "lo": 1024, "hi": 1536, "chunk": 1, "every": 1},
        # a mixed batch of short and long requests in which every eighth brings a prompt chunk
        {"name": "map_mixed_1024", "op": "map", "requests": 1024, "lo": 0, "hi": 4096, "chunk": 1024, "every": 8},
        # the decode rows of that batch as the QKV product leaves them (fp32, q and k beside v)
        {"name": "rope_decode_512", "op": "rope", "tokens": 512, "nq": 32, "nkv": 8, "d": 128, "rot": 128,
         "interleaved": False, "factor": 1.0, "far": 1536, "in": "f32", "out": "bf16"},
        # a long prompt of a model with interleaved pairs, half of each head rotated, positions stretched
        {"name": "rope_chunk_8192", "op": "rope", "tokens": 8192, "nq": 64, "nkv": 8, "d": 128, "rot": 64,
         "interleaved": True, "factor": 8.0, "far": 131072, "in": "bf16", "out": "bf16"},
        # one new token for each decode request, into pages that hold older slots: k as the rotation leaves it, v as
        # the QKV product does
        {"name": "append_decode_512", "op": "append", "tokens": 512, "nkv": 8, "d": 128, "run": 1, "k": "bf16",
         "v": "f32"},
        # a prompt: whole pages in a row
        {"name": "append_chunk_8192", "op": "append", "tokens": 8192, "nkv": 8, "d": 128, "run": 1024, "k": "bf16",
         "v": "bf16"},
        # a short cached prefix of the tiny layer, an odd number of rows
        {"name": "read_prefix_45", "op": "read", "tokens": 45, "nkv": 2, "d": 64, "run": 45, "out": "f32"},
        # cached prefixes of a batch, for attention of new prompts over them
        {"name": "read_prefix_32768", "op": "read", "tokens": 32768, "nkv": 8, "d": 128, "run": 2048, "out": "bf16"},
        # the tiny layer's decode batch: latency
        {"name": "attn_tiny_8", "op": "attn", "requests": 8, "lo": 16, "hi": 64, "median": 0, "empty": 0,
         "nq": 4, "nkv": 2, "d": 64},
        # the benchmark's decode batch
        {"name": "attn_512x1280", "op": "attn", "requests": 512, "lo": 1024, "hi": 1536, "median": 0, "empty": 0,
         "nq": 32, "nkv": 8, "d": 128},
        # ragged contexts, a few rows of the batch not in use
        {"name": "attn_ragged_512", "op": "attn", "requests": 512, "lo": 1, "hi": 2048, "median": 512, "empty": 5,
         "nq": 32, "nkv": 8, "d": 128},
        # two long conversations
        {"name": "attn_long_2x131072", "op": "attn", "requests": 2, "lo": 120000, "hi": 131072, "median": 0,
         "empty": 0, "nq": 64, "nkv": 8, "d": 128},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["map", "rope", "append", "read", "attn", "attn"])
    if op == "map":
        R, chunk = _log_int(rng, 1, 1024), _log_int(rng, 1, 1024)
        return {"op": op, "requests": R, "lo": 0, "hi": _log_int(rng, 16, 4096), "chunk": chunk,
                "every": max(rng.randint(1, 16), R * chunk // 131072 + 1)}
    nkv = rng.choice([1, 2, 4, 5, 8])
    d = rng.choice([64, 128, 128])
    if op == "rope":
        return {"op": op, "tokens": _log_int(rng, 1, 8192), "nq": nkv * rng.randint(1, 8), "nkv": nkv, "d": d,
                "rot": rng.choice([d, d, d // 2, d // 4]), "interleaved": rng.random() < 0.5,
                "factor": rng.choice([1.0, 1.0, 4.0, 8.0]), "far": _log_int(rng, 16, 131072),
                "in": rng.choice(["f32", "bf16"]), "out": "bf16"}
    if op in ("append", "read"):
        T = _log_int(rng, 1, 8192 if op == "append" else 32768)
        c = {"op": op, "tokens": T, "nkv": nkv, "d": d, "run": min(T, rng.choice([1, 7, 100, 1024]))}
        for name in ("k", "v") if op == "append" else ("out",):
            c[name] = rng.choice(["f32", "bf16"])
        return c
    R = _log_int(rng, 1, 512)
    most = min(131072, 512 * 1536 * 8 * 128 // (R * nkv * d))
    hi = _log_int(rng, 16, most)
    return {"op": op, "requests": R, "lo": rng.choice([1, (hi + 1) // 2]), "hi": hi,
            "median": rng.choice([0, 0, max(1, hi // 4)]), "empty": rng.choice([0, 0, min(2, R - 1)]),
            "nq": nkv * rng.randint(1, 8), "nkv": nkv, "d": d}


# --- sizes that follow from a case -----------------------------------------------------------------


def _lengths(case):
    """Keys of each request: the case's own, whatever the seed of the values."""
    r = random.Random("lengths of %s" % sorted((k, v) for k, v in case.items() if k != "name"))
    lens = []
    for _ in range(case["requests"]):
        n = case["median"] * math.exp(r.gauss(0.0, 1.0)) if case.get("median") else r.randint(case["lo"], case["hi"])
        lens.append(int(min(max(round(n), case["lo"]), case["hi"])))
    for i in range(case.get("empty", 0)):
        lens[(7 * i + 3) % len(lens)] = 0
    return lens


def _new_tokens(case):
    return [case["chunk"] if i % case["every"] == 0 else 1 for i in range(case["requests"])]


def _pages(n):
    return (n + PAGE - 1) // PAGE


def _rows(case):
    """Elements of one row of K and V together, and the bytes that the cache holds of them."""
    n = 2 * case["nkv"] * case["d"]
    return n, n // 2 + n // GROUP * 2


def work(case):
    op = case["op"]
    if op == "map":
        old, new = _lengths(case), _new_tokens(case)
        R, T = case["requests"], sum(new)
        held = sum(_pages(c) for c in old)
        pages = sum(_pages(c + n) for c, n in zip(old, new))
        reads = 8 * R + 4 * pages                    # lengths; old table entries, free pages for the new ones
        writes = 8 * R + 4 * pages + 4 * (pages - held) + 8 * T
        return {"bytes": reads + writes, "flops": 0}
    if op == "rope":
        T, heads = case["tokens"], case["nq"] + case["nkv"]
        size = sum(4 if case[k] == "f32" else 2 for k in ("in", "out"))
        return {"bytes": T * (heads * case["d"] * size + 4) + 4 * case["rot"], "flops": 3 * T * heads * case["rot"]}
    n, held = _rows(case) if op != "attn" else (0, 0)
    if op == "append":  # rows in, codes written and read back, rows out
        size = sum(4 if case[k] == "f32" else 2 for k in ("k", "v"))
        return {"bytes": case["tokens"] * (n // 2 * size + 2 * held + 2 * n + 4),
                "flops": 4 * case["tokens"] * n}
    if op == "read":
        return {"bytes": case["tokens"] * (held + n * (4 if case["out"] == "f32" else 2) + 4),
                "flops": case["tokens"] * n}
    lens = _lengths(case)
    keys, R = sum(lens), case["requests"]
    return {"bytes": keys * _rows(case)[1] + 4 * sum(_pages(x) for x in lens) + R * (4 * case["nq"] * case["d"] + 8),
            "flops": 4 * keys * case["nq"] * case["d"]}


# --- the 4-bit cache, plain ------------------------------------------------------------------------


def _parts(pool, nkv, d):
    """Views of a pool [pages, nkv, 2, 9 d] uint8: K codes [page, head, slot, t, j, h, b], K scales, V codes
    [page, head, e, t, g, j, h, b], V scales [page, head, slot, j]."""
    ng = d // GROUP
    k, v = pool[:, :, 0], pool[:, :, 1]
    scales = [x[..., 8 * d:].view(torch.bfloat16).unflatten(-1, (PAGE, ng)) for x in (k, v)]
    return (k[..., :8 * d].unflatten(-1, (PAGE, 4, ng, 2, 2)), scales[0],
            v[..., :8 * d].unflatten(-1, (2, 4, 8, ng, 2, 2)), scales[1])


def _nibbles(x):
    return torch.stack((x & 15, x >> 4), -1)


def _k_columns(codes, scale):
    """[..., t, j, h, b] codes and [..., j] scales -> [..., d] fp32."""
    c = _nibbles(codes).to(torch.float32) - 8.0                    # t, j, h, b, p % 2
    n = c.dim()
    c = c.permute(*range(n - 5), n - 4, n - 5, n - 2, n - 1, n - 3)   # j, t, b, p % 2, h
    return (c.flatten(-4) * scale.to(torch.float32).unsqueeze(-1)).flatten(-2)


def _v_columns(codes, scale):
    """[..., g, j, b] codes and [..., j] scales -> [..., d] fp32."""
    c = _nibbles(codes).to(torch.float32) - 8.0                    # g, j, b, p % 2
    c = c.transpose(-4, -3)
    return (c.flatten(-3) * scale.to(torch.float32).unsqueeze(-1)).flatten(-2)


def _quantise(x):
    """Rows [..., d] -> codes [..., d] uint8 in 1..15 and bf16 scales [..., d / 32]. The quotient is taken in 64
    bits, where a value next to a border keeps its side."""
    g = x.to(torch.float32).unflatten(-1, (-1, GROUP))
    a = g.abs().amax(-1).to(torch.bfloat16).to(torch.float32)
    s = (a / 7.0).to(torch.bfloat16)
    s = torch.where(a < SMALLEST, torch.zeros_like(s), s)
    s = torch.where(a <= LARGEST, s, torch.full_like(s, math.nan))
    c = torch.round(g.double() / s.double().unsqueeze(-1))
    c = torch.where((s > 0).unsqueeze(-1), c, torch.zeros_like(c)).clamp(-7, 7)
    return (c + 8).to(torch.uint8).flatten(-2), s


def _pack_k(codes):
    """[..., d] -> [..., t, j, h, b]."""
    c = codes.unflatten(-1, (-1, 4, 2, 2, 2))                      # j, t, b, p % 2, h
    n = c.dim()
    c = c.permute(*range(n - 5), n - 4, n - 5, n - 1, n - 3, n - 2)
    return c[..., 0] | (c[..., 1] << 4)


def _pack_v(codes):
    """[..., d] -> [..., g, j, b]."""
    c = codes.unflatten(-1, (-1, 8, 2, 2)).transpose(-4, -3)       # g, j, b, p % 2
    return c[..., 0] | (c[..., 1] << 4)


def _store(pool, nkv, d, page, slot, k, v):
    """Rows [n, nkv, d] of K and V into the slots."""
    kc, ks, vc, vs = _parts(pool, nkv, d)
    codes, scale = _quantise(k)
    kc[page, :, slot] = _pack_k(codes)
    ks[page, :, slot] = scale
    codes, scale = _quantise(v)
    vc[page, :, slot // 8, slot % 8 // 2, :, :, slot % 2] = _pack_v(codes)
    vs[page, :, slot] = scale


def _load(pool, nkv, d, page, slot):
    """Rows [n, nkv, d] fp32 of K and V at the slots."""
    kc, ks, vc, vs = _parts(pool, nkv, d)
    return (_k_columns(kc[page, :, slot], ks[page, :, slot]),
            _v_columns(vc[page, :, slot // 8, slot % 8 // 2, :, :, slot % 2], vs[page, :, slot]))


def _load_pages(pool, nkv, d, page):
    """Whole pages [..., nkv, 16, d] fp32 of K and V."""
    kc, ks, vc, vs = _parts(pool, nkv, d)
    k = _k_columns(kc[page], ks[page])
    v = vc[page]                                                   # ..., e, t, g, j, h, b
    n = v.dim()
    v = v.permute(*range(n - 4), n - 2, n - 4, n - 3, n - 1).flatten(-6, -4)
    return k, _v_columns(v, vs[page])


# --- inputs ----------------------------------------------------------------------------------------


def _normal(gen, shape, dtype=torch.float32):
    return torch.randn(shape, device="cuda", generator=gen, dtype=torch.float32).to(dtype)


def _filled_pool(gen, pages, nkv, d):
    """Pages of rows as projections leave them: columns of unequal spread, quantised."""
    pool = torch.empty((pages, nkv, 2, 9 * d), dtype=torch.uint8, device="cuda")
    kc, ks, vc, vs = _parts(pool, nkv, d)
    spread = torch.exp(0.5 * _normal(gen, (2, nkv, 1, d)))
    step = max(1, (1 << 27) // (nkv * PAGE * d))
    for at in range(0, pages, step):
        n = min(step, pages - at)
        for which in (0, 1):
            codes, scale = _quantise(_normal(gen, (n, nkv, PAGE, d)) * spread[which])
            if which == 0:
                kc[at:at + n], ks[at:at + n] = _pack_k(codes), scale
            else:
                packed = _pack_v(codes).unflatten(2, (2, 4, 2))    # page, head, e, t, h, g, j, b
                vc[at:at + n], vs[at:at + n] = packed.permute(0, 1, 2, 3, 5, 6, 4, 7), scale
    return pool


def _frequencies(rot, factor):
    """Rotary frequencies theta^(-2 i / rot), stretched for long contexts by wavelength: long waves (more than 8192
    positions) turn `factor` times slower, short ones (under 2048) as before, those between in a smooth blend."""
    f = 500000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    if factor != 1.0:
        turns = 8192.0 * f / (2.0 * math.pi)
        blend = ((turns - 1.0) / (4.0 - 1.0)).clamp(0.0, 1.0)
        f = f * ((1.0 - blend) / factor + blend)
    return f


def _slots(gen, tokens, run):
    """Runs of `run` consecutive slots that start on a page of their own, in scattered pages; a run that is no
    multiple of a page starts at any slot of its first page."""
    per = _pages(run) + 1
    runs = (tokens + run - 1) // run
    pages = torch.randperm(runs * per, device="cuda", generator=gen).view(runs, per)
    first = torch.randint(0, PAGE, (runs, 1), device="cuda", generator=gen) if run % PAGE else 0
    at = torch.arange(run, device="cuda") + first
    slot = torch.gather(pages, 1, (at // PAGE).expand(runs, run)) * PAGE + at % PAGE
    return slot.flatten()[:tokens].to(torch.int32), runs * per


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    s = {"case": case, "status": torch.zeros(1, dtype=torch.int32, device="cuda")}
    if op == "map":
        old, new = _lengths(case), _new_tokens(case)
        before, after = [_pages(c) for c in old], [_pages(c + n) for c, n in zip(old, new)]
        width = max(after) + 3
        spare = sum(after) - sum(before) + 5
        total = sum(before) + spare
        ids = torch.randperm(total, device="cuda", generator=gen).to(torch.int32)
        table = torch.full((len(old), width), -1, dtype=torch.int32, device="cuda")
        held = torch.tensor(before, device="cuda").unsqueeze(1) > torch.arange(width, device="cuda")
        table[held] = ids[spare:]
        i32 = lambda n: torch.full((n,), -1, dtype=torch.int32, device="cuda")  # noqa: E731
        s |= {"ctx": torch.tensor(old, dtype=torch.int32, device="cuda"),
              "new": torch.tensor(new, dtype=torch.int32, device="cuda"), "table": table, "free": ids[:spare].clone(),
              "free_count": torch.tensor([spare], dtype=torch.int32, device="cuda"), "pages": total,
              "kv_len": i32(len(old)), "indptr": i32(len(old) + 1), "indices": i32(sum(after) + 8),
              "slots": i32(sum(new) + 8), "positions": i32(sum(new) + 8), "left": i32(1)}
    elif op == "rope":
        T, nq, nkv, d = case["tokens"], case["nq"], case["nkv"], case["d"]
        out = DTYPES[case["out"]][0]
        s |= {"qkv": _normal(gen, (T, (nq + 2 * nkv) * d), DTYPES[case["in"]][0]),
              "positions": torch.randint(0, case["far"], (T,), device="cuda", generator=gen, dtype=torch.int32),
              "freq": _frequencies(case["rot"], case["factor"]).cuda(),
              "q": torch.empty((T, nq, d), dtype=out, device="cuda"),
              "k": torch.empty((T, nkv, d), dtype=out, device="cuda")}
    elif op in ("append", "read"):
        T, nkv, d = case["tokens"], case["nkv"], case["d"]
        s["slots"], s["pages"] = _slots(gen, T, case["run"])
        s["pool"] = _filled_pool(gen, s["pages"], nkv, d)
        out = torch.bfloat16 if op == "append" else DTYPES[case["out"]][0]
        s["k"], s["v"] = (torch.empty((T, nkv, d), dtype=out, device="cuda") for _ in range(2))
        if op == "append":  # k rotated and on its own, v beside q and k in the product's rows
            s["new_k"] = _normal(gen, (T, nkv, d), DTYPES[case["k"]][0])
            s["new_v"] = _normal(gen, (T, 6 * nkv, d), DTYPES[case["v"]][0])[:, 5 * nkv:]
    else:
        lens = _lengths(case)
        R, nq, nkv, d = case["requests"], case["nq"], case["nkv"], case["d"]
        counts = [_pages(n) for n in lens]
        starts = [0]
        for n in counts:
            starts.append(starts[-1] + n)
        s["pages"] = max(1, starts[-1])
        s |= {"pool": _filled_pool(gen, s["pages"], nkv, d), "width": max(1, max(counts)),
              "kv_len": torch.tensor(lens, dtype=torch.int32, device="cuda"),
              "indptr": torch.tensor(starts, dtype=torch.int32, device="cuda"),
              "indices": torch.randperm(s["pages"], device="cuda", generator=gen).to(torch.int32),
              "q": _normal(gen, (R, nq, d), torch.bfloat16),
              "out": torch.empty((R, nq, d), dtype=torch.bfloat16, device="cuda")}
    return s


# --- one pass --------------------------------------------------------------------------------------


def _plain_map(s):
    ctx, new, table = s["ctx"].long(), s["new"].long(), s["table"]
    before, after = (ctx + PAGE - 1) // PAGE, (ctx + new + PAGE - 1) // PAGE
    need = after - before
    ends = need.cumsum(0)
    fits = (need == 0) | (ends <= s["free_count"])
    column = torch.arange(table.shape[1], device="cuda")
    fresh = fits.unsqueeze(1) & (column >= before.unsqueeze(1)) & (column < after.unsqueeze(1))
    taken = (ends - need).unsqueeze(1) + column - before.unsqueeze(1)
    page = s["free"][(s["free_count"] - 1 - taken).clamp(0, s["free"].numel() - 1)]
    table[:] = torch.where(fresh, page, table)
    pages = torch.where(fits, after, before)
    s["kv_len"][:] = torch.where(fits, ctx + new, ctx)
    s["indptr"][0] = 0
    s["indptr"][1:] = pages.cumsum(0)
    used = table[column < pages.unsqueeze(1)]
    s["indices"][:used.numel()] = used
    row = torch.repeat_interleave(torch.arange(ctx.numel(), device="cuda"), new)
    at = torch.arange(row.numel(), device="cuda") - (new.cumsum(0) - new)[row] + ctx[row]
    s["positions"][:row.numel()] = at
    slot = table[row, (at // PAGE).clamp(max=table.shape[1] - 1)] * PAGE + at % PAGE
    s["slots"][:row.numel()] = torch.where(fits[row], slot, -1)
    s["left"][0] = s["free_count"][0] - need[fits].sum()


def _rotate(x, cos, sin, rot, interleaved):
    """x [T, heads, d] fp32; cos, sin [T, 1, rot / 2]."""
    turned, rest = x[..., :rot], x[..., rot:]
    if interleaved:
        a, b = turned[..., 0::2], turned[..., 1::2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = turned[..., :rot // 2], turned[..., rot // 2:]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((turned, rest), -1)


def _plain_rope(s):
    c = s["case"]
    T, nq, nkv, d = c["tokens"], c["nq"], c["nkv"], c["d"]
    angle = s["positions"].double().unsqueeze(1) * s["freq"]
    cos, sin = (t.to(torch.float32).unsqueeze(1) for t in (angle.cos(), angle.sin()))
    rows = s["qkv"][:, :(nq + nkv) * d].to(torch.float32).view(T, nq + nkv, d)
    rows = _rotate(rows, cos, sin, c["rot"], c["interleaved"]).to(s["q"].dtype)
    s["q"][:], s["k"][:] = rows[:, :nq], rows[:, nq:]


def _plain_attention(s):
    c = s["case"]
    R, nq, nkv, d = c["requests"], c["nq"], c["nkv"], c["d"]
    column = torch.arange(s["width"], device="cuda")
    at = s["indptr"][:-1].long().unsqueeze(1) + column
    page = s["indices"][at.clamp(max=s["indices"].numel() - 1)].long()
    k, v = _load_pages(s["pool"], nkv, d, page)                    # R, width, nkv, 16, d
    q = s["q"].to(torch.float32).view(R, 1, nkv, nq // nkv, d)
    x = torch.matmul(q, k.transpose(-1, -2)) * (1.0 / math.sqrt(d))   # R, width, nkv, G, 16
    key = column.view(-1, 1, 1, 1) * PAGE + torch.arange(PAGE, device="cuda")
    seen = key < s["kv_len"].view(R, 1, 1, 1, 1)
    x = x.masked_fill(~seen, -math.inf)
    top = x.amax((1, 4), keepdim=True)
    w = torch.exp(x - torch.where(top > -math.inf, top, torch.zeros_like(top)))
    w = w / w.sum((1, 4), keepdim=True).clamp(min=1e-30)
    s["out"][:] = torch.matmul(w, v).sum(1).view(R, nq, d).to(torch.bfloat16)


_workspaces = {}


def _own(s):
    import intra_device_overlapped_b200 as nf
    c, op = s["case"], s["case"]["op"]
    stream = torch.cuda.current_stream().cuda_stream
    status = s["status"].data_ptr()
    if op == "map":
        nf.check(nf.nf_op_page_map(
            s["ctx"].data_ptr(), s["new"].data_ptr(), c["requests"], s["table"].data_ptr(), s["table"].shape[1],
            s["free"].data_ptr(), s["free"].numel(), s["free_count"].data_ptr(), s["pages"], s["kv_len"].data_ptr(),
            s["indptr"].data_ptr(), s["indices"].data_ptr(), s["indices"].numel(), s["slots"].data_ptr(),
            s["positions"].data_ptr(), s["slots"].numel(), s["left"].data_ptr(), status, stream))
        return
    nkv, d = c["nkv"], c["d"]
    if op == "rope":
        nq, rows = c["nq"], s["qkv"]
        nf.check(nf.nf_op_rope(
            rows.data_ptr(), rows.stride(0), s["q"].data_ptr(), nq * d, nq,
            rows.data_ptr() + nq * d * rows.element_size(), rows.stride(0), s["k"].data_ptr(), nkv * d, nkv,
            DTYPES[c["in"]][1], DTYPES[c["out"]][1], s["positions"].data_ptr(), c["tokens"], d, c["rot"],
            c["interleaved"], s["freq"].data_ptr(), 1.0, stream))
    elif op in ("append", "read"):
        if op == "append":
            nf.check(nf.nf_op_kv4_append(
                s["new_k"].data_ptr(), s["new_k"].stride(0), DTYPES[c["k"]][1], s["new_v"].data_ptr(),
                s["new_v"].stride(0), DTYPES[c["v"]][1], s["slots"].data_ptr(), c["tokens"], s["pool"].data_ptr(), s["pages"], nkv, d,
                status, stream))
        nf.check(nf.nf_op_kv4_read(
            s["pool"].data_ptr(), s["pages"], s["slots"].data_ptr(), c["tokens"], nkv, d, s["k"].data_ptr(), nkv * d,
            s["v"].data_ptr(), nkv * d, DTYPES[c.get("out", "bf16")][1], status, stream))
    else:
        size = nf.nf_kv4_workspace_bytes(c["nq"], nkv, d)
        place = (size, torch.cuda.current_device(), stream)
        held = _workspaces.get(place)
        if held is None:  # zeroed once on the stream that uses it, kept by the program for all its calls there
            held = _workspaces[place] = torch.zeros(size, dtype=torch.uint8, device="cuda")
        nf.check(nf.nf_op_kv4_decode_attention(
            s["q"].data_ptr(), c["nq"] * d, s["out"].data_ptr(), c["nq"] * d, s["pool"].data_ptr(), s["pages"],
            s["kv_len"].data_ptr(), s["indptr"].data_ptr(), s["indices"].data_ptr(), c["requests"], c["nq"], nkv, d,
            0.0, held.data_ptr(), size, status, 0, stream))


def run(s):
    op = s["case"]["op"]
    if own:
        _own(s)
    elif op == "map":
        _plain_map(s)
    elif op == "rope":
        _plain_rope(s)
    elif op == "attn":
        _plain_attention(s)
    else:
        c, slot = s["case"], s["slots"].long()
        page, slot = slot // PAGE, slot % PAGE
        if op == "append":
            _store(s["pool"], c["nkv"], c["d"], page, slot, s["new_k"], s["new_v"])
        k, v = _load(s["pool"], c["nkv"], c["d"], page, slot)
        s["k"][:], s["v"][:] = k, v
    names = {"map": ("kv_len", "indptr", "indices", "table", "slots", "positions", "left"), "rope": ("q", "k"),
             "append": ("k", "v"), "read": ("k", "v"), "attn": ("out",)}
    return {n: s[n] for n in names[op]}


# --- the definitions in 64 bits --------------------------------------------------------------------


def _place(d):
    """Byte and half of the byte of every (slot, column) in a K and in a V tile, from the layout's formulas."""
    slot, col = torch.meshgrid(torch.arange(PAGE), torch.arange(d), indexing="ij")
    j, r = col // 32, col % 32
    t, p, h = r // 8, r % 8 // 2, r % 2
    k = slot * (d // 2) + t * (d // 8) + 4 * j + 2 * h + p // 2, p % 2
    g, p = r // 4, r % 4
    e, t, h = slot // 8, slot % 8 // 2, slot % 2
    v = e * 4 * d + t * d + g * (d // 8) + 4 * j + 2 * h + p // 2, p % 2
    return [tuple(x.cuda() for x in pair) for pair in (k, v)]


def _tiles64(tiles, place):
    """Tiles [..., 9 d] uint8 -> values [..., 16, d] in 64 bits."""
    byte, half = place
    d = byte.shape[1]
    code = (tiles[..., byte.flatten()].int() >> (4 * half.flatten())) % 16 - 8
    scale = tiles[..., 8 * d:].contiguous().view(torch.bfloat16).double()
    return code.double().unflatten(-1, (PAGE, d)) * scale.unflatten(-1, (PAGE, -1)).repeat_interleave(32, -1)


def _held64(x):
    """What the cache holds of rows x, in 64 bits."""
    x = x.double().unflatten(-1, (-1, 32))
    a = x.abs().amax(-1, keepdim=True).to(torch.bfloat16).double()
    s = (a / 7).to(torch.bfloat16).double()
    held = torch.clamp(torch.round(x / s), -7, 7) * s
    return torch.where(a < SMALLEST, 0.0, torch.where(a <= LARGEST, held, math.nan)).flatten(-2)


def exact(case, seed):
    op = case["op"]
    if op == "map":
        return None
    s = prepare(case, seed)
    d = case["d"]
    if op == "rope":
        T, nq, nkv, half = case["tokens"], case["nq"], case["nkv"], case["rot"] // 2
        x = s["qkv"].double()[:, :(nq + nkv) * d].reshape(T, nq + nkv, d)
        i = torch.arange(half, device="cuda")
        a, b = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + half)
        turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                           s["positions"].double().view(T, 1, 1) * s["freq"])
        z = torch.complex(x[..., a], x[..., b]) * turn
        x[..., a], x[..., b] = z.real, z.imag
        return {"q": x[:, :nq], "k": x[:, nq:]}
    if op == "append":
        return {"k": _held64(s["new_k"]), "v": _held64(s["new_v"])}
    places = _place(d)
    slot = s["slots"].long() if op == "read" else None
    if op == "read":
        rows = torch.arange(slot.numel(), device="cuda")
        at = range(0, slot.numel(), 2048)
        pick = lambda which: torch.cat([  # noqa: E731
            _tiles64(s["pool"][slot[i:i + 2048] // PAGE, :, which], places[which])[
                rows[:slot[i:i + 2048].numel()], :, slot[i:i + 2048] % PAGE] for i in at])
        return {"k": pick(0), "v": pick(1)}
    nq, nkv = case["nq"], case["nkv"]
    out = torch.zeros((case["requests"], nq, d), dtype=torch.float64, device="cuda")
    starts = s["indptr"].tolist()
    for r, n in enumerate(_lengths(case)):
        if n == 0:
            continue
        tiles = s["pool"][s["indices"][starts[r]:starts[r] + _pages(n)].long()]
        for h in range(nkv):
            K, V = (_tiles64(tiles[:, h, w], places[w]).flatten(0, 1)[:n] for w in (0, 1))
            q = s["q"][r].double().view(nkv, -1, d)[h]
            w = torch.softmax(q @ K.T / math.sqrt(d), -1)
            out[r].view(nkv, -1, d)[h] = w @ V
    return {"out": out}
