"""Operators around the 4-bit KV cache on the GPU, through the C ABI, against plain 64-bit implementations."""
import math

import numpy as np
import pytest
import torch

import kv4_reference as ref

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF16, F32 = 0, 1
TORCH = {BF16: torch.bfloat16, F32: torch.float32}
HALF_STEP = {BF16: 2.0 ** -8, F32: 2.0 ** -24}  # a rounding's largest relative error


@pytest.fixture(scope="module")
def nf():
    import intra_device_overlapped_b200 as m
    return m


def _dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
    return t if dtype is None else t.to(dtype)


def _i32(a):
    return _dev(np.asarray(a, dtype=np.int32))


def _status():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


def _host(t):
    return t.double().cpu().numpy()


# --- page tables ------------------------------------------------------------------------------------


def _run_map(nf, ctx, new, table, free, count, num_pages, page_cap, token_cap, stream=0):
    R, stride = table.shape
    d = {"kv_len": _i32([-7] * max(R, 1)), "indptr": _i32([-7] * (R + 1)), "indices": _i32([-7] * (page_cap + 3)),
         "slots": _i32([-7] * (token_cap + 3)), "positions": _i32([-7] * (token_cap + 3)), "left": _i32([-7]),
         "table": _i32(table if R else [[-1] * stride]), "status": _status()}
    c, n, f, k = _i32(ctx if R else [0]), (None if new is None else _i32(new if R else [0])), _i32(free), _i32([count])
    nf.check(nf.nf_op_page_map(c.data_ptr(), 0 if n is None else n.data_ptr(), R, d["table"].data_ptr(), stride,
                               f.data_ptr(), len(free), k.data_ptr(), num_pages, d["kv_len"].data_ptr(),
                               d["indptr"].data_ptr(), d["indices"].data_ptr(), page_cap, d["slots"].data_ptr(),
                               d["positions"].data_ptr(), token_cap, d["left"].data_ptr(), d["status"].data_ptr(),
                               stream), "page_map")
    torch.cuda.synchronize()
    return {k2: v.cpu().numpy() for k2, v in d.items()}


def _same_map(got, want, R):
    assert (int(got["status"][0]) in want["status"]) if want["status"] else got["status"][0] == 0
    assert got["kv_len"][:R].tolist() == want["kv_len"]
    assert got["indptr"].tolist() == want["indptr"]
    for name in ("indices", "slots", "positions"):
        n = len(want[name])
        assert got[name][:n].tolist() == want[name], name
        assert (got[name][n:] == -7).all(), name       # rows behind the last one stay as they are
    assert int(got["left"][0]) == want["left"]
    assert np.array_equal(got["table"][:R], want["table"])


def _batch(rng, R, most, new_most, spare, stride_extra=2):
    ctx = rng.integers(0, most + 1, R)
    new = rng.integers(0, new_most + 1, R)
    b, a = -(-ctx // 16), -(-(ctx + new) // 16)
    held, need = int(b.sum()), int((a - b).sum())
    ids = rng.permutation(held + need + spare + 4)
    table = np.full((R, (int(a.max()) if R else 0) + stride_extra), -1)
    at = 0
    for r in range(R):
        table[r, :b[r]] = ids[at:at + b[r]]
        at += b[r]
    return ctx, new, table, ids[held:held + max(need + spare, 1)], need + spare, len(ids)


@pytest.mark.parametrize("R,most,new_most", [(0, 0, 0), (1, 0, 1), (1, 40, 200), (5, 33, 3), (37, 100, 40),
                                             (513, 300, 20), (1025, 64, 1), (5000, 40, 2), (16384, 20, 1)])
def test_page_map(nf, R, most, new_most):
    rng = np.random.default_rng(R * 131 + most)
    ctx, new, table, free, count, ids = _batch(rng, R, most, new_most, 3)
    pages, tokens = int((-(-(ctx + new) // 16)).sum()), int(new.sum())
    for page_cap, token_cap in ((pages, tokens), (pages + 5, tokens + 9)):
        got = _run_map(nf, ctx, new, table, free, count, ids, page_cap, token_cap)
        _same_map(got, ref.page_map(ctx, new, table, free, count, ids, page_cap, token_cap), R)


def test_page_map_one_token_each(nf):
    rng = np.random.default_rng(3)
    ctx, _, table, _, _, ids = _batch(rng, 200, 90, 0, 0)
    free = np.arange(ids, ids + 200)
    got = _run_map(nf, ctx, None, table, free, 150, ids + 200, 2000, 200)
    _same_map(got, ref.page_map(ctx, [1] * 200, table, free, 150, ids + 200, 2000, 200), 200)


@pytest.mark.parametrize("spare", [-1, -7, -60, -1000000])
def test_page_map_refuses_requests_without_pages(nf, spare):
    rng = np.random.default_rng(17)
    ctx, new, table, free, count, ids = _batch(rng, 90, 50, 60, 0)
    count = max(0, count + spare)
    got = _run_map(nf, ctx, new, table, free, count, ids, 4000, 9000)
    want = ref.page_map(ctx, new, table, free, count, ids, 4000, 9000)
    assert 3 in want["status"]
    _same_map(got, want, 90)


@pytest.mark.parametrize("fault", ["negative", "row", "row_new", "huge", "page_id", "free_id", "count", "pages", "tokens"])
def test_page_map_reports_bad_input(nf, fault):
    rng = np.random.default_rng(29)
    ctx, new, table, free, count, ids = _batch(rng, 60, 70, 30, 5)
    page_cap, token_cap = 2000, 3000
    if fault == "negative":
        ctx[7], new[20] = -1, -3
    elif fault == "row":
        ctx[9] = 16 * table.shape[1] + 1
    elif fault == "row_new":
        ctx[9], new[9] = 16 * table.shape[1] - 5, 6
    elif fault == "huge":
        ctx[9], new[9] = 2 ** 31 - 1, 1
    elif fault == "page_id":
        ctx[4] = max(ctx[4], 20)
        table[4, 1] = ids + 3
    elif fault == "free_id":
        free[-2] = -5
    elif fault == "count":
        count = len(free) + 9
    elif fault == "pages":
        page_cap = 11
    else:
        token_cap = 23
    got = _run_map(nf, ctx, new, table, free, count, ids, page_cap, token_cap)
    want = ref.page_map(ctx, new, table, free, count, ids, page_cap, token_cap)
    assert 6 in want["status"]
    _same_map(got, want, 60)


# --- rotary positions -------------------------------------------------------------------------------


def _freqs(rot, theta=500000.0):
    return theta ** (-2.0 * np.arange(rot // 2) / rot)


def _check_rope(got, x, positions, freq, scale, rot, inter, out_dtype):
    """Against 64 bits. cos and sin are within 2^-22 (their argument, at most 1 half turn, is rounded to 2^-24 of
    itself: 2^-24 pi; sincospif adds under 2 of their units, 2^-23), times scale; two products and a sum round by
    2^-24 each; the result rounds once to its type."""
    want = ref.rope(x, positions, freq, scale, rot, inter)
    size = np.abs(want)
    bound = HALF_STEP[out_dtype] * size
    i = np.arange(rot // 2)
    a, b = (2 * i, 2 * i + 1) if inter else (i, i + rot // 2)
    pair = np.abs(x[..., a]) + np.abs(x[..., b])
    for c in (a, b):
        bound[..., c] += pair * abs(scale) * (2.0 ** -22 + 3 * 2.0 ** -24)
    err = np.abs(_host(got) - want)
    assert (err <= bound * (1 + 2.0 ** -7) + 1e-40).all(), float((err - bound).max())


ROPE = [  # T, nq, nkv, d, rot, interleaved, in, out
    (1, 4, 2, 64, 64, 0, BF16, BF16), (7, 32, 8, 128, 128, 0, F32, BF16), (33, 8, 1, 128, 64, 1, BF16, BF16),
    (5, 3, 3, 80, 80, 0, F32, F32), (5, 3, 3, 80, 20, 1, BF16, F32), (9, 1, 0, 6, 2, 0, BF16, BF16),
    (9, 0, 5, 128, 96, 1, F32, BF16), (300, 64, 8, 128, 128, 1, BF16, BF16), (2, 2, 1, 256, 256, 0, F32, F32),
    (3, 2, 2, 512, 512, 0, BF16, BF16), (1500, 4, 2, 64, 32, 0, F32, BF16), (13, 5, 1, 34, 34, 1, BF16, BF16),
    (4099, 2, 1, 128, 128, 0, BF16, BF16)]


@pytest.mark.parametrize("T,nq,nkv,d,rot,inter,idt,odt", ROPE)
def test_rope(nf, T, nq, nkv, d, rot, inter, idt, odt):
    rng = np.random.default_rng(T + d)
    rows = _dev(rng.standard_normal((T, (nq + 2 * nkv) * d)).astype(np.float32), TORCH[idt])  # q, k, v in a row
    pos = rng.integers(0, 131072, T)
    pos[0] = 131071 if T > 1 else 3
    freq = _freqs(rot)
    p, f = _i32(pos), _dev(freq)
    q = torch.full((T, nq * d + 3), -7.0, dtype=TORCH[odt], device=DEV)
    k = torch.full((T, nkv * d), -7.0, dtype=TORCH[odt], device=DEV)
    nf.check(nf.nf_op_rope(rows.data_ptr(), rows.stride(0), q.data_ptr(), q.stride(0), nq,
                           rows.data_ptr() + nq * d * rows.element_size(), rows.stride(0), k.data_ptr(), k.stride(0),
                           nkv, idt, odt, p.data_ptr(), T, d, rot, inter, f.data_ptr(), 1.25))
    torch.cuda.synchronize()
    x = _host(rows).reshape(T, nq + 2 * nkv, d)
    assert (q[:, nq * d:] == -7.0).all()
    for got, part in ((q[:, :nq * d].reshape(T, nq, d), x[:, :nq]), (k.reshape(T, nkv, d), x[:, nq:nq + nkv])):
        if part.size:
            _check_rope(got, part, pos, freq, 1.25, rot, inter, odt)


@pytest.mark.parametrize("d,rot,inter,dt,offset", [(128, 128, 0, BF16, 0), (128, 32, 1, F32, 0), (64, 48, 0, BF16, 1),
                                                   (128, 64, 0, F32, 3), (66, 22, 1, BF16, 5)])
def test_rope_in_place_and_odd_offsets(nf, d, rot, inter, dt, offset):
    T, nq, nkv = 17, 3, 2
    rng = np.random.default_rng(d + rot)
    width = (nq + nkv) * d + offset
    buf = _dev(rng.standard_normal(T * width + offset).astype(np.float32), TORCH[dt])
    before = buf.clone()
    rows = buf[offset:].view(T, width)
    pos = rng.integers(-50, 4000, T)   # negative positions turn the other way
    freq = _freqs(rot, 10000.0)
    p, f = _i32(pos), _dev(freq)
    kp = rows.data_ptr() + nq * d * rows.element_size()
    nf.check(nf.nf_op_rope(rows.data_ptr(), width, rows.data_ptr(), width, nq, kp, width, kp, width, nkv, dt, dt,
                           p.data_ptr(), T, d, rot, inter, f.data_ptr()))
    torch.cuda.synchronize()
    x = _host(before[offset:].view(T, width)[:, :(nq + nkv) * d]).reshape(T, nq + nkv, d)
    _check_rope(rows[:, :(nq + nkv) * d].reshape(T, nq + nkv, d), x, pos, freq, 1.0, rot, inter, dt)
    assert torch.equal(rows[:, (nq + nkv) * d:], before[offset:].view(T, width)[:, (nq + nkv) * d:])
    assert torch.equal(buf[:offset], before[:offset])


# --- rows of the cache ------------------------------------------------------------------------------


def _garbage(rng, pages, nkv, d):
    return rng.integers(0, 256, pages * nkv * 18 * d, dtype=np.uint8)


def _append(nf, k, v, slots, pool, pages, nkv, d, status, stream=0):
    dtype = {torch.bfloat16: BF16, torch.float32: F32}
    nf.check(nf.nf_op_kv4_append(k.data_ptr(), k.stride(0), dtype[k.dtype], v.data_ptr(), v.stride(0), dtype[v.dtype],
                                 slots.data_ptr(), slots.numel(), pool.data_ptr(), pages, nkv, d, status.data_ptr(),
                                 stream), "append")


@pytest.mark.parametrize("T,nkv,d,kt,vt", [
    (1, 1, 64, BF16, BF16), (1, 8, 128, F32, F32), (17, 2, 64, F32, BF16), (40, 5, 128, BF16, F32),
    (64, 8, 128, BF16, BF16), (301, 3, 128, F32, BF16), (700, 1, 64, BF16, F32), (2048, 8, 128, F32, F32)])
def test_append_writes_the_defined_bytes_and_no_others(nf, T, nkv, d, kt, vt):
    rng = np.random.default_rng(T * 3 + d)
    pages = T // 16 + 3
    raw = _garbage(rng, pages, nkv, d)
    slots = rng.permutation(pages * 16)[:T]
    if T > 4:
        slots[3] = -1
    spread = np.exp(rng.standard_normal((1, nkv, d)))
    k = _dev((rng.standard_normal((T, nkv, d)) * spread).astype(np.float32), TORCH[kt])
    rows = _dev(rng.standard_normal((T, 3 * nkv, d)).astype(np.float32), TORCH[vt])
    v = rows[:, 2 * nkv:]
    pool, status = _dev(raw), _status()
    _append(nf, k, v, _i32(slots), pool, pages, nkv, d, status)
    torch.cuda.synchronize()
    want = ref.Pool(pages, nkv, d, raw)
    want.write(slots, _host(k), _host(v))
    assert int(status) == 0
    assert np.array_equal(pool.cpu().numpy(), want.raw.reshape(-1))


def test_append_on_borders_and_special_values(nf):
    """Exact ties go to the even code, values one fp32 step beside them to their side, tiny groups are zeros,
    groups with an infinity, a NaN or more than 2^60 read back as NaN, their neighbours as ever."""
    d, nkv = 128, 2
    rows = []
    for s in (1.0, 0.25, 2.0 ** -40, 1.078125, 3.0 * 2.0 ** 20, 2.0 ** 57):
        g = np.zeros(32)
        g[0] = 7 * s   # scale: bf16(bf16(7 s) / 7)
        sc = float(ref.to_bf16(ref.to_bf16(7 * s) / 7))
        ties = [(n + 0.5) * sc for n in range(-7, 7)]
        g[1:15] = ties
        g32 = g.astype(np.float32)
        g32[15:29] = np.nextafter(np.array(ties, dtype=np.float32), np.float32(np.inf))
        g32[29:32] = np.nextafter(np.array(ties[:3], dtype=np.float32), np.float32(-np.inf))
        rows.append(g32)
    special = [np.full(32, 2.0 ** -61), np.full(32, 2.0 ** -60), np.zeros(32), np.full(32, 2.0 ** 60),
               np.full(32, 1.01 * 2.0 ** 60), np.full(32, 3e38), np.r_[np.inf, np.ones(31)], np.r_[np.ones(31), -np.inf],
               np.r_[np.ones(5), np.nan, np.ones(26)], np.r_[np.nan, np.full(31, np.inf)], np.full(32, -0.0),
               np.full(32, 1e-45), np.r_[-7.0, np.full(31, 0.5)], np.full(32, 3.4e38)]
    rows += [np.asarray(x, dtype=np.float32) for x in special]
    while len(rows) % (nkv * 4):
        rows.append(np.ones(32, dtype=np.float32))
    x = np.stack(rows).reshape(-1, nkv, d)
    T = len(x)
    k, v = _dev(x), _dev(x[::-1].copy())
    pool, status, slots = torch.zeros(2 * nkv * 18 * d, dtype=torch.uint8, device=DEV), _status(), _i32(range(5, 5 + T))
    _append(nf, k, v, slots, pool, 2, nkv, d, status)
    want = ref.Pool(2, nkv, d)
    want.write(range(5, 5 + T), x.astype(np.float64), x[::-1].astype(np.float64))
    assert np.array_equal(pool.cpu().numpy(), want.raw.reshape(-1))
    out = [torch.empty((T, nkv, d), dtype=torch.float32, device=DEV) for _ in range(2)]
    nf.check(nf.nf_op_kv4_read(pool.data_ptr(), 2, slots.data_ptr(), T, nkv, d, out[0].data_ptr(), nkv * d,
                               out[1].data_ptr(), nkv * d, F32, status.data_ptr()))
    torch.cuda.synchronize()
    for got, w in zip(out, want.rows(np.arange(5, 5 + T))):
        assert np.array_equal(_host(got), w, equal_nan=True)     # 3 bits of code by 8 of scale: exact in fp32
    assert int(status) == 0
    back = _host(out[0])
    over = np.isnan(back.reshape(-1, 32)).all(1)
    assert np.array_equal(np.isnan(back.reshape(-1, 32)).any(1), over) and 0 < over.sum() < len(over)


@pytest.mark.parametrize("T,nkv,d,dt", [(1, 1, 64, F32), (45, 2, 64, F32), (33, 5, 128, BF16), (3000, 8, 128, BF16),
                                        (100, 8, 128, F32)])
def test_read(nf, T, nkv, d, dt):
    rng = np.random.default_rng(T + nkv)
    pages = T // 16 + 2
    p = ref.Pool(pages, nkv, d, _garbage(rng, pages, nkv, d))
    p.raw[..., 8 * d + 1::2] = 0x3E + p.raw[..., 8 * d + 1::2] % 4   # scales around 1
    slots = rng.permutation(pages * 16)[:T]
    want = p.rows(slots)
    if T > 8:
        slots[5] = -1
    pool, status = _dev(p.raw.reshape(-1)), _status()
    kd = torch.full((T, nkv * d + 8), 9.0, dtype=TORCH[dt], device=DEV)
    vd = torch.full((T, nkv * d), 9.0, dtype=TORCH[dt], device=DEV)
    sl = _i32(slots)
    nf.check(nf.nf_op_kv4_read(pool.data_ptr(), pages, sl.data_ptr(), T, nkv, d, kd.data_ptr(), kd.stride(0),
                               vd.data_ptr(), vd.stride(0), dt, status.data_ptr()))
    torch.cuda.synchronize()
    assert int(status) == 0 and (kd[:, nkv * d:] == 9.0).all()
    for got, w in ((kd[:, :nkv * d], want[0]), (vd, want[1])):
        w = torch.from_numpy(w.reshape(T, -1)).to(torch.float32).to(TORCH[dt])   # exact in fp32, one rounding
        if T > 8:
            w[5] = 9.0
        assert torch.equal(got.cpu(), w)


def test_rows_outside_the_pool_are_reported_and_skipped(nf):
    nkv, d, pages, T = 2, 128, 3, 6
    rng = np.random.default_rng(5)
    raw = _garbage(rng, pages, nkv, d)
    k = _dev(rng.standard_normal((T, nkv, d)).astype(np.float32))
    for bad in ([48], [-2], [2 ** 31 - 1], [-2 ** 31]):
        slots = [7, 40] + bad + [1, 2, 3]
        pool, status = _dev(raw), _status()
        _append(nf, k, k, _i32(slots), pool, pages, nkv, d, status)
        want = ref.Pool(pages, nkv, d, raw)
        want.write(slots, _host(k), _host(k))
        assert np.array_equal(pool.cpu().numpy(), want.raw.reshape(-1)) and int(status) == nf.NF_ERR_DEVICE_BOUNDS
        status.zero_()
        out = torch.full((T, nkv, d), 9.0, device=DEV)
        sl = _i32(slots)
        nf.check(nf.nf_op_kv4_read(pool.data_ptr(), pages, sl.data_ptr(), T, nkv, d, out.data_ptr(), nkv * d,
                                   out.data_ptr(), nkv * d, F32, status.data_ptr()))
        torch.cuda.synchronize()
        assert (out[2] == 9.0).all() and (out[0] != 9.0).any() and int(status) == nf.NF_ERR_DEVICE_BOUNDS


# --- attention --------------------------------------------------------------------------------------


class Cache:
    """A 4-bit pool of random rows with requests of given lengths on scattered pages."""

    def __init__(self, lens, nkv, d, seed=0, spread=1.0, extra=2, v_scale=1.0):
        self.lens, self.nkv, self.d = list(lens), nkv, d
        rng = np.random.default_rng(seed)
        counts = [-(-n // 16) for n in lens]
        self.pages = sum(counts) + extra
        codes = rng.integers(1, 16, (self.pages, nkv, 2, 8 * d), dtype=np.uint8)
        codes |= rng.integers(1, 16, codes.shape, dtype=np.uint8) << 4
        scale = 0.15 * np.exp(0.5 * rng.standard_normal((self.pages, nkv, 2, d // 2)))
        scale[:, :, 0] *= spread
        scale[:, :, 1] *= v_scale
        raw = np.concatenate([codes, ref.to_bits(scale).view(np.uint8)], -1)
        self.host = ref.Pool(self.pages, nkv, d, raw)
        ids = rng.permutation(self.pages)
        self.indptr = np.concatenate([[0], np.cumsum(counts)])
        self.indices = ids[:max(1, self.indptr[-1])]
        # slots behind each request's last key: what an unwritten slot may hold (NaN scales among it)
        for r, n in enumerate(lens):
            if n % 16:
                page = self.indices[self.indptr[r + 1] - 1]
                for s in range(n % 16, 16):
                    at = 8 * d + s * (d // 32) * 2
                    self.host.raw[page, :, :, at:at + d // 32 * 2] = 0xFF
        self.upload()

    def upload(self):
        self.pool = _dev(self.host.raw.reshape(-1))
        self.dev = [_i32(self.lens if self.lens else [0]), _i32(self.indptr), _i32(self.indices)]

    def keys(self, r):
        pages = self.indices[self.indptr[r]:self.indptr[r + 1]]
        k, v = self.host.pages64(pages)
        n = self.lens[r]
        flat = lambda x: x.transpose(1, 0, 2, 3).reshape(self.nkv, -1, self.d)[:, :n]  # noqa: E731
        return flat(k), flat(v)


def _workspace(nf, nq, nkv, d):
    return torch.zeros(nf.nf_kv4_workspace_bytes(nq, nkv, d), dtype=torch.uint8, device=DEV)


def _attend(nf, c, q, out, ws, status, scale=0.0, sm=0, stream=0, R=None):
    nq = q.shape[1]
    nf.check(nf.nf_op_kv4_decode_attention(
        q.data_ptr(), q.stride(0), out.data_ptr(), out.stride(0), c.pool.data_ptr(), c.pages, c.dev[0].data_ptr(),
        c.dev[1].data_ptr(), c.dev[2].data_ptr(), len(c.lens) if R is None else R, nq, c.nkv, c.d, scale, ws.data_ptr(),
        ws.numel(), status.data_ptr(), sm, stream), "kv4 attention")


def _check_attention(c, q, got, scale=None, rows=None):
    """Against 64 bits, element by element. The output rounds once to bf16 (2^-8 of it); each weight rounds to
    fp16 (2^-11), and again when scaled by V's scale. A score is an fp32 sum of q (code + 8) less one of 8 q: at
    most |q| times 15 + 8 scales a column. Its roundings, in units of 2^-23 of that: 2 for the tensor-core steps of a
    group and 1 for that of the biases, 5 for the 10 additions of a group's bias, 1/2 for its split in three terms, 2 for 4 joins of groups:
    less than 11. (A scale is a seventh of its group's largest value or less; the bound takes the value itself for it,
    for steps of the tensor core that lose more.) A weight's relative error is twice (numerator, sum) that of its
    exponent; ex2 adds 2^-22 and the sums 2^-22 more. With S the group's largest scale so far, f in [2^3, 2^5) / S and
    the largest weight w at 2^4 or more, neither w nor w s f can be nearer than fp16's least step allows, 2^-25. Times
    |code| <= 8, over f and the sum of the weights (at least 2^4), that is 2^-26 of S (s <= S) and 2^-29 of S for each
    key; s f below 2^-14 may be off by as much, for all keys together 2^-14 8 / f <= 2^-14 S."""
    d, nkv = c.d, c.nkv
    G = q.shape[1] // nkv
    sc = 1.0 / math.sqrt(d) if scale is None else scale
    qh, gh = _host(q), _host(got)
    num = den = 0.0
    for r in range(len(c.lens)) if rows is None else rows:
        if c.lens[r] == 0:
            assert (gh[r] == 0.0).all()
            continue
        K, V = c.keys(r)
        for h in range(nkv):
            qq = qh[r, h * G:(h + 1) * G]
            want, mass = ref.attention(qq, K[h], V[h], sc)
            unit = np.abs(K[h]).reshape(len(K[h]), -1, 32).max(-1).repeat(32, -1)    # at least a scale, or a zero group
            x_err = 11 * 2.0 ** -23 * sc * (np.abs(qq) @ (23 * unit).T).max(-1)
            bound = 2.0 ** -8 * np.abs(want) + (2.0 ** -10 + 2 * x_err[:, None] + 2.0 ** -21) * mass
            # (some code of a group of 32 is not 0: its largest value is at least its scale)
            largest = np.abs(V[h]).max(0).reshape(-1, 32).max(-1).repeat(32)
            bound += (2.0 ** -14 + (2.0 ** -26 + 2.0 ** -29) * len(V[h])) * largest
            err = np.abs(gh[r, h * G:(h + 1) * G] - want)
            assert (err <= bound * (1 + 2.0 ** -6)).all(), (r, h, float((err / bound).max()))
            num, den = num + (err ** 2).sum(), den + (want ** 2).sum()
    if den:
        # over all elements the 2-norm of the bf16 roundings is at most 2^-8; the weights' errors are independent
        # and far below
        assert math.sqrt(num / den) <= 2.0 ** -8


SHAPES = [  # lengths, nq, nkv, d
    ([1], 1, 1, 64), ([1, 2, 15, 16, 17, 0, 31, 32, 33], 4, 2, 64), ([0, 0, 5], 8, 8, 128),
    ([64, 100, 1], 32, 8, 128), ([257, 3, 640, 0, 17], 15, 5, 128), ([1000] * 3, 14, 2, 64), ([500, 700], 24, 4, 128),
    (list(range(0, 75)), 6, 1, 128), ([5000], 8, 1, 128), ([4096, 1, 3000], 64, 8, 128), ([20011], 7, 1, 64),
    ([333] * 40, 32, 8, 128), ([9] * 700, 2, 2, 64),
    # fewer (request, KV head) pairs than SMs, of equal lengths and of very different ones
    ([300 + i for i in range(18)], 8, 8, 128), ([9000] + [3] * 16 + [0], 16, 8, 128), ([2000, 1, 40] * 5, 18, 9, 64)]


@pytest.mark.parametrize("lens,nq,nkv,d", SHAPES, ids=lambda x: str(x)[:20] if isinstance(x, list) else str(x))
def test_attention(nf, lens, nq, nkv, d):
    c = Cache(lens, nkv, d, seed=len(lens) + nq)
    R = len(lens)
    rng = np.random.default_rng(R)
    wide_q = _dev(rng.standard_normal((R + 2, nq * d + 24)).astype(np.float32), torch.bfloat16)
    q = wide_q[:R, 8:8 + nq * d].unflatten(1, (nq, d))
    wide_out = torch.full((R + 2, nq * d + 16), -7.0, dtype=torch.bfloat16, device=DEV)
    out = wide_out[:R, :nq * d].unflatten(1, (nq, d))
    ws, status = _workspace(nf, nq, nkv, d), _status()
    _attend(nf, c, q, out, ws, status)
    torch.cuda.synchronize()
    assert int(status) == 0
    first = out.clone()
    _check_attention(c, q, out)
    assert (wide_out[:R, nq * d:] == -7.0).all() and (wide_out[R:] == -7.0).all()
    for sm in (0, 1, 5):   # again (the workspace as the call left it), and on few SMs
        out.fill_(float("nan"))
        _attend(nf, c, q, out, ws, status, sm=sm)
        torch.cuda.synchronize()
        if sm == 0:
            assert torch.equal(out, first)
        _check_attention(c, q, out, rows=range(min(R, 12)))
    _attend(nf, c, q, q, ws, status)   # in place
    torch.cuda.synchronize()
    assert torch.equal(q, first)


@pytest.mark.parametrize("scale,spread", [(0.02, 1.0), (1.0, 1.0), (3.0, 4.0)])
def test_attention_scale_and_peaked_rows(nf, scale, spread):
    """From almost equal weights to one key that takes all: the running maximum moves far."""
    c = Cache([700, 33, 1], 2, 128, seed=5, spread=spread)
    q = _dev(np.random.default_rng(1).standard_normal((3, 8, 128)).astype(np.float32), torch.bfloat16)
    out, ws, status = torch.empty_like(q), _workspace(nf, 8, 2, 128), _status()
    _attend(nf, c, q, out, ws, status, scale=scale)
    torch.cuda.synchronize()
    _check_attention(c, q, out, scale=float(np.float32(scale)))


@pytest.mark.parametrize("qs,vs", [(2.0 ** 40, 2.0 ** -30), (2.0 ** -40, 2.0 ** 30), (2.0 ** -126, 2.0 ** 57),
                                   (1.0, 2.0 ** -50), (2.0 ** 20, 1.0)])
def test_attention_at_far_magnitudes(nf, qs, vs):
    """Large and small q (K scaled against it, so that the scores stay ordinary) and V."""
    spread = min(max(1.0 / qs, 2.0 ** -50), 2.0 ** 50)
    c = Cache([200, 17], 2, 128, seed=6, spread=spread, v_scale=vs)
    x = np.random.default_rng(1).standard_normal((2, 4, 128)) * qs
    q = _dev(x.astype(np.float32), torch.bfloat16)
    out, ws, status = torch.empty_like(q), _workspace(nf, 4, 2, 128), _status()
    _attend(nf, c, q, out, ws, status)
    torch.cuda.synchronize()
    _check_attention(c, q, out)


@pytest.mark.parametrize("qs", [2.0 ** 60, 2.0 ** 100, 2.0 ** 112, 2.0 ** 118, 2.0 ** 122])
def test_attention_of_huge_scores_takes_the_largest(nf, qs):
    """Scores up to 2^80, far apart: one key has all the weight, the others' underflow."""
    c = Cache([200, 17, 33], 2, 128, seed=16, spread=2.0 ** -45)
    x = np.random.default_rng(3).standard_normal((3, 8, 128)) * qs
    q = _dev(x.astype(np.float32), torch.bfloat16)
    out, ws, status = torch.empty_like(q), _workspace(nf, 8, 2, 128), _status()
    _attend(nf, c, q, out, ws, status)
    torch.cuda.synchronize()
    qh, gh = _host(q), _host(out)
    for r in range(3):
        K, V = c.keys(r)
        for h in range(8):
            s = K[h // 4] @ qh[r, h] / math.sqrt(128)
            order = np.argsort(s)
            # the rounding of a score (_check_attention) cannot change the order, and the next weight is below 2^-100
            err = 11 * 2.0 ** -23 * 23 * (np.abs(K[h // 4]).max() * np.abs(qh[r, h]).sum()) / math.sqrt(128)
            if s[order[-1]] - s[order[-2]] <= 2 * err + 100:
                continue
            want = V[h // 4][order[-1]]
            # one weight, 1 of 1 but for the roundings to fp16 and that of the output
            bound = (2.0 ** -8 + 2.0 ** -10) * np.abs(want) + 2.0 ** -13 * np.abs(V[h // 4]).max()
            assert (np.abs(gh[r, h] - want) <= bound).all(), (r, h)


def test_attention_mixed_v_scales_in_one_row(nf):
    """V scales that differ by 2^60 between keys and groups: small groups keep their own precision."""
    c = Cache([300, 40], 1, 128, seed=9)
    sc = c.host.raw[:, :, 1, 8 * 128:]
    f = ref.from_bits(np.ascontiguousarray(sc).view(np.uint16)).reshape(c.pages, 1, 16, 4)
    f = np.where(np.isnan(f), 1.0, f) * np.array([2.0 ** -30, 1.0, 2.0 ** 30, 2.0 ** -5])
    sc[...] = ref.to_bits(f).view(np.uint8).reshape(sc.shape)
    c.upload()
    q = _dev(np.random.default_rng(1).standard_normal((2, 8, 128)).astype(np.float32), torch.bfloat16)
    out, ws, status = torch.empty_like(q), _workspace(nf, 8, 1, 128), _status()
    _attend(nf, c, q, out, ws, status)
    torch.cuda.synchronize()
    _check_attention(c, q, out)


def test_attention_propagates_nan_of_seen_keys_only(nf):
    """A NaN scale in a visible V group reaches that group's columns of its KV head's rows; in a visible K
    group, all columns; slots behind the length (NaN here everywhere) reach nothing."""
    c = Cache([50, 50, 50], 2, 128, seed=3)
    page = c.indices[c.indptr[0] + 1]
    c.host.raw[page, 1, 1, 8 * 128 + (5 * 4 + 2) * 2:][:2] = [0xC0, 0x7F]     # request 0, head 1, V slot 5, group 2
    page = c.indices[c.indptr[2]]
    c.host.raw[page, 0, 0, 8 * 128 + (3 * 4 + 1) * 2:][:2] = [0xC0, 0x7F]     # request 2, head 0, K
    c.upload()
    q = _dev(np.random.default_rng(1).standard_normal((3, 4, 128)).astype(np.float32), torch.bfloat16)
    out, ws, status = torch.empty_like(q), _workspace(nf, 4, 2, 128), _status()
    _attend(nf, c, q, out, ws, status)
    torch.cuda.synchronize()
    nan = torch.isnan(out).cpu().numpy()
    want = np.zeros_like(nan)
    want[0, 2:, 64:96] = True
    want[2, :2] = True
    assert np.array_equal(nan, want)
    _check_attention(c, q, out, rows=[1])


def test_attention_reports_bad_lengths_and_pages(nf):
    c = Cache([40, 40, 40, 40, 40], 2, 128, seed=4)
    q = _dev(np.random.default_rng(1).standard_normal((5, 4, 128)).astype(np.float32), torch.bfloat16)
    ws = _workspace(nf, 4, 2, 128)
    clean = c.indices.copy()
    for fault in ("negative", "long", "page", "page_negative", "indptr"):
        lens, indices, indptr = list(c.lens), clean.copy(), c.indptr.copy()
        kept = 40
        if fault == "negative":
            lens[2], kept = -5, 0
        elif fault == "long":
            lens[2], kept = 49, 48        # one key more than its three pages hold
        elif fault == "page":
            indices[c.indptr[2] + 1] = c.pages
        elif fault == "page_negative":
            indices[c.indptr[2] + 1] = -3
        else:
            indptr[3] = indptr[2] - 1     # a row that ends before it starts
            kept = 0
        c.dev = [_i32(lens), _i32(indptr), _i32(indices)]
        out, status = torch.full_like(q, float("nan")), _status()
        _attend(nf, c, q, out, ws, status)
        torch.cuda.synchronize()
        assert int(status) == nf.NF_ERR_DEVICE_BOUNDS, fault
        got = _host(out)[2]
        K, V = c.host.pages64(clean[c.indptr[2]:c.indptr[3]])
        K, V = (x.transpose(1, 0, 2, 3).reshape(2, -1, 128) for x in (K, V))
        seen = np.arange(48) < kept
        if "page" in fault:
            seen[16:32] = False
        if fault == "long":
            assert np.isnan(got).all()    # it reads slots that hold NaN here
        else:
            for h in range(2):
                want, mass = ref.attention(_host(q)[2, 2 * h:2 * h + 2], K[h][seen], V[h][seen], 128 ** -0.5)
                assert (np.abs(got[2 * h:2 * h + 2] - want) <= 2.0 ** -7 * np.abs(want) + 2.0 ** -8 * mass).all(), fault
        if fault != "indptr":
            _check_attention(c, q, out, rows=[0, 1, 3, 4])


def test_attention_far_into_a_large_pool(nf):
    """Pages beyond byte 2^32 of the pool."""
    nkv, d, pages = 8, 128, 240000                 # 4.4 GB
    nb = nf.nf_kv4_page_bytes(nkv, d)
    assert pages * nb > 2 ** 32
    small = Cache([100, 40], nkv, d, seed=8, extra=0)
    pool = torch.empty(pages * nb, dtype=torch.uint8, device=DEV)
    far = pages - 1 - 3 * np.arange(small.pages)
    view = pool.view(pages, nb)
    view[torch.from_numpy(far).to(DEV)] = _dev(small.host.raw.reshape(small.pages, -1))
    q = _dev(np.random.default_rng(1).standard_normal((2, 32, d)).astype(np.float32), torch.bfloat16)
    out, ws, status = torch.empty_like(q), _workspace(nf, 32, nkv, d), _status()
    idx = _i32(far[small.indices])
    nf.check(nf.nf_op_kv4_decode_attention(q.data_ptr(), 32 * d, out.data_ptr(), 32 * d, pool.data_ptr(), pages,
                                           small.dev[0].data_ptr(), small.dev[1].data_ptr(), idx.data_ptr(), 2, 32, nkv,
                                           d, 0.0, ws.data_ptr(), ws.numel(), status.data_ptr()))
    torch.cuda.synchronize()
    assert int(status) == 0
    _check_attention(small, q, out)
    # rows written and read there
    slots = _i32([int(far[0]) * 16 + 15, (pages - 1) * 16 + 14])
    x = _dev(np.random.default_rng(2).standard_normal((2, nkv, d)).astype(np.float32))
    _append(nf, x, x, slots, pool, pages, nkv, d, status)
    back = [torch.empty_like(x) for _ in range(2)]
    nf.check(nf.nf_op_kv4_read(pool.data_ptr(), pages, slots.data_ptr(), 2, nkv, d, back[0].data_ptr(), nkv * d,
                               back[1].data_ptr(), nkv * d, F32, status.data_ptr()))
    torch.cuda.synchronize()
    codes, scale = ref.quantise(_host(x))
    assert int(status) == 0
    for b in back:
        assert np.array_equal(_host(b), ref.values(codes, scale))


def test_attention_ordinary_length_row_among_many_empty(nf):
    lens = [0] * 3000
    lens[1234], lens[2999] = 200, 3
    c = Cache(lens, 2, 64, seed=1)
    q = _dev(np.random.default_rng(1).standard_normal((3000, 4, 64)).astype(np.float32), torch.bfloat16)
    out, ws, status = torch.full_like(q, float("nan")), _workspace(nf, 4, 2, 64), _status()
    _attend(nf, c, q, out, ws, status)
    torch.cuda.synchronize()
    assert int(status) == 0
    _check_attention(c, q, out, rows=[1234, 2999])
    out[1234] = out[2999] = 0
    assert (out == 0).all()


@pytest.mark.parametrize("R,nq,nkv", [(16384, 2, 1), (16383, 1, 1), (3, 2048, 256), (150, 256, 256)])
def test_attention_at_the_limits(nf, R, nq, nkv):
    """The most requests and the most heads that a call takes."""
    rng = np.random.default_rng(R + nkv)
    lens = rng.integers(0, 41, R)
    lens[-1] = 700 if R < 100 else 90
    c = Cache([int(n) for n in lens], nkv, 64, seed=R)
    q = _dev(rng.standard_normal((R, nq, 64)).astype(np.float32), torch.bfloat16)
    out, ws, status = torch.full_like(q, float("nan")), _workspace(nf, nq, nkv, 64), _status()
    _attend(nf, c, q, out, ws, status)
    torch.cuda.synchronize()
    assert int(status) == 0
    rows = [0, R - 1] if R < 200 else [0, R - 1, *rng.integers(0, R, 300)]
    _check_attention(c, q, out, rows=rows)
    gone = torch.from_numpy(lens == 0).to(DEV)
    assert (out[gone] == 0).all() and out[~gone].isfinite().all()


# --- together ---------------------------------------------------------------------------------------


class Step:
    """Decode steps over a 4-bit cache from the rows that the QKV product leaves: every operator, in order."""

    def __init__(self, nf, R, nq, nkv, d, hidden, pages, stride, lens, seed=0):
        self.nf, self.R, self.nq, self.nkv, self.d, self.hidden, self.pages, self.stride = (
            nf, R, nq, nkv, d, hidden, pages, stride)
        rng = np.random.default_rng(seed)
        self.width = (nq + 2 * nkv) * d
        self.w = _dev((rng.standard_normal((self.width, hidden)) * 0.08).astype(np.float32), torch.bfloat16)
        self.x = torch.zeros((R, hidden), dtype=torch.bfloat16, device=DEV)
        self.rows = torch.zeros((R, self.width), dtype=torch.float32, device=DEV)
        self.q = torch.zeros((R, nq, d), dtype=torch.bfloat16, device=DEV)
        self.k = torch.zeros((R, nkv, d), dtype=torch.bfloat16, device=DEV)
        self.out = torch.zeros((R, nq, d), dtype=torch.bfloat16, device=DEV)
        self.pool = torch.full((pages * nf.nf_kv4_page_bytes(nkv, d),), 0xFF, dtype=torch.uint8, device=DEV)
        self.table = torch.full((R, stride), -1, dtype=torch.int32, device=DEV)
        self.free = _i32(rng.permutation(pages))
        self.count, self.left = _i32([pages]), _i32([0])
        self.lens = _i32(lens)
        self.kv_len, self.indptr = _i32([0] * R), _i32([0] * (R + 1))
        self.indices, self.slots, self.positions = _i32([0] * (R * stride)), _i32([0] * R), _i32([0] * R)
        self.freq = _dev(_freqs(d))
        self.ws, self.status = _workspace(nf, nq, nkv, d), _status()

    def run(self, stream=0):
        nf, R, nq, nkv, d = self.nf, self.R, self.nq, self.nkv, self.d
        p = lambda t: t.data_ptr()  # noqa: E731
        nf.check(nf.nf_op_page_map(p(self.lens), 0, R, p(self.table), self.stride, p(self.free), self.free.numel(),
                                   p(self.count), self.pages, p(self.kv_len), p(self.indptr), p(self.indices),
                                   self.indices.numel(), p(self.slots), p(self.positions), R, p(self.left),
                                   p(self.status), stream), "map")
        nf.check(nf.nf_op_gemm_bf16(p(self.x), p(self.w), p(self.rows), R, self.width, self.hidden, 0, stream), "gemm")
        nf.check(nf.nf_op_rope(p(self.rows), self.width, p(self.q), nq * d, nq, p(self.rows) + 4 * nq * d, self.width,
                               p(self.k), nkv * d, nkv, F32, BF16, p(self.positions), R, d, d, 0, p(self.freq), 1.0,
                               stream), "rope")
        nf.check(nf.nf_op_kv4_append(p(self.k), nkv * d, BF16, p(self.rows) + 4 * (nq + nkv) * d, self.width, F32,
                                     p(self.slots), R, p(self.pool), self.pages, nkv, d, p(self.status), stream),
                 "append")
        nf.check(nf.nf_op_kv4_decode_attention(p(self.q), nq * d, p(self.out), nq * d, p(self.pool), self.pages,
                                               p(self.kv_len), p(self.indptr), p(self.indices), R, nq, nkv, d, 0.0,
                                               p(self.ws), self.ws.numel(), p(self.status), 0, stream), "attention")

    def advance(self):
        self.lens.copy_(self.kv_len)
        self.count.copy_(self.left)


def _steps(seed, n, R, hidden):
    rng = np.random.default_rng(seed)
    return [_dev(rng.standard_normal((R, hidden)).astype(np.float32), torch.bfloat16) for _ in range(n)]


def test_decode_steps_together(nf):
    """40 decode steps of 5 requests, each operator feeding the next; the whole history recomputed in 64 bits."""
    R, nq, nkv, d, hidden, n = 5, 8, 2, 64, 256, 40
    s = Step(nf, R, nq, nkv, d, hidden, pages=20, stride=4, lens=[0] * R)
    freq, w = _freqs(d), None
    hist = [([], []) for _ in range(R)]
    for i, x in enumerate(_steps(1, n, R, hidden)):
        s.x.copy_(x)
        s.run()
        torch.cuda.synchronize()
        assert int(s.status) == 0
        w = _host(s.w) if w is None else w
        rows = _host(x) @ w.T
        k = ref.rope(rows[:, nq * d:(nq + nkv) * d].reshape(R, nkv, d), np.full(R, i), freq, 1.0, d, False)
        v = rows[:, (nq + nkv) * d:].reshape(R, nkv, d)
        q = _host(s.q)
        want_q = ref.rope(rows[:, :nq * d].reshape(R, nq, d), np.full(R, i), freq, 1.0, d, False)
        # a product of 256 fp32 terms (2^-23 each of at most the sum of their sizes), rope, one bf16 rounding
        size = (np.abs(_host(x)) @ np.abs(w).T)[:, :nq * d].reshape(R, nq, d).max()
        assert np.abs(q - want_q).max() <= 2.0 ** -8 * np.abs(want_q).max() + 260 * 2.0 ** -23 * size
        back = [torch.empty((R, nkv, d), dtype=torch.float32, device=DEV) for _ in range(2)]
        nf.check(nf.nf_op_kv4_read(s.pool.data_ptr(), s.pages, s.slots.data_ptr(), R, nkv, d, back[0].data_ptr(),
                                   nkv * d, back[1].data_ptr(), nkv * d, F32, s.status.data_ptr()))
        torch.cuda.synchronize()
        out = _host(s.out)
        for which, (exact, held) in enumerate(((k, _host(back[0])), (v, _host(back[1])))):
            top = np.abs(exact.reshape(R, nkv, -1, 32)).max(-1).repeat(32, -1).reshape(R, nkv, d)
            # half a step of a seventh of the largest; largest, scale (twice) and k are rounded to bf16, by 2^-8 each;
            # and fp32 noise of the product across a border
            assert (np.abs(held - exact) <= top * (0.5 / 7 + 4 * 2.0 ** -8 + 1e-4)).all()
            for r in range(R):
                hist[r][which].append(held[r])
        for r in range(R):
            K, V = (np.stack(h).transpose(1, 0, 2) for h in hist[r])
            for h in range(nkv):
                want, mass = ref.attention(q[r, 4 * h:4 * h + 4], K[h], V[h], d ** -0.5)
                assert (np.abs(out[r, 4 * h:4 * h + 4] - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -9 * mass).all()
        assert s.kv_len.tolist() == [i + 1] * R and int(s.left) == 20 - R * (-(-(i + 1) // 16))
        s.advance()


def test_captured_steps_replay_to_the_same_bits(nf):
    """Two graphs with workspaces of their own, replayed in turn on two streams, against plain calls."""
    R, nq, nkv, d, hidden = 6, 32, 8, 128, 512
    lens = [0, 15, 16, 300, 1000, 77]
    xs = _steps(7, 3, R, hidden)

    def fresh(seed):
        s = Step(nf, R, nq, nkv, d, hidden, pages=200, stride=70, lens=lens, seed=seed)
        rng = np.random.default_rng(seed)
        b = [-(-n // 16) for n in lens]
        for r in range(R):   # pages of the cached tokens, filled
            s.table[r, :b[r]] = s.free[sum(b[:r]):sum(b[:r + 1])]
        s.free = s.free[sum(b):].clone()
        s.count.fill_(s.free.numel())
        rows = _dev(rng.standard_normal((200 * 16, nkv, d)).astype(np.float32))
        _append(nf, rows, rows, _i32(range(200 * 16)), s.pool, 200, nkv, d, s.status)
        torch.cuda.synchronize()
        return s

    want = []
    for seed in (1, 2):
        s = fresh(seed)
        for x in xs:
            s.x.copy_(x)
            s.run()
            s.advance()
            torch.cuda.synchronize()
            want.append(s.out.clone())
        assert int(s.status) == 0
    steps = [fresh(1), fresh(2)]
    graphs, streams = [], [torch.cuda.Stream(DEV) for _ in range(2)]
    for s, st in zip(steps, streams):
        keep = [t.clone() for t in (s.table, s.pool)]
        s.x.copy_(xs[0])
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            s.run(st.cuda_stream)          # once before the capture, then put back
            st.synchronize()
            s.table.copy_(keep[0])
            s.pool.copy_(keep[1])
            st.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=st):
                s.run(st.cuda_stream)
                s.advance()
        graphs.append(g)
    for i, x in enumerate(xs):
        for s, g, st in zip(steps, graphs, streams):
            with torch.cuda.stream(st):
                s.x.copy_(x)
                g.replay()
        torch.cuda.synchronize()
        for j, s in enumerate(steps):
            assert int(s.status) == 0
            assert torch.equal(s.out, want[3 * j + i]), (i, j)
    del graphs


def test_calls_from_two_streams_at_once(nf):
    """Ordinary calls that overlap on two streams, a workspace each."""
    caches = [Cache([900, 30, 0, 411], 8, 128, seed=s) for s in (1, 2)]
    q = [_dev(np.random.default_rng(s).standard_normal((4, 32, 128)).astype(np.float32), torch.bfloat16) for s in (1, 2)]
    ws = [_workspace(nf, 32, 8, 128) for _ in range(2)]
    outs = [torch.full_like(x, float("nan")) for x in q]
    streams, status = [torch.cuda.Stream(DEV) for _ in range(2)], _status()
    torch.cuda.synchronize()
    for _ in range(30):
        for i in (0, 1):
            _attend(nf, caches[i], q[i], outs[i], ws[i], status, stream=streams[i].cuda_stream)
    torch.cuda.synchronize()
    assert int(status) == 0
    for i in (0, 1):
        _check_attention(caches[i], q[i], outs[i])


@pytest.mark.parametrize("op,extra", [("kv4_decode_attention", []), ("kv4_decode_attention", ["--requests", "3", "--sm", "2"]),
                                      ("kv4_append", []), ("kv4_read", ["--rows", "9"]), ("rope", []), ("page_map", [])])
def test_each_operation_timed_alone(nf, op, extra, capsys):
    from intra_device_overlapped_b200 import opbench
    got = opbench.main(["--op", op, "--workload", "tiny_layer", "--reps", "2", *extra])
    assert got["us"] > 0 and got["bytes"] > 0 and op in capsys.readouterr().out


def test_host_memory_is_refused(nf):
    host = torch.zeros(1 << 16, dtype=torch.uint8).pin_memory()
    dev = torch.zeros(1 << 16, dtype=torch.uint8, device=DEV)
    h, g = host.data_ptr(), dev.data_ptr()
    bad = nf.NF_ERR_INVALID_ARGUMENT
    assert nf.nf_op_kv4_append(h, 64, 0, g, 64, 0, g, 1, g, 1, 1, 64, g) == bad
    assert nf.nf_op_kv4_read(g, 1, h, 1, 1, 64, g, 64, g, 64, 0, g) == bad
    assert nf.nf_op_rope(g, 64, h, 64, 1, 0, 0, 0, 0, 0, 0, 0, g, 1, 64, 64, 0, g) == bad
    size = nf.nf_kv4_workspace_bytes(1, 1, 64)
    ws = torch.zeros(size, dtype=torch.uint8, device=DEV)
    assert nf.nf_op_kv4_decode_attention(g, 64, g, 64, g, 1, h, g, g, 1, 1, 1, 64, 0.0, ws.data_ptr(), size, g) == bad
    assert nf.nf_op_page_map(g, h, 1, g, 1, g, 1, g, 1, g, g, g, 1, g, g, 1, g + 4096, g) == bad
    torch.cuda.synchronize()
