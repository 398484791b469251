"""What attention over the 4-bit KV cache may lose: roundings counted one by one, outliers among keys and columns."""
import math

import numpy as np
import pytest
import torch

import kv4_reference as ref
from test_gpu_kv4 import Cache, _attend, _dev, _host, _status, _workspace

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nf():
    import intra_device_overlapped_b200 as m
    return m


def _scales(c, which):
    """View [pages, nkv, 16, d / 32] of a host pool's scales as bf16 bits (a copy: _put stores it)."""
    raw = np.ascontiguousarray(c.host.raw[:, :, which, 8 * c.d:]).view(np.uint16)
    return raw.reshape(c.pages, c.nkv, 16, c.d // 32)


def _put(c, which, bits):
    c.host.raw[:, :, which, 8 * c.d:] = np.ascontiguousarray(bits).view(np.uint8).reshape(c.pages, c.nkv, -1)


def _run(nf, c, q, scale=0.0, sm=0):
    out, ws, status = torch.full_like(q, float("nan")), _workspace(nf, q.shape[1], c.nkv, c.d), _status()
    _attend(nf, c, q, out, ws, status, scale=scale, sm=sm)
    torch.cuda.synchronize()
    assert int(status) == 0
    return out


def _check(c, q, got, scale=None, rows=None):
    """Against 64 bits, column by column, relative to the sums of weight times |V| ("mass") alone. A weight times a
    scale of V rounds to fp16 once (2^-11); the output rounds to bf16 (2^-8). A score is an fp32 sum of q (code + 8) less
    one of 8 q: 23 scales a column at most, rounded in units of 2^-23 of that 11 times at most (2 tensor-core steps of
    a group, 1 for that of the biases, 5 for the 10 additions of a group's bias, 1/2 for its split in three terms, 2 for
    4 joins of groups), and q's columns are off by 2^-24 of the largest of their 32 at most. A weight's relative error is
    twice that of its exponent (numerator, sum); ex2 adds 2^-22 and the sums 2^-22 more. What is too small for fp16
    comes to 2^-12 of the largest mass of the 32 columns."""
    d, nkv = c.d, c.nkv
    G = q.shape[1] // nkv
    sc = 1.0 / math.sqrt(d) if scale is None else scale
    qh, gh = _host(q), _host(got)
    worst = 0.0
    for r in range(len(c.lens)) if rows is None else rows:
        K, V = c.keys(r)
        for h in range(nkv):
            qq = qh[r, h * G:(h + 1) * G]
            want, mass = ref.attention(qq, K[h], V[h], sc)
            unit = np.abs(K[h]).reshape(len(K[h]), -1, 32).max(-1).repeat(32, -1)
            most = np.abs(qq).reshape(G, -1, 32).max(-1).repeat(32, -1)
            x_err = sc * ((11 * 2.0 ** -23 * 23 * np.abs(qq) + 2.0 ** -24 * most) @ unit.T).max(-1)
            group = mass.reshape(G, -1, 32).max(-1).repeat(32, -1)
            bound = 2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 2 * x_err[:, None] + 2.0 ** -21) * mass + 2.0 ** -12 * group
            err = np.abs(gh[r, h * G:(h + 1) * G] - want)
            assert (err <= bound * (1 + 2.0 ** -6) + 1e-37).all(), (r, h, float((err / (bound + 1e-37)).max()))
            worst = max(worst, float((err / (bound + 1e-37)).max()))
    return worst


def test_a_weight_rounds_once(nf):
    """Two keys whose values are opposite and whose weights differ by 2^-8 at most: the output's own rounding is far below
    the weights'. (The sum of two roundings of 2^-11 each is above the bound for one (request, head, group) in 70.)"""
    R, nkv, d = 96, 2, 128
    c = Cache([2] * R, nkv, d, seed=11)
    rng = np.random.default_rng(12)
    pages = c.indices
    for which in (0, 1):
        byte, half = c.host.byte[which], c.host.half[which]
        tile = c.host.raw[:, :, which]
        codes = (tile[:, :, byte[0]] >> (4 * half[0])) % 16     # [pages, nkv, d] of slot 0
        other = codes if which == 0 else 16 - codes
        for slot, new in ((0, codes), (1, other)):
            new = new.copy()
            if which == 0:
                new[..., 0] = 15
            for hf in (0, 1):
                cols = np.nonzero(half[slot] == hf)[0]
                b = byte[slot, cols]
                keep = 0xF0 if hf == 0 else 0x0F
                tile[:, :, b] = (tile[:, :, b] & keep) | (new[..., cols] << (4 * hf)).astype(np.uint8)
        bits = _scales(c, which).copy()
        bits[:, :, 0] = 0x3E00 + rng.integers(0, 127, bits[:, :, 0].shape)   # 1/8 .. 1/4, any mantissa
        bits[:, :, 1] = bits[:, :, 0] + (1 if which == 0 else 0)             # the next score beside the first's
        _put(c, which, bits)
    c.upload()
    q = torch.zeros((R, 16, d), dtype=torch.bfloat16, device="cuda:0")
    q[..., 0] = _dev(rng.standard_normal((R, 16)).astype(np.float32) * 2, torch.bfloat16)
    out = _run(nf, c, q)
    assert pages.size == R
    qh, gh = _host(q), _host(out)
    for r in range(R):
        K, V = c.keys(r)
        assert np.array_equal(V[:, 0], -V[:, 1])
        for h in range(nkv):
            qq = qh[r, 8 * h:8 * h + 8]
            want, mass = ref.attention(qq, K[h], V[h], d ** -0.5)
            # _check's terms, without the loss of weights too small for fp16: these are not
            x_err = d ** -0.5 * 11 * 2.0 ** -23 * 23 * (np.abs(qq) @ np.abs(K[h]).T).max(-1)[:, None]
            bound = 2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 2 * x_err + 2.0 ** -21) * mass
            err = np.abs(gh[r, 8 * h:8 * h + 8] - want)
            assert (err <= bound).all(), (r, h, float((err - bound).max()))


def _set_key(c, r, at, which, head, scales=None, codes=None):
    """Key `at` of request r: its scales (one per group, None: as they are) and codes [d] in -7..7."""
    page, slot = c.indices[c.indptr[r] + at // 16], at % 16
    tile = c.host.raw[page, head, which]
    if scales is not None:
        n = 8 * c.d + slot * (c.d // 32) * 2
        for j, s in enumerate(scales):
            if s is not None:
                tile[n + 2 * j:n + 2 * j + 2] = ref.to_bits(np.array([s])).view(np.uint8)
    if codes is not None:
        for hf in (0, 1):
            cols = np.nonzero(c.host.half[which, slot] == hf)[0]
            b = c.host.byte[which, slot, cols]
            tile[b] = (tile[b] & (0xF0 if hf == 0 else 0x0F)) | ((codes[cols] + 8) << (4 * hf)).astype(np.uint8)


def _biased(c, q, keys, log2_weight, head):
    """The keys' scores at `head` lower by `log2_weight` than they would be at 0: column 0 of q is 4 for every head."""
    d = c.d
    codes = np.zeros(d, dtype=np.int64)
    codes[0] = -7
    for r, at in keys:
        scale = log2_weight * math.log(2) * math.sqrt(d) / (4 * 7)
        _set_key(c, r, at, 0, head, scales=[scale] + [0.0] * (d // 32 - 1), codes=codes)


OUTLIERS = [  # log2 of the weight that a key loses, log2 of its values' magnitude
    (100, 40), (60, 57), (30, 30), (20, 18), (40, 25), (12, 10), (40, 17), (25, 24), (0, 17), (0, -40)]


@pytest.mark.parametrize("lens,nq,nkv,d", [([2, 16, 40], 8, 2, 128), ([700, 33], 12, 2, 64), ([3000], 8, 1, 128),
                                           ([90, 100, 17, 64] * 12, 16, 4, 128)], ids=str)
@pytest.mark.parametrize("below,above", OUTLIERS)
def test_keys_of_little_weight_and_large_values(nf, lens, nq, nkv, d, below, above):
    """Keys with values 2^above times the others' and weights 2^-below of theirs, in some groups of columns or all: they
    count for what they are, and so do the others."""
    rng = np.random.default_rng(below * 64 + abs(above) + len(lens))
    c = Cache(lens, nkv, d, seed=below + len(lens), spread=0.5)
    q = rng.standard_normal((len(lens), nq, d))
    q[..., 0] = 4.0
    ng = d // 32
    for r, n in enumerate(lens):
        for head in range(nkv):
            keys = sorted({int(x) for x in rng.integers(0, n, max(1, n // 300))} - ({0} if n == 2 else set()))
            _biased(c, q, [(r, k) for k in keys], below, head)
            groups = range(ng) if (r + head) % 2 else [head % ng, ng - 1]
            for k in keys:
                _set_key(c, r, k, 1, head, [0.15 * 2.0 ** above if j in groups else None for j in range(ng)])
    c.upload()
    q = _dev(q.astype(np.float32), torch.bfloat16)
    for sm in (0, 3):
        _check(c, q, _run(nf, c, q, sm=sm), rows=range(min(len(lens), 6)))


@pytest.mark.parametrize("lens,nq,nkv,d", [([2], 1, 1, 64), ([40, 300], 8, 2, 128), ([2500] * 3, 16, 2, 128)], ids=str)
@pytest.mark.parametrize("weight", [20, 35, 60])
def test_the_key_that_weighs_most_has_no_values(nf, lens, nq, nkv, d, weight):
    """One key takes nearly all the weight and holds zeros in some groups: the others' values are what is left there. A
    group without values in any key is exactly 0."""
    rng = np.random.default_rng(weight)
    c = Cache(lens, nkv, d, seed=weight, spread=0.25)
    q = rng.standard_normal((len(lens), nq, d)) * 0.5
    q[..., 0] = 4.0
    ng = d // 32
    for r, n in enumerate(lens):
        for head in range(nkv):
            k = int(rng.integers(0, n))
            _biased(c, q, [(r, at) for at in range(n) if at != k], weight, head)
            _set_key(c, r, k, 1, head, [0.0 if j % 2 == 0 else None for j in range(ng)])
            if ng == 4:
                for at in range(n):
                    _set_key(c, r, at, 1, head, [None, None, None, 0.0])
    c.upload()
    q = _dev(q.astype(np.float32), torch.bfloat16)
    out = _run(nf, c, q)
    _check(c, q, out)
    if ng == 4:
        assert (out[..., 96:] == 0).all() and (out[..., :32] != 0).any()


def test_outliers_beside_missing_pages_and_nan(nf):
    """A key of large values and no weight in a request with a page outside the pool, and one with a NaN scale."""
    c = Cache([70, 70], 1, 128, seed=21)
    q = np.random.default_rng(4).standard_normal((2, 8, 128))
    q[..., 0] = 4.0
    for r in (0, 1):
        _biased(c, q, [(r, 5)], 80, 0)
        _set_key(c, r, 5, 1, 0, [2.0 ** 35] * 4)
    _set_key(c, 1, 9, 1, 0, [None, math.nan, None, None])
    c.upload()
    clean = c.indices.copy()
    c.indices[c.indptr[0] + 2] = c.pages + 7
    c.dev[2] = torch.from_numpy(c.indices.astype(np.int32)).cuda()
    q = _dev(q.astype(np.float32), torch.bfloat16)
    out, ws, status = torch.full_like(q, float("nan")), _workspace(nf, 8, 1, 128), _status()
    _attend(nf, c, q, out, ws, status)
    torch.cuda.synchronize()
    assert int(status) == nf.NF_ERR_DEVICE_BOUNDS
    nan = torch.isnan(out).cpu().numpy()
    assert nan[1, :, 32:64].all() and nan.sum() == 8 * 32
    c.indices = clean
    K, V = (x[0, np.r_[0:32, 48:70]] for x in c.keys(0))
    keep = lambda r: (K[None], V[None])  # noqa: E731
    c.keys = keep
    _check(c, q, out, rows=[0])


@pytest.mark.parametrize("lens,nq,nkv,d", [([1, 5, 64], 8, 2, 128), ([900], 3, 1, 64), ([200] * 30, 16, 8, 128)], ids=str)
@pytest.mark.parametrize("down", [9, 11, 12, 14, 20, 30, 45, 70])
def test_columns_of_small_q_meet_large_k(nf, lens, nq, nkv, d, down):
    """q's columns of one group are 2^-down of the others, K's 2^down of theirs: they make the scores alike. One row of
    q has zeros there, one nothing but them."""
    rng = np.random.default_rng(down + len(lens))
    c = Cache(lens, nkv, d, seed=down)
    at = d // 32 - 1
    bits = _scales(c, 0).copy()
    f = ref.from_bits(bits)
    half = down // 2
    f = np.where(np.isnan(f), f, f * 2.0 ** np.where(np.arange(d // 32) == at, half, half - down))
    _put(c, 0, ref.to_bits(f))
    c.upload()
    q = rng.standard_normal((len(lens), nq, d)) * 2.0 ** (down - half)
    q[..., 32 * at:] *= 2.0 ** -down
    q[0, 0, 32 * at:] = 0.0
    q[0, -1, :32 * at] = 0.0
    q = _dev(q.astype(np.float32), torch.bfloat16)
    out = _run(nf, c, q)
    _check(c, q, out, rows=range(min(len(lens), 5)))
    _run(nf, c, q, sm=2)


@pytest.mark.parametrize("lens,nq,nkv", [([40, 900, 7], 8, 2), ([60] * 40, 24, 8)], ids=str)
def test_outliers_in_place_and_called_again(nf, lens, nq, nkv):
    """The output over q, call after call with one workspace, gives the same bits; the workspace's counters are at 0 again."""
    d = 128
    c = Cache(lens, nkv, d, seed=31)
    q = np.random.default_rng(6).standard_normal((len(lens), nq, d))
    q[..., 0] = 4.0
    for r in range(0, len(lens), 2):
        for head in range(nkv):
            _biased(c, q, [(r, 3)], 70, head)
            _set_key(c, r, 3, 1, head, [2.0 ** 30] * 4)
    c.upload()
    q = _dev(q.astype(np.float32), torch.bfloat16)
    want = _run(nf, c, q)
    _check(c, q, want, rows=range(min(len(lens), 6)))
    ws, status = _workspace(nf, nq, nkv, d), _status()
    for _ in range(3):
        both = q.clone()
        _attend(nf, c, both, both, ws, status)
        torch.cuda.synchronize()
        assert torch.equal(both, want) and int(status) == 0
        assert (ws.view(torch.int32)[:2 * 16 * 160] == 0).all()


@pytest.mark.parametrize("value", [math.nan, math.inf, 3e38])
def test_one_head_of_q_that_is_no_ordinary_row(nf, value):
    """NaN, an infinity or the largest numbers in one head's q: the other heads are as ever."""
    c = Cache([300, 20], 2, 128, seed=41)
    q = _dev(np.random.default_rng(7).standard_normal((2, 10, 128)).astype(np.float32), torch.bfloat16)
    want = _run(nf, c, q)
    odd = q.clone()
    odd[:, 7, 40] = value
    out = _run(nf, c, odd)
    others = [h for h in range(10) if h != 7]
    keep = q.clone()
    keep[:, 7] = 0
    _check(c, keep, torch.where(torch.arange(10, device="cuda").view(1, 10, 1) == 7, _run(nf, c, keep), out))
    assert torch.equal(out[:, :5], want[:, :5])     # another KV head: the same bits
    assert out[:, others].isfinite().all() and (math.isfinite(value) or out[:, 7].isnan().all())
