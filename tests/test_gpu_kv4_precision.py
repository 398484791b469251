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
