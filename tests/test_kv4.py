"""Operators around the 4-bit KV cache, host side: refusals, frequencies, the layout's formulas. CPU only.

The pointers below are never followed: every call is refused, by its arguments or (without a device, or
with a pointer that no device owns) before a launch.
"""
import math

import numpy as np
import pytest
import torch

import intra_device_overlapped_b200 as nf
import kv4_reference as ref

P = 4096  # an aligned address that is nobody's memory


def _rope(**kw):
    a = dict(q=P, qs=512, qo=P * 2, qos=512, nq=4, k=P * 3, ks=256, ko=P * 4, kos=256, nkv=2, idt=0, odt=0, pos=P * 5,
             T=3, d=128, rot=128, inter=0, freq=P * 6, scale=1.0)
    a.update(kw)
    return nf.nf_op_rope(a["q"], a["qs"], a["qo"], a["qos"], a["nq"], a["k"], a["ks"], a["ko"], a["kos"], a["nkv"],
                         a["idt"], a["odt"], a["pos"], a["T"], a["d"], a["rot"], a["inter"], a["freq"], a["scale"])


def _append(read=False, **kw):
    a = dict(k=P, ks=256, v=P * 2, vs=256, dt=0, vdt=0, slots=P * 3, T=3, pool=P * 4, pages=5, nkv=2, d=128, status=P * 5)
    a.update(kw)
    if read:
        return nf.nf_op_kv4_read(a["pool"], a["pages"], a["slots"], a["T"], a["nkv"], a["d"], a["k"], a["ks"], a["v"],
                                 a["vs"], a["dt"], a["status"])
    return nf.nf_op_kv4_append(a["k"], a["ks"], a["dt"], a["v"], a["vs"], a["vdt"], a["slots"], a["T"], a["pool"],
                               a["pages"], a["nkv"], a["d"], a["status"])


def _attn(**kw):
    a = dict(q=P, qs=1024, out=P * 2, os=1024, pool=P * 3, pages=5, kv=P * 4, ip=P * 5, ix=P * 6, R=3, nq=8, nkv=2,
             d=128, scale=0.0, ws=P * 7, size=None, status=P * 8, sm=0)
    a.update(kw)
    size = nf.nf_kv4_workspace_bytes(8, 2, 128) if a["size"] is None else a["size"]
    return nf.nf_op_kv4_decode_attention(a["q"], a["qs"], a["out"], a["os"], a["pool"], a["pages"], a["kv"], a["ip"],
                                         a["ix"], a["R"], a["nq"], a["nkv"], a["d"], a["scale"], a["ws"], size,
                                         a["status"], a["sm"])


def _map(**kw):
    a = dict(ctx=P, new=0, R=3, table=P * 2, stride=8, free=P * 3, cap=9, count=P * 4, pages=50, kv=P * 5, ip=P * 6,
             ix=P * 7, pcap=30, slots=P * 8, pos=P * 9, tcap=30, left=P * 10, status=P * 11)
    a.update(kw)
    return nf.nf_op_page_map(a["ctx"], a["new"], a["R"], a["table"], a["stride"], a["free"], a["cap"], a["count"],
                             a["pages"], a["kv"], a["ip"], a["ix"], a["pcap"], a["slots"], a["pos"], a["tcap"],
                             a["left"], a["status"])


BAD, UNSUP = nf.NF_ERR_INVALID_ARGUMENT, nf.NF_ERR_UNSUPPORTED


@pytest.mark.parametrize("call", [_rope, _append, lambda: _append(True), _attn, _map])
def test_memory_of_no_device_is_refused(call):
    assert call() == (BAD if torch.cuda.is_available() else nf.NF_ERR_CUDA)


@pytest.mark.parametrize("kw,want", [
    (dict(q=0), BAD), (dict(qo=0), BAD), (dict(k=0), BAD), (dict(ko=0), BAD), (dict(pos=0), BAD), (dict(freq=0), BAD),
    (dict(T=-1), BAD), (dict(nq=-1), BAD), (dict(nkv=-1), BAD), (dict(d=127), BAD), (dict(rot=63), BAD),
    (dict(rot=0), BAD), (dict(rot=130), BAD), (dict(inter=2), BAD), (dict(idt=2), BAD), (dict(odt=-1), BAD),
    (dict(qs=511), BAD), (dict(kos=255), BAD), (dict(q=P + 1), BAD), (dict(ko=P * 4 + 2, odt=1), BAD),
    (dict(pos=P * 5 + 2), BAD), (dict(freq=P * 6 + 4), BAD), (dict(scale=math.nan), BAD),
    (dict(qo=P, qos=520), BAD), (dict(ko=P * 3, odt=1), BAD),
    (dict(d=514, rot=2, qs=4096, qos=4096, ks=4096, kos=4096), UNSUP), (dict(T=0), 0),
    (dict(nq=0, nkv=0, q=0, k=0, qo=0, ko=0), 0)])
def test_rope_refusals(kw, want):
    assert _rope(**kw) == want


@pytest.mark.parametrize("read", [False, True])
@pytest.mark.parametrize("kw,want", [
    (dict(k=0), BAD), (dict(v=0), BAD), (dict(slots=0), BAD), (dict(pool=0), BAD), (dict(status=0), BAD),
    (dict(T=-1), BAD), (dict(pages=0), BAD), (dict(pages=nf.NF_KV4_MAX_PAGES + 1), BAD), (dict(dt=2, vdt=2), BAD),
    (dict(nkv=0), BAD), (dict(d=0), BAD), (dict(d=96), UNSUP), (dict(nkv=257, ks=1 << 20, vs=1 << 20), UNSUP),
    (dict(ks=252), BAD), (dict(vs=258), BAD), (dict(k=P + 4), BAD), (dict(v=P + 8, dt=1, vdt=1), BAD), (dict(pool=P + 8), BAD),
    (dict(ks=260), BAD), (dict(slots=P * 3 + 2), BAD), (dict(status=P * 5 + 1), BAD), (dict(T=1 << 30), BAD),
    (dict(T=0), 0)])
def test_row_refusals(read, kw, want):
    assert _append(read, **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(q=0), BAD), (dict(out=0), BAD), (dict(pool=0), BAD), (dict(kv=0), BAD), (dict(ip=0), BAD), (dict(ix=0), BAD),
    (dict(ws=0), BAD), (dict(status=0), BAD), (dict(pages=0), BAD), (dict(R=-1), BAD),
    (dict(R=nf.NF_KV4_MAX_REQUESTS + 1), BAD), (dict(nq=0), BAD), (dict(nq=9), BAD), (dict(nkv=0), BAD),
    (dict(d=96), UNSUP), (dict(nq=18, qs=4096, os=4096), UNSUP), (dict(scale=-1.0), BAD), (dict(scale=math.nan), BAD),
    (dict(scale=math.inf), BAD), (dict(out=P, os=1032), BAD), (dict(scale=3e38), BAD), (dict(pages=(1 << 30) + 1, nkv=2), BAD),
    (dict(pages=1 << 26, nkv=32, nq=32, qs=4096, os=4096, size=1 << 30), BAD), (dict(kv=P * 4 + 1), BAD),
    (dict(ip=P * 5 + 2), BAD), (dict(ix=P * 6 + 2), BAD), (dict(status=P * 8 + 2), BAD),
    (dict(qs=1016), BAD), (dict(os=1028), BAD), (dict(q=P + 8), BAD),
    (dict(out=P * 2 + 8), BAD), (dict(pool=P * 3 + 8), BAD), (dict(ws=P * 7 + 128), BAD), (dict(size=16), BAD),
    (dict(sm=-1), BAD), (dict(R=0), 0)])
def test_attention_refusals(kw, want):
    assert _attn(**kw) == want


@pytest.mark.parametrize("kw", [
    dict(ctx=0), dict(table=0), dict(free=0), dict(count=0), dict(kv=0), dict(ip=0), dict(ix=0), dict(slots=0),
    dict(pos=0), dict(left=0), dict(status=0), dict(R=-1), dict(R=nf.NF_KV4_MAX_REQUESTS + 1), dict(stride=0),
    dict(cap=-1), dict(pcap=-1), dict(tcap=-1), dict(pages=0), dict(pages=nf.NF_KV4_MAX_PAGES + 1),
    dict(left=P * 4),
    # arrays that are written and overlap others
    dict(kv=P), dict(kv=P + 8), dict(new=P * 5), dict(ip=P * 3 + 32), dict(slots=P * 9 - 4), dict(pos=P * 8 + 116),
    dict(table=P * 3 - 92), dict(left=P * 5 + 8), dict(left=P * 7 + 116), dict(kv=P * 6 + 12), dict(ix=P * 8 - 116),
    # not aligned to their elements
    dict(ctx=P + 1), dict(new=P * 12 + 2), dict(table=P * 2 + 2), dict(count=P * 4 + 3), dict(slots=P * 8 + 2)])
def test_page_map_refusals(kw):
    assert _map(**kw) == BAD


def test_page_map_arrays_next_to_one_another_are_taken():
    assert _map(kv=P + 12, left=P * 9 - 4, table=P * 3 - 96) == (BAD if torch.cuda.is_available() else nf.NF_ERR_CUDA)


def test_sizes():
    assert nf.nf_kv4_page_bytes(8, 128) == 8 * 2 * 9 * 128
    assert nf.nf_kv4_page_bytes(1, 64) == 2 * 9 * 64
    assert nf.nf_kv4_page_bytes(0, 64) == -BAD and nf.nf_kv4_page_bytes(2, 80) == -UNSUP
    assert nf.nf_kv4_workspace_bytes(32, 8, 128) > 0
    assert nf.nf_kv4_workspace_bytes(33, 8, 128) == -BAD and nf.nf_kv4_workspace_bytes(72, 8, 128) == -UNSUP


@pytest.mark.parametrize("d", [64, 128])
def test_every_code_has_a_place_of_its_own(d):
    for which in (0, 1):
        at = {ref.place(which, s, c, d) for s in range(16) for c in range(d)}
        assert len(at) == 16 * d and all(0 <= b < 8 * d for b, _ in at)
        owner = {}
        for s in range(16):
            for c in range(d):
                assert owner.setdefault(ref.place(which, s, c, d)[0], s) == s  # no byte of two slots


def _freq(**kw):
    c = dict(theta=10000.0, rot_dim=128, scaling=0, factor=1.0, low=1.0, high=4.0, original_positions=8192)
    c.update(kw)
    return nf.nf_rope_frequencies(nf.nf_rope_config(**c))


def _plain(theta, rot):
    return np.array([theta ** (-2.0 * i / rot) for i in range(rot // 2)])


# The host forms each frequency with a pow (under 1 ulp, 2^-52) and at most five more roundings, the reference
# likewise: 16 * 2^-53 covers both.
REL = 16 * 2.0 ** -53


@pytest.mark.parametrize("rot", [2, 64, 128, 80])
def test_plain_and_linear_frequencies(rot):
    st, f, m = _freq(rot_dim=rot)
    assert st == 0 and m == 1.0
    np.testing.assert_allclose(f, _plain(10000.0, rot), rtol=REL)
    st, g, m = _freq(rot_dim=rot, scaling=nf.NF_ROPE_LINEAR, factor=4.0)
    assert st == 0 and m == 1.0
    np.testing.assert_allclose(g, np.array(f) / 4.0, rtol=REL)


def test_ntk_keeps_the_first_wave_and_stretches_the_last():
    _, f, _ = _freq()
    st, g, m = _freq(scaling=nf.NF_ROPE_NTK, factor=8.0)
    assert st == 0 and m == 1.0 and g[0] == f[0] == 1.0
    assert math.isclose(g[-1], f[-1] / 8.0, rel_tol=1e-12)  # theta' = theta * 8^(128/126): its 126/128-th power
    assert all(g[i] / f[i] >= g[i + 1] / f[i + 1] for i in range(63))


def test_wavelength_bands():
    f = _plain(500000.0, 128)
    st, g, m = _freq(theta=500000.0, scaling=nf.NF_ROPE_WAVELENGTH, factor=8.0)
    assert st == 0 and m == 1.0
    seen = set()
    for a, b in zip(f, g):
        turns = 8192 * a / (2 * math.pi)
        if turns >= 4.0:
            want, band = a, "kept"
        elif turns <= 1.0:
            want, band = a / 8.0, "stretched"
        else:
            k = (turns - 1.0) / 3.0
            want, band = (1 - k) * a / 8.0 + k * a, "between"
        seen.add(band)
        assert math.isclose(b, want, rel_tol=4 * REL)  # k cancels up to two bits more
    assert seen == {"kept", "stretched", "between"}


def test_yarn_bands_and_factor():
    rot, theta, span = 128, 10000.0, 4096
    f = _plain(theta, rot)
    st, g, m = _freq(scaling=nf.NF_ROPE_YARN, factor=16.0, low=1.0, high=32.0, original_positions=span)
    assert st == 0 and m == np.float32(0.1 * math.log(16.0) + 1.0)
    index = lambda turns: rot * math.log(span / (turns * 2 * math.pi)) / (2 * math.log(theta))  # noqa: E731
    first, last = math.floor(index(32.0)), math.ceil(index(1.0))
    assert 0 < first < last < rot // 2
    for i in range(rot // 2):
        k = min(max((i - first) / (last - first), 0.0), 1.0)
        assert math.isclose(g[i], k * f[i] / 16.0 + (1 - k) * f[i], rel_tol=REL)
    assert g[first] == f[first] and math.isclose(g[last], f[last] / 16.0, rel_tol=REL)


@pytest.mark.parametrize("kw", [
    dict(rot_dim=3), dict(rot_dim=0), dict(rot_dim=514), dict(theta=0.0), dict(theta=math.inf), dict(scaling=5),
    dict(scaling=1, factor=0.5), dict(scaling=1, factor=math.nan), dict(scaling=2, rot_dim=2, factor=2.0),
    dict(scaling=3, factor=2.0, original_positions=0), dict(scaling=3, factor=2.0, low=4.0),
    dict(scaling=4, factor=2.0, low=0.0), dict(scaling=4, factor=2.0, theta=1.0), dict(scaling=4, factor=2.0, high=math.inf)])
def test_frequency_refusals(kw):
    assert _freq(**kw)[0] == BAD


def test_config_struct_matches_the_header(tmp_path):
    import test_abi_layout
    import ctypes
    names = test_abi_layout.STRUCTS
    try:
        test_abi_layout.STRUCTS = ["nf_rope_config"]
        c = test_abi_layout.c_layout(tmp_path)
    finally:
        test_abi_layout.STRUCTS = names
    assert ctypes.sizeof(nf.nf_rope_config) == c["nf_rope_config"]
    for field, _ in nf.nf_rope_config._fields_:
        assert getattr(nf.nf_rope_config, field).offset == c[f"nf_rope_config.{field}"]
