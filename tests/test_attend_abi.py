"""Refusals of the attention block's operators without a GPU: every argument that
include/moe.h rules out returns its code on the host, before any CUDA call
(the addresses here are never dereferenced), and the host's frequency tables."""
import ctypes
import math

import numpy as np
import pytest

import expert_routing_grouped_gb300 as moe

A = 1 << 20
AREA = 1 << 26
INF, NAN = float("inf"), float("nan")


def addr(i):
    return A + i * AREA


def rope(**kw):
    d = dict(x=addr(0), pos=addr(1), freqs=addr(2), T=4, heads=5, D=128, R=128, il=0, inv=0, m=1.0,
             dt=1, out=addr(3), xs=0, xhs=0, os=0, ohs=0)
    d.update(kw)
    return moe.lib.moe_rope(d["x"], d["pos"], d["freqs"], d["T"], d["heads"], d["D"], d["R"], d["il"],
                            d["inv"], d["m"], d["dt"], d["out"], d["xs"], d["xhs"], d["os"], d["ohs"],
                            None)


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(T=(1 << 24) + 1), dict(heads=0), dict(D=0), dict(D=1025, R=2), dict(R=0), dict(R=-2),
    dict(R=63), dict(R=130), dict(heads=1 << 14), dict(m=NAN), dict(m=INF), dict(dt=2), dict(dt=-1),
    dict(x=None), dict(pos=None), dict(freqs=None), dict(out=None), dict(x=addr(0) + 1),
    dict(out=addr(3) + 1), dict(dt=0, x=addr(0) + 2), dict(pos=addr(1) + 2), dict(freqs=addr(2) + 4),
    dict(xs=639), dict(xhs=127), dict(os=639), dict(ohs=64), dict(xs=-640), dict(xs=(1 << 32) + 1),
    dict(xhs=130, xs=640), dict(xs=128, xhs=384), dict(out=addr(0) + 64), dict(out=addr(0), os=648),
    dict(out=addr(1)), dict(out=addr(2) - 8), dict(out=addr(0) + 128),
])
def test_rope_refuses(kw):
    assert rope(**kw) == moe.MOE_ERR_ARG


def test_rope_dry_run():
    assert rope(T=0, x=None, pos=None, freqs=None, out=None) == moe.MOE_OK
    assert rope(T=0, R=3) == moe.MOE_ERR_ARG


@pytest.mark.parametrize("args", [
    (0, 1e4, 0, 1.0, 0, 32, 1), (7, 1e4, 0, 1.0, 0, 32, 1), (1026, 1e4, 0, 1.0, 0, 32, 1),
    (64, 0.5, 0, 1.0, 0, 32, 1), (64, NAN, 0, 1.0, 0, 32, 1), (64, INF, 0, 1.0, 0, 32, 1),
    (64, 1e4, 4, 1.0, 0, 32, 1), (64, 1e4, -1, 1.0, 0, 32, 1), (64, 1e4, 1, 0.5, 0, 32, 1),
    (64, 1e4, 1, NAN, 0, 32, 1), (2, 1e4, 2, 4.0, 0, 32, 1), (64, 1e4, 3, 4.0, 0, 32, 1),
    (64, 1e4, 3, 4.0, 4096, 1, 1), (64, 1e4, 3, 4.0, 4096, 32, -1), (64, 1e4, 3, 4.0, NAN, 32, 1),
    (64, 1e4, 3, 4.0, 4096, INF, 1),
])
def test_rope_freqs_refuses(args):
    buf = (ctypes.c_double * 1024)()
    assert moe.lib.moe_rope_freqs(*args, buf, None) == moe.MOE_ERR_ARG
    assert moe.lib.moe_rope_freqs(64, 1e4, 0, 1.0, 0, 32, 1, None, None) == moe.MOE_ERR_ARG


@pytest.mark.parametrize("rot", [2, 10, 64, 128, 1024])
def test_rope_freqs_values(rot):
    """Against the formulas; a few units of f64 each."""
    i = np.arange(rot // 2)
    f, m = moe.rope_freqs(rot, 1e6)
    assert m == 1 and np.allclose(f, 1e6 ** (-2.0 * i / rot), rtol=1e-14, atol=0)
    f, m = moe.rope_freqs(rot, 1e6, moe.ROPE_LINEAR, 8.0)
    assert m == 1 and np.allclose(f, 1e6 ** (-2.0 * i / rot) / 8, rtol=1e-14, atol=0)
    f, m = moe.rope_freqs(rot, 1e4, moe.ROPE_PARTS, 16.0, 4096, 32, 1)
    assert m == np.float32(0.1 * math.log(16.0) + 1)
    for j in i:
        g = 1e4 ** (-2.0 * j / rot)
        turns = 4096 * g / (2 * math.pi)
        keep = 1.0 if turns >= 32 else 0.0 if turns <= 1 else (turns - 1) / 31
        assert math.isclose(f[j], g * keep + g / 16 * (1 - keep), rel_tol=1e-13)
    if rot > 2:   # by base: the first pair as it was, the last one slowed by the factor
        f, m = moe.rope_freqs(rot, 1e4, moe.ROPE_BASE, 4.0)
        assert f[0] == 1 and math.isclose(f[-1], 1e4 ** (-(rot - 2.0) / rot) / 4, rel_tol=1e-13)


def append(**kw):
    d = dict(k=addr(0), v=addr(1), cache=addr(2), pages=addr(3), off=addr(4), len=addr(5), T=6, S=3,
             Hkv=2, D=128, P=16, np=8, mp=4, dt=1, ks=0, vs=0)
    d.update(kw)
    return moe.lib.moe_kv4_append(d["k"], d["v"], d["cache"], d["pages"], d["off"], d["len"], d["T"], d["S"],
                                  d["Hkv"], d["D"], d["P"], d["np"], d["mp"], d["dt"], d["ks"], d["vs"],
                                  None)


BATCH = [dict(T=-1), dict(S=0), dict(S=65536), dict(Hkv=0), dict(Hkv=1025), dict(D=96), dict(D=0), dict(P=8),
         dict(P=48), dict(P=512), dict(P=0), dict(np=0), dict(mp=0), dict(mp=(1 << 26) + 1), dict(off=None),
         dict(pages=None), dict(len=None), dict(cache=None), dict(cache=addr(2) + 8),
         dict(pages=addr(3) + 2), dict(off=addr(4) + 1), dict(len=addr(5) + 2)]


@pytest.mark.parametrize("kw", BATCH + [
    dict(T=(1 << 24) + 1), dict(T=1 << 24, Hkv=32), dict(dt=2), dict(k=None), dict(v=None),
    dict(k=addr(0) + 8), dict(v=addr(1) + 2), dict(ks=255), dict(ks=260), dict(vs=254), dict(vs=-256),
    dict(ks=(1 << 32) + 8), dict(dt=0, ks=258), dict(cache=addr(0)), dict(cache=addr(1) + 64),
    dict(cache=addr(3) - 1024), dict(cache=addr(4)), dict(cache=addr(5)),
])
def test_append_refuses(kw):
    assert append(**kw) == moe.MOE_ERR_ARG


def test_append_dry_run():
    assert append(T=0, k=None, v=None, cache=None, pages=None, len=None, off=None) == moe.MOE_OK
    assert append(T=0, D=80) == moe.MOE_ERR_ARG


def attention(**kw):
    d = dict(q=addr(0), cache=addr(2), pages=addr(3), off=addr(4), len=addr(5), T=6, S=3, mq=0, H=8,
             Hkv=2, D=128, P=16, np=8, mp=4, scale=0.1, cap=0.0, win=0, causal=1, out=addr(1), qs=0,
             os=0, ws=addr(6), nb=AREA, status=addr(8))
    d.update(kw)
    return moe.lib.moe_kv4_attention(d["q"], d["cache"], d["pages"], d["off"], d["len"], d["T"], d["S"],
                                     d["mq"], d["H"], d["Hkv"], d["D"], d["P"], d["np"], d["mp"],
                                     d["scale"], d["cap"], d["win"], d["causal"], d["out"], d["qs"],
                                     d["os"], d["ws"], d["nb"], d["status"], None)


@pytest.mark.parametrize("kw", BATCH + [
    dict(T=(1 << 19) + 1), dict(mq=-1), dict(H=0), dict(H=9), dict(H=1026), dict(scale=NAN),
    dict(scale=INF), dict(cap=-1.0), dict(cap=NAN), dict(cap=INF), dict(win=-1), dict(q=None),
    dict(out=None), dict(q=addr(0) + 8), dict(out=addr(1) + 2), dict(ws=addr(6) + 8),
    dict(status=addr(8) + 2), dict(qs=1023), dict(qs=1028), dict(os=512), dict(os=-1024),
    dict(os=(1 << 31) + 8), dict(out=addr(0)), dict(out=addr(0) + 64), dict(out=addr(2)),
    dict(out=addr(3)), dict(out=addr(4)), dict(out=addr(5)), dict(out=addr(8) - 16),
])
def test_attention_refuses(kw):
    assert attention(**kw) == moe.MOE_ERR_ARG


def test_attention_dry_run():
    assert attention(T=0, q=None, cache=None, pages=None, len=None, out=None, off=None, ws=None, nb=0) == 0
    assert attention(T=0, H=7) == moe.MOE_ERR_ARG


def test_attention_columns_that_meet():
    """Query and result as columns of one wider tensor: a byte into the neighbour's is refused."""
    assert attention(out=addr(0) + 2048 - 16, qs=4096, os=4096) == moe.MOE_ERR_ARG


def test_page_bytes():
    assert moe.kv4_page_bytes(16, 1, 64) == 16 * 72 and moe.kv4_page_bytes(64, 8, 128) == 64 * 8 * 144
    for bad in ((8, 1, 64), (16, 0, 64), (16, 1025, 64), (16, 1, 96), (0, 1, 64), (24, 1, 64)):
        assert moe.kv4_page_bytes(*bad) == 0


def test_workspace():
    """0 for sizes that the call refuses; a smaller one, none, or one that meets an
    operand is refused."""
    good = dict(T=6, n_seq=3, n_heads=8, n_kv_heads=2, head_dim=128, page_size=16, max_pages=4)
    assert moe.kv4_workspace(**good) == 0   # 64 tokens at most: nothing to cut
    good["max_pages"] = mp = 1024
    need = moe.kv4_workspace(**good)
    assert need > 0
    for bad in (dict(T=0), dict(T=-1), dict(T=(1 << 19) + 1), dict(n_seq=0), dict(n_heads=9), dict(n_heads=1026),
                dict(head_dim=96), dict(page_size=8), dict(max_pages=0), dict(max_pages=(1 << 26) + 1),
                dict(max_q=-1)):
        assert moe.kv4_workspace(**{**good, **bad}) == 0
    assert attention(mp=mp, nb=need - 1) == moe.MOE_ERR_NOMEM and attention(mp=mp, nb=0) == moe.MOE_ERR_NOMEM
    assert attention(mp=mp, ws=None, nb=0) == moe.MOE_ERR_ARG and attention(mp=mp, ws=None) == moe.MOE_ERR_ARG
    for i in (0, 1, 2, 3, 4, 5, 8):   # q, out, cache, pages, q_off, kv_len, status
        assert attention(mp=mp, ws=addr(i) - 16) == moe.MOE_ERR_ARG


@pytest.mark.parametrize("H,Hkv", [(8, 8), (96, 8), (40, 1)])
def test_workspace_is_enough_for_fewer(H, Hkv):
    """What T rows need is enough for a known max_q, and for as many single rows."""
    for T, S in ((1, 1), (64, 64), (300, 5), (4096, 1)):
        all_ = moe.kv4_workspace(T, S, H, Hkv, 128, 64, 2048)
        for mq in (1, 3, 16, 4096):
            assert moe.kv4_workspace(T, S, H, Hkv, 128, 64, 2048, max_q=mq) <= all_
