"""Refusals of the dense operators without a GPU: every argument that
include/moe.h rules out returns its code on the host, before any CUDA call
(the addresses here are never dereferenced)."""
import pytest

import expert_routing_grouped_gb300 as moe

A = 1 << 20   # an aligned address; areas 64 MB apart do not overlap
AREA = 1 << 26


def addr(i):
    return A + i * AREA


def norm(**kw):
    d = dict(x=addr(0), resid=addr(1), resid_out=addr(2), gain=addr(3), T=4, H=512, eps=1e-6,
             x_dtype=1, resid_dtype=0, out_dtype=2, group=0, out=addr(4), scale=addr(5), xs=0,
             rs=0, ros=0, os=0)
    d.update(kw)
    return moe.lib.moe_add_rmsnorm(d["x"], d["resid"], d["resid_out"], d["gain"], d["T"], d["H"],
                                   d["eps"], d["x_dtype"], d["resid_dtype"], d["out_dtype"],
                                   d["group"], d["out"], d["scale"], d["xs"], d["rs"], d["ros"],
                                   d["os"], None)


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(H=0), dict(H=4), dict(H=520), dict(H=32768 + 16), dict(eps=-1e-6),
    dict(eps=float("nan")), dict(x_dtype=2), dict(x_dtype=-1), dict(resid_dtype=2),
    dict(out_dtype=0), dict(out_dtype=3), dict(group=16), dict(group=256), dict(group=-32),
    dict(H=544, group=64), dict(out_dtype=1, group=32), dict(x=None), dict(out=None),
    dict(scale=None), dict(resid=None), dict(resid_out=None), dict(x=addr(0) + 8),
    dict(resid=addr(1) + 4), dict(resid_out=addr(2) + 4), dict(gain=addr(3) + 4),
    dict(out=addr(4) + 8), dict(scale=addr(5) + 2), dict(xs=511), dict(xs=516), dict(rs=514),
    dict(ros=510), dict(os=520), dict(xs=-512),
    dict(out=addr(0)), dict(out=addr(1) + 64), dict(out=addr(2)), dict(out=addr(3) + 16),
    dict(scale=addr(0)), dict(scale=addr(1)), dict(scale=addr(2)), dict(scale=addr(3)),
    dict(scale=addr(4)), dict(resid_out=addr(1) + 64), dict(resid_out=addr(1), ros=1024),
    dict(resid_out=addr(0)), dict(resid_out=addr(3)),
])
def test_add_rmsnorm_refuses(kw):
    assert norm(**kw) == moe.MOE_ERR_ARG


def test_add_rmsnorm_dry_run():
    assert norm(T=0, x=None, resid=None, resid_out=None, gain=None, out=None, scale=None) == 0
    assert norm(T=0, group=48) == moe.MOE_ERR_ARG


def linear(**kw):
    d = dict(x=addr(0), xsc=None, w=addr(1), wsc=None, bias=addr(2), resid=addr(3), out=addr(4),
             T=4, N=100, K=512, dtype=1, out_dtype=0, act=0, xs=0, ws=0, rs=0, os=0,
             status=addr(5))
    d.update(kw)
    return moe.lib.moe_linear(d["x"], d["xsc"], d["w"], d["wsc"], d["bias"], d["resid"], d["out"],
                              d["T"], d["N"], d["K"], d["dtype"], d["out_dtype"], d["act"],
                              d["xs"], d["ws"], d["rs"], d["os"], d["status"], None)


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(T=(1 << 19) + 1), dict(N=0), dict(N=(1 << 19) + 1), dict(K=0), dict(K=4),
    dict(K=516), dict(K=(1 << 19) + 8), dict(dtype=0), dict(dtype=3), dict(out_dtype=2),
    dict(act=-1), dict(act=4), dict(act=3), dict(act=3, N=104), dict(x=None), dict(w=None),
    dict(out=None), dict(xsc=addr(6)), dict(wsc=addr(6)), dict(dtype=2),
    dict(dtype=2, xsc=addr(6)), dict(dtype=2, wsc=addr(6)),
    dict(dtype=2, K=520, xsc=addr(6), wsc=addr(7)), dict(x=addr(0) + 8), dict(w=addr(1) + 2),
    dict(bias=addr(2) + 2), dict(out=addr(4) + 2), dict(resid=addr(3) + 1),
    dict(status=addr(5) + 2), dict(dtype=2, xsc=addr(6) + 1, wsc=addr(7)), dict(xs=504),
    dict(xs=516), dict(ws=516), dict(ws=-512), dict(rs=99), dict(os=64), dict(out=addr(0) + 64),
    dict(out=addr(1)), dict(out=addr(2)), dict(out=addr(5) - 4),
    dict(resid=addr(4) + 4), dict(resid=addr(4), rs=200),
    dict(dtype=2, xsc=addr(4), wsc=addr(7)), dict(dtype=2, xsc=addr(6), wsc=addr(4) + 16),
])
def test_linear_refuses(kw):
    assert linear(**kw) == moe.MOE_ERR_ARG


def test_linear_dry_run():
    assert linear(T=0, x=None, w=None, out=None, bias=None, resid=None) == 0
    assert linear(T=0, K=12) == moe.MOE_ERR_ARG


def balance(**kw):
    d = dict(z=addr(0), bias=addr(1), idx=addr(2), mask=addr(3), off=addr(4), T=64, E=16, k=2,
             S=3, z_dtype=0, mode=0, alpha=0.01, grad=addr(5), zs=0, loss=addr(6),
             counts=addr(7), tokens=addr(8), prob=addr(9), dz=addr(10), dzs=0, ws=addr(11),
             nb=1 << 20)
    d.update(kw)
    return moe.lib.moe_balance_loss(d["z"], d["bias"], d["idx"], d["mask"], d["off"], d["T"],
                                    d["E"], d["k"], d["S"], d["z_dtype"], d["mode"], d["alpha"],
                                    d["grad"], d["zs"], d["loss"], d["counts"], d["tokens"],
                                    d["prob"], d["dz"], d["dzs"], d["ws"], d["nb"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(E=0), -2), (dict(E=1025), -2), (dict(k=0), -2), (dict(k=17), -2),
    (dict(E=64, k=33), -2), (dict(mode=3), -2), (dict(mode=-1), -2), (dict(T=-1), -4),
    (dict(S=0), -4), (dict(S=65536), -4), (dict(off=None), -4), (dict(z_dtype=2), -4),
    (dict(alpha=float("inf")), -4), (dict(alpha=float("nan")), -4),
    (dict(T=1 << 25, k=4, nb=1 << 40), -4), (dict(zs=15), -4), (dict(dzs=8), -4),
    (dict(zs=-16), -4), (dict(loss=None), -4), (dict(counts=None), -4), (dict(tokens=None), -4),
    (dict(prob=None), -4), (dict(z=None), -4), (dict(idx=None), -4), (dict(ws=None), -4),
    (dict(nb=16), -1), (dict(z=addr(0) + 2), -4), (dict(z=addr(0) + 1, z_dtype=1), -4),
    (dict(dz=addr(10) + 2), -4), (dict(bias=addr(1) + 1), -4), (dict(idx=addr(2) + 2), -4),
    (dict(off=addr(4) + 2), -4), (dict(grad=addr(5) + 2), -4), (dict(loss=addr(6) + 2), -4),
    (dict(ws=addr(11) + 2), -4), (dict(dz=addr(0) + 64), -4), (dict(dz=addr(0), dzs=32), -4),
    (dict(ws=addr(0)), -4), (dict(ws=addr(10) + 128), -4), (dict(ws=addr(7)), -4),
    (dict(loss=addr(0)), -4), (dict(prob=addr(10)), -4), (dict(counts=addr(2)), -4),
    (dict(tokens=addr(7)), -4), (dict(prob=addr(7)), -4), (dict(dz=addr(2)), -4),
    (dict(dz=addr(3)), -4), (dict(loss=addr(5)), -4), (dict(counts=addr(4)), -4),
])
def test_balance_refuses(kw, code):
    assert balance(**kw) == code


def test_balance_workspace_sizes():
    ws = moe.balance_workspace
    assert ws(0, 8, 1) == 0 and ws(4, 0, 1) == 0 and ws(4, 1025, 1) == 0 and ws(4, 8, 0) == 0
    assert 0 < ws(1, 8, 1) <= ws(64, 8, 1) <= ws(1 << 20, 8, 1)
    # bounded whatever T: at most 456 runs of tokens, and one for each segment
    assert ws(1 << 25, 1024, 64) <= (456 + 64) * (2 * 1024 + 4) * 4
    assert balance(nb=ws(64, 16, 3) - 1) == moe.MOE_ERR_NOMEM


def test_balance_dry_run():
    assert balance(T=0, z=None, idx=None, loss=None, ws=None, nb=0) == 0
    assert balance(T=0, mode=5) == moe.MOE_ERR_ROUTING


def test_columns_of_one_tensor_that_meet():
    """Column slices of one wider tensor (one row stride) may be apart; these
    are not: a row further, or a byte into the neighbour's columns.  (Slices
    that are apart are accepted: the GPU tests use them.)"""
    base, H, wide = addr(0), 512, 4 * 512
    cols = dict(x=base, resid=base + H * 4, resid_out=base + 2 * H * 4, x_dtype=0, xs=wide, rs=wide,
                ros=wide, os=4 * wide)
    assert norm(out=base + wide * 4, **cols) == moe.MOE_ERR_ARG
    assert norm(out=base + 4 * wide - 496, **cols) == moe.MOE_ERR_ARG
    assert linear(x=base, out=base + 512 * 2, resid=base + 512 * 2 + 200, xs=2048, os=1024, rs=1024,
                  bias=None) == moe.MOE_ERR_ARG
    assert linear(x=base, out=base + 1000, xs=2048, os=1024, resid=None, bias=None) == moe.MOE_ERR_ARG
    assert balance(z=base, dz=base + 60, zs=64, dzs=64) == moe.MOE_ERR_ARG
