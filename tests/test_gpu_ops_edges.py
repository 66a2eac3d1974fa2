"""Edges of the dense operators on the GPU, against their 64-bit forms
(ops_ref.py): values at the ends of f32's range, masks beside gradients that
are not finite, sizes whose launches differ from the small ones', the accuracy
of f32 outputs, and products that give up.

Tolerances come from the arithmetic, as in test_gpu_ops.py, whose checks are
used here."""
import numpy as np
import pytest
import torch

import ops_ref as ref
from test_gpu_ops import (DT, E4M3, SENT, check_balance, check_linear, check_norm, gen,
                          make_balance, make_linear, randn, run_balance, run_linear, run_norm)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    import expert_routing_grouped_gb300 as m
    return m


# ------------------------------------------------------------ add_rmsnorm --

def four_squares(d):
    """Four whole numbers up to 256 whose squares add up to d."""
    for a in range(min(256, int(d ** 0.5)), -1, -1):
        for b in range(min(a, int((d - a * a) ** 0.5)), -1, -1):
            rest = d - a * a - b * b
            c = int(rest ** 0.5)
            while c >= 0 and 2 * c * c >= rest:
                e = int(round((rest - c * c) ** 0.5))
                if c <= 256 and e <= 256 and e * e == rest - c * c:
                    return a, b, c, e
                c -= 1
    raise AssertionError(d)


def whole_rows(T, H, seed):
    """Rows of whole numbers below 257 whose mean square is 64^2 exactly."""
    rs = np.random.RandomState(seed)
    rows = np.zeros((T, H))
    for t in range(T):
        while True:
            v = rs.randint(-109, 110, H - 4)
            d = H * 4096 - int((v * v).sum())
            if 0 <= d <= 200000:
                break
        rows[t] = np.concatenate([v, four_squares(d)])
    return torch.tensor(rows, dtype=torch.float32, device="cuda")


@pytest.mark.parametrize("group", [0, 32, 64, 128])
@pytest.mark.parametrize("with_gain", [False, True])
@pytest.mark.parametrize("dtype", [0, 1])
def test_add_rmsnorm_codes_are_the_rounded_quotients(moe, group, with_gain, dtype):
    """Where nothing before the quotient rounds (whole numbers, a root mean
    square of 64 and eps 0: 1 / rms is a power of two, and r * gain is rounded
    once whatever the order), the scale is f32(max |n| / 448) and every code is
    e4m3(f32(n / scale)) bit for bit -- at exact ties, which whole numbers meet
    often, too."""
    T, H = 400, 512
    x = whole_rows(T, H, 7 + group)
    gain = 1 + 0.2 * randn(gen(3), H) if with_gain else None
    out, scale, _ = run_norm(moe, x.to(DT[dtype]), None, gain, 2, group, eps=0.0)
    n = (x if gain is None else x * gain) / 64
    want = n.cpu().view(T, -1, group or H)
    sc = want.abs().amax(2) / 448.0
    assert torch.equal(scale.cpu().view(T, -1), sc)
    codes = (want / sc[:, :, None]).clamp(-448, 448).to(E4M3).view(T, H)
    assert torch.equal(out.cpu().view(torch.uint8), codes.view(torch.uint8))


# Rows of more than 4096 values in batches of 304 rows and more: at most 512
# threads a row, each with two, four or eight pieces.
@pytest.mark.parametrize("T,H", [(304, 4096 + 16), (310, 12288), (305, 20000), (304, 32768)])
@pytest.mark.parametrize("out_dtype,group", [(1, 0), (2, 0), (2, 32)])
def test_add_rmsnorm_many_long_rows(moe, T, H, out_dtype, group):
    if group:
        H = H // group * group
    g = gen(T + H)
    x = (3 * randn(g, T, H)).bfloat16()
    resid = 5 * randn(g, T, H)
    gain = 1 + 0.3 * randn(g, H)
    out, scale, rout = run_norm(moe, x, resid, gain, out_dtype, group)
    check_norm(x, resid, gain, out, scale, rout, out_dtype, group)


def wide(T, n, extra, dtype):
    """A whole buffer of T rows of n + extra values, all SENT, and its first n columns."""
    full = torch.full((T, n + extra), SENT, device="cuda").to(dtype)
    return full, full[:, :n]


@pytest.mark.parametrize("T", [1, 5])
@pytest.mark.parametrize("H", [192, 4096 + 32])
def test_padding_of_every_row_is_left_alone(moe, T, H):
    """Also behind the last row's end."""
    g = gen(T)
    for out_dtype, group in ((1, 0), (2, 0), (2, 32)):
        x, resid = randn(g, T, H).bfloat16(), randn(g, T, H)
        full, out = wide(T, H, 32, DT[out_dtype])
        rfull, rout = wide(T, H, 32, torch.float32)
        scale = torch.full((T * (H // (group or H)) + 8,), SENT, device="cuda")
        moe.add_rmsnorm(x, T, H, 1e-6, out, resid=resid, resid_out=rout,
                        scale=scale if out_dtype == 2 else None, group=group, out_dtype=out_dtype,
                        out_stride=H + 32, resid_out_stride=H + 32)
        assert bool((full[:, H:].float() == SENT).all()) and bool((rfull[:, H:] == SENT).all())
        assert bool((scale[T * (H // (group or H)):] == SENT).all())
    for rows in (T, 20 * T):   # few tokens, and the tensor-core form
        for out_dtype in (0, 1):
            x, w, sx, sw, b, r = make_linear(g, rows, 64, 37, 1, 0, out_dtype, False, False)
            full, out = wide(rows, 37, 3, DT[out_dtype])
            moe.linear(x, w, rows, 37, 64, out, out_dtype=out_dtype, out_stride=40)
            assert bool((full[:, 37:].float() == SENT).all())
    for E in (7, 64):
        z, idx, _, _ = make_balance(g, T, E, 2, 0)
        full, dz = wide(T, E, 4, torch.float32)
        f = dict(device="cuda")
        ws = torch.empty(moe.balance_workspace(T, E), dtype=torch.uint8, **f)
        moe.balance_loss(z, idx, T, E, 2, torch.empty(1, **f), torch.empty(1, E, dtype=torch.int32, **f),
                         torch.empty(1, dtype=torch.int32, **f), torch.empty(1, E, **f), ws, dz=dz,
                         dz_stride=E + 4)
        assert bool((full[:, E:] == SENT).all()) and bool((full[:, :E] != SENT).all())


# ------------------------------------------------------------------ linear --

# Relative error of a whole f32 result, |out - y| / |y| over all its elements.
# A truncating addition to an accumulator loses between nothing and one unit in
# the last place (2^-23) of the running sum, half of it on average.  A segment
# of K is at most 48 additions (of 16 bf16 products), in each factor of a SwiGLU
# 28; the additions of the segments, to nearest, are far below.  With operands of
# both signs a running sum averages 2/3 of its end: 48 * 2^-24 * 2/3 = 1.9e-6,
# SwiGLU 2 * 28 * 2^-24 * 2/3 = 2.2e-6 times the activation's slope of at most
# 1.13.  e4m3 products hold 8 significant bits and lose far less, so their longer
# segments meet the same bound.  One accumulator for all of K = 14336 would lose
# 896 * 2^-24 * 2/3 = 3.6e-5.
PLAIN_REL, SWIGLU_REL = 2e-6, 3e-6


def one_sign_rel(dtype, act):
    """Operands of one sign: every loss adds up, whole units at most, and a
    running sum averages half of its end.  e4m3 segments: 192 additions of 32
    products, which then hold more bits than the accumulator has left."""
    adds = 192 if dtype == 2 else 28 if act == 3 else 48
    return adds * 2.0 ** -23 / 2 * (2 * 1.13 if act == 3 else 1)


@pytest.mark.parametrize("one_sign", [False, True])
@pytest.mark.parametrize("dtype", [1, 2])
@pytest.mark.parametrize("T,K,N,act", [
    (1, 4096, 256, 0), (4, 14336, 512, 0), (9, 14336, 256, 3), (16, 131072, 64, 0), (3, 524288 - 256, 40, 0),
    (16, 262144, 16, 3), (24, 4096, 512, 0), (40, 14336, 256, 3), (130, 14336, 512, 0), (200, 131072, 64, 0),
    (64, 131072, 32, 3), (200, 524288, 64, 0), (700, 14336, 1024, 0), (1200, 6144, 1536, 3)])
def test_linear_f32_outputs_are_f32_sums(moe, T, K, N, act, dtype, one_sign):
    g = gen(T + N)
    x, w, sx, sw, b, r = make_linear(g, T, K, N, dtype, act, 0, False, False)
    if one_sign:
        x, w = x.float().abs().to(x.dtype), w.float().abs().to(w.dtype)
    out, st = run_linear(moe, x, w, sx, sw, None, None, N, dtype, 0, act)
    y, _ = ref.linear(x, w, N, act, sx, sw)
    rel = float((out.double() - y).norm() / y.norm())
    bound = one_sign_rel(dtype, act) if one_sign else SWIGLU_REL if act == 3 else PLAIN_REL
    assert int(st) == 0 and rel <= bound, rel


def test_linear_pairs_back_to_back(moe):
    """Products in the CTA-pair form one after another, between them kernels
    that take the same SMs: the same bits each time."""
    g = gen(31)
    T, K, N = 4096, 256, 2048
    x, w, _, _, _, _ = make_linear(g, T, K, N, 1, 0, 0, False, False)
    out, st = run_linear(moe, x, w, None, None, None, None, N, 1, 0, 0)
    check_linear(out, st, x, w, None, None, None, None, N, 0)
    few, _ = run_linear(moe, x[:40], w, None, None, None, None, N, 1, 0, 0)
    outs = [torch.empty_like(out) for _ in range(3)]
    small = torch.empty_like(few)
    norm = torch.empty(T, K, dtype=torch.bfloat16, device="cuda")
    for i in range(200):
        moe.linear(x, w, T, N, K, outs[i % 3])
        if i % 2:
            moe.linear(x[:40], w, 40, N, K, small)
        else:
            moe.add_rmsnorm(x, T, K, 1e-6, norm)
    for o in outs:
        assert torch.equal(o, out)
    assert torch.equal(small, few)


@pytest.mark.parametrize("T,K,N", [(40, 8192, 256), (1000, 2048, 320), (4096, 1024, 4096)])
def test_linear_wait_limit(moe, T, K, N):
    """The limit set through the call (split, one CTA per tile, CTA pairs): the
    product returns and its status word says 2; with the default back the next
    one is right, and a product of another thread never saw the limit."""
    import threading
    g = gen(T)
    x, w, _, _, _, _ = make_linear(g, T, K, N, 1, 0, 0, False, False)
    others = []
    moe.linear_wait_limit(0)
    try:
        for _ in range(20):   # also where the operands lie in L2
            out, status = run_linear(moe, x, w, None, None, None, None, N, 1, 0, 0)
            assert int(status) == 2
        t = threading.Thread(target=lambda: others.append(
            run_linear(moe, x, w, None, None, None, None, N, 1, 0, 0)))
        t.start()
        t.join()
    finally:
        moe.linear_wait_limit(2000000)
    for out, status in others + [run_linear(moe, x, w, None, None, None, None, N, 1, 0, 0)]:
        check_linear(out, status, x, w, None, None, None, None, N, 0)


@pytest.mark.parametrize("T,K,N", [(40, 8192, 256), (1000, 2048, 320), (4096, 1024, 4096)])
def test_linear_that_gave_up_without_a_status_word(moe, T, K, N):
    """The device's word says so, once; a status word of the caller's own keeps
    it out of there."""
    g = gen(T)
    x, w, _, _, _, _ = make_linear(g, T, K, N, 1, 0, 0, False, False)
    out = torch.empty(T, N, device="cuda")
    assert moe.linear_status() == 0
    moe.linear_wait_limit(0)
    try:
        moe.linear(x, w, T, N, K, out)
        assert moe.linear_status() == 2 and moe.linear_status() == 0
        _, status = run_linear(moe, x, w, None, None, None, None, N, 1, 0, 0)
        assert moe.linear_status() == 0 and int(status) == 2
    finally:
        moe.linear_wait_limit(2000000)
    moe.linear(x, w, T, N, K, out)
    assert moe.linear_status() == 0
    check_linear(out, torch.zeros(1), x, w, None, None, None, None, N, 0)


def test_linear_environment_does_not_reach_the_kernels(moe, monkeypatch):
    """MOE_LINEAR_NO_WAIT: not without a status word, and not where the process
    inherited it."""
    import os
    import subprocess
    import sys
    g = gen(3)
    T, K, N = 40, 4096, 256
    x, w, _, _, _, _ = make_linear(g, T, K, N, 1, 0, 0, False, False)
    want, status = run_linear(moe, x, w, None, None, None, None, N, 1, 0, 0)
    check_linear(want, status, x, w, None, None, None, None, N, 0)
    out = torch.zeros_like(want)
    monkeypatch.setenv("MOE_LINEAR_NO_WAIT", "1")
    moe.linear(x, w, T, N, K, out)
    assert torch.equal(out, want)
    here = os.path.dirname(os.path.abspath(__file__))
    code = ("import sys; sys.path[:0] = [%r, %r]\n"
            "import test_gpu_ops as t, expert_routing_grouped_gb300 as moe\n"
            "x, w = t.make_linear(t.gen(3), 40, 4096, 256, 1, 0, 0, False, False)[:2]\n"
            "out, status = t.run_linear(moe, x, w, None, None, None, None, 256, 1, 0, 0)\n"
            "t.check_linear(out, status, x, w, None, None, None, None, 256, 0)\n"
            % (os.path.dirname(here), here))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=200)
    assert r.returncode == 0, r.stderr[-2000:]


# ------------------------------------------------------------ balance loss --

@pytest.mark.parametrize("level", [-87.0, -84.0, -60.0, -30.0, 10.0])
@pytest.mark.parametrize("T,E,dtype,extra", [
    (1, 8, 0, 0), (40, 8, 0, 0), (6, 64, 1, 0), (9, 7, 0, 0), (12, 128, 0, 1), (30, 256, 1, 0),
    (700, 128, 0, 0), (700, 160, 1, 0)])
def test_balance_sigmoid_of_far_logits(moe, T, E, dtype, extra, level):
    """Sigmoids near the ends of f32's range (all of them at least 2^-126) and a
    large gradient from above, as a scaled loss has: probabilities and gradient
    are the formula's."""
    g = gen(T + E)
    z = (level + 0.25 * torch.rand(T, E, generator=g, device="cuda")).to(DT[dtype])
    k = 2
    idx = torch.randint(0, E, (T, k), generator=g, dtype=torch.int32, device="cuda")
    grad = torch.full((1,), 65536.0, device="cuda")
    got = run_balance(moe, z, idx, None, None, None, k, 1, grad=grad, extra=extra)
    check_balance(got, z, idx, None, None, None, k, 1, grad=grad)
    assert bool(got[4].isfinite().all())


@pytest.mark.parametrize("mode", [0, 1])
@pytest.mark.parametrize("T,E,dtype", [(20, 8, 0), (20, 64, 1), (20, 60, 0), (20, 7, 1), (20, 256, 0),
                                       (2000, 64, 0), (2000, 64, 1), (700, 256, 1)])
def test_balance_masked_rows_stay_zero_whatever_comes_from_above(moe, T, E, dtype, mode):
    """grad, bias or a masked row's own logits may be anything: dz of a masked
    row is 0, and a segment without kept tokens has loss and prob 0."""
    g = gen(E)
    z, idx, _, _ = make_balance(g, T, E, 2, dtype)
    m = (torch.arange(T, device="cuda") % 3 != 1).to(torch.uint8)
    z[m == 0] = torch.tensor([float("nan"), float("inf"), -float("inf"), 1.0], device="cuda").to(
        z.dtype).repeat(E)[:E]
    for up in (float("inf"), float("nan"), 2.0):
        grad = torch.full((1,), up, device="cuda")
        dz = run_balance(moe, z, idx, None, m, None, 2, mode, grad=grad)[4]
        assert bool((dz[m == 0] == 0).all())
    got = run_balance(moe, z, idx, None, m, None, 2, mode, grad=torch.full((1,), 2.0, device="cuda"))
    kept = z.clone()
    kept[m == 0] = 0
    check_balance(got, kept, idx, None, m, None, 2, mode, grad=torch.full((1,), 2.0))
    bias = torch.full((E,), float("nan"), device="cuda")
    none = torch.zeros_like(m)
    loss, counts, tokens, prob, dz = run_balance(moe, z, idx, bias, none, None, 2, mode)
    assert float(loss) == 0 and int(tokens) == 0 and int(counts.sum()) == 0
    assert bool((prob == 0).all()) and bool((dz == 0).all())


# Chunks of the pass above 32 tokens (T > 14592) and of the histograms above
# 256 (T > 16384), and several rows of one warp in a segment.
@pytest.mark.parametrize("T,E,k,S,dtype,mode", [
    (16389, 256, 8, 24, 1, 1), (16389, 64, 4, 5, 0, 0), (40001, 64, 2, 7, 1, 0), (40001, 130, 4, 3, 0, 1),
    (40001, 8, 2, 1, 0, 0), (70000, 32, 2, 11, 0, 1)])
@pytest.mark.parametrize("mask", [False, True])
def test_balance_long_batches(moe, T, E, k, S, dtype, mode, mask):
    g = gen(T + E)
    z, idx, off, m = make_balance(g, T, E, k, dtype, S, mask)
    bias = 0.3 * randn(g, E)
    grad = 1 + 0.1 * randn(g, S)
    got = run_balance(moe, z, idx, bias, m, off, k, mode, grad=grad)
    check_balance(got, z, idx, bias, m, off, k, mode, grad=grad)
    plain = run_balance(moe, z, idx, bias, m, off, k, mode, want_dz=False)
    check_balance(plain, z, idx, bias, m, off, k, mode)
    for a, b in zip(got[:4], plain[:4]):   # with and without a gradient, the same bits
        assert torch.equal(a, b)


def test_balance_disorder_with_more_segments_than_tokens(moe):
    """An array whose order would make every other of 65534 segments all 127
    tokens long is worked on as if they were empty; the same count of segments
    in order is summed as ever."""
    T, E, k, S = 127, 64, 2, 65534
    z, idx, _, _ = make_balance(gen(1), T, E, k, 0)
    off = torch.tensor([0, T] * S, dtype=torch.int32, device="cuda")[:S + 1]
    loss, counts, tokens, prob, dz = run_balance(moe, z, idx, None, None, off, k, 0)
    assert int(tokens.sum()) == 0 and int(counts.sum()) == 0 and bool((dz == SENT).all())
    S = 600
    off = torch.full((S + 1,), 120, dtype=torch.int32, device="cuda")
    off[:300] = 3
    got = run_balance(moe, z, idx, None, None, off, k, 0)
    check_balance(got, z, idx, None, None, off, k, 0)


def test_balance_of_no_tokens_is_zero(moe):
    """T = 0: every segment is empty, and its results are an empty segment's,
    in a captured call too."""
    E, S = 16, 5
    f = dict(device="cuda")
    loss, prob = torch.full((S + 1,), SENT, **f), torch.full((S + 1, E), SENT, **f)
    counts = torch.full((S + 1, E), 77, dtype=torch.int32, **f)
    tokens = torch.full((S + 1,), 77, dtype=torch.int32, **f)
    off = torch.zeros(S + 1, dtype=torch.int32, **f)
    z, idx = torch.empty(0, E, **f), torch.empty(0, 2, dtype=torch.int32, **f)
    ws = torch.empty(0, dtype=torch.uint8, **f)

    def call():
        moe.balance_loss(z, idx, 0, E, 2, loss, counts, tokens, prob, ws, seq_off=off, n_seq=S)

    def check():
        for t, fill in ((loss, SENT), (prob, SENT), (counts, 77), (tokens, 77)):
            assert bool((t[:S] == 0).all()) and bool((t[S:] == fill).all())

    call()
    check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for t, fill in ((loss, SENT), (prob, SENT), (counts, 77), (tokens, 77)):
        t.fill_(fill)
    graph.replay()
    check()
