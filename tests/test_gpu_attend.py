"""The attention block's operators on the GPU against their 64-bit forms
(attend_ref.py).  Tolerances come from the arithmetic: a rounding to type t is
off by at most half a step, eps(t) / 2 of the value; the rest is derived beside
each check."""
import math

import numpy as np
import pytest
import torch

import attend_ref as ref

pytestmark = pytest.mark.gpu

DT = {0: torch.float32, 1: torch.bfloat16}
SENT = 72.0


@pytest.fixture(scope="module")
def moe():
    import expert_routing_grouped_gb300 as m
    return m


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


# -------------------------------------------------------------------- rope --

def check_rope(out, x, pos, freqs, rot, il, inv, m):
    y, size = ref.rope(x, pos, freqs, rot, il, inv, m)
    # Sine and cosine in f32: their own error (2 units of 2^-24), the angle's
    # rounding to f32 (2^-25 half turns, pi 2^-25) and its lowest 32 bits (2^-33
    # turns), the product with mscale; then two products and a sum: under 8 units
    # of 2^-24 of |u| + |v|.
    tol = 8 * 2.0 ** -24 * size + ref.half_step(out.dtype) * y.abs() * 1.0001 + 2.0 ** -133
    d = (out.double() - y).abs()
    assert bool((d <= tol).all()), float((d / tol).max())
    assert torch.equal(out[..., rot:], x[..., rot:])


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("il,inv", [(False, False), (True, False), (False, True), (True, True)])
@pytest.mark.parametrize("T,heads,D,rot", [
    (1, 1, 2, 2), (1, 104, 128, 64), (3, 5, 128, 128), (7, 3, 80, 40), (2, 4, 96, 48), (5, 2, 65, 34),
    (33, 9, 64, 2), (2, 2, 1024, 1024), (300, 40, 128, 128), (4, 3, 256, 200), (4097, 16, 64, 64),
    (2, 300, 1024, 1022), (1, 1000, 6, 4), (37, 1, 72, 24)])
def test_rope(moe, T, heads, D, rot, il, inv, dtype):
    g = gen(T + heads + D)
    x = randn(g, T, heads, D).to(DT[dtype])
    pos = torch.randint(0, 1 << 20, (T,), generator=g, device="cuda", dtype=torch.int32)
    f, _ = moe.rope_freqs(rot, 1e4)
    freqs = torch.from_numpy(f).cuda()
    out = torch.full_like(x, SENT)
    moe.rope(x, pos, freqs, T, heads, D, out, rot_dim=rot, interleaved=il, inverse=inv, mscale=1.25,
             dtype=dtype)
    check_rope(out, x, pos, freqs, rot, il, inv, 1.25)
    y = x.clone()   # in place: the same bits
    moe.rope(y, pos, freqs, T, heads, D, y, rot_dim=rot, interleaved=il, inverse=inv, mscale=1.25,
             dtype=dtype)
    assert torch.equal(y, out)


def test_rope_far_positions(moe):
    """The ends of int32, and frequencies of any size and sign, against exact integers."""
    pos = [0, 1, -1, 5, 10 ** 6, 2 ** 24 + 1, 2 ** 31 - 1, -2 ** 31, -12345678]
    freqs = [1.0, 0.3, 1e-7, 2.0 ** -60, 6.25, 1000.1, -0.7, 0.0, 5e-324, 2 * math.pi]
    x = torch.zeros(len(pos), 1, 20, device="cuda")
    x[..., :10] = 1   # u = 1, v = 0: the result is (cos, sin)
    out = torch.empty_like(x)
    moe.rope(x, torch.tensor(pos, dtype=torch.int32, device="cuda"),
             torch.tensor(freqs, dtype=torch.float64, device="cuda"), len(pos), 1, 20, out, dtype=0)
    from decimal import Decimal, getcontext
    getcontext().prec = 60
    pi = Decimal("3.14159265358979323846264338327950288419716939937510582097494")
    for a, p in enumerate(pos):
        for b, f in enumerate(freqs):
            turns = Decimal(p) * Decimal(f) / (2 * pi)
            ang = float((turns - turns.to_integral_value()) * 2 * pi)
            # pos 2^-64 turns of the fraction and 2^-62 of 1000 radians at 2^31: under 2^-30
            tol = 8 * 2.0 ** -24
            assert abs(float(out[a, 0, b]) - math.cos(ang)) <= tol, (p, f)
            assert abs(float(out[a, 0, 10 + b]) - math.sin(ang)) <= tol, (p, f)


def test_rope_fused_row_strides_and_untouched(moe):
    """Query and key heads of a fused row in place; heads-first tensors; the rest stays."""
    g = gen(4)
    T, H, Hkv, D, rot = 11, 6, 2, 64, 32
    row = (H + 2 * Hkv) * D + 24
    for dtype in (0, 1):
        x = randn(g, T, row).to(DT[dtype])
        before = x.clone()
        pos = torch.arange(T, dtype=torch.int32, device="cuda") + 1000
        freqs = torch.from_numpy(moe.rope_freqs(rot, 1e4)[0]).cuda()
        moe.rope(x, pos, freqs, T, H + Hkv, D, x, rot_dim=rot, dtype=dtype, x_stride=row, out_stride=row)
        n = (H + Hkv) * D
        check_rope(x[:, :n].reshape(T, -1, D), before[:, :n].reshape(T, -1, D), pos, freqs, rot, False,
                   False, 1.0)
        assert torch.equal(x[:, n:], before[:, n:])
        # [heads][T][D] to [T][heads][D + 8]
        y = randn(g, 5, T, D).to(DT[dtype])
        out = torch.full((T, 5, D + 8), SENT, device="cuda").to(DT[dtype])
        moe.rope(y, pos, freqs, T, 5, D, out, rot_dim=rot, interleaved=True, dtype=dtype, x_stride=D,
                 x_head_stride=T * D, out_stride=5 * (D + 8), out_head_stride=D + 8)
        check_rope(out[..., :D], y.transpose(0, 1), pos, freqs, rot, True, False, 1.0)
        assert bool((out[..., D:] == SENT).all())
        # elements at odd addresses
        z = randn(g, T * 3 * D + 1).to(DT[dtype])[1:].view(T, 3, D)
        out = torch.empty(T * 3 * D + 1, device="cuda", dtype=DT[dtype])[1:].view(T, 3, D)
        moe.rope(z, pos, freqs, T, 3, D, out, rot_dim=rot, dtype=dtype)
        check_rope(out, z, pos, freqs, rot, False, False, 1.0)


def test_rope_gradient(moe):
    """inverse is the transposed operator: <turn(x), g> = <x, turn_back(g)> for
    every pair of basis directions, and differences along random directions."""
    g = gen(6)
    T, heads, D, rot = 3, 2, 16, 12
    pos = torch.tensor([0, 77, 123456], dtype=torch.int32, device="cuda")
    freqs = torch.from_numpy(moe.rope_freqs(rot, 1e4)[0]).cuda()
    for il in (False, True):
        def turn(v, inv):
            out = torch.empty_like(v)
            moe.rope(v, pos, freqs, T, heads, D, out, rot_dim=rot, interleaved=il, inverse=inv,
                     mscale=1.5, dtype=0)
            return out
        x, up, way = randn(g, T, heads, D), randn(g, T, heads, D), randn(g, T, heads, D)
        grad = turn(up, True).double()
        # the operator is linear: a difference over a step of 1 is the derivative
        d = ((turn(x + way, False).double() - turn(x, False).double()) * up.double()).sum()
        size = float((up.abs().double() * (x.abs() + way.abs()).double()).sum()) * 3
        assert abs(float(d - (grad * way.double()).sum())) <= 32 * 2.0 ** -24 * size
        formula, s = ref.rope(up, pos, freqs, rot, il, True, 1.5)
        assert bool(((grad - formula).abs() <= 8 * 2.0 ** -24 * s + 2.0 ** -24 * formula.abs()).all())


def test_rope_scaled_and_nonfinite(moe):
    g = gen(7)
    f, m = moe.rope_freqs(64, 1e6, moe.ROPE_PARTS, 8.0, 32768)
    freqs = torch.from_numpy(f).cuda()
    x = randn(g, 4, 3, 64)
    pos = torch.tensor([0, 5, 200000, 262143], dtype=torch.int32, device="cuda")
    out = torch.empty_like(x)
    moe.rope(x, pos, freqs, 4, 3, 64, out, mscale=m, dtype=0)
    check_rope(out, x, pos, freqs, 64, False, False, m)
    x[1, 2, 7] = float("inf")
    x[2, 0, 40] = float("nan")
    moe.rope(x, pos, freqs, 4, 3, 64, out, mscale=m, dtype=0)
    bad = ~torch.isfinite(out)
    want = torch.zeros_like(bad)
    want[1, 2, [7, 39]] = True
    want[2, 0, [8, 40]] = True
    assert torch.equal(bad, want)


# ------------------------------------------------------------- kv4_append --

def batch(new, cache):
    off = [0]
    for n in new:
        off.append(off[-1] + n)
    return torch.tensor(off, dtype=torch.int32, device="cuda"), off


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page,Hkv,new,have", [
    (16, 1, [1], [1]), (16, 2, [5, 0, 1, 16], [5, 3, 40, 16]), (64, 3, [70, 1], [70, 64]),
    (256, 1, [300], [511]), (32, 8, [33, 32, 31], [100, 32, 64]), (128, 5, [1] * 70, list(range(1, 71)))])
def test_append(moe, page, Hkv, new, have, D, dtype):
    g = gen(page + D)
    c = ref.Cache(g, have, Hkv, D, page)
    off, o = batch(new, c)
    T = o[-1]
    x = randn(g, 2, T, Hkv, D) * torch.exp(randn(g, 2, 1, Hkv, D))
    x = x.to(DT[dtype])
    k, v = x[0], x[1]
    k[0, 0, :64] = 3.7          # one value only
    v[T - 1, Hkv - 1, 3] = 1e9  # far beyond float16
    k[T // 2, 0, 5] = float("-inf")
    v[T // 2, 0, 0] = float("nan")
    want = ref.Cache.__new__(ref.Cache)
    want.__dict__.update(c.__dict__)
    want.bytes = c.bytes.clone()
    for s in range(len(new)):
        for which, rows in ((0, k), (1, v)):
            want.put(s, which, have[s] - new[s], rows[o[s]:o[s + 1]].float())
    moe.kv4_append(k, v, c.bytes, c.pages, c.kv_len, T, Hkv, D, page, c.n_pages, c.max_pages, q_off=off,
                   n_seq=len(new), dtype=dtype)
    for which in (0, 1):
        a, b = c.part(which), want.part(which)
        assert torch.equal(a[0], b[0])
        sa, sb = a[1].contiguous().view(torch.float16), b[1].contiguous().view(torch.float16)
        assert bool(((sa == sb) | (sa.isnan() & sb.isnan())).all())


def test_append_one_row_each_strided(moe):
    """Without q_off one row a sequence; K and V as columns of a fused row."""
    g = gen(3)
    have, Hkv, D, page = [1, 17, 32, 100], 2, 64, 16
    c = ref.Cache(g, have, Hkv, D, page)
    want = c.bytes.clone()
    fused = randn(g, 4, 5 * Hkv * D).bfloat16()
    k, v = fused[:, Hkv * D:2 * Hkv * D], fused[:, 3 * Hkv * D:4 * Hkv * D]
    moe.kv4_append(k, v, c.bytes, c.pages, c.kv_len, 4, Hkv, D, page, c.n_pages, c.max_pages,
                   k_stride=fused.stride(0), v_stride=fused.stride(0))
    got, c.bytes = c.bytes, want
    for s, n in enumerate(have):
        c.put(s, 0, n - 1, k[s].reshape(1, Hkv, D).float())
        c.put(s, 1, n - 1, v[s].reshape(1, Hkv, D).float())
    assert torch.equal(got, want)


def test_append_drops_what_has_no_place(moe):
    """Negative positions, holes, rows in no sequence, offsets and lengths out of range."""
    g = gen(5)
    Hkv, D, page = 1, 64, 16
    c = ref.Cache(g, [40, 4], Hkv, D, page)
    c.pages[0, 1] = -1
    before = c.bytes.clone()
    k, v = randn(g, 2, 48, Hkv, D).bfloat16()
    # rows 2..41 are sequence 0 (positions 0..39; 16..31 in a hole), 42..47 sequence 1 (-2..3)
    off = torch.tensor([2, 42, 48], dtype=torch.int32, device="cuda")
    moe.kv4_append(k, v, c.bytes, c.pages, c.kv_len, 48, Hkv, D, page, c.n_pages, c.max_pages, q_off=off,
                   n_seq=2)
    got, c.bytes = c.bytes, before
    for which, x in ((0, k), (1, v)):
        c.put(0, which, 0, x[2:18].float())
        c.put(0, which, 32, x[34:42].float())
        c.put(1, which, 0, x[44:48].float())
    assert torch.equal(got, before)
    # offsets beyond T, lengths beyond the table or negative: nothing outside the cache is touched
    wide = torch.full((got.numel() + 4096,), 7, dtype=torch.uint8, device="cuda")
    body = wide[2048:2048 + got.numel()]
    for off, n in (([-5, 60, 1 << 30], [1 << 30, -7]), ([48, 0, 20], [40, 4])):
        moe.kv4_append(k, v, body, c.pages, torch.tensor(n, dtype=torch.int32, device="cuda"), 48, Hkv, D,
                       page, c.n_pages, c.max_pages,
                       q_off=torch.tensor(off, dtype=torch.int32, device="cuda"), n_seq=2)
        assert bool((wide[:2048] == 7).all()) and bool((wide[2048 + got.numel():] == 7).all())


# ---------------------------------------------------------- kv4_attention --

def run(moe, q, c, new, off=None, softcap=0.0, window=0, causal=True, scale=None, max_q=0, out=None,
        stream=None):
    T, H, D = q.shape
    if out is None:
        out = torch.full((T, H, D), SENT, device="cuda").bfloat16()
    n = moe.kv4_workspace(T, len(new), H, c.Hkv, D, c.page, c.max_pages, max_q=max_q)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda") if n else None
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    moe.kv4_attention(q, c.bytes, c.pages, c.kv_len, T, H, c.Hkv, D, c.page, c.n_pages, c.max_pages, out,
                      ws, q_off=off, n_seq=len(new), max_q=max_q, scale=scale, softcap=softcap,
                      window=window, causal=causal, q_stride=q.stride(0), out_stride=out.stride(0),
                      status=status, stream=stream)
    assert int(status) == 0
    return out


def check(out, q, c, o, softcap=0.0, window=0, causal=True, scale=None, holes=()):
    scale = q.shape[2] ** -0.5 if scale is None else scale
    for s in range(len(o) - 1):
        if o[s + 1] == o[s]:
            continue
        seen = torch.ones(c.have[s], dtype=torch.bool, device="cuda")
        for hs, first, end in holes:
            if hs == s:
                seen[first:end] = False
        y, bound = ref.attend(q[o[s]:o[s + 1]], c.K[s], c.V[s], scale, softcap, window, causal, seen)
        got = out[o[s]:o[s + 1]].double()
        tol = bound + ref.half_step(torch.bfloat16) * (y.abs() + bound) + 2.0 ** -133
        ok = ((got - y).abs() <= tol) | (torch.isnan(got) & torch.isnan(y))
        assert bool(ok.all()), (s, int((~ok).sum()), float(torch.nan_to_num((got - y).abs() / tol).max()))


LENS = [[1], [2, 1], [15, 16, 17], [31, 32, 33, 1, 0, 64], [127, 128, 129], [255, 256, 257, 300], [700, 5],
        [1500], [4097, 1]]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,Hkv", [(1, 1), (8, 2), (5, 1), (12, 1), (16, 1), (36, 4), (6, 6), (24, 1), (40, 1)])
@pytest.mark.parametrize("have", LENS)
def test_decode(moe, have, H, Hkv, D):
    g = gen(sum(have) + H + D)
    page = [16, 32, 64, 128, 256][(sum(have) + H) % 5]
    c = ref.Cache(g, have, Hkv, D, page)
    q = (1.5 * randn(g, len(have), H, D)).bfloat16()
    out = run(moe, q, c, have)
    check(out, q, c, list(range(len(have) + 1)))


@pytest.mark.parametrize("softcap,window,causal", [(0.0, 0, False), (20.0, 0, True), (0.0, 7, True),
                                                   (0.0, 100, False), (5.0, 33, True)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("new,have", [
    ([1, 1, 1], [300, 20, 1]), ([2, 3, 4, 1], [40, 3, 513, 1]), ([8, 0, 5], [600, 7, 100]),
    ([20, 1, 9], [20, 400, 300]), ([130], [130]), ([33, 70], [500, 70]), ([300], [777])])
def test_masks(moe, new, have, page, D, softcap, window, causal):
    """Single tokens, a few, prompts and mixtures under every mask."""
    g = gen(sum(have) + page + D)
    H, Hkv = 8, 2
    c = ref.Cache(g, have, Hkv, D, page)
    off, o = batch(new, c)
    q = (2 * randn(g, o[-1], H, D)).bfloat16()
    out = run(moe, q, c, new, off, softcap, window, causal, scale=0.2)
    check(out, q, c, o, softcap, window, causal, scale=0.2)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,Hkv", [(1, 1), (3, 1), (12, 2), (7, 7), (48, 1), (200, 1)])
@pytest.mark.parametrize("new,have", [([17], [17]), ([64, 64], [64, 200]), ([127, 1, 2], [1000, 1000, 50]),
                                      ([257], [300]), ([5, 128, 0, 129], [2000, 128, 9, 129])])
def test_heads(moe, new, have, H, Hkv, D):
    """Shared heads of any number against rows of any number."""
    g = gen(sum(have) + H)
    c = ref.Cache(g, have, Hkv, D, 64)
    off, o = batch(new, c)
    q = (1.5 * randn(g, o[-1], H, D)).bfloat16()
    check(run(moe, q, c, new, off), q, c, o)
    out = run(moe, q, c, new, off, max_q=max(new))
    check(out, q, c, o)


@pytest.mark.parametrize("new", [[1, 1], [3, 2], [70, 40]])
@pytest.mark.parametrize("D", [64, 128])
def test_rows_that_see_nothing(moe, new, D):
    """No tokens, more rows than tokens, holes that leave nothing: zeros."""
    g = gen(8)
    H, Hkv, page = 4, 2, 16
    c = ref.Cache(g, [0, 40], Hkv, D, page)
    off, o = batch(new, c)
    q = randn(g, o[-1], H, D).bfloat16()
    out = run(moe, q, c, new, off)
    assert bool((out[:o[1]] == 0).all())
    check(out[o[1]:], q[o[1]:], type("C", (), dict(have=[40], K=[c.K[1]], V=[c.V[1]])), [0, new[1]]) \
        if new[1] <= 40 else None
    c.kv_len[1] = 1
    out = run(moe, q, c, new, off)
    assert bool((out[o[1]:o[2] - 1] == 0).all())   # negative positions
    assert not bool((out[o[2] - 1] == 0).all())
    c.kv_len[1] = 40
    for holes in ([0], [1], [0, 2], [0, 1, 2]):
        pages = c.pages.clone()
        for i, h in enumerate(holes):
            c.pages[1, h] = [-1, c.n_pages, -2 ** 31][i]
        out = run(moe, q, c, new, off)
        if new[1] <= 40:
            one = type("C", (), dict(have=[40], K=[c.K[1]], V=[c.V[1]]))
            check(out[o[1]:], q[o[1]:], one, [0, new[1]], holes=[(0, 16 * h, 16 * h + 16) for h in holes])
        if len(holes) == 3:
            assert bool((out == 0).all())
        c.pages = pages


@pytest.mark.parametrize("new,have", [([1, 1], [70, 30]), ([4, 3], [70, 30]), ([40, 30], [70, 30]),
                                      ([200], [260])])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("window", [0, 20])
def test_nan_reaches_only_who_sees_it(moe, new, have, D, window):
    g = gen(9)
    H, Hkv, page = 6, 2, 32
    c = ref.Cache(g, have, Hkv, D, page)
    off, o = batch(new, c)
    x = randn(g, 1, Hkv, D)
    for s, which, token in ((0, 0, 5), (0, 1, have[0] - 1), (0, 1, have[0] // 2)):
        y = x.clone()
        y[0, 1, 3] = float("nan")
        (c.K if which == 0 else c.V)[s][token] = c.put(s, which, token, y)[0]
    q = randn(g, o[-1], H, D).bfloat16()
    out = run(moe, q, c, new, off, window=window)
    check(out, q, c, o, window=window)
    # and queries: an infinity or a NaN stays in its row and head
    q2 = q.clone()
    q2[0, 0, 1], q2[0, 3, 2] = float("nan"), float("inf")
    out2 = run(moe, q2, c, new, off, window=window)
    same = torch.ones(o[-1], H, dtype=torch.bool, device="cuda")
    same[0, 0] = same[0, 3] = False
    assert bool(out2[0, 0].isnan().all()) and bool(out2[0, 3].isnan().all())
    a, b = out[same], out2[same]
    assert bool(((a == b) | (a.isnan() & b.isnan())).all())


@pytest.mark.parametrize("size", [1e-3, 1.0, 300.0])
@pytest.mark.parametrize("new", [[1], [3], [50]])
def test_sizes_of_values(moe, new, size):
    """Small and large keys and values (queries the other way round)."""
    g = gen(10)
    c = ref.Cache(g, [400], 1, 128, 16, size=size)
    q = (randn(g, new[0], 4, 128) / size).bfloat16()
    off, o = batch(new, c)
    check(run(moe, q, c, new, off), q, c, o)


@pytest.mark.parametrize("new", [[1, 1, 1], [2, 4, 3], [40, 9, 60]])
def test_strides_and_untouched(moe, new):
    """Query as a column slice of a fused row; rows in no sequence and past max_q stay."""
    g = gen(11)
    H, Hkv, D = 4, 2, 64
    have = [90, 70, 60]
    c = ref.Cache(g, have, Hkv, D, 16)
    total = sum(new)
    fused = randn(g, total + 5, 3 * H * D + 8).bfloat16()
    q = fused[:, H * D:2 * H * D].unflatten(1, (H, D))
    out = torch.full((total + 5, H + 1, D), SENT, device="cuda").bfloat16()
    off = torch.tensor([2] + [2 + sum(new[:i + 1]) for i in range(3)], dtype=torch.int32, device="cuda")
    run(moe, q, c, new, off, out=out[:, :H])
    o = [0] + [sum(new[:i + 1]) for i in range(3)]
    check(out[2:2 + total, :H], q[2:2 + total], c, o)
    assert bool((out[:, H] == SENT).all()) and bool((out[:2] == SENT).all()) and bool((out[2 + total:] == SENT).all())
    top = max(new)
    if top > 1:
        part = torch.full((total + 5, H + 1, D), SENT, device="cuda").bfloat16()
        run(moe, q, c, new, off, out=part[:, :H], max_q=top - 1)
        for s in range(3):
            a, n = 2 + o[s], min(new[s], top - 1)
            assert torch.equal(part[a:a + n, :H].float(), out[a:a + n, :H].float())
            assert bool((part[a + n:2 + o[s + 1]] == SENT).all())


def test_offsets_and_lengths_out_of_range(moe):
    """Clamped: nothing outside the operands is touched, and the call ends."""
    g = gen(12)
    H, Hkv, D, page = 4, 2, 64, 16
    c = ref.Cache(g, [90, 70, 60], Hkv, D, page)
    c.pages[c.pages < 0] = 0
    q = randn(g, 30, H, D).bfloat16()
    for off, n in (([0, 1 << 30, 5, 30], [1 << 30, -5, 60]), ([-9, -3, 40, 7], [90, 70, 60]),
                   ([30, 20, 10, 0], [1 << 30, 1 << 30, 1 << 30])):
        c.kv_len = torch.tensor(n, dtype=torch.int32, device="cuda")
        wide = torch.full((34, H, D), SENT, device="cuda").bfloat16()
        run(moe, q, c, [1] * 3, torch.tensor(off, dtype=torch.int32, device="cuda"), out=wide[2:32])
        assert bool((wide[:2] == SENT).all()) and bool((wide[32:] == SENT).all())


@pytest.mark.parametrize("new,have", [([1, 1], [5000, 300]), ([3], [3000]), ([300, 1, 5], [1300, 900, 40])])
def test_repeats_bitwise_graph_and_streams(moe, new, have):
    """The same bits on every call, in a graph whose lengths change between replays, on another stream."""
    g = gen(13)
    H, Hkv, D = 8, 2, 128
    c = ref.Cache(g, have, Hkv, D, 64)
    off, o = batch(new, c)
    q = randn(g, o[-1], H, D).bfloat16()
    first = run(moe, q, c, new, off)
    for _ in range(3):
        assert torch.equal(run(moe, q, c, new, off), first)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = run(moe, q, c, new, off, stream=side)
    side.synchronize()
    assert torch.equal(other, first)
    out = torch.zeros_like(q)
    n = moe.kv4_workspace(o[-1], len(new), H, Hkv, D, 64, c.max_pages)
    ws = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.kv4_attention(q, c.bytes, c.pages, c.kv_len, o[-1], H, Hkv, D, 64, c.n_pages, c.max_pages, out,
                          ws, q_off=off, n_seq=len(new))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first)
    shorter = [max(n, m // 2) for n, m in zip(new, have)]
    c.kv_len.copy_(torch.tensor(shorter, dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    one = type("C", (), dict(have=shorter, K=[k[:n] for k, n in zip(c.K, shorter)],
                             V=[v[:n] for v, n in zip(c.V, shorter)]))
    check(out, q, one, o)


def test_many_sequences(moe):
    """A large ragged batch of single tokens, some without any tokens, and one long one."""
    g = gen(14)
    H, Hkv, D = 8, 4, 64
    have = [int(v) for v in torch.randint(0, 90, (1100,), generator=g, device="cuda")]
    have[700] = 9000
    c = ref.Cache(g, have, Hkv, D, 16)
    q = randn(g, len(have), H, D).bfloat16()
    out = run(moe, q, c, have)
    for s in [0, 1, 2, 500, 699, 700, 701, 1098, 1099] + [i for i, n in enumerate(have) if n in (0, 1, 16)]:
        one = type("C", (), dict(have=[have[s]], K=[c.K[s]], V=[c.V[s]]))
        check(out[s:s + 1], q[s:s + 1], one, [0, 1])


def test_attention_block_together(moe):
    """One block's attention half as a user runs it, for a prompt and then single
    tokens: norm -> QKV product -> rotary -> cache -> attention -> output product
    onto the stream, every step against 64 bits on what the step before it gave."""
    g = gen(15)
    hid, H, Hkv, D, page, S = 512, 8, 2, 64, 16, 2
    wide = (H + 2 * Hkv) * D
    w_qkv = (randn(g, wide, hid) / hid ** 0.5).bfloat16()
    w_o = (randn(g, hid, H * D) / (H * D) ** 0.5).bfloat16()
    freqs = torch.from_numpy(moe.rope_freqs(D, 1e4)[0]).cuda()
    have = [37, 20]
    c = ref.Cache(g, [n + 3 for n in have], Hkv, D, page)
    c.bytes.fill_(255)
    c.K = [torch.zeros(0, Hkv, D, dtype=torch.float64, device="cuda") for _ in have]
    c.V = [torch.zeros(0, Hkv, D, dtype=torch.float64, device="cuda") for _ in have]
    length = [0, 0]
    for new in (have, [1, 1], [1, 1], [1, 1]):
        length = [a + b for a, b in zip(length, new)]
        off, o = batch(new, c)
        T = o[-1]
        c.kv_len.copy_(torch.tensor(length, dtype=torch.int32))
        pos = torch.cat([torch.arange(n - m, n) for m, n in zip(new, length)]).to(torch.int32).cuda()
        stream = randn(g, T, hid)
        x = torch.zeros(T, hid, device="cuda")
        normed = torch.empty(T, hid, dtype=torch.bfloat16, device="cuda")
        moe.add_rmsnorm(x, T, hid, 1e-6, normed, resid=stream, resid_out=stream, x_dtype=0)
        qkv = torch.empty(T, wide, dtype=torch.bfloat16, device="cuda")
        moe.linear(normed, w_qkv, T, wide, hid, qkv, out_dtype=moe.BF16)
        plain = qkv.clone()
        moe.rope(qkv, pos, freqs, T, H + Hkv, D, qkv, x_stride=wide, out_stride=wide)
        heads = (H + Hkv) * D
        check_rope(qkv[:, :heads].reshape(T, -1, D), plain[:, :heads].reshape(T, -1, D), pos, freqs, D,
                   False, False, 1.0)
        k, v = qkv[:, H * D:heads], qkv[:, heads:]
        moe.kv4_append(k, v, c.bytes, c.pages, c.kv_len, T, Hkv, D, page, c.n_pages, c.max_pages, q_off=off,
                       n_seq=S, k_stride=wide, v_stride=wide)
        for s in range(S):
            rows = slice(o[s], o[s + 1])
            for kept, fresh in ((c.K, k), (c.V, v)):
                y = ref.values(*ref.quantise(fresh[rows].reshape(-1, Hkv, D).float()))
                kept[s] = torch.cat([kept[s], y])
        c.have = length
        q = qkv[:, :H * D].unflatten(1, (H, D))
        att = run(moe, q, c, new, off, max_q=max(new))
        check(att, q, c, o)
        before = stream.clone()
        moe.linear(att, w_o, T, hid, H * D, stream, resid=stream)
        want = before.double() + att.view(T, -1).double() @ w_o.double().t()
        size = att.view(T, -1).double().abs() @ w_o.double().abs().t()
        assert bool(((stream.double() - want).abs() <= (H * D / 8 + 32) * 2.0 ** -23 * size + 2.0 ** -23 * want.abs()).all())


# ------------------------------------------------- waits, captures, far addresses --

def test_attention_waits_give_up(moe):
    """A wait limit of 0 gives up: the status word says so, with none moe_linear_status
    does; nothing hangs, and the next call is right."""
    g = gen(16)
    for H, Hkv, D, new, have in ((8, 2, 128, [300, 20], [700, 500]), (40, 1, 64, [1, 1], [900, 2000])):
        c = ref.Cache(g, have, Hkv, D, 32)
        off, o = batch(new, c)
        T = o[-1]
        q = randn(g, T, H, D).bfloat16()
        out = torch.zeros_like(q)
        n = moe.kv4_workspace(T, len(new), H, Hkv, D, 32, c.max_pages)
        ws = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")

        def call(st):
            moe.kv4_attention(q, c.bytes, c.pages, c.kv_len, T, H, Hkv, D, 32, c.n_pages, c.max_pages, out, ws,
                              q_off=off, n_seq=len(new), status=st)
            torch.cuda.synchronize()

        assert moe.linear_status() == 0
        moe.linear_wait_limit(0)
        try:
            call(status)
            assert int(status) == 2 and moe.linear_status() == 0
            call(None)
            assert moe.linear_status() == 2 and moe.linear_status() == 0
        finally:
            moe.linear_wait_limit(2000000)
        status.zero_()
        call(status)
        assert int(status) == 0
        check(out, q, c, o)


def test_two_streams_at_once(moe):
    """Different calls on two streams, each with its own workspace, many times over."""
    g = gen(17)
    jobs = []
    for H, Hkv, D, new, have in ((12, 1, 128, [1, 1], [3000, 50]), (8, 2, 64, [150], [400])):
        c = ref.Cache(g, have, Hkv, D, 64)
        off, o = batch(new, c)
        q = randn(g, o[-1], H, D).bfloat16()
        n = moe.kv4_workspace(o[-1], len(new), H, Hkv, D, 64, c.max_pages)
        jobs.append((c, off, o, q, torch.empty_like(q), torch.empty(max(n, 16), dtype=torch.uint8, device="cuda"),
                     torch.cuda.Stream(), len(new)))
    torch.cuda.synchronize()
    for _ in range(20):
        for c, off, o, q, out, ws, st, n in jobs:
            moe.kv4_attention(q, c.bytes, c.pages, c.kv_len, o[-1], q.shape[1], c.Hkv, q.shape[2], 64, c.n_pages,
                              c.max_pages, out, ws, q_off=off, n_seq=n, stream=st)
    torch.cuda.synchronize()
    for c, off, o, q, out, ws, st, n in jobs:
        check(out, q, c, o)


@pytest.mark.parametrize("new", [[1], [40]])
def test_far_pages_and_rows(moe, new):
    """Pages past 4 GB of a cache, rows of q past 4 GB: appended to and attended."""
    g = gen(18)
    H, Hkv, D, page, have = 8, 8, 128, 256, [700]
    c = ref.Cache(g, have, Hkv, D, page, spare=0)
    n_pages = (5 << 30) // moe.kv4_page_bytes(page, Hkv, D)
    far = torch.empty(n_pages, *c.bytes.shape[1:], dtype=torch.uint8, device="cuda")
    last = torch.arange(n_pages - c.n_pages, n_pages, device="cuda")
    far[last] = c.bytes
    c.bytes, c.pages, c.n_pages = far, (c.pages + (n_pages - c.n_pages)).to(torch.int32), n_pages
    n = new[0]
    x = randn(g, 2, n, Hkv, D).bfloat16()
    off, o = batch(new, c)
    moe.kv4_append(x[0], x[1], c.bytes, c.pages, c.kv_len, n, Hkv, D, page, c.n_pages, c.max_pages, q_off=off,
                   n_seq=1)
    for kept, rows in ((c.K, x[0]), (c.V, x[1])):
        kept[0][have[0] - n:] = ref.values(*ref.quantise(rows.float()))
    if n == 1:
        q = randn(g, 1, H, D).bfloat16()
    else:
        stride = (1 << 27) + 64   # 40 rows: 10 GB apart
        wide = torch.empty(stride * (n - 1) + H * D, dtype=torch.bfloat16, device="cuda")
        q = wide.as_strided((n, H, D), (stride, D, 1))
        q.copy_(randn(g, n, H, D))
    check(run(moe, q, c, new, off), q, c, o)


def test_first_call_inside_a_capture():
    """A process whose first calls are captured: attributes and lookups work there."""
    import subprocess
    import sys
    code = """
import torch, expert_routing_grouped_gb300 as moe
torch.cuda.init()
D, H, Hkv, P = 64, 4, 2, 16
k = torch.randn(40, Hkv, D, device='cuda').bfloat16()
q = torch.randn(40, H, D, device='cuda').bfloat16()
cache = torch.zeros(4, moe.kv4_page_bytes(P, Hkv, D), dtype=torch.uint8, device='cuda')
pages = torch.tensor([[2, 0, 3, 1]], dtype=torch.int32, device='cuda')
n = torch.tensor([40], dtype=torch.int32, device='cuda')
off = torch.tensor([0, 40], dtype=torch.int32, device='cuda')
out = torch.zeros_like(q)
ws = torch.empty(max(16, moe.kv4_workspace(40, 1, H, Hkv, D, P, 4)), dtype=torch.uint8, device='cuda')
f = torch.ones(D // 2, dtype=torch.float64, device='cuda')
pos = torch.arange(40, dtype=torch.int32, device='cuda')
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    moe.rope(q, pos, f, 40, H, D, q)
    moe.kv4_append(k, k, cache, pages, n, 40, Hkv, D, P, 4, 4, q_off=off, n_seq=1)
    moe.kv4_attention(q, cache, pages, n, 40, H, Hkv, D, P, 4, 4, out, ws, q_off=off, n_seq=1)
g.replay()
torch.cuda.synchronize()
assert bool(out.isfinite().all()) and float(out.abs().max()) > 0
"""
    subprocess.run([sys.executable, "-c", code], check=True, timeout=300)


@pytest.mark.parametrize("window", [(1 << 31) - 1, (1 << 30) + 5, 1 << 30])
@pytest.mark.parametrize("H,new,have", [(2, [5, 3, 1], [3, 40, 1]), (4, [70, 40], [50, 60])])
def test_widest_windows(moe, H, new, have, window):
    """Windows as wide as int32 goes, with rows at negative positions: no window at all."""
    g = gen(19)
    c = ref.Cache(g, have, 2, 128, 16)
    off, o = batch(new, c)
    q = randn(g, o[-1], H, 128).bfloat16()
    for causal in (True, False):
        out = run(moe, q, c, new, off, window=window, causal=causal)
        assert torch.equal(out, run(moe, q, c, new, off, causal=causal))
        check(out, q, c, o, causal=causal)


@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("D", [64, 128])
def test_extreme_scales(moe, n, D):
    """Factors beyond f32: scores of 0 stay 0, a cap of nearly nothing levels all
    weights, and a row whose scores are all far below 0 still sees its tokens."""
    g = gen(20)
    c = ref.Cache(g, [90], 1, D, 16)
    off, o = batch([n], c)
    q = randn(g, n, 1, D).bfloat16()
    zero = torch.zeros_like(q)
    for x, kw in ((zero, dict(scale=3e38)), (zero, dict(scale=-2e38, softcap=1e-30)), (q, dict(scale=0.0)),
                  (q, dict(scale=0.0, softcap=1e-40)), (q, dict(scale=1.0, softcap=1e-40)),
                  (q, dict(scale=2.0 ** -140))):
        check(run(moe, x, c, [n], off, **kw), x, c, o, **kw)
    # Keys 1, 2, 3, ... times -2^100: the first token alone has weight.
    rows = (1 + torch.arange(90.0, device="cuda"))[:, None, None].expand(90, 1, D)
    assert torch.equal(c.put(0, 0, 0, rows), rows.double())
    q = torch.full_like(q, -2.0 ** 100)
    out = run(moe, q, c, [n], off).double()
    want = c.V[0][0].double()
    least = want.unflatten(1, (-1, 64)).amin(2, keepdim=True).expand(1, D // 64, 64).flatten(1)
    # weight 1 (or 1 step, whose rounding meets the code), V and out rounded
    tol = (2.0 ** -10 + 2.0 ** -8) * want.abs() * 1.01 + 2.0 ** -11 * (want - least)
    assert bool(((out - want).abs() <= tol).all())


def test_offsets_out_of_order(moe):
    """Offsets in any order: rows outside the call's and pages that are not the
    sequences' own stay as they were, and the next ordered call is right."""
    g = gen(21)
    H, Hkv, D, page, T = 8, 2, 64, 16, 400
    n = 40
    c = ref.Cache(g, [60] * n, Hkv, D, page)
    q = randn(g, T, H, D).bfloat16()
    x = randn(g, 2, T, Hkv, D).bfloat16()
    held = c.bytes.clone()
    own = torch.zeros(c.n_pages, dtype=torch.bool, device="cuda")
    own[c.pages[:, :4].reshape(-1).long()] = True
    rng = np.random.default_rng(5)
    for _ in range(8):
        off = torch.from_numpy(rng.integers(-100, T + 100, n + 1).astype(np.int32)).cuda()
        area = torch.full((T + 200, H, D), SENT, device="cuda").bfloat16()
        run(moe, q, c, [0] * n, off, out=area[100:100 + T])
        assert bool((area[:100] == SENT).all()) and bool((area[100 + T:] == SENT).all())
        moe.kv4_append(x[0], x[1], c.bytes, c.pages, c.kv_len, T, Hkv, D, page, c.n_pages, c.max_pages,
                       q_off=off, n_seq=n)
        assert torch.equal(c.bytes[~own], held[~own])
        c.bytes.copy_(held)
    new = [10] * n
    off, o = batch(new, c)
    check(run(moe, q, c, new, off), q, c, o)


@pytest.mark.parametrize("H,Hkv,D,new,have", [
    (1024, 1024, 64, [1], [20]), (1024, 1, 64, [2, 1], [70, 300]), (1024, 1, 128, [1], [40]),
    (1024, 64, 128, [1, 1], [90, 3]), (1008, 63, 64, [2], [33])])
def test_most_heads(moe, H, Hkv, D, new, have):
    """As many query heads as a call takes, each with its own KV head or all with one."""
    g = gen(22)
    c = ref.Cache(g, have, Hkv, D, 16)
    off, o = batch(new, c)
    q = randn(g, o[-1], H, D).bfloat16()
    check(run(moe, q, c, new, off), q, c, o)


def test_most_sequences(moe):
    """65535 sequences of one token each, appended and attended: each sees itself alone."""
    g = gen(23)
    n, H, D, page = 65535, 2, 64, 16
    pages = torch.randperm(n, generator=g, device="cuda").to(torch.int32)[:, None].contiguous()
    cache = torch.full((n, moe.kv4_page_bytes(page, 1, D)), 255, dtype=torch.uint8, device="cuda")
    length = torch.ones(n, dtype=torch.int32, device="cuda")
    x = randn(g, 2, n, 1, D).bfloat16()
    moe.kv4_append(x[0], x[1], cache, pages, length, n, 1, D, page, n, 1)
    q = randn(g, n, H, D).bfloat16()
    out = torch.empty_like(q)
    need = moe.kv4_workspace(n, n, H, 1, D, page, 1)
    work = torch.empty(need, dtype=torch.uint8, device="cuda") if need else None
    moe.kv4_attention(q, cache, pages, length, n, H, 1, D, page, n, 1, out, work)
    v = ref.values(*ref.quantise(x[1].float())).expand(n, H, D)
    # weight 1, so step c rounds as in attend's bound; V and the result round once
    least = v.amin(2, keepdim=True)
    tol = (2.0 ** -10 + 2.0 ** -8) * v.abs() * 1.01 + 2.0 ** -11 * (v - least) + 2.0 ** -24
    assert bool(((out.double() - v).abs() <= tol).all())
