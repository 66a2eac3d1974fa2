"""Attention over the 4-bit cache where values differ in size: a row's result must
not depend on what it does not see, nor lose bits to what hardly counts.  The bound
here (`close`) counts each token's error with that token's own weight, and only
the tokens that the row sees."""
import math

import pytest
import torch

import attend_ref as ref
from test_gpu_attend import batch, gen, randn, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    import expert_routing_grouped_gb300 as m
    return m


def held(c, s, which):
    """(lo, step code) of a sequence's tokens as the cache holds them, f64 [n][Hkv][D]."""
    n, P = c.have[s], c.page
    pos = torch.arange(n, device="cuda")
    page = c.pages[s].long()[pos // P]
    codes, scale = c.part(which)
    b = codes[page, :, pos % P]
    b = torch.stack([b & 15, b >> 4], -1).flatten(-2).double().unflatten(-1, (-1, ref.GROUP))
    sc = scale[page, :, pos % P].contiguous().view(torch.float16).double().unflatten(-1, (-1, 2))
    lo = sc[..., 1:].expand(b.shape)
    return lo.flatten(-2), (sc[..., :1] * b).flatten(-2), sc[..., 0]


def close(out, q, c, s, scale=None, softcap=0.0, window=0, causal=True):
    """The rows q [n][H][D] of sequence s against the definition in 64 bits.

    A score of token j is off by e_j: sums of 16 products that truncate (2^-23 of what
    they hold), the exponent's argument (2^-20 of 1 + |score|), with more than 16
    columns the keys' rounding to float16 (2^-11).  Weights off by e_j move the
    result by sum p_j (e^e_j - 1) (|V_j| + |out|).  With at most 16 columns w step is
    rounded (2^-11 of what it adds, and 2^-32 of the largest product where it is
    small); with more w and V are, w to no less than 2^-25 of the largest.  Then f32
    sums and the result's own rounding."""
    n, H, D = q.shape
    G = H // c.Hkv
    few = n * G <= 16
    L = c.have[s]
    scale = D ** -0.5 if scale is None else scale
    klo, kst, _ = held(c, s, 0)
    vlo, vst, vstep = held(c, s, 1)
    pos = (L - n + torch.arange(n, device="cuda"))[:, None]
    key = torch.arange(L, device="cuda")
    see = key <= pos if causal else torch.ones(n, L, dtype=torch.bool, device="cuda")
    if window:
        see = see & (key > pos - window)
    for h in range(H):
        i = h // G
        K, V = (klo + kst)[:, i], (vlo + vst)[:, i]
        kabs, vabs = (klo.abs() + kst)[:, i], (vlo.abs() + vst)[:, i]
        qh = q[:, h].double()
        x = qh @ K.t() * scale
        if softcap:
            x = softcap * torch.tanh(x / softcap)
        p = torch.softmax(torch.where(see, x, torch.full_like(x, -math.inf)), 1)
        y = p @ V
        e = (D / 8 + 16) * 2.0 ** -23 * (qh.abs() @ kabs.t()) * abs(scale) + 2.0 ** -20 * (1 + x.abs())
        if not few:
            e = e + 2.0 ** -11 * (qh.abs() @ K.abs().t()) * abs(scale)
        move = p * torch.expm1(e) * 1.05
        bound = move @ V.abs() + move.sum(1, keepdim=True) * y.abs()
        sums = (L / 8 + 64) * 2.0 ** -23
        if few:
            most = (p[:, :, None] * vstep[:, i]).amax(1).repeat_interleave(ref.GROUP, 1)
            bound = bound + 2.0 ** -11 * (p @ vst[:, i]) + L * 15 * 2.0 ** -32 * most + sums * (p @ vabs)
        else:
            least = torch.minimum(p, 2.0 ** -25 * p.amax(1, keepdim=True))
            bound = bound + (2.0 ** -10 + sums) * (p @ V.abs()) + least @ V.abs()
        bound = bound + sums * y.abs()
        tol = bound + ref.half_step(torch.bfloat16) * (y.abs() + bound) + 2.0 ** -133
        d = (out[:, h].double() - y).abs()
        assert bool((d <= tol).all()), (h, float((d / tol).max()), float(((out[:, h].double() - y).norm() / y.norm())))


def put_row(c, s, token, k, v):
    """One token's K and V, [Hkv][D] each."""
    for which, x in ((0, k), (1, v)):
        if x is not None:
            c.put(s, which, token, x[None])


@pytest.mark.parametrize("ratio", [1e-2, 1e-3, 1e-5])
@pytest.mark.parametrize("n,H", [(1, 4), (3, 4), (1, 12), (9, 4)])
@pytest.mark.parametrize("have", [70, 5000])
def test_halves_of_different_size(moe, have, n, H, ratio):
    """The second 64 dimensions of V much smaller than the first, and the other way round."""
    g = gen(31)
    c = ref.Cache(g, [have], 2, 128, 64)
    size = torch.tensor([[300.0, 300 * ratio], [300 * ratio, 300.0]], device="cuda").repeat_interleave(64, 1)
    c.put(0, 1, 0, randn(g, have, 2, 128) * size)
    q = (1.5 * randn(g, n, 2 * H, 128)).bfloat16()
    off, _ = batch([n], c)
    close(run(moe, q, c, [n], off), q, c, 0)


@pytest.mark.parametrize("size", [1.0, 0.02, 1e-3])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,H", [(1, 4), (2, 2), (3, 5), (7, 4)])
@pytest.mark.parametrize("where", ["window", "window edge", "causal", "far", "far late"])
def test_one_huge_token(moe, where, n, H, D, size):
    """A token whose V is at the cache's limit: outside the window of all rows or of
    all but the first, hidden from all rows but the last, or seen with hardly any weight."""
    g = gen(32)
    have, window = 3000, 1000
    c = ref.Cache(g, [have], 1, D, 16)
    c.put(0, 1, 0, size * randn(g, have, 1, D))
    q = (1.5 * randn(g, n, H, D)).bfloat16()
    huge = size * randn(g, 1, D)
    huge[0, 5::7] = float("inf")
    huge[0, 6::7] = -1e30
    kw = dict(window=window) if where.startswith("window") else {}
    token = {"window": have - n - window, "window edge": have - n - window + 1, "causal": have - 1, "far": 5,
             "far late": 2000}[where]
    k = None
    if where.startswith("far"):   # a score of about -45
        q = q.abs()
        k = torch.full((1, D), -45 * D ** 0.5 / float(q.float().sum(2).mean()), device="cuda")
    put_row(c, 0, token, k, huge)
    off, _ = batch([n], c)
    close(run(moe, q, c, [n], off, **kw), q, c, 0, **kw)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,H", [(1, 4), (2, 7), (5, 4)])
@pytest.mark.parametrize("rise", [0.0, 0.4, -0.4])
def test_maximum_that_moves(moe, rise, n, H, D):
    """Scores that rise or fall by far more than a step over the tokens while V's size
    goes the other way, and a first token with all the weight and V = 0."""
    g = gen(33)
    have = 700
    c = ref.Cache(g, [have], 1, D, 32)
    at = torch.arange(have, device="cuda")
    q = (1.5 * randn(g, n, H, D)).bfloat16().abs()
    mean = float(q.float().sum(2).mean())
    # token t scores about rise t
    c.put(0, 0, 0, (randn(g, have, 1, D) * 0.3 + (rise * at * D ** 0.5 / mean)[:, None, None]))
    c.put(0, 1, 0, randn(g, have, 1, D) * torch.exp(-rise / 4 * (at - have / 2))[:, None, None].clamp(1e-3, 1e4))
    if rise == 0:
        put_row(c, 0, 0, torch.full((1, D), 30 * D ** 0.5 / mean, device="cuda"), torch.zeros(1, D, device="cuda"))
    off, _ = batch([n], c)
    close(run(moe, q, c, [n], off), q, c, 0)


@pytest.mark.parametrize("softcap,scale", [
    (5.0, 0.1), (30.0, 0.1), (30.0, 2.0), (1e3, 0.1), (1e3, 20.0), (1e4, 0.1), (1e5, 0.1), (1e6, 0.1), (1e6, 8.0),
    (1e9, 0.1), (1e20, 0.1), (1e30, 0.1), (1e38, 0.1), (3e38, 0.1), (1e-3, 0.1)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,H", [(1, 4), (3, 4), (9, 4)])
def test_caps_of_any_size(moe, n, H, D, softcap, scale):
    """A cap costs a score 2^-20 of itself, not of the cap: one far above all scores
    changes nothing that counts."""
    g = gen(34)
    c = ref.Cache(g, [300], 1, D, 16)
    q = (1.5 * randn(g, n, H, D)).bfloat16()
    off, _ = batch([n], c)
    kw = dict(softcap=softcap, scale=scale)
    close(run(moe, q, c, [n], off, **kw), q, c, 0, **kw)


def test_append_reads_no_other_rows(moe):
    """Rows in no sequence are not read: with 70 rows of 2^20 in sequences the call takes
    less time than the memory needs to read all 8.6 GB (1.09 ms at the 7.9 TB/s that it
    is rated for)."""
    g = gen(35)
    T, Hkv, D, page = 1 << 20, 8, 128, 16
    have, new = [50, 40, 1], [40, 29, 1]
    c = ref.Cache(g, have, Hkv, D, page)
    want = c.bytes.clone()
    k, v = torch.empty(2, T, Hkv, D, device="cuda")
    off = torch.tensor([1000, 1040, 1069, 1070], dtype=torch.int32, device="cuda")
    k[1000:1070], v[1000:1070] = randn(g, 2, 70, Hkv, D)
    best = math.inf
    for _ in range(5):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        moe.kv4_append(k, v, c.bytes, c.pages, c.kv_len, T, Hkv, D, page, c.n_pages, c.max_pages, q_off=off,
                       n_seq=3, dtype=0)
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b))
    got, c.bytes = c.bytes, want
    at = 1000
    for s in range(3):
        for which, x in ((0, k), (1, v)):
            c.put(s, which, have[s] - new[s], x[at:at + new[s]])
        at += new[s]
    assert torch.equal(got, want)
    assert best < 1.0, best
