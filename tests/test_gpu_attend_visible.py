"""Attention over the 4-bit cache: which tokens each row sees, exactly, at the lengths
where keys are cut into spans and parts and rings and page look-ahead come round.

With scale 0 all scores are 0, so a row's result is the mean of V over what it sees.
V is 15 in dimension (j // 64) mod D of token j and 0 elsewhere (lo 0, step 1, code 15:
exact), so that 15 count / n counts the tokens seen of every block of 64.  What rounds
is the mean, to bf16 (2^-8), and f32 sums of whole numbers ((L / 8 + 64) 2^-23): under
0.55 of a token where two blocks share a dimension, so one lost or met twice shows."""
import pytest
import torch

import attend_ref as ref
from test_gpu_attend import batch, gen, randn, run
from test_gpu_attend_edges import close

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    import expert_routing_grouped_gb300 as m
    return m


# heads, KV heads, new rows and lengths: at most 16 columns, more, and both
CASES = [
    (8, 2, [1], [8100]), (4, 1, [1, 2, 4], [5000, 300, 4097]), (12, 1, [1], [7000]), (3, 3, [1, 1], [4160, 2047]),
    (8, 2, [40], [6000]), (16, 1, [9, 3], [5000, 4500]), (4, 2, [300], [4100]), (32, 1, [1, 1], [3000, 8000]),
    (8, 2, [1, 20, 2, 70], [4097, 5000, 2600, 3000]),
]
MASKS = [(0, True), (700, True), (3000, True), (0, False), (1000, False), (33, True)]


def counting_cache(g, have, Hkv, D, page):
    c = ref.Cache(g, have, Hkv, D, page)
    for s, n in enumerate(have):
        v = torch.zeros(n, Hkv, D, device="cuda")
        at = torch.arange(n, device="cuda")
        v[at, :, (at // 64) % D] = 15
        # rows of zeros in the other group: lo 0, step 0
        assert torch.equal(c.put(s, 1, 0, v), v.double())
    return c


def seen_by(n, L, window, causal):
    pos = (L - n + torch.arange(n, device="cuda"))[:, None]
    key = torch.arange(L, device="cuda")
    see = key <= pos if causal else torch.ones(n, L, dtype=torch.bool, device="cuda")
    if window:
        see = see & (key > pos - window)
    return see


def check_counts(out, see, D, bad=None):
    """out [n][heads][D] of rows that see [n][L]; bad [n]: rows that have to be NaN."""
    n, L = see.shape
    block = torch.nn.functional.one_hot((torch.arange(L, device="cuda") // 64) % D, D).double()
    count, total = see.double() @ block, see.sum(1, keepdim=True).double()
    got = out.double() * total[:, None] / 15
    if bad is not None:
        assert bool(out[bad].isnan().all()) and bool(out[~bad].isfinite().all())
        got, count = got[~bad], count[~bad]
    tol = (2.0 ** -8 * 1.01 + (L / 8 + 64) * 2.0 ** -23) * count
    assert float(tol.max() if tol.numel() else 0) < 0.55   # of a token
    assert bool(((got - count[:, None]).abs() <= tol[:, None]).all()), float((got - count[:, None]).abs().max())


@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("window,causal", MASKS)
@pytest.mark.parametrize("H,Hkv,new,have", CASES)
def test_seen_tokens_counted(moe, H, Hkv, new, have, window, causal, D, page):
    g = gen(51)
    c = counting_cache(g, have, Hkv, D, page)
    off, o = batch(new, c)
    q = randn(g, o[-1], H, D).bfloat16()
    for cap in (0.0, 20.0, 1e4):
        out = run(moe, q, c, new, off, window=window, causal=causal, scale=0.0, softcap=cap)
        for s, n in enumerate(new):
            check_counts(out[o[s]:o[s + 1]], seen_by(n, have[s], window, causal), D)


@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("window,causal", [(0, True), (1500, True), (0, False)])
@pytest.mark.parametrize("H,Hkv,new,have", CASES)
def test_holes_far_from_the_start(moe, H, Hkv, new, have, window, causal, D, page):
    """Pages without a place, one and two in a row, past the first turn of every ring."""
    g = gen(52)
    c = counting_cache(g, have, Hkv, D, page)
    off, o = batch(new, c)
    q = randn(g, o[-1], H, D).bfloat16()
    ids = [-1, c.n_pages, 2 ** 31 - 1, -2 ** 31]
    gone = []
    for s, n in enumerate(have):
        lost = torch.zeros(n, dtype=torch.bool, device="cuda")
        for i, token in enumerate((5, 1040, 1090, 1110, 2064, 2500, 2560, 2999, n - 1 - page)):
            if 0 <= token < n:
                first = token // page
                c.pages[s, first] = ids[i % 4]
                lost[first * page:(first + 1) * page] = True
        gone.append(lost)
    out = run(moe, q, c, new, off, window=window, causal=causal, scale=0.0)
    for s, n in enumerate(new):
        check_counts(out[o[s]:o[s + 1]], seen_by(n, have[s], window, causal) & ~gone[s], D)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("window", [0, 40, 900])
@pytest.mark.parametrize("H,Hkv,new,have", CASES)
def test_nan_far_from_the_start(moe, H, Hkv, new, have, window, D):
    """Tokens with a NaN in K or V of the last KV head: the rows that see one are NaN
    there, all others count what they see."""
    g = gen(53)
    page = 32
    c = counting_cache(g, have, Hkv, D, page)
    off, o = batch(new, c)
    q = randn(g, o[-1], H, D).bfloat16()
    x = torch.zeros(1, Hkv, D, device="cuda")
    x[0, -1, D - 1] = float("nan")
    places = [[], [3], [n_ for n_ in (1040, 2065)], [2999]]
    for s, n in enumerate(have):
        at = [t for t in places[(s + 2) % 4] if t < n - 1] + [n - new[s] - 30]
        nan = torch.zeros(n, dtype=torch.bool, device="cuda")
        for i, t in enumerate(at):
            if t >= 0:
                keep = c.part(i % 2)[0].clone(), c.part(i % 2)[1].clone()
                c.put(s, i % 2, t, x)
                # only the last head's token: the others' codes and scales come back
                for part, was in zip(c.part(i % 2), keep):
                    part[:, :-1] = was[:, :-1]
                nan[t] = True
        c.nan = getattr(c, "nan", []) + [nan]
    out = run(moe, q, c, new, off, window=window, scale=0.0)
    G = H // Hkv
    for s, n in enumerate(new):
        see = seen_by(n, have[s], window, True)
        bad = (see & c.nan[s]).any(1)
        rows = out[o[s]:o[s + 1]]
        check_counts(rows[:, H - G:], see, D, bad)
        if G < H:
            check_counts(rows[:, :H - G], see, D)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("window,causal,softcap", [(0, True, 0.0), (700, True, 0.0), (3000, True, 30.0),
                                                   (0, False, 0.0), (1000, False, 100.0)])
@pytest.mark.parametrize("H,Hkv,new,have", CASES)
def test_weights_at_length(moe, H, Hkv, new, have, window, causal, softcap, D):
    """Scores that differ, under the bound that counts each token with its own weight."""
    g = gen(54)
    c = ref.Cache(g, have, Hkv, D, 64)
    off, o = batch(new, c)
    q = (1.5 * randn(g, o[-1], H, D)).bfloat16()
    kw = dict(window=window, causal=causal, softcap=softcap)
    out = run(moe, q, c, new, off, **kw)
    for s in range(len(new)):
        close(out[o[s]:o[s + 1]], q[o[s]:o[s + 1]], c, s, **kw)


def test_one_long_among_many_sequences(moe):
    """More sequences than a block looks over at its start: the long one's every token."""
    g = gen(55)
    H, Hkv, D, page = 4, 2, 64, 16
    have = [1 + i % 40 for i in range(1100)]
    have[700], have[3] = 8000, 2500
    c = counting_cache(g, have, Hkv, D, page)
    q = randn(g, len(have), H, D).bfloat16()
    out = run(moe, q, c, have, scale=0.0)
    for s in [0, 1, 2, 3, 4, 699, 700, 701, 1098, 1099]:
        check_counts(out[s:s + 1], seen_by(1, have[s], 0, True), D)
