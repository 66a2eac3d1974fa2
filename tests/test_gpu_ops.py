"""The dense operators on the GPU against their 64-bit forms (ops_ref.py).

Tolerances come from the arithmetic: a rounding to type t is off by at most
half a step, eps(t) / 2 of the value; what f32 sums may add is derived beside
each check."""
import ctypes

import numpy as np
import pytest
import torch

import ops_ref as ref

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn
DT = {0: torch.float32, 1: torch.bfloat16, 2: E4M3}
F32, BF16 = 0, 1
SENT = 72.0   # fills what a call must leave alone (exact in every type)


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


def strided(t, extra):
    """t as the first columns of wider rows filled with SENT."""
    if not extra:
        return t
    full = torch.full((t.shape[0], t.shape[1] + extra), SENT, device=t.device).to(t.dtype)
    full[:, :t.shape[1]] = t
    return full[:, :t.shape[1]]


def padding_untouched(t, extra):
    if extra:
        full = t.as_strided((t.shape[0], t.stride(0)), (t.stride(0), 1)) if t.shape[0] > 1 else None
        if full is not None:   # the last row's padding lies past the view
            assert bool((full[:-1, t.shape[1]:].float() == SENT).all())


# ------------------------------------------------------------ add_rmsnorm --

# Row statistics: a sum of H squares in f32, at most 32 fmaf in a thread, 5
# shuffle levels and 32 warps: under 128 units of 2^-24, halved by the root;
# the root, the division, gain and product add under 16.
STAT = 96 * 2.0 ** -24


def run_norm(moe, x, resid, gain, out_dtype, group, eps=1e-6, extra=0, in_place=False, stream=None):
    T, H = x.shape
    code = {torch.float32: 0, torch.bfloat16: 1}
    out = strided(torch.full((T, H), SENT, device="cuda").to(DT[out_dtype]), extra)
    gs = group or H
    scale = torch.full((T, H // gs), SENT, device="cuda") if out_dtype == 2 else None
    rout = None
    if resid is not None:
        rout = resid if in_place else strided(torch.full((T, H), SENT, device="cuda").to(resid.dtype), extra)
    st = lambda t: 0 if t is None else t.stride(0)  # noqa: E731
    moe.add_rmsnorm(x, T, H, eps, out, resid=resid, resid_out=rout, gain=gain, scale=scale,
                    group=group, x_dtype=code[x.dtype],
                    resid_dtype=0 if resid is None else code[resid.dtype], out_dtype=out_dtype,
                    x_stride=st(x), resid_stride=st(resid), resid_out_stride=st(rout),
                    out_stride=st(out), stream=stream)
    return out, scale, rout


def check_norm(x, resid, gain, out, scale, rout, out_dtype, group, eps=1e-6):
    H = x.shape[1]
    n, new, sc = ref.norm(x, resid, gain, eps, (group or H) if out_dtype == 2 else None)
    if resid is not None:
        assert torch.equal(rout, new)
    if out_dtype == 1:
        tol = (ref.half_step(torch.bfloat16) + STAT) * n.abs() + 2.0 ** -133
        assert bool(((out.double() - n).abs() <= tol).all())
        return
    assert bool(((scale.double() - sc).abs() <= STAT * sc).all())
    q = out.double().view(n.shape[0], -1, group or H)
    v = n.view_as(q) / scale.double()[:, :, None]
    # half a step of a normal, or of the subnormals below 2^-6 (steps of 2^-9)
    tol = torch.clamp(2.0 ** -4 * v.abs(), min=2.0 ** -10) + 2 * STAT * v.abs()
    assert bool(((q - v).abs() <= tol).all())


@pytest.mark.parametrize("T,H", [(1, 16), (3, 32), (1, 6144), (5, 2048), (7, 4096 + 16), (2, 8192),
                                 (3, 8192 + 48), (2, 20000), (1, 32768), (333, 512)])
@pytest.mark.parametrize("xt,rt", [(0, 0), (1, 0), (0, 1), (1, 1), (0, None), (1, None)])
@pytest.mark.parametrize("out_dtype", [1, 2])
def test_add_rmsnorm(moe, T, H, xt, rt, out_dtype):
    g = gen(T * 7 + H)
    x = (3 * randn(g, T, H)).to(DT[xt])
    resid = None if rt is None else (5 * randn(g, T, H)).to(DT[rt])
    gain = 1 + 0.3 * randn(g, H) if (T + H) % 2 else None
    out, scale, rout = run_norm(moe, x, resid, gain, out_dtype, 0)
    check_norm(x, resid, gain, out, scale, rout, out_dtype, 0)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("T,H", [(1, 128), (4, 1024 + 128), (9, 6144), (2, 12800), (1, 32768)])
def test_add_rmsnorm_groups(moe, group, T, H):
    g = gen(group + H)
    x = randn(g, T, H).bfloat16()
    # groups of very different sizes, one of them zero
    resid = randn(g, T, H) * torch.exp(4 * randn(g, H // group)).repeat_interleave(group)
    x[0, :group] = 0
    resid[0, :group] = 0
    gain = randn(g, H)
    out, scale, rout = run_norm(moe, x, resid, gain, 2, group)
    check_norm(x, resid, gain, out, scale, rout, 2, group)
    assert float(scale[0, 0]) == 2.0 ** -126 and bool((out[0, :group].float() == 0).all())


@pytest.mark.parametrize("out_dtype,group", [(1, 0), (2, 0), (2, 64)])
def test_add_rmsnorm_strides_in_place_and_untouched(moe, out_dtype, group):
    g = gen(3)
    T, H = 6, 704
    x = strided(randn(g, T, H).bfloat16(), 40)
    resid = strided(randn(g, T, H), 12)
    before = resid.clone()
    out, scale, rout = run_norm(moe, x, resid, None, out_dtype, group, extra=64, in_place=True)
    check_norm(x, before, None, out, scale, rout, out_dtype, group)
    padding_untouched(out, 64)
    padding_untouched(resid, 12)
    out2, scale2, rout2 = run_norm(moe, x, before, None, out_dtype, group, extra=64)
    padding_untouched(rout2, 64)
    assert torch.equal(out.float(), out2.float()) and torch.equal(rout, rout2)


def test_add_rmsnorm_matches_plain_norm(moe):
    """Without residual and gain it is moe_rmsnorm_bf16's formula."""
    g = gen(5)
    x = randn(g, 9, 6144)
    a, _, _ = run_norm(moe, x, None, None, 1, 0)
    b = torch.empty(9, 6144, dtype=torch.bfloat16, device="cuda")
    moe.rmsnorm_bf16(x, 9, 6144, 1e-6, b)
    # the two sum in different orders: at most one bf16 step apart, rarely
    d = (a.float() - b.float()).abs()
    assert bool((d <= 2.0 ** -7 * b.float().abs()).all())
    assert float((d > 0).float().mean()) < 0.01


@pytest.mark.parametrize("group", [0, 32])
def test_add_rmsnorm_nonfinite_rows(moe, group):
    """NaN and infinity stay in their rows; zeros and the smallest normals work."""
    H = 512
    x = randn(gen(9), 6, H)
    x[1, 40] = float("nan")
    x[2, 50] = float("inf")
    x[3] = 0
    x[4] = 2.0 ** -126
    out, scale, _ = run_norm(moe, x, None, None, 2, group)
    o = out.float()
    assert bool(o[1].isnan().all()) and bool(scale[1].isnan().all())
    hit = slice(0, H) if group == 0 else slice(32, 64)   # infinity times 0, in its group
    assert bool(o[2, hit].isnan().all())
    rest = torch.cat([o[2, :hit.start], o[2, hit.stop:]])
    assert bool((rest == 0).all())
    assert bool((o[3] == 0).all()) and bool((scale[3] == 2.0 ** -126).all())
    fine = [0, 4, 5]
    check_norm(x[fine], None, None, out[fine], scale[fine], None, 2, group)


# ------------------------------------------------------------------ linear --

def make_linear(g, T, K, N, dtype, act, out_dtype, bias, resid):
    rows = 2 * N if act == 3 else N
    x, w = randn(g, T, K), randn(g, rows, K) / K ** 0.5
    sx = sw = None
    if dtype == 2:
        sx = x.abs().amax(1) / 448
        sw = w.abs().amax(1) / 448
        x, w = x / sx[:, None], w / sw[:, None]
    x, w = x.to(DT[dtype]), w.to(DT[dtype])
    b = randn(g, rows) if bias else None
    r = (2 * randn(g, T, N)).to(DT[out_dtype]) if resid else None
    return x, w, sx, sw, b, r


def run_linear(moe, x, w, sx, sw, b, r, N, dtype, out_dtype, act, extra=0, in_place=False,
               stream=None, out=None):
    T, K = x.shape
    if out is None:
        out = r if in_place else strided(torch.full((T, N), SENT, device="cuda").to(DT[out_dtype]), extra)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    moe.linear(x, w, T, N, K, out, dtype=dtype, out_dtype=out_dtype, act=act, x_scale=sx,
               w_scale=sw, bias=b, resid=r, x_stride=x.stride(0), w_stride=w.stride(0),
               resid_stride=0 if r is None else r.stride(0), out_stride=out.stride(0),
               status=status, stream=stream)
    return out, status


def check_linear(out, status, x, w, sx, sw, b, r, N, act, resid=None):
    y, err = ref.linear(x, w, N, act, sx, sw, b, r if resid is None else resid)
    tol = err + ref.half_step(out.dtype) * (y.abs() + err) + 2.0 ** -133
    bad = ((out.double() - y).abs() > tol)
    assert int(status) == 0
    assert not bool(bad.any()), (int(bad.sum()), float(((out.double() - y).abs() / tol).max()))


SHAPES = [(1, 8, 1), (1, 512, 64), (2, 48, 7), (3, 6144, 256), (7, 1040, 33), (8, 4096, 100),
          (9, 256, 130), (16, 2064, 257), (17, 512, 48), (31, 14336, 96), (32, 72, 1000),
          (33, 640, 129), (64, 2048, 65), (65, 1024, 384), (127, 136, 255), (128, 512, 128),
          (129, 2056, 640), (200, 1000, 511), (256, 64, 2048), (257, 4096, 136), (300, 24, 1111),
          (512, 768, 1024), (1000, 520, 320), (1537, 256, 777), (2048, 1024, 2064)]


@pytest.mark.parametrize("dtype", [1, 2])
@pytest.mark.parametrize("T,K,N", SHAPES)
def test_linear_shapes(moe, T, K, N, dtype):
    if dtype == 2:
        K = (K + 15) // 16 * 16
    g = gen(T + K + N)
    x, w, sx, sw, b, r = make_linear(g, T, K, N, dtype, 0, 0, False, False)
    out, status = run_linear(moe, x, w, sx, sw, b, r, N, dtype, 0, 0)
    check_linear(out, status, x, w, sx, sw, b, r, N, 0)


@pytest.mark.parametrize("dtype", [1, 2])
@pytest.mark.parametrize("out_dtype", [0, 1])
@pytest.mark.parametrize("act", [0, 1, 2, 3])
@pytest.mark.parametrize("bias,resid", [(False, True), (True, False), (True, True)])
@pytest.mark.parametrize("T", [1, 5, 16, 40, 130, 700])
def test_linear_epilogues(moe, T, dtype, out_dtype, act, bias, resid):
    K, N = 528, 208
    g = gen(100 + T + act)
    x, w, sx, sw, b, r = make_linear(g, T, K, N, dtype, act, out_dtype, bias, resid)
    out, status = run_linear(moe, x, w, sx, sw, b, r, N, dtype, out_dtype, act)
    check_linear(out, status, x, w, sx, sw, b, r, N, act)


@pytest.mark.parametrize("dtype", [1, 2])
@pytest.mark.parametrize("T,act", [(4, 0), (4, 3), (50, 2), (50, 3), (400, 0), (400, 3)])
def test_linear_strides_in_place_and_untouched(moe, T, act, dtype):
    K, N = 400, 144
    g = gen(T + act)
    x, w, sx, sw, b, r = make_linear(g, T, K, N, dtype, act, 0, True, True)
    x, w, r = strided(x, 48), strided(w, 16), strided(r, 3)
    before = r.clone()
    out, status = run_linear(moe, x, w, sx, sw, b, r, N, dtype, 0, act, in_place=True)
    check_linear(out, status, x, w, sx, sw, b, r, N, act, resid=before)
    padding_untouched(out, 3)
    # out of place onto rows of another stride: the same values
    other, status = run_linear(moe, x, w, sx, sw, b, before, N, dtype, 0, act, extra=5)
    padding_untouched(other, 5)
    assert torch.equal(other, out)


@pytest.mark.parametrize("T,N", [(1, 4096), (6, 512), (100, 256), (600, 512)])
def test_linear_repeats_bitwise_and_rows_do_not_mix(moe, T, N):
    """The same bits on every call; a NaN row of x or w stays in its row or column."""
    g = gen(T)
    x, w, sx, sw, b, r = make_linear(g, T, 1024, N, 1, 0, 0, False, False)
    a, _ = run_linear(moe, x, w, None, None, None, None, N, 1, 0, 0)
    for _ in range(3):
        c, _ = run_linear(moe, x, w, None, None, None, None, N, 1, 0, 0)
        assert torch.equal(a, c)
    w[N // 2, 7] = float("nan")
    if T > 1:
        x[T // 2, 9] = float("inf")
    c, _ = run_linear(moe, x, w, None, None, None, None, N, 1, 0, 0)
    keep_r = torch.arange(T, device="cuda") != (T // 2 if T > 1 else -1)
    keep_c = torch.arange(N, device="cuda") != N // 2
    assert bool(c[:, N // 2].isnan().all())
    assert torch.equal(c[keep_r][:, keep_c], a[keep_r][:, keep_c])
    if T > 1:
        assert not bool(c[T // 2].isfinite().any())


# ------------------------------------------------------------ balance loss --

def run_balance(moe, z, idx, bias, mask, off, k, mode, alpha=0.01, grad=None, want_dz=True,
                extra=0, in_place=False, stream=None):
    T, E = z.shape
    S = 1 if off is None else len(off) - 1
    f = dict(device="cuda")
    loss, prob = torch.full((S,), SENT, **f), torch.full((S, E), SENT, **f)
    counts = torch.full((S, E), 77, dtype=torch.int32, **f)
    tokens = torch.full((S,), 77, dtype=torch.int32, **f)
    dz = None
    if want_dz:
        dz = z if in_place else strided(torch.full((T, E), SENT, **f).to(z.dtype), extra)
    ws = torch.empty(moe.balance_workspace(T, E, S), dtype=torch.uint8, **f)
    moe.balance_loss(z, idx, T, E, k, loss, counts, tokens, prob, ws, bias=bias, mask=mask,
                     seq_off=off, n_seq=S, z_dtype=0 if z.dtype == torch.float32 else 1,
                     router_mode=mode, alpha=alpha, dz=dz, grad=grad, z_stride=z.stride(0),
                     dz_stride=0 if dz is None else dz.stride(0), stream=stream)
    return loss, counts, tokens, prob, dz


def check_balance(got, z, idx, bias, mask, off, k, mode, alpha=0.01, grad=None):
    loss, counts, tokens, prob, dz = got
    T, E = z.shape
    rl, rc, rt, rp, rdz, size = ref.balance(z, idx, bias, mask, off, k, mode, alpha, grad)
    assert torch.equal(counts.cpu().long(), rc) and torch.equal(tokens.cpu().long(), rt)
    # p: expf (2 units), the rounding of z + bias and of z - max (units of
    # 2^-24 times their size, taken as absolute errors of the exponent), a
    # positive sum of E terms over 32 slots and 5 levels, a division; mean:
    # positive sums: at most T / 8 rows in a warp, then under 64 partials.
    fin = z.cpu().double()
    big = float(fin[fin.abs() < 1e30].abs().max()) + (0 if bias is None else float(bias.abs().max()))
    rel = (4 * big + 64) * 2.0 ** -24
    srel = rel + (T / 8 + 64) * 2.0 ** -24
    assert bool(((prob.cpu().double() - rp).abs() <= srel * rp + 1e-37).all())
    assert bool(((loss.cpu().double() - rl).abs() <= (srel + E / 32 * 2.0 ** -24) * rl.abs() + 1e-37).all())
    if dz is None:
        return
    inside = torch.zeros(T, dtype=torch.bool)
    for s, rows in ref.segments(T, off, None):
        inside[rows] = True
    d = dz.cpu().double()
    assert bool((d[~inside] == SENT).all())
    tol = 4 * rel * size + ref.half_step(z.dtype) * rdz.abs() + 1e-37
    assert bool(((d - rdz).abs() <= tol)[inside].all())


def make_balance(g, T, E, k, dtype, S=1, mask=False):
    z = (1.5 * randn(g, T, E) + randn(g, E)).to(DT[dtype])
    idx = torch.topk(z.float(), k, dim=1).indices.to(torch.int32)
    off = None
    if S > 1:
        cut = np.sort(np.random.RandomState(T + S).randint(0, T + 1, S + 1))
        off = torch.tensor(cut, dtype=torch.int32, device="cuda")
    m = (torch.rand(T, generator=g, device="cuda") < 0.8).to(torch.uint8) if mask else None
    return z, idx, off, m


@pytest.mark.parametrize("mode", [0, 1, 2])
@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("T,E,k,S,mask", [
    (1, 1, 1, 1, False), (1, 8, 2, 1, False), (2, 64, 8, 1, True), (33, 60, 4, 1, False),
    (100, 7, 3, 5, True), (257, 256, 8, 1, True), (600, 160, 6, 9, True), (500, 1024, 16, 3, False),
    (3000, 33, 2, 40, True), (5001, 128, 8, 2, False), (64, 500, 32, 64, True)])
def test_balance(moe, T, E, k, S, mask, dtype, mode):
    g = gen(T + E)
    z, idx, off, m = make_balance(g, T, E, k, dtype, S, mask)
    bias = 0.3 * randn(g, E) if E % 2 == 0 else None
    grad = randn(g, S) if T % 2 else None
    got = run_balance(moe, z, idx, bias, m, off, k, mode, grad=grad)
    check_balance(got, z, idx, bias, m, off, k, mode, grad=grad)
    plain = run_balance(moe, z, idx, bias, m, off, k, mode, want_dz=False)
    for a, b in zip(got[:4], plain[:4]):   # with and without a gradient, the same bits
        assert torch.equal(a, b)


@pytest.mark.parametrize("mode", [0, 1])
def test_balance_gradient_against_differences(moe, mode):
    """d loss / d z by central differences of the f64 loss with fixed counts."""
    g = gen(2)
    T, E, k = 12, 16, 3
    z, idx, off, m = make_balance(g, T, E, k, 0)
    bias = 0.5 * randn(g, E)
    dz = run_balance(moe, z, idx, bias, None, None, k, mode)[4].cpu().double()
    zc, b, h = z.cpu().double(), bias.cpu(), 1e-4
    c = torch.bincount(idx.cpu().reshape(-1).long(), minlength=E).double()

    def loss(v):
        return float(0.01 * E / (k * T) * (c * ref.probs(v, b, mode).mean(0)).sum())

    for t, e in [(0, 0), (3, 5), (7, 15), (11, 8)]:
        up, dn = zc.clone(), zc.clone()
        up[t, e] += h
        dn[t, e] -= h
        diff = (loss(up) - loss(dn)) / (2 * h)
        # differences: h^2 / 6 of a third derivative below 0.01 * 16 * 6, and
        # f64 rounding 1e-16 / h; the kernel: f32 units of terms below 0.2
        assert abs(float(dz[t, e]) - diff) < 1e-8 / 6 + 1e-11 + 64 * 2.0 ** -24 * 0.2


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("mode", [0, 1])
def test_balance_masked_values(moe, mode, dtype):
    """Masked experts (-infinity, the lowest value), rows with nothing left,
    dropped slots, and NaN in padding rows."""
    g = gen(8)
    T, E, k = 40, 64, 4
    z, idx, off, m = make_balance(g, T, E, k, dtype)
    m = torch.ones(T, dtype=torch.uint8, device="cuda")
    z[0, 10:20] = float("-inf")
    z[1, 5:] = torch.finfo(z.dtype).min
    z[2] = float("-inf")
    z[3] = torch.finfo(z.dtype).min
    z[4] = float("nan")
    m[4] = 0
    z[5] = float("inf")
    m[5] = 0
    idx[6, 2:] = -1
    idx[7] = -1
    idx[8, 0] = E
    idx[9, 1] = 2 ** 31 - 1
    idx[10, 0] = -2 ** 31
    idx[11] = idx[11, 0]          # the same expert in every slot
    got = run_balance(moe, z, idx, None, m, None, k, mode)
    check_balance(got, z, idx, None, m, None, k, mode)
    dz = got[4].float()
    assert bool((dz[4] == 0).all()) and bool((dz[5] == 0).all()) and bool((dz[2] == 0).all())
    # an unmasked NaN row reaches the loss, as in the formula
    m[4] = 1
    got = run_balance(moe, z, idx, None, m, None, k, mode)
    assert bool(got[0].isnan().all()) and bool(got[4][4].isnan().all())
    assert not bool(got[4][[0, 1, 2, 3] + list(range(6, T))].isnan().any())


def test_balance_everything_masked_and_empty_segments(moe):
    g = gen(4)
    T, E, k = 50, 32, 2
    z, idx, _, _ = make_balance(g, T, E, k, 0)
    m = torch.zeros(T, dtype=torch.uint8, device="cuda")
    loss, counts, tokens, prob, dz = run_balance(moe, z, idx, None, m, None, k, 0)
    assert float(loss) == 0 and int(tokens) == 0 and int(counts.sum()) == 0
    assert bool((prob == 0).all()) and bool((dz == 0).all())
    off = torch.tensor([0, 0, 10, 10, 10, 40, 40], dtype=torch.int32, device="cuda")
    got = run_balance(moe, z, idx, None, None, off, k, 0)
    check_balance(got, z, idx, None, None, off, k, 0)
    assert got[0].cpu().tolist()[0] == 0 and got[2].cpu().tolist() == [0, 10, 0, 0, 30, 0]


def test_balance_strides_in_place_repeats(moe):
    g = gen(6)
    T, E, k = 700, 100, 5
    z, idx, off, m = make_balance(g, T, E, k, 0, 6, True)
    z = strided(z, 28)
    got = run_balance(moe, z, idx, None, m, off, k, 0, extra=3)
    check_balance(got, z, idx, None, m, off, k, 0)
    padding_untouched(got[4], 3)
    # the same call gives the same bits (the odd stride of dz above and rows of
    # whole 16-byte pieces are different variants, which sum in another order)
    for extra in (0, 3):
        once, again = (run_balance(moe, z, idx, None, m, off, k, 0, extra=extra) for _ in range(2))
        check_balance(once, z, idx, None, m, off, k, 0)
        for a, b in zip(once, again):
            assert torch.equal(a, b)
    inside = slice(int(off[0]), int(off[-1]))
    zc = z.clone()
    want = run_balance(moe, zc, idx, None, m, off, k, 0)
    here = run_balance(moe, zc, idx, None, m, off, k, 0, in_place=True)
    for a, b in zip(here[:4], want):
        assert torch.equal(a, b)
    assert torch.equal(here[4][inside], want[4][inside])
    assert torch.equal(zc[:int(off[0])], z[:int(off[0])])


def test_balance_perfectly_even_batch_has_loss_alpha(moe):
    T, E = 64, 16
    z = torch.zeros(T, E, device="cuda")
    idx = (torch.arange(T * 2, device="cuda", dtype=torch.int32) % E).view(T, 2)
    loss, counts, _, _, dz = run_balance(moe, z, idx, None, None, None, 2, 0, alpha=0.5)
    assert abs(float(loss) - 0.5) < 1e-6 and bool((counts == T * 2 // E).all())
    assert bool((dz == 0).all())


# ------------------------------------------------ streams, graphs, together --

def ops_call(moe, s, stream=None):
    run_norm_into = moe.add_rmsnorm
    run_norm_into(s["x"], s["T"], s["H"], 1e-6, s["q"], resid=s["r"], resid_out=s["r2"],
                  gain=s["gain"], scale=s["sc"], x_dtype=1, resid_dtype=0, out_dtype=2, stream=stream)
    moe.linear(s["q"], s["w"], s["T"], s["N"], s["H"], s["h"], dtype=2, out_dtype=0,
               x_scale=s["sc"], w_scale=s["ws"], stream=stream)
    moe.balance_loss(s["h"], s["idx"], s["T"], s["N"], 4, s["loss"], s["counts"], s["tokens"],
                     s["prob"], s["work"], n_seq=1, alpha=0.1, dz=s["dz"], stream=stream)


def ops_state(moe, seed, T=48, H=512, N=64):
    g = gen(seed)
    w = randn(g, N, H)
    f = dict(device="cuda")
    ws = w.abs().amax(1) / 448
    h = torch.empty(T, N, **f)
    return dict(T=T, H=H, N=N, x=randn(g, T, H).bfloat16(), r=randn(g, T, H), r2=torch.empty(T, H, **f),
                gain=1 + 0.1 * randn(g, H), q=torch.empty(T, H, dtype=E4M3, **f),
                sc=torch.empty(T, **f), w=(w / ws[:, None]).to(E4M3), ws=ws, h=h,
                idx=torch.randint(0, N, (T, 4), generator=g, dtype=torch.int32, **f),
                loss=torch.empty(1, **f), counts=torch.empty(1, N, dtype=torch.int32, **f),
                tokens=torch.empty(1, dtype=torch.int32, **f), prob=torch.empty(1, N, **f),
                work=torch.empty(moe.balance_workspace(T, N, 1), dtype=torch.uint8, **f),
                dz=torch.empty_like(h))


OUTS = ("r2", "sc", "h", "loss", "counts", "tokens", "prob", "dz")


@pytest.mark.parametrize("T", [1, 8, 48, 300])
def test_ops_captured_replayed_and_two_streams(moe, T):
    """Replays of a captured graph and calls on two streams at once give the
    eager calls' bits: no call keeps anything for the next or shares scratch."""
    a, b = ops_state(moe, 1, T), ops_state(moe, 2, T)
    for s in (a, b):
        ops_call(moe, s)
    torch.cuda.synchronize()
    want = [{k: s[k].clone() for k in OUTS} for s in (a, b)]
    graphs = []
    for s in (a, b):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            ops_call(moe, s)
        graphs.append(gr)

    def clear():
        for s in (a, b):
            for k in OUTS:
                s[k].zero_()
        torch.cuda.synchronize()

    clear()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        with torch.cuda.stream(s1):
            graphs[0].replay()
        with torch.cuda.stream(s2):
            graphs[1].replay()
    torch.cuda.synchronize()
    for s, w in zip((a, b), want):
        for k in OUTS:
            assert torch.equal(s[k], w[k]), k
    clear()
    for _ in range(5):
        ops_call(moe, a, stream=s1)
        ops_call(moe, b, stream=s2)
    torch.cuda.synchronize()
    for s, w in zip((a, b), want):
        for k in OUTS:
            assert torch.equal(s[k], w[k]), k


@pytest.mark.parametrize("T", [1, 6, 70, 600])
def test_ops_together_around_a_router(moe, T):
    """A dense layer's half step and the router behind it, as they are used:
    norm in 8 bits -> SwiGLU product -> down product onto the stream -> norm ->
    router logits -> selection -> balance loss and gradient."""
    H, I, E, k = 512, 768, 64, 8
    g = gen(T)
    x, resid = randn(g, T, H).bfloat16(), 2 * randn(g, T, H)
    gain = 1 + 0.1 * randn(g, H)
    w13 = randn(g, 2 * I, H) / H ** 0.5
    s13 = w13.abs().amax(1) / 448
    w13 = (w13 / s13[:, None]).to(E4M3)
    w2 = (randn(g, H, I) / I ** 0.5).bfloat16()
    wr = (randn(g, E, H) / H ** 0.5).bfloat16()
    q, sc, r1 = run_norm(moe, x, resid, gain, 2, 0)
    check_norm(x, resid, gain, q, sc, r1, 2, 0)
    h, st = run_linear(moe, q, w13, sc.view(-1), s13, None, None, I, 2, 1, 3)
    check_linear(h, st, q, w13, sc.view(-1), s13, None, None, I, 3)
    before = r1.clone()
    r2, st = run_linear(moe, h, w2, None, None, None, r1, H, 1, 0, 0, in_place=True)
    check_linear(r2, st, h, w2, None, None, None, None, H, 0, resid=before)
    n, _, _ = run_norm(moe, r2, None, gain, 1, 0)
    check_norm(r2, None, gain, n, None, None, 1, 0)
    z, st = run_linear(moe, n, wr, None, None, None, None, E, 1, 0, 0)
    check_linear(z, st, n, wr, None, None, None, None, E, 0)
    idx = torch.empty(T, k, dtype=torch.int32, device="cuda")
    wt = torch.empty(T, k, device="cuda")
    moe.route_noalloc(n, T, H, E, k, moe.X_BF16, moe.ROUTER_SOFTMAX, 1.0, wr.float(), None, idx, wt)
    # the router picks by the same logits: each choice is within rounding of the k-th largest
    kth = torch.topk(z, k, dim=1).values[:, -1:]
    assert bool((torch.gather(z, 1, idx.long()) >= kth - 1e-4 * z.abs().max()).all())
    got = run_balance(moe, z, idx, None, None, None, k, 0)
    check_balance(got, z, idx, None, None, None, k, 0)


def test_ops_device_refusals_leave_outputs(moe):
    """A refused call launches nothing."""
    x = torch.zeros(4, 512, device="cuda", dtype=torch.bfloat16)
    out = torch.full((4, 512), SENT, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(moe.MoeError) as e:
        moe.add_rmsnorm(x, 4, 512, -1.0, out)
    assert e.value.code == moe.MOE_ERR_ARG
    with pytest.raises(moe.MoeError):
        moe.linear(x, x, 4, 4, 500, out, out_dtype=1)
    ws = torch.empty(16, dtype=torch.uint8, device="cuda")
    one = torch.zeros(64, device="cuda")
    ids = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    with pytest.raises(moe.MoeError) as e:
        moe.balance_loss(x, ids, 4, 512, 2, one, ids, ids, one, ws, z_dtype=1)
    assert e.value.code == moe.MOE_ERR_NOMEM
    torch.cuda.synchronize()
    assert bool((out.float() == SENT).all())


@pytest.mark.parametrize("T", [1, 5, 16, 40, 600])
@pytest.mark.parametrize("act", [0, 3])
def test_linear_e4m3_every_code(moe, T, act):
    """Every e4m3 code on both sides, subnormals, zeros and (in single rows)
    NaN codes among them: a NaN reaches its row of w's outputs or its token,
    and nothing else."""
    K, N = 512, 256
    rows = 2 * N if act == 3 else N
    g = gen(T)
    codes = torch.randint(0, 256, (T + rows, K), generator=g, device="cuda", dtype=torch.int32)
    codes[(codes & 127) == 127] = 3
    x, w = codes[:T].to(torch.uint8), codes[T:].to(torch.uint8)
    w[0, :256] = torch.tensor([c if c & 127 != 127 else 0 for c in range(256)], dtype=torch.uint8, device="cuda")
    sx = 2.0 ** torch.randint(-8, 0, (T,), generator=g, device="cuda").float()
    sw = 2.0 ** torch.randint(-12, -4, (rows,), generator=g, device="cuda").float()
    out, st = run_linear(moe, x.view(E4M3), w.view(E4M3), sx, sw, None, None, N, 2, 0, act)
    check_linear(out, st, x.view(E4M3), w.view(E4M3), sx, sw, None, None, N, act)
    w[7, K - 1] = 0x7F
    w[rows - 3, 0] = 0xFF
    bad, st = run_linear(moe, x.view(E4M3), w.view(E4M3), sx, sw, None, None, N, 2, 0, act)
    cols = sorted({7, (rows - 3) % N})
    keep = [n for n in range(N) if n not in cols]
    assert bool(bad[:, cols].isnan().all()) and torch.equal(bad[:, keep], out[:, keep])
    w[7, K - 1] = 1
    w[rows - 3, 0] = 1
    x[T - 1, 3] = 0x7F
    bad, st = run_linear(moe, x.view(E4M3), w.view(E4M3), sx, sw, None, None, N, 2, 0, act)
    assert bool(bad[T - 1].isnan().all()) and not bool(bad[:T - 1].isnan().any())


# Large products: several tiles for each CTA pair, pairs whose second half has
# no rows, many K segments, tiles of two widths.
@pytest.mark.parametrize("dtype", [1, 2])
@pytest.mark.parametrize("out_dtype", [0, 1])
@pytest.mark.parametrize("T,K,N,act", [(3001, 512, 4097, 0), (2500, 1040, 4112, 3), (4096, 272, 2048, 1),
                                       (600, 14336, 4096, 0), (2049, 4096, 1300, 2), (8200, 128, 1024, 0)])
def test_linear_large(moe, T, K, N, act, dtype, out_dtype):
    g = gen(T + N)
    x, w, sx, sw, b, r = make_linear(g, T, K, N, dtype, act, out_dtype, True, True)
    out, st = run_linear(moe, x, w, sx, sw, b, r, N, dtype, out_dtype, act)
    check_linear(out, st, x, w, sx, sw, b, r, N, act)
    again, st = run_linear(moe, x, w, sx, sw, b, r, N, dtype, out_dtype, act)
    assert torch.equal(out, again)


def test_linear_random_shapes(moe):
    """Sixty seeded shapes over the whole range of forms and tilings."""
    rs = np.random.RandomState(17)
    for i in range(60):
        T = int(np.exp(rs.uniform(0, np.log(3000))))
        K = 16 * int(np.exp(rs.uniform(0, np.log(260))))
        act = int(rs.randint(4))
        N = int(np.exp(rs.uniform(0, np.log(2500))))
        if act == 3:
            N = (N + 15) // 16 * 16
        dtype, out_dtype, bias, resid = 1 + i % 2, int(rs.randint(2)), bool(rs.randint(2)), bool(rs.randint(2))
        x, w, sx, sw, b, r = make_linear(gen(i), T, K, N, dtype, act, out_dtype, bias, resid)
        out, st = run_linear(moe, x, w, sx, sw, b, r, N, dtype, out_dtype, act)
        try:
            check_linear(out, st, x, w, sx, sw, b, r, N, act)
        except AssertionError as e:
            raise AssertionError("T=%d K=%d N=%d act=%d dtype=%d out=%d: %s" % (T, K, N, act, dtype, out_dtype, e))


@pytest.mark.parametrize("T", [3, 20])
def test_ops_offsets_past_32_bits(moe, T):
    """Row strides that put the last rows past 2^31 elements and 2^32 bytes."""
    far = (1 << 31) // (T - 1) // 16 * 16 + 64
    H, N, E = 256, 64, 32
    g = gen(T)
    big = torch.empty((T - 1) * far + 4096, dtype=torch.bfloat16, device="cuda")

    def spread(t, at):
        v = big.as_strided((T, t.shape[1]), (far, 1), at)
        v.copy_(t)
        return v

    x = spread(randn(g, T, H).bfloat16(), 0)
    w = (randn(g, N, H) / 16).bfloat16()
    resid = spread(randn(g, T, N).bfloat16(), 512)
    out = spread(torch.zeros(T, N, device="cuda"), 1024)
    _, st = run_linear(moe, x, w, None, None, None, resid, N, 1, 1, 0, out=out)
    check_linear(out, st, x, w, None, None, None, resid, N, 0)
    n = spread(torch.zeros(T, H, device="cuda"), 1536)
    rout = spread(torch.zeros(T, H, device="cuda"), 2048)
    r = spread(randn(g, T, H).bfloat16(), 2560)
    moe.add_rmsnorm(x, T, H, 1e-6, n, resid=r, resid_out=rout, resid_dtype=1, x_stride=far,
                    resid_stride=far, resid_out_stride=far, out_stride=far)
    check_norm(x, r, None, n, None, rout, 1, 0)
    z = spread(randn(g, T, E).bfloat16(), 3104)
    dz = spread(torch.zeros(T, E, device="cuda"), 3584)
    idx = torch.randint(0, E, (T, 2), generator=g, device="cuda", dtype=torch.int32)
    loss, prob = torch.empty(1, device="cuda"), torch.empty(1, E, device="cuda")
    counts = torch.empty(1, E, dtype=torch.int32, device="cuda")
    tokens = torch.empty(1, dtype=torch.int32, device="cuda")
    ws = torch.empty(moe.balance_workspace(T, E), dtype=torch.uint8, device="cuda")
    moe.balance_loss(z, idx, T, E, 2, loss, counts, tokens, prob, ws, z_dtype=1, alpha=0.01, dz=dz,
                     z_stride=far, dz_stride=far)
    check_balance((loss, counts, tokens, prob, dz), z, idx, None, None, None, 2, 0)


def test_ops_from_two_threads(moe):
    """Calls from two host threads at once, each on its own stream."""
    import threading
    a, b = ops_state(moe, 5, 300), ops_state(moe, 6, 20)
    for s in (a, b):
        ops_call(moe, s)
    torch.cuda.synchronize()
    want = [{k: s[k].clone() for k in OUTS} for s in (a, b)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    bad = []

    def go(s, st):
        try:
            for _ in range(50):
                ops_call(moe, s, stream=st)
        except Exception as e:   # noqa: BLE001
            bad.append(e)

    ts = [threading.Thread(target=go, args=v) for v in zip((a, b), streams)]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    torch.cuda.synchronize()
    assert not bad
    for s, w in zip((a, b), want):
        for k in OUTS:
            assert torch.equal(s[k], w[k]), k


def test_ops_first_call_inside_a_capture():
    """A process whose first calls are captured (no call before to set anything up)."""
    import os
    import subprocess
    import sys
    here = os.path.dirname(os.path.abspath(__file__))
    code = ("import sys; sys.path[:0] = [%r, %r]\n"
            "import torch, expert_routing_grouped_gb300 as moe, test_gpu_ops as t\n"
            "states = [t.ops_state(moe, 1, T) for T in (1, 40, 2000)]\n"
            "gr = torch.cuda.CUDAGraph()\n"
            "with torch.cuda.graph(gr):\n"
            "    for s in states: t.ops_call(moe, s)\n"
            "gr.replay(); torch.cuda.synchronize()\n"
            "got = [{k: s[k].clone() for k in t.OUTS} for s in states]\n"
            "for s in states: t.ops_call(moe, s)\n"
            "torch.cuda.synchronize()\n"
            "assert all(torch.equal(g[k], s[k]) for g, s in zip(got, states) for k in t.OUTS)\n"
            % (os.path.dirname(here), here))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=200)
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.parametrize("S,E", [(7, 64), (34, 256), (300, 64), (3000, 64)])
def test_balance_many_segments(moe, S, E):
    """More segments than a warp looks at once, many of them empty or of one
    token, in each of the kernels' forms."""
    T, k = 9000, 4
    g = gen(S)
    z, idx, _, m = make_balance(g, T, E, k, 0, 1, True)
    rs = np.random.RandomState(S)
    cuts = [np.sort(rs.randint(0, T + 1, S + 1)), np.minimum(np.arange(S + 1) * 2, T),
            np.concatenate([np.zeros(S // 2, int), np.full(S + 1 - S // 2, T)])]
    for cut in cuts:
        off = torch.tensor(cut, dtype=torch.int32, device="cuda")
        got = run_balance(moe, z, idx, None, m, off, k, 1)
        check_balance(got, z, idx, None, m, off, k, 1)
        plain = run_balance(moe, z, idx, None, m, off, k, 1, want_dz=False)
        for a, b in zip(got[:4], plain[:4]):
            assert torch.equal(a, b)


def test_balance_disordered_segments_stay_in_bounds(moe):
    """seq_off that is not what the header asks for: any values, but nothing
    outside the outputs is written."""
    T, E, k = 5000, 64, 2
    z, idx, _, _ = make_balance(gen(3), T, E, k, 0)
    for bad in ([5000, 0, 9999, -7, 100], [-2 ** 31, 2 ** 31 - 1, 3, 3, 4000], [10, 5, 4, 3, 2]):
        off = torch.tensor(bad, dtype=torch.int32, device="cuda")
        for n, dt in ((T, True), (300, False)):
            buf = torch.full((n + 2, E), SENT, device="cuda")
            S = len(bad) - 1
            f = dict(device="cuda")
            outs = [torch.full((S * c + 2,), 72, dtype=d, **f)
                    for c, d in ((1, torch.float32), (E, torch.int32), (1, torch.int32), (E, torch.float32))]
            nb = moe.balance_workspace(n, E, S)
            ws = torch.full((nb + 64,), 0x55, dtype=torch.uint8, **f)
            moe.balance_loss(z, idx, n, E, k, outs[0][1:], outs[1][1:], outs[2][1:], outs[3][1:], ws[:nb],
                             seq_off=off, n_seq=S, dz=buf[1:] if dt else None)
            torch.cuda.synchronize()
            assert bool((buf[0] == SENT).all()) and bool((buf[-1] == SENT).all())
            assert bool((ws[nb:] == 0x55).all())
            for o in outs:
                assert int(o[0]) == 72 and int(o[-1]) == 72


@pytest.mark.parametrize("mode", [0, 1])
def test_balance_long_segment_among_short_ones(moe, mode):
    """One segment with nearly all the tokens is summed like any other; in an
    array whose order would make every other segment that long, none is."""
    T, E, k, S = 6000, 64, 2, 600
    z, idx, _, _ = make_balance(gen(mode), T, E, k, 0)
    bias = None if mode else randn(gen(7), E)
    for at in (0, 300, S - 1):
        off = torch.full((S + 1,), 5900, dtype=torch.int32, device="cuda")
        off[:at + 1] = 7
        off[S] = T if at < S - 1 else 5900
        got = run_balance(moe, z, idx, bias, None, off, k, mode)
        check_balance(got, z, idx, bias, None, off, k, mode)
    off = torch.tensor([0, T] * S, dtype=torch.int32, device="cuda")[:S + 1]
    loss, counts, tokens, prob, dz = run_balance(moe, z, idx, bias, None, off, k, mode)
    assert int(tokens.sum()) == 0 and int(counts.sum()) == 0 and bool((dz == SENT).all())


def test_ops_on_columns_of_one_tensor(moe):
    """Operands and results side by side in the rows of one tensor."""
    g = gen(12)
    T, H, N = 50, 256, 96
    wide = torch.full((T, 4 * 1024), SENT, device="cuda").bfloat16()
    x, out, n, rout, resid = (wide[:, a:a + c] for a, c in ((0, H), (H, N), (512, H), (1024, H), (2048, H)))
    x.copy_(randn(g, T, H))
    resid.copy_(randn(g, T, H))
    w = (randn(g, N, H) / 16).bfloat16()
    _, st = run_linear(moe, x, w, None, None, None, None, N, 1, 1, 0, out=out)
    check_linear(out, st, x, w, None, None, None, None, N, 0)
    moe.add_rmsnorm(x, T, H, 1e-6, n, resid=resid, resid_out=rout, resid_dtype=1, x_stride=4096,
                    resid_stride=4096, resid_out_stride=4096, out_stride=4096)
    check_norm(x, resid, None, n, None, rout, 1, 0)
    for a, b in ((H + N, 512), (768, 1024), (1280, 2048), (2304, 4096)):
        assert bool((wide[:, a:b].float() == SENT).all())


@pytest.mark.parametrize("T,K,N", [(40, 8192, 256), (1000, 2048, 320), (1500, 1024, 777), (4096, 1024, 4096)])
@pytest.mark.parametrize("out_dtype", [0, 1])
def test_linear_waits_give_up(moe, monkeypatch, T, K, N, out_dtype):
    """With a limit of 0 every wait that is not complete when first tested gives
    up (split, one CTA per tile, CTA pairs): the call returns, the status word
    says 2, and the next call is right.  No fault and no hang: the roles stop,
    drain their copies and MMAs, free their tensor memory and return."""
    g = gen(T)
    x, w, sx, sw, b, r = make_linear(g, T, K, N, 1, 0, out_dtype, False, False)
    monkeypatch.setenv("MOE_LINEAR_NO_WAIT", "1")
    out, status = run_linear(moe, x, w, sx, sw, b, r, N, 1, out_dtype, 0)
    torch.cuda.synchronize()
    assert int(status) == 2
    monkeypatch.delenv("MOE_LINEAR_NO_WAIT")
    out, status = run_linear(moe, x, w, sx, sw, b, r, N, 1, out_dtype, 0)
    check_linear(out, status, x, w, sx, sw, b, r, N, 0)
