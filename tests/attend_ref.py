"""Plain 64-bit forms of the attention block's operators (rope, kv4_append,
kv4_attention), written from their formulas, and the error bounds their tests
hold the kernels to."""
import math

import torch

GROUP = 64


def rope(x, pos, freqs, rot, interleaved, inverse, mscale):
    """(y, size): y in f64, size[...] = mscale (|u| + |v|) of each turned element
    (0 where an element is copied)."""
    x = x.double()
    a = pos.double()[:, None] * freqs.double()
    c, s = torch.cos(a)[:, None] * mscale, torch.sin(a)[:, None] * mscale * (-1 if inverse else 1)
    half = rot // 2
    iu = torch.arange(half) * 2 if interleaved else torch.arange(half)
    iv = iu + (1 if interleaved else half)
    u, v = x[..., iu], x[..., iv]
    y, size = x.clone(), torch.zeros_like(x)
    y[..., iu], y[..., iv] = u * c - v * s, u * s + v * c
    size[..., iu] = size[..., iv] = mscale * (u.abs() + v.abs())
    return y, size


def quantise(x):
    """uint8 codes and float16 (step, lo) [..., D / 64, 2], as the header defines them."""
    g = x.float().unflatten(-1, (-1, GROUP))
    bad = torch.isnan(g).any(-1, keepdim=True)
    g = torch.where(torch.isnan(g), torch.zeros_like(g), g).clamp(-60000.0, 60000.0)
    lo = g.amin(-1, keepdim=True).half()
    step = ((g.amax(-1, keepdim=True) - lo.float()).clamp(min=0) / torch.full_like(lo, 15.0).float()).half()
    c = torch.round((g - lo.float()) / step.float()).clamp(0, 15)
    c = torch.where((step > 0) & ~bad, c, torch.zeros_like(c)).to(torch.uint8)
    nan = torch.full_like(lo, float("nan"))
    return c.flatten(-2), torch.cat([torch.where(bad, nan, step), torch.where(bad, nan, lo)], -1)


def values(codes, scale):
    """What codes [..., D] and (step, lo) stand for, f64."""
    c = codes.double().unflatten(-1, (-1, GROUP))
    return (scale[..., 1:].double() + scale[..., :1].double() * c).flatten(-2)


class Cache:
    """A paged cache with `have[s]` tokens of sequence s, in pages of any order;
    every byte that belongs to no token is 0xFF (NaN scales)."""

    def __init__(self, g, have, Hkv, D, page, spare=2, size=1.0, max_pages=None, device="cuda"):
        self.Hkv, self.D, self.page, self.have = Hkv, D, page, list(have)
        need = [-(-n // page) for n in have]
        self.n_pages = sum(need) + spare
        self.max_pages = max_pages or max(max(need), 1)
        order = torch.randperm(self.n_pages, generator=g, device=device).to(torch.int32)
        # entries past a sequence's pages: ids far out of range
        self.pages = torch.full((len(have), self.max_pages), 1 << 30, dtype=torch.int32, device=device)
        at = 0
        for s, n in enumerate(need):
            self.pages[s, :n] = order[at:at + n]
            at += n
        self.kv_len = torch.tensor(self.have, dtype=torch.int32, device=device)
        self.bytes = torch.full((self.n_pages, Hkv, page * D * 9 // 8), 255, dtype=torch.uint8, device=device)
        self.K, self.V = [], []
        for s, n in enumerate(have):
            x = size * torch.randn(2, n, Hkv, D, generator=g, device=device)
            x = x * torch.exp(0.3 * torch.randn(2, 1, Hkv, D, generator=g, device=device)) + 0.5
            self.K.append(self.put(s, 0, 0, x[0]))
            self.V.append(self.put(s, 1, 0, x[1]))

    def part(self, which):
        """Views of the codes [page][Hkv][slot][D / 2] and scales [...][D / 16] of K (0) or V (1)."""
        P, D = self.page, self.D
        lead = self.bytes.shape[:2]
        codes = self.bytes[..., which * P * D // 2:(which + 1) * P * D // 2].unflatten(-1, (P, D // 2))
        first = P * D + which * P * D // 16
        return codes, self.bytes[..., first:first + P * D // 16].unflatten(-1, (P, D // 16))

    def put(self, s, which, first, x):
        """Rows x [n][Hkv][D] at positions first .. of sequence s; returns what they became (f64)."""
        codes, scale = quantise(x)
        pos = torch.arange(first, first + x.shape[0], device=x.device)
        page = self.pages[s].long()[pos // self.page]
        c, sc = self.part(which)
        c[page, :, pos % self.page] = codes[..., 0::2] | (codes[..., 1::2] << 4)
        sc[page, :, pos % self.page] = scale.flatten(-2).contiguous().view(torch.uint8)
        return values(codes, scale)


def attend(q, K, V, scale, softcap, window, causal, seen=None):
    """(out, bound) of the last rows q [n][H][D] of one sequence with K, V
    [len][Hkv][D], in f64; seen [len]: False for tokens in holes.

    The bound counts, per row: keys, values and weights rounded to float16 (half
    a step, 2^-11 of the value), f32 sums that truncate (a unit, 2^-23, for every
    16 products), a few roundings of the exponent's argument.  A score off by d
    moves every weight by at most exp(2 d) - 1 of itself, numerator and sum
    together; small weights round by 2^-25 of the largest.  Where the weights
    carry the scales, w step is what is rounded and meets the code, not the
    value: step c = V - lo, and lo is the least value of the token's 64 (whose
    code is 0), so that rounding counts 2^-11 w (V - least)."""
    n, H, D = q.shape
    L, Hkv = K.shape[:2]
    G = H // Hkv
    o = torch.zeros(n, H, D, dtype=torch.float64, device=q.device)
    bound = torch.zeros_like(o)
    pos = (L - n + torch.arange(n, device=q.device))[:, None]
    key = torch.arange(L, device=q.device)
    see = key <= pos if causal else torch.ones(n, L, dtype=torch.bool, device=q.device)
    if window:
        see = see & (key > pos - window)
    if seen is not None:
        see = see & seen
    for h in range(H):
        k, v = K[:, h // G], V[:, h // G]
        qh = q[:, h].double()
        x = qh @ k.t() * scale
        mag = qh.abs() @ k.abs().t() * abs(scale)
        if softcap:
            x = softcap * torch.tanh(x / softcap)
        x = torch.where(see, x, torch.full_like(x, -math.inf))
        top = x.amax(1, keepdim=True) if L else torch.full((n, 1), -math.inf, device=q.device, dtype=torch.float64)
        none = top == -math.inf
        w = torch.exp(x - torch.where(none, torch.zeros_like(top), top))
        w = torch.where(see, w, torch.zeros_like(w))
        l = w.sum(1, keepdim=True)
        p = w / torch.where(l == 0, torch.ones_like(l), l)
        # a row that does not see a token takes nothing from it, whatever it holds
        vv = torch.where(torch.isnan(v), torch.zeros_like(v), v)
        o[:, h] = p @ vv
        nanv = torch.isnan(v).any(1)
        o[:, h] = torch.where((see & nanv).any(1, keepdim=True), torch.full_like(o[:, h], math.nan), o[:, h])
        e = (2.0 ** -11 + (D / 8 + 16) * 2.0 ** -23) * torch.where(see, mag, torch.zeros_like(mag))
        e = torch.nan_to_num(e).amax(1, keepdim=True) if L else torch.zeros_like(l)
        e = e + 2.0 ** -20 * (1 + (softcap if softcap else torch.nan_to_num(top.abs(), posinf=0.0)))
        rel = torch.expm1(2 * e) + 2.0 ** -10 + (L / 8 + 64) * 2.0 ** -23
        above = vv.unflatten(1, (-1, GROUP))
        above = (above - above.amin(2, keepdim=True)).flatten(1)
        bound[:, h] = rel * (p @ vv.abs()) + 2.0 ** -11 * (p @ above) + 2.0 ** -24 * L * (vv.abs().amax(0) if L else 0)
    return o, bound


def half_step(dtype):
    return torch.finfo(dtype).eps / 2
