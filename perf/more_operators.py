"""The operators of an attention block beside the MoE layer, as cases that can be measured.

Three operators: rotary positions (rope), the rows of K and V put into a paged
cache in 4 bits (kv4_append), and attention over that cache for single tokens,
a few drafted tokens and prompts (kv4_attention).  `own` chooses between their
plain form in elementary torch operations and the library's calls.

The cache is uint8 [n_pages][Hkv][page * D * 9 / 8].  A block holds, for the
page's tokens in order: K codes [page][D / 2], V codes [page][D / 2] (the even
value in the low 4 bits), then K's and V's float16 (step, lo) [page][D / 64][2].
A code c stands for lo + step * c.
"""
import math
import random

import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2}
CODE = {"f32": 0, "bf16": 1}
GROUP = 64
THETA = 1e6


def _rope(name, T, heads, D, rot, interleaved, dtype, factor=1.0, inverse=False, start=0):
    return {"name": name, "op": "rope", "T": T, "heads": heads, "D": D, "rot": rot,
            "interleaved": interleaved, "dtype": dtype, "factor": factor, "inverse": inverse,
            "start": start}


def _append(name, T, n_seq, kv, Hkv, D, page, dtype):
    return {"name": name, "op": "append", "T": T, "n_seq": n_seq, "kv": kv, "Hkv": Hkv, "D": D,
            "page": page, "dtype": dtype}


def _attend(name, T, n_seq, kv, H, Hkv, D, page, ragged=False, window=0, softcap=0.0, causal=True):
    return {"name": name, "op": "attend", "T": T, "n_seq": n_seq, "kv": kv, "H": H, "Hkv": Hkv,
            "D": D, "page": page, "ragged": ragged, "window": window, "softcap": softcap,
            "causal": causal}


def listed():
    return [
        # One decoded token: 96 query and 8 key heads of one row, half of each head turned.
        _rope("rope 1x104x128 part", 1, 104, 128, 64, True, "bf16", start=100000),
        # A prefill chunk: 32 query and 8 key heads, whole heads in the half layout.
        _rope("rope 4096x40x128", 4096, 40, 128, 128, False, "bf16"),
        # The gradient of f32 rows at far positions with scaled frequencies, an odd part of odd heads.
        _rope("rope 1037x20x80 f32 back", 1037, 20, 80, 40, False, "f32", factor=8.0, inverse=True,
              start=900000),
        # One new token for each sequence of a decode batch.
        _append("append 64x8x128", 64, 64, 8192, 8, 128, 16, "bf16"),
        # A prompt's rows into an empty cache.
        _append("append 8192x8x128", 8192, 1, 8192, 8, 128, 64, "bf16"),
        # A ragged batch of f32 rows onto sequences that have a past.
        _append("append 1037x4x64 f32", 1037, 24, 500, 4, 64, 16, "f32"),
        # One decoded token over a short context: launches and latency.
        _attend("decode 1x4096 96/8", 1, 1, 4096, 96, 8, 128, 64),
        # A decode batch over contexts of different lengths.
        _attend("decode 64x8192 32/8", 64, 64, 8192, 32, 8, 128, 16, ragged=True),
        # One decoded token over a long context.
        _attend("decode 1x131072 96/8", 1, 1, 131072, 96, 8, 128, 64),
        # Four drafted tokens verified at once in each of four sequences.
        _attend("verify 4x4x16384 96/8", 16, 4, 16384, 96, 8, 128, 64),
        # A prompt attends to itself.
        _attend("prompt 8192 32/8", 8192, 1, 8192, 32, 8, 128, 64),
        # Chunks of ragged prompts, small heads without sharing, a window and capped scores.
        _attend("chunks 2043 16/16 window cap", 2043, 6, 4096, 16, 16, 64, 32, ragged=True,
                window=1024, softcap=30.0),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over the logarithm."""
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi))) + 0.5)))


def draw(rng):
    op = rng.choice(["rope", "append", "attend", "attend"])
    if op == "rope":
        D = rng.choice([64, 80, 96, 128, 256])
        heads = _log(rng, 1, 128)
        dtype = rng.choice(["f32", "bf16"])
        T = _log(rng, 1, min(8192, 4096 * 40 * 128 * 2 // (heads * D * SIZE[dtype])))
        c = _rope(None, T, heads, D, rng.choice([D, D // 2, 2 * rng.randint(1, D // 2)]),
                  rng.random() < 0.5, dtype, rng.choice([1.0, 1.0, 4.0, 8.0, 32.0]),
                  rng.random() < 0.3, _log(rng, 1, 1 << 20) - 1)
    elif op == "append":
        dtype = rng.choice(["f32", "bf16"])
        D, Hkv = rng.choice([64, 128]), rng.randint(1, 16)
        T = _log(rng, 1, 8192 * 8 * 128 * 2 // (Hkv * D * SIZE[dtype]))
        n_seq = min(T, _log(rng, 1, 64))
        c = _append(None, T, n_seq, -(-T // n_seq) * 2 + _log(rng, 1, 4096), Hkv, D,
                    rng.choice([16, 32, 64, 128, 256]), dtype)
    else:
        D, Hkv = rng.choice([64, 128, 128]), rng.choice([1, 2, 3, 4, 5, 8, 8, 16])
        H = Hkv * rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 12, 16])
        kind = rng.choice(["decode", "decode", "few", "prompt"])
        per = {"decode": 1, "few": rng.randint(2, 8), "prompt": _log(rng, 9, 8192)}[kind]
        most = {"decode": 128, "few": 32, "prompt": 8}[kind]
        n_seq = _log(rng, 1, most)
        kv = _log(rng, per, 131072)
        c = _attend(None, 0, n_seq, kv, H, Hkv, D, rng.choice([16, 32, 64, 128, 256]),
                    rng.random() < 0.5, _log(rng, 16, 8192) if rng.random() < 0.3 else 0,
                    rng.choice([0.0, 0.0, 30.0, 50.0]), rng.random() < 0.9)
        # no more bytes or products than the largest listed cases
        c["n_seq"] = n_seq = max(1, min(n_seq, 64 * 8192 * 8 * 128 // (kv * Hkv * D)))
        c["T"] = n_seq * per
        most = 8192 * 4096 * 32 * 128
        while c["T"] > n_seq and c["T"] * kv * H * D > most:
            c["T"] = max(n_seq, c["T"] // 2)
    del c["name"]
    return c


def _lengths(c):
    """(new tokens, tokens in the cache) of each sequence: fixed by the case, not by the seed."""
    T, S = c["T"], c["n_seq"]
    rng = random.Random(T * 31 + S * 7 + c["kv"])
    if T == S:
        new = [1] * S
    elif c.get("ragged", True) and S > 1:
        cut = sorted(rng.randint(0, T) for _ in range(S - 1))
        new = [b - a for a, b in zip([0] + cut, cut + [T])]
    else:
        new = [T // S + (1 if s < T % S else 0) for s in range(S)]
    if c.get("ragged", True) and S > 1:
        have = [max(n, _log(rng, max(1, c["kv"] // 16), c["kv"])) for n in new]
        have[rng.randrange(S)] = max(c["kv"], max(new))
    else:
        have = [max(n, c["kv"]) for n in new]
    return new, have


# ------------------------------------------------------------------ inputs --

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def prepare(case, seed):
    return {"rope": _prepare_rope, "append": _prepare_append, "attend": _prepare_attend}[case["op"]](case, seed)


def _freqs(rot, factor):
    """Radians per position of each pair: fast pairs as they are, slow ones
    slowed by `factor`, a ramp between 32 and 1 turns in 32768 positions."""
    out = []
    for i in range(rot // 2):
        f = THETA ** (-2.0 * i / rot)
        turns = 32768 * f / (2 * math.pi)
        keep = min(1.0, max(0.0, (turns - 1) / 31))
        out.append(f * (keep + (1 - keep) / factor))
    return out


def _prepare_rope(c, seed):
    g = _gen(seed)
    s = dict(c)
    s["x"] = _randn(g, c["T"], c["heads"], c["D"]).to(DT[c["dtype"]])
    first = c["start"] + int(torch.randint(0, 64, (1,), generator=g, device="cuda"))
    s["pos"] = torch.arange(first, first + c["T"], device="cuda", dtype=torch.int32)
    s["freqs"] = torch.tensor(_freqs(c["rot"], c["factor"]), dtype=torch.float64, device="cuda")
    s["mscale"] = 0.1 * math.log(c["factor"]) + 1
    s["out"] = torch.empty_like(s["x"])
    return s


def _batch(s, c, g):
    """Lengths, offsets and a page table whose pages lie in any order."""
    new, have = _lengths(c)
    P, S = c["page"], c["n_seq"]
    need = [-(-n // P) for n in have]
    s["max_pages"], s["n_pages"] = max(need), sum(need)
    order = torch.randperm(s["n_pages"], generator=g, device="cuda").to(torch.int32)
    table = torch.full((S, s["max_pages"]), -1, dtype=torch.int32, device="cuda")
    at = 0
    for q, n in enumerate(need):
        table[q, :n] = order[at:at + n]
        at += n
    off = [0]
    for n in new:
        off.append(off[-1] + n)
    s["new"], s["have"], s["need"], s["off"], s["max_q"] = new, have, need, off, max(new)
    s["pages"] = table
    s["kv_len"] = torch.tensor(have, dtype=torch.int32, device="cuda")
    s["q_off"] = None if c["T"] == S else torch.tensor(off, dtype=torch.int32, device="cuda")
    s["cache"] = torch.zeros(s["n_pages"], c["Hkv"], P * c["D"] * 9 // 8, dtype=torch.uint8, device="cuda")


def _fill(s, c, g):
    """A cache of quantised rows whose channels differ in size and offset, as keys' do."""
    P, D, Hkv = c["page"], c["D"], c["Hkv"]
    size, mean = torch.exp(0.4 * _randn(g, 2, Hkv, 1, D)), 0.5 * _randn(g, 2, Hkv, 1, D)
    step = max(1, (1 << 26) // (Hkv * P * D))
    for a in range(0, s["n_pages"], step):
        n = min(step, s["n_pages"] - a)
        for which in (0, 1):
            x = _randn(g, n, Hkv, P, D) * size[which] + mean[which]
            codes, scale = _quantise(x)
            _put(s["cache"][a:a + n], which, codes, scale, P, D)


def _put(blocks, which, codes, scale, P, D):
    """Whole pages of codes [..., P, D] and (step, lo) [..., P, D / 64, 2]."""
    half, side = P * D // 2, P * D // 16
    lead = codes.shape[:-2]
    packed = codes[..., 0::2] | (codes[..., 1::2] << 4)
    blocks[..., which * half:(which + 1) * half] = packed.reshape(*lead, half)
    raw = scale.contiguous().view(torch.uint8).reshape(*lead, side)
    blocks[..., P * D + which * side:P * D + (which + 1) * side] = raw


def _prepare_append(c, seed):
    g = _gen(seed)
    s = dict(c)
    _batch(s, c, g)
    chan = torch.exp(0.5 * _randn(g, 2, 1, c["Hkv"], c["D"]))
    kv = _randn(g, 2, c["T"], c["Hkv"], c["D"]) * chan
    s["k"], s["v"] = kv[0].to(DT[c["dtype"]]), kv[1].to(DT[c["dtype"]])
    return s


def _prepare_attend(c, seed):
    g = _gen(seed)
    s = dict(c)
    _batch(s, c, g)
    _fill(s, c, g)
    s["q"] = (1.5 * _randn(g, c["T"], c["H"], c["D"])).bfloat16()
    s["out"] = torch.empty_like(s["q"])
    s["work_"] = None
    return s


# ------------------------------------------------------------- one pass --

def run(state):
    if own:
        return {"rope": _own_rope, "append": _own_append, "attend": _own_attend}[state["op"]](state)
    return {"rope": _plain_rope, "append": _plain_append, "attend": _plain_attend}[state["op"]](state)


def _own_rope(s):
    import expert_routing_grouped_gb300 as moe
    moe.rope(s["x"], s["pos"], s["freqs"], s["T"], s["heads"], s["D"], s["out"], rot_dim=s["rot"],
             interleaved=s["interleaved"], inverse=s["inverse"], mscale=s["mscale"],
             dtype=CODE[s["dtype"]])
    return s["out"]


def _own_append(s):
    import expert_routing_grouped_gb300 as moe
    moe.kv4_append(s["k"], s["v"], s["cache"], s["pages"], s["kv_len"], s["T"], s["Hkv"], s["D"],
                   s["page"], s["n_pages"], s["max_pages"], q_off=s["q_off"], n_seq=s["n_seq"],
                   dtype=CODE[s["dtype"]])
    return _held(s)


def _own_attend(s):
    import expert_routing_grouped_gb300 as moe
    if s["work_"] is None:   # kept by the program, as long as its sizes do not change
        n = moe.kv4_workspace(s["T"], s["n_seq"], s["H"], s["Hkv"], s["D"], s["page"], s["max_pages"],
                              max_q=s["max_q"])
        s["work_"] = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
    moe.kv4_attention(s["q"], s["cache"], s["pages"], s["kv_len"], s["T"], s["H"], s["Hkv"], s["D"],
                      s["page"], s["n_pages"], s["max_pages"], s["out"], s["work_"],
                      q_off=s["q_off"], n_seq=s["n_seq"], max_q=s["max_q"], softcap=s["softcap"],
                      window=s["window"], causal=s["causal"])
    return s["out"]


def _held(s):
    """The cache's two parts: the codes' bytes, and the (step, lo) of every group."""
    split = s["page"] * s["D"]
    return s["cache"][..., :split], s["cache"].view(torch.float16)[..., split // 2:]


def _plain_rope(s):
    x, R = s["x"].float(), s["rot"]
    a = s["pos"].double()[:, None] * s["freqs"]   # far positions: angles in 64 bits
    if s["inverse"]:
        a = -a
    cos, sin = (torch.cos(a) * s["mscale"]).float()[:, None], (torch.sin(a) * s["mscale"]).float()[:, None]
    if s["interleaved"]:
        u, v = x[..., 0:R:2], x[..., 1:R:2]
    else:
        u, v = x[..., :R // 2], x[..., R // 2:R]
    y = x.clone()
    if s["interleaved"]:
        y[..., 0:R:2], y[..., 1:R:2] = u * cos - v * sin, u * sin + v * cos
    else:
        y[..., :R // 2], y[..., R // 2:R] = u * cos - v * sin, u * sin + v * cos
    return y.to(s["x"].dtype)


def _quantise(x):
    """Codes [..., D] (uint8) and (step, lo) [..., D / 64, 2] (float16) of f32 rows."""
    v = x.float().unflatten(-1, (-1, GROUP)).clamp(-60000.0, 60000.0)
    lo = v.amin(-1, keepdim=True).half()
    fifteen = torch.full_like(lo, 15.0, dtype=torch.float32)   # a tensor: divided, not multiplied by 1 / 15
    step = ((v.amax(-1, keepdim=True) - lo.float()).clamp(min=0.0) / fifteen).half()
    c = torch.round((v - lo.float()) / step.float()).clamp(0.0, 15.0)
    c = torch.where(step > 0, c, torch.zeros_like(c))
    return c.to(torch.uint8).flatten(-2), torch.cat([step, lo], -1)


def _plain_append(s):
    P, D, Hkv = s["page"], s["D"], s["Hkv"]
    at = torch.arange(s["T"], device="cuda")
    if s["q_off"] is None:
        seq, pos = at, s["kv_len"].long() - 1
    else:
        off = s["q_off"].long()
        seq = torch.bucketize(at, off[1:], right=True)
        pos = s["kv_len"].long()[seq] - off[seq + 1] + at
    page, slot = s["pages"].long()[seq, pos // P], pos % P
    flat = s["cache"].view(s["n_pages"], Hkv, -1)
    for which, x in ((0, s["k"]), (1, s["v"])):
        codes, scale = _quantise(x)
        packed = codes[..., 0::2] | (codes[..., 1::2] << 4)
        part = flat[..., which * P * D // 2:(which + 1) * P * D // 2].view(s["n_pages"], Hkv, P, D // 2)
        part[page, :, slot] = packed
        first = P * D + which * P * D // 16
        part = flat[..., first:first + P * D // 16].view(s["n_pages"], Hkv, P, D // 16)
        part[page, :, slot] = scale.flatten(-2).view(torch.uint8)
    return _held(s)


def _rows(s, q):
    """K and V of sequence q in f32, [Hkv][tokens][D] each."""
    P, D, n = s["page"], s["D"], s["have"][q]
    blocks = s["cache"][s["pages"][q, :s["need"][q]].long()]
    out = []
    for which in (0, 1):
        b = blocks[..., which * P * D // 2:(which + 1) * P * D // 2].reshape(-1, s["Hkv"], P, D // 2)
        codes = torch.stack([b & 15, b >> 4], -1).flatten(-2).float()
        first = P * D + which * P * D // 16
        sc = blocks[..., first:first + P * D // 16].contiguous().view(torch.float16).float()
        sc = sc.view(-1, s["Hkv"], P, D // GROUP, 2)
        v = sc[..., 1:] + sc[..., :1] * codes.unflatten(-1, (D // GROUP, GROUP))
        out.append(v.flatten(-2).permute(1, 0, 2, 3).reshape(s["Hkv"], -1, D)[:, :n])
    return out


def _plain_attend(s):
    D, Hkv, G = s["D"], s["Hkv"], s["H"] // s["Hkv"]
    out = torch.empty_like(s["q"])
    for b in range(s["n_seq"]):
        n, t0, nq = s["have"][b], s["off"][b], s["new"][b]
        if nq == 0:
            continue
        K, V = _rows(s, b)
        key = torch.arange(n, device="cuda")
        for a in range(0, nq, 1024):
            m = min(1024, nq - a)
            q = s["q"][t0 + a:t0 + a + m].float().view(m, Hkv, G, D).permute(1, 2, 0, 3)
            x = torch.matmul(q.reshape(Hkv, G * m, D), K.transpose(1, 2)) / math.sqrt(D)
            if s["softcap"]:
                x = s["softcap"] * torch.tanh(x / s["softcap"])
            pos = (n - nq + a + torch.arange(m, device="cuda"))[:, None]
            see = key <= (pos if s["causal"] else n)
            if s["window"]:
                see = see & (key > pos - s["window"])
            see = see.repeat(G, 1)
            x = x.masked_fill(~see, -math.inf)
            top = x.amax(-1, keepdim=True)
            e = torch.exp(x - torch.where(top > -math.inf, top, torch.zeros_like(top)))
            sums = e.sum(-1, keepdim=True)
            o = torch.matmul(e, V) / torch.where(sums > 0, sums, torch.ones_like(sums))
            out[t0 + a:t0 + a + m] = o.view(Hkv, G, m, D).permute(2, 0, 1, 3).reshape(m, -1, D).bfloat16()
            del x, e, see
    return out


# ------------------------------------------------------------ what it costs --

def work(case):
    c = case
    if c["op"] == "rope":
        n = c["T"] * c["heads"]
        return {"bytes": 2 * n * c["D"] * SIZE[c["dtype"]] + 4 * c["T"] + 4 * c["rot"], "flops": 3 * n * c["rot"]}
    D, Hkv = c["D"], c["Hkv"]
    if c["op"] == "append":
        n = 2 * c["T"] * Hkv * D
        return {"bytes": n * SIZE[c["dtype"]] + n * 9 // 16, "flops": 6 * n}
    rows = pairs = 0
    for nq, n in zip(*_lengths(c)):
        if nq == 0:
            continue
        first = max(0, n - nq - c["window"] + 1) if c["window"] else 0
        rows += n - first
        w = c["window"] or n
        for p in range(n - nq, n):   # one query at position p
            end = p + 1 if c["causal"] else n
            pairs += end - max(0, p + 1 - w)
    return {"bytes": rows * Hkv * D * 9 // 8 + 4 * c["T"] * c["H"] * D, "flops": 4 * pairs * c["H"] * D}


# ------------------------------------------------------- the definition, f64 --

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "attend" and work(case)["flops"] > 4e12:
        return None
    return {"rope": _exact_rope, "append": _exact_append, "attend": _exact_attend}[case["op"]](s)


def _exact_rope(s):
    half = s["rot"] // 2
    turn = torch.polar(torch.full((s["T"], half), s["mscale"], dtype=torch.float64, device="cuda"),
                       torch.outer(s["pos"].double(), s["freqs"]))
    if s["inverse"]:
        turn = turn.conj()
    x = s["x"].double()
    head, rest = x.split([s["rot"], s["D"] - s["rot"]], dim=2)
    pairs = head.unflatten(2, (half, 2)) if s["interleaved"] else head.unflatten(2, (2, half)).transpose(2, 3)
    turned = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn.unsqueeze(1))
    if not s["interleaved"]:
        turned = turned.transpose(2, 3)
    return torch.cat([turned.flatten(2), rest], dim=2)


def _exact_append(s):
    P, D = s["page"], s["D"]
    side = _held(s)[1].double().view(s["n_pages"], s["Hkv"], 2, P, D // GROUP, 2)
    pages = s["pages"].tolist()
    for which, x in enumerate((s["k"], s["v"])):
        g = x.double().view(s["T"], s["Hkv"], D // GROUP, GROUP).clamp(-60000, 60000)
        low = g.min(dim=3).values
        kept = low.half().double()   # the step is defined from the kept lo
        step = torch.clamp(g.max(dim=3).values - kept, min=0) / 15
        pair = torch.stack([step, low], dim=3)
        for b in range(s["n_seq"]):
            first = s["have"][b] - s["new"][b]
            i = 0
            while i < s["new"][b]:
                p = first + i
                n = min(P - p % P, s["new"][b] - i)
                t = s["off"][b] + i
                side[pages[b][p // P], :, which, p % P:p % P + n] = pair[t:t + n].transpose(0, 1)
                i += n
    return None, side.view(s["n_pages"], s["Hkv"], -1)


def _exact_attend(s):
    P, D, Hkv = s["page"], s["D"], s["Hkv"]
    G = s["H"] // Hkv
    out = torch.zeros(s["T"], s["H"], D, dtype=torch.float64, device="cuda")
    shift = torch.tensor([0, 4], dtype=torch.uint8, device="cuda")
    for b in range(s["n_seq"]):
        n, nq = s["have"][b], s["new"][b]
        if nq == 0:
            continue
        ids = s["pages"][b][:s["need"][b]].long()
        for h in range(Hkv):
            raw = s["cache"][ids, h]
            side = raw[:, P * D:].contiguous().view(torch.float16).double().view(-1, 2, P, D // GROUP, 2)
            codes = raw[:, :P * D].reshape(-1, 2, P, D // 2)
            kv = []
            for w in (0, 1):
                c = torch.bitwise_right_shift(codes[:, w].unsqueeze(-1), shift).bitwise_and(15)
                c = c.reshape(-1, GROUP)[:n * (D // GROUP)].double()
                low = side[:, w].reshape(-1, 2)[:n * (D // GROUP)]
                kv.append(torch.addcmul(low[:, 1:], c, low[:, :1]).reshape(n, D))
            K, V = kv
            for a in range(0, nq, 1024):
                t = torch.arange(a, min(a + 1024, nq), device="cuda")
                rows = s["off"][b] + t
                q = s["q"][rows, h * G:(h + 1) * G].double().flatten(0, 1)
                z = (q @ K.T) * D ** -0.5
                if s["softcap"]:
                    z = torch.tanh(z / s["softcap"]) * s["softcap"]
                back = (n - nq + t).repeat_interleave(G)[:, None] - torch.arange(n, device="cuda")
                if s["causal"]:
                    z[back < 0] = -math.inf
                if s["window"]:
                    z[back >= s["window"]] = -math.inf
                w = torch.exp(z - torch.logsumexp(z, dim=1, keepdim=True))
                out[rows, h * G:(h + 1) * G] = torch.nan_to_num(w @ V).view(len(t), G, D)
    return out
