"""The dense operators around the MoE layer, as cases that can be measured.

Three operators: the RMS norm that adds into the residual stream and can round
to 8 bits (add_rmsnorm), the matrix product with bias, activation and residual
in its epilogue (linear), and the router's balance loss with per-expert counts
and the gradient of the logits (balance_loss).  `own` chooses between their
plain form in elementary torch operations and the library's calls.
"""
import math

import torch

own = False

E4M3 = torch.float8_e4m3fn
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": E4M3}
SIZE = {"f32": 4, "bf16": 2, "e4m3": 1}
CODE = {"f32": 0, "bf16": 1, "e4m3": 2}
ACT = {"none": 0, "silu": 1, "gelu": 2, "swiglu": 3}
EPS = 1e-6
ALPHA = 0.01


def _norm(name, T, H, x, resid, out, group=0, gain=True):
    return {"name": name, "op": "norm", "T": T, "H": H, "x": x, "resid": resid, "out": out,
            "group": group, "gain": gain}


def _linear(name, T, K, N, dtype, out, act="none", bias=False, resid=False):
    return {"name": name, "op": "linear", "T": T, "K": K, "N": N, "dtype": dtype, "out": out,
            "act": act, "bias": bias, "resid": resid}


def _balance(name, T, E, k, mode, dtype, grad, n_seq=1, mask=False):
    return {"name": name, "op": "balance", "T": T, "E": E, "k": k, "mode": mode, "dtype": dtype,
            "grad": grad, "n_seq": n_seq, "mask": mask}


def listed():
    return [
        # One decoded token's pre-norm between two stacked layers.
        _norm("norm 1x6144 bf16", 1, 6144, "f32", "f32", "bf16"),
        # The pre-norm of a prefill chunk whose next product runs in 8 bits.
        _norm("norm 4096x6144 e4m3", 4096, 6144, "bf16", "f32", "e4m3"),
        # A ragged batch on a bf16 residual stream, one scale per 128 values.
        _norm("norm 1037x4096 e4m3/128", 1037, 4096, "bf16", "bf16", "e4m3", group=128, gain=False),
        # One decoded token through a dense FFN's gate and up products.
        _linear("linear 1x6144x2048 swiglu", 1, 6144, 2048, "bf16", "bf16", "swiglu"),
        # Four drafted tokens verified at once: an FFN's down product in 8 bits onto the stream.
        _linear("linear 4x14336x4096 e4m3", 4, 14336, 4096, "e4m3", "f32", resid=True),
        # A short ragged prompt, odd output width, bias and activation.
        _linear("linear 203x2048x1027 gelu", 203, 2048, 1027, "bf16", "bf16", "gelu", bias=True),
        # The down product of a prefill chunk, added into the f32 residual stream.
        _linear("linear 2048x14336x4096", 2048, 14336, 4096, "bf16", "f32", resid=True),
        # The gate and up products of a prefill chunk in 8 bits.
        _linear("linear 4096x4096x14336 e4m3", 4096, 4096, 14336, "e4m3", "bf16", "swiglu"),
        # A small batch's loss and gradient, where launches count.
        _balance("balance 64x64 step", 64, 64, 8, 0, "f32", True),
        # Padded sequences of different lengths in one batch, bf16 logits, loss and gradient.
        _balance("balance 16389x256 seq step", 16389, 256, 8, 1, "bf16", True, n_seq=24, mask=True),
        # Loss and counts of a large batch without a gradient (watching the balance).
        _balance("balance 65536x256 loss", 65536, 256, 8, 1, "f32", False),
        # Loss, counts and gradient of a large batch.
        _balance("balance 65536x256 step", 65536, 256, 8, 1, "f32", True),
    ]


def _log(rng, lo, hi, step=1):
    """A whole multiple of `step` between lo and hi, spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return min(hi // step * step, max(-(-lo // step) * step, int(v / step + 0.5) * step))


def draw(rng):
    op = rng.choice(["norm", "linear", "balance"])
    if op == "norm":
        out = rng.choice(["bf16", "e4m3", "e4m3"])
        group = rng.choice([0, 0, 32, 64, 128]) if out == "e4m3" else 0
        H = _log(rng, 256, 16384, max(16, group))
        T = _log(rng, 1, min(8192, 4096 * 6144 // H))
        c = _norm(None, T, H, rng.choice(["f32", "bf16"]), rng.choice(["none", "f32", "bf16"]), out,
                  group, rng.random() < 0.7)
        if T * H * _norm_bytes(c) > 4096 * 6144 * 11:
            c["T"] = max(1, 4096 * 6144 * 11 // (H * _norm_bytes(c)))
    elif op == "linear":
        dtype = rng.choice(["bf16", "e4m3"])
        act = rng.choice(["none", "silu", "gelu", "swiglu"])
        T = _log(rng, 1, 8192)
        K = _log(rng, 128, 14336, 16)
        N = _log(rng, 64, 14336, 16 if act == "swiglu" else 1)
        rows = N * (2 if act == "swiglu" else 1)
        T = max(1, min(T, 4096 * 4096 * 28672 // (K * rows)))
        c = _linear(None, T, K, N, dtype, rng.choice(["f32", "bf16"]), act, rng.random() < 0.5,
                    rng.random() < 0.5)
    else:
        E = rng.choice([8, 16, 60, 64, 128, 160, 256, 384, 512, 1024])
        T = _log(rng, 16, 65536 * 256 // max(E, 256))
        n_seq = min(T, _log(rng, 1, 64))
        c = _balance(None, T, E, rng.randint(1, min(E, 16)), rng.choice([0, 1, 2]),
                     rng.choice(["f32", "bf16"]), rng.random() < 0.7, n_seq, rng.random() < 0.5)
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs --

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _rows_e4m3(v):
    """v in 8 bits, one scale a row: (e4m3 rows, f32 scales)."""
    s = (v.abs().amax(1) / 448).clamp(min=2.0 ** -126)
    return (v / s[:, None]).to(E4M3), s


def prepare(case, seed):
    return {"norm": _prepare_norm, "linear": _prepare_linear, "balance": _prepare_balance}[case["op"]](case, seed)


def _prepare_norm(c, seed):
    g = _gen(seed)
    T, H = c["T"], c["H"]
    s = dict(c)
    # rows of different sizes with a few outlying channels, as residual streams have them
    chan = torch.exp(0.5 * _randn(g, H))
    size = torch.exp(0.5 * _randn(g, T, 1))
    s["x_"] = (_randn(g, T, H) * chan * size).to(DT[c["x"]])
    s["resid_"] = None if c["resid"] == "none" else (4 * _randn(g, T, H) * chan * size).to(DT[c["resid"]])
    s["gain_"] = 1 + 0.2 * _randn(g, H) if c["gain"] else None
    s["resid_out"] = None if c["resid"] == "none" else torch.empty_like(s["resid_"])
    s["out_"] = torch.empty(T, H, dtype=DT[c["out"]], device="cuda")
    groups = H // c["group"] if c["group"] else 1
    s["scale"] = torch.empty(T, groups, device="cuda") if c["out"] == "e4m3" else None
    return s


def _prepare_linear(c, seed):
    g = _gen(seed)
    T, K, N = c["T"], c["K"], c["N"]
    rows = 2 * N if c["act"] == "swiglu" else N
    s = dict(c)
    x, w = _randn(g, T, K), _randn(g, rows, K) / math.sqrt(K)
    s["x_scale"] = s["w_scale"] = None
    if c["dtype"] == "e4m3":
        x, s["x_scale"] = _rows_e4m3(x)
        w, s["w_scale"] = _rows_e4m3(w)
    s["x_"], s["w_"] = x.to(DT[c["dtype"]]), w.to(DT[c["dtype"]])
    s["bias_"] = 0.5 * _randn(g, rows) if c["bias"] else None
    s["resid_"] = (2 * _randn(g, T, N)).to(DT[c["out"]]) if c["resid"] else None
    s["out_"] = torch.empty(T, N, dtype=DT[c["out"]], device="cuda")
    return s


def _prepare_balance(c, seed):
    g = _gen(seed)
    T, E, k, S = c["T"], c["E"], c["k"], c["n_seq"]
    s = dict(c)
    # popular and rare experts: a fixed offset per expert under the tokens' own logits
    z = _randn(g, T, E) + 1.2 * _randn(g, E)
    s["z"] = z.to(DT[c["dtype"]])
    s["bias_"] = 0.1 * _randn(g, E)
    s["idx"] = torch.topk(s["z"].float() + s["bias_"], k, dim=1).indices.to(torch.int32)
    cut = torch.sort(torch.randint(0, T + 1, (S - 1,), generator=g, device="cuda")).values if S > 1 else None
    ends = [torch.zeros(1, dtype=torch.int64, device="cuda")] + ([cut] if S > 1 else []) + \
        [torch.full((1,), T, dtype=torch.int64, device="cuda")]
    s["seq_off"] = torch.cat(ends).to(torch.int32)
    s["mask"] = (torch.rand(T, generator=g, device="cuda") < 0.9).to(torch.uint8) if c["mask"] else None
    s["up"] = 1 + 0.1 * _randn(g, S) if c["grad"] else None   # the gradient that comes from above
    f = {"device": "cuda"}
    s["loss"], s["prob"] = torch.empty(S, **f), torch.empty(S, E, **f)
    s["counts"] = torch.empty(S, E, dtype=torch.int32, **f)
    s["tokens"] = torch.empty(S, dtype=torch.int32, **f)
    s["dz"] = torch.empty_like(s["z"]) if c["grad"] else None
    # scratch for the partial sums: sized by the caller, as the library's header says
    s["work"] = torch.empty((3 * 1024 + S) * (2 * E + 4) + 1024, dtype=torch.float32, **f)
    return s


# ------------------------------------------------------------- one pass --

def run(state):
    if own:
        return {"norm": _own_norm, "linear": _own_linear, "balance": _own_balance}[state["op"]](state)
    return {"norm": _plain_norm, "linear": _plain_linear, "balance": _plain_balance}[state["op"]](state)


def _own_norm(s):
    import expert_routing_grouped_gb300 as moe
    r = s["resid"]
    moe.add_rmsnorm(s["x_"], s["T"], s["H"], EPS, s["out_"], resid=s["resid_"], resid_out=s["resid_out"],
                    gain=s["gain_"], scale=s["scale"], group=s["group"], x_dtype=CODE[s["x"]],
                    resid_dtype=0 if r == "none" else CODE[r], out_dtype=CODE[s["out"]])
    return s["out_"], s["scale"], s["resid_out"]


def _own_linear(s):
    import expert_routing_grouped_gb300 as moe
    moe.linear(s["x_"], s["w_"], s["T"], s["N"], s["K"], s["out_"], dtype=CODE[s["dtype"]],
               out_dtype=CODE[s["out"]], act=ACT[s["act"]], x_scale=s["x_scale"],
               w_scale=s["w_scale"], bias=s["bias_"], resid=s["resid_"])
    return s["out_"]


def _own_balance(s):
    import expert_routing_grouped_gb300 as moe
    moe.balance_loss(s["z"], s["idx"], s["T"], s["E"], s["k"], s["loss"], s["counts"], s["tokens"],
                     s["prob"], s["work"], bias=s["bias_"], mask=s["mask"], seq_off=s["seq_off"],
                     n_seq=s["n_seq"], z_dtype=CODE[s["dtype"]], router_mode=s["mode"], alpha=ALPHA,
                     dz=s["dz"], grad=s["up"])
    return s["loss"], s["counts"], s["tokens"], s["prob"], s["dz"]


def _plain_norm(s):
    r = s["x_"].float()
    new = None
    if s["resid_"] is not None:
        new = (s["resid_"].float() + r).to(DT[s["resid"]])
        r = new.float()
    n = r * torch.rsqrt((r * r).mean(1, keepdim=True) + EPS)
    if s["gain_"] is not None:
        n = n * s["gain_"]
    if s["out"] != "e4m3":
        return n.to(DT[s["out"]]), None, new
    v = n.view(s["T"], -1, s["group"] or s["H"])
    scale = (v.abs().amax(2) / 448).clamp(min=2.0 ** -126)
    return (v / scale[:, :, None]).to(E4M3).view(s["T"], s["H"]), scale, new


def _act(y, act, N):
    if act == "silu":
        return y * torch.sigmoid(y)
    if act == "gelu":
        return 0.5 * y * (1 + torch.erf(y * math.sqrt(0.5)))
    if act == "swiglu":
        return y[:, :N] * torch.sigmoid(y[:, :N]) * y[:, N:]
    return y


def _plain_linear(s):
    y = s["x_"].float() @ s["w_"].float().t()
    if s["x_scale"] is not None:
        y = y * s["x_scale"][:, None] * s["w_scale"]
    if s["bias_"] is not None:
        y = y + s["bias_"]
    y = _act(y, s["act"], s["N"])
    if s["resid_"] is not None:
        y = y + s["resid_"].float()
    return y.to(DT[s["out"]])


def _plain_balance(s):
    T, E, k, S = s["T"], s["E"], s["k"], s["n_seq"]
    seg = torch.bucketize(torch.arange(T, device="cuda"), s["seq_off"][1:].long(), right=True)
    keep = torch.ones(T, device="cuda") if s["mask"] is None else s["mask"].float()
    z = s["z"].float()
    if s["mode"] == 1:
        sg = torch.sigmoid(z)
        p = sg / sg.sum(1, keepdim=True)
    else:
        e = torch.exp(z + s["bias_"] - (z + s["bias_"]).amax(1, keepdim=True))
        p = e / e.sum(1, keepdim=True)
    p = p * keep[:, None]
    # long sums in 64 bits
    tokens = torch.zeros(S, dtype=torch.float64, device="cuda").index_add_(0, seg, keep.double())
    some = tokens.clamp(min=1)
    prob = torch.zeros(S, E, dtype=torch.float64, device="cuda").index_add_(0, seg, p.double()) / some[:, None]
    counts = torch.zeros(S * E, dtype=torch.float64, device="cuda").index_add_(
        0, (seg[:, None] * E + s["idx"].long()).view(-1), keep.double()[:, None].expand(T, k).reshape(-1)).view(S, E)
    loss = ALPHA * E / (k * some) * (counts * prob).sum(1)
    dz = None
    if s["dz"] is not None:
        # sum_e p_e (c_i - c_e): the mean taken off the counts changes nothing but the rounding
        a = s["up"].double()[:, None] * ALPHA * E / (k * some * some)[:, None] * (counts - counts.mean(1, keepdim=True))
        a = a.float()[seg]
        dz = p * (a - (p * a).sum(1, keepdim=True))
        if s["mode"] == 1:
            dz = dz * (1 - sg)
        dz = dz.to(DT[s["dtype"]])
    return loss.float(), counts.to(torch.int32), tokens.to(torch.int32), prob.float(), dz


# ------------------------------------------------------------ what it costs --

def _norm_bytes(c):
    """Bytes of one element: x and the old residual read, the new one and the output written."""
    return SIZE[c["x"]] + (2 * SIZE[c["resid"]] if c["resid"] != "none" else 0) + SIZE[c["out"]]


def work(case):
    c = case
    T = c["T"]
    if c["op"] == "norm":
        groups = (c["H"] // c["group"] if c["group"] else 1) if c["out"] == "e4m3" else 0
        return {"bytes": T * c["H"] * _norm_bytes(c) + 4 * T * groups + (4 * c["H"] if c["gain"] else 0),
                "flops": 6 * T * c["H"]}
    if c["op"] == "linear":
        rows = c["N"] * (2 if c["act"] == "swiglu" else 1)
        b = (T + rows) * c["K"] * SIZE[c["dtype"]] + T * c["N"] * SIZE[c["out"]] * (2 if c["resid"] else 1)
        if c["dtype"] == "e4m3":
            b += 4 * (T + rows)
        return {"bytes": b + (4 * rows if c["bias"] else 0), "flops": 2 * T * c["K"] * rows}
    z = T * c["E"] * SIZE[c["dtype"]]
    return {"bytes": z * (2 if c["grad"] else 1) + 4 * T * c["k"] + (T if c["mask"] else 0) + 8 * c["n_seq"] * c["E"],
            "flops": T * c["E"] * (12 if c["grad"] else 6)}


# ------------------------------------------------------- the definition, f64 --

def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "linear": _exact_linear, "balance": _exact_balance}[case["op"]](s)


def _exact_norm(s):
    x = s["x_"].double()
    new = x if s["resid_"] is None else s["resid_"].double() + x
    if s["resid"] == "bf16":   # the norm is of the stream as it is kept
        new = new.to(torch.bfloat16).double()
    rms = torch.sqrt(torch.square(new).sum(1) / s["H"] + EPS)
    n = new / rms[:, None]
    if s["gain_"] is not None:
        n = torch.einsum("th,h->th", n, s["gain_"].double())
    new = None if s["resid_"] is None else new
    if s["out"] != "e4m3":
        return n, None, new
    parts = n.unflatten(1, (-1, s["group"] or s["H"]))
    scale = torch.maximum(parts.amax(2), -parts.amin(2)).div(448).clamp_min(2.0 ** -126)
    return torch.div(parts, scale.unsqueeze(2)).flatten(1), scale, new


def _exact_linear(s):
    x, w = s["x_"].double(), s["w_"].double()
    if s["x_scale"] is not None:
        x.mul_(s["x_scale"].double().unsqueeze(1))
        w.mul_(s["w_scale"].double().unsqueeze(1))
    y = torch.mm(x, w.T)
    if s["bias_"] is not None:
        y.add_(s["bias_"].double().unsqueeze(0))
    if s["act"] == "silu":
        y = y / (1 + torch.exp(-y))
    elif s["act"] == "gelu":
        y = y * 0.5 * torch.special.erfc(-y / math.sqrt(2))
    elif s["act"] == "swiglu":
        gate, up = y.split(s["N"], dim=1)
        y = up * gate / (1 + torch.exp(-gate))
    return y if s["resid_"] is None else y + s["resid_"].double()


def _exact_balance(s):
    T, E, k, S = s["T"], s["E"], s["k"], s["n_seq"]
    off = s["seq_off"].tolist()
    z = s["z"].double()
    loss, prob = torch.zeros(S, dtype=torch.float64), torch.zeros(S, E, dtype=torch.float64)
    dz = torch.zeros(T, E, dtype=torch.float64, device="cuda")
    for q in range(S):
        rows = torch.arange(off[q], off[q + 1], device="cuda")
        if s["mask"] is not None:
            rows = rows[s["mask"][rows] != 0]
        n = len(rows)
        if n == 0:
            continue
        zq = z[rows]
        if s["mode"] == 1:
            sig = 1 / (1 + torch.exp(-zq))
            p = sig / sig.sum(1, keepdim=True)
        else:
            p = torch.softmax(zq + s["bias_"].double(), dim=1)
        c = torch.bincount(s["idx"][rows].reshape(-1).long(), minlength=E).double()
        mean = p.sum(0) / n
        loss[q] = ALPHA * E / (k * n) * torch.dot(c, mean)
        prob[q] = mean
        if s["dz"] is not None:
            a = float(s["up"][q]) * ALPHA * E / (float(k) * n * n) * c
            d = p * (a - torch.mv(p, a)[:, None])
            dz[rows] = d * (1 - sig) if s["mode"] == 1 else d
    return loss, None, None, prob, None if s["dz"] is None else dz
