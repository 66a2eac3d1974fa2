"""Plain 64-bit forms of the dense operators (add_rmsnorm, linear,
balance_loss), written from their formulas, and the error bounds their tests
hold the kernels to."""
import torch

E4M3_MAX = 448.0
TINY = 2.0 ** -126


def norm(x, resid, gain, eps, group=None):
    """(n, resid_out, scale): n unrounded f64; scale per group (None: no 8-bit output)."""
    r = x.double()
    new = None
    if resid is not None:
        new = (resid.float() + x.float()).to(resid.dtype)   # defined as the f32 sum, then resid's type
        r = new.double()
    n = r / torch.sqrt((r * r).mean(1, keepdim=True) + eps)
    if gain is not None:
        n = n * gain.double()
    scale = None
    if group is not None:
        scale = (n.view(n.shape[0], -1, group).abs().amax(2) / E4M3_MAX).clamp(min=TINY)
    return n, new, scale


def act(kind, a, N):
    """kind as the library's codes: none, silu, gelu, swiglu."""
    if kind == 1:
        return a * torch.sigmoid(a)
    if kind == 2:
        return 0.5 * a * (1 + torch.erf(a / 2 ** 0.5))
    if kind == 3:
        return a[:, :N] * torch.sigmoid(a[:, :N]) * a[:, N:]
    return a


def linear(x, w, N, kind, sx=None, sw=None, bias=None, resid=None):
    """(y, bound): y in f64 and how far a kernel with f32 sums may be from it
    before its output is rounded.

    Every tensor-core instruction adds at least 16 products to a running sum
    that never exceeds S = sum |x||w|, truncating at most twice by one unit of
    f32 (2^-23 S each); partial sums of warps or blocks add a few more:
    (K / 8 + 32) 2^-23 S covers them.  Scales, bias and the activation round a
    handful of times more (16 units); the activations' slopes stay below 1.13,
    and a SwiGLU product carries each factor's error times the other factor."""
    xd, wd = x.double(), w.double()
    if sx is not None:
        xd, wd = xd * sx.double()[:, None], wd * sw.double()[:, None]
    a = xd @ wd.t()
    S = xd.abs() @ wd.abs().t()
    K = x.shape[1]
    err = (K / 8 + 32) * 2.0 ** -23 * S
    if bias is not None:
        a = a + bias.double()
    err = err + 16 * 2.0 ** -24 * (a.abs() + S)
    y = act(kind, a, N)
    if kind == 3:
        g, u, eg, eu = a[:, :N], a[:, N:], err[:, :N], err[:, N:]
        err = 1.13 * eg * (u.abs() + eu) + (g * torch.sigmoid(g)).abs() * eu
    else:
        err = 1.13 * err
    err = err + 16 * 2.0 ** -24 * y.abs()
    if resid is not None:
        y = y + resid.double()
    return y, err


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def segments(T, seq_off, mask):
    """[(segment, kept rows)] on the CPU."""
    off = [0, T] if seq_off is None else [int(v) for v in seq_off]
    out = []
    for s in range(len(off) - 1):
        rows = torch.arange(off[s], off[s + 1])
        if mask is not None:
            rows = rows[mask.cpu()[rows] != 0]
        out.append((s, rows))
    return out


def probs(z, bias, mode):
    z = z.double()
    if mode == 1:
        sg = torch.sigmoid(z)
        tot = sg.sum(1, keepdim=True)
        return torch.where(tot > 0, sg / tot, torch.zeros_like(sg))
    l = z if bias is None else z + bias.double()
    m = l.amax(1, keepdim=True)
    m = torch.where(torch.isinf(m) & (m < 0), torch.zeros_like(m), m)
    e = torch.exp(l - m)
    tot = e.sum(1, keepdim=True)
    return torch.where(tot > 0, e / tot, torch.zeros_like(e))


def balance(z, idx, bias, mask, seq_off, k, mode, alpha, grad=None):
    """(loss, counts, tokens, prob, dz, size) on the CPU in f64; dz is zero
    outside the kept rows, size[t][i] the sum of the magnitudes that dz[t][i]
    is the difference of."""
    z, idx = z.cpu(), idx.cpu()
    T, E = z.shape
    S = 1 if seq_off is None else len(seq_off) - 1
    loss, prob = torch.zeros(S, dtype=torch.float64), torch.zeros(S, E, dtype=torch.float64)
    counts, tokens = torch.zeros(S, E, dtype=torch.int64), torch.zeros(S, dtype=torch.int64)
    dz, size = torch.zeros(T, E, dtype=torch.float64), torch.zeros(T, E, dtype=torch.float64)
    b = None if bias is None else bias.cpu()
    for s, rows in segments(T, seq_off, mask):
        n = len(rows)
        tokens[s] = n
        if n == 0:
            continue
        p = probs(z[rows], b, mode)
        ids = idx[rows].reshape(-1).long()
        c = torch.bincount(ids[(ids >= 0) & (ids < E)], minlength=E)
        counts[s] = c
        prob[s] = p.sum(0) / n
        loss[s] = alpha * E / (k * n) * (c.double() * prob[s]).sum()
        up = 1.0 if grad is None else float(grad[s])
        a = up * alpha * E / (k * n * n) * c.double()
        slope = 1 - torch.sigmoid(z[rows].double()) if mode == 1 else 1.0
        dz[rows] = p * slope * (a - (p * a).sum(1, keepdim=True))
        size[rows] = p * slope * (a.abs() + (p * a.abs()).sum(1, keepdim=True))
    return loss, counts, tokens, prob, dz, size
