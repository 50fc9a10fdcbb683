"""Definitions in 64 bits of the operators around the label head (group norm,
dropout, policy and preference losses), with bounds of what float32 arithmetic in
their kernels may be off by.

u = 2^-24 is half a unit of float32.  Sums of n terms are off by at most 8 sqrt(n) u
of the sum of their magnitudes (roundings of either sign; n is the longest chain of
additions, never more than the terms)."""
import numpy as np
import torch

U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24}
u = 2.0 ** -24


def rounded(bound, value, dtype):
    return bound + U[dtype] * (value.abs() + bound) + TINY[dtype]


def frames(x, lengths):
    B, T = x.shape[:2]
    n = torch.full((B,), T, device=x.device) if lengths is None else lengths.long().clamp(0, T)
    return n, torch.arange(T, device=x.device) < n[:, None]


def _act(h, act):
    """(act(h), act'(h), a bound of |act''|)"""
    if act == "silu":
        s = torch.sigmoid(h)
        return h * s, s * (1 + h * (1 - s)), 0.5
    if act == "relu":
        return h.clamp(min=0), (h > 0).double(), 0.0
    return h, torch.ones_like(h), 0.0


class GroupNorm:
    """Everything of a call [B, T, C], in 64 bits; e_*: bounds."""

    def __init__(self, x, G, w, b, lengths, eps, act):
        B, T, C = x.shape
        D = C // G
        self.shape, self.G, self.D, self.act, self.dtype = (B, T, C), G, D, act, x.dtype
        n, live = frames(x, lengths)
        self.live = live[:, :, None, None]
        zero = torch.zeros((), dtype=torch.float64, device=x.device)
        xd = torch.where(self.live, x.double().view(B, T, G, D), zero)
        M = (n * D).clamp(min=1).double()[:, None, None, None]
        self.M, self.n = M, n
        mean = xd.sum((1, 3), keepdim=True) / M
        dev = torch.where(self.live, xd - mean, zero)
        var = (dev * dev).sum((1, 3), keepdim=True) / M
        r = 1 / torch.sqrt(var + eps)
        self.mean, self.r = mean, r
        self.w = (torch.ones(C, device=x.device) if w is None else w).double().view(G, D)
        self.b = (torch.zeros(C, device=x.device) if b is None else b).double().view(G, D)
        self.depth = 8 * (T / 4 + 64) ** 0.5 * u  # a thread joins its rows by fours, then the threads, then the blocks
        self.e_mean = self.depth * (xd.abs().sum((1, 3), keepdim=True) / M + mean.abs())
        # squared distances are positive; the mean's error enters squared, each distance is rounded
        self.e_r = self.depth + 4 * u + (self.e_mean * r) ** 2  # relative
        self.xh = dev * r
        self.e_xh = self.e_mean * r + (self.e_r + 4 * u) * self.xh.abs()
        self.h = self.xh * self.w + self.b
        self.e_h = self.w.abs() * self.e_xh + 4 * u * ((self.w * self.xh).abs() + self.b.abs())
        y, self.slope, curve = _act(self.h, act)
        self.y = torch.where(self.live, y, zero)
        # the exponential's argument is rounded: relative |h| u log2(e), and a few units for it and the division
        sig = (12 + 4 * self.h.abs()) * u if act == "silu" else 0.0
        self.e_y = torch.where(self.live, 1.1 * self.e_h + sig * y.abs(), zero)
        self.e_slope = curve * self.e_h + sig * (1 + self.h.abs())
        if act == "relu":  # which side of 0 an h next to it is on
            self.e_slope = (self.h.abs() <= self.e_h).double()

    def flat(self, t):
        return t.reshape(self.shape)

    def backward(self, dy):
        B, T, C = self.shape
        zero = torch.zeros((), dtype=torch.float64, device=dy.device)
        g = torch.where(self.live, dy.double().view(B, T, self.G, self.D), zero)
        d = g * self.slope
        e_d = g.abs() * (self.e_slope + 4 * u * self.slope.abs())
        t, e_t = d * self.w, self.w.abs() * (e_d + 2 * u * d.abs())
        xh, exh, M, r = self.xh, self.e_xh, self.M, self.r

        def mean(v):
            return v.sum((1, 3), keepdim=True) / M

        dx = torch.where(self.live, r * (t - mean(t) - xh * mean(t * xh)), zero)
        tx = (t * xh).abs()
        e_m0 = mean(e_t) + (self.depth + 4 * u) * mean(t.abs())
        e_m1 = mean(e_t * xh.abs() + t.abs() * exh) + (self.depth + 4 * u) * mean(tx)
        e_dx = r * (e_t + e_m0 + xh.abs() * e_m1 + exh * mean(tx) + 6 * u * (t.abs() + mean(t.abs()) + xh.abs() * mean(tx)))
        e_dx = torch.where(self.live, e_dx + self.e_r * dx.abs(), zero)
        depth = 8 * (T + B + 64) ** 0.5 * u
        dw, db = (d * xh).sum((0, 1)), d.sum((0, 1))
        e_dw = (e_d * xh.abs() + d.abs() * exh).sum((0, 1)) + depth * (d * xh).abs().sum((0, 1))
        e_db = e_d.sum((0, 1)) + depth * d.abs().sum((0, 1))
        return (self.flat(dx), dw.view(-1), db.view(-1)), (self.flat(e_dx), e_dw.view(-1), e_db.view(-1))


# ---- dropout

def philox(ctr, key):
    """Philox4x32-10 of uint32 arrays [4, n], keys [2]: [4, n]."""
    c = [np.asarray(v, np.uint64) for v in ctr]
    k = [int(v) for v in key]
    m = np.uint64(0xFFFFFFFF)
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), b & m, (a >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), a & m]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return np.stack(c)


def kept(first, n, p, seed, offset):
    """Whether elements first .. first + n - 1 are kept, and the factor (float32)."""
    i = np.arange(first, first + n, dtype=np.uint64)
    q = np.unique(i // np.uint64(8))
    seed, offset = seed % 2 ** 64, offset % 2 ** 64
    w = philox([q & np.uint64(0xFFFFFFFF), q >> np.uint64(32), np.full_like(q, offset & 0xFFFFFFFF),
                np.full_like(q, offset >> 32)], (seed & 0xFFFFFFFF, seed >> 32))
    j = i % np.uint64(8)
    word = w[(j // np.uint64(2)).astype(int), (i // np.uint64(8) - q[0]).astype(int)]
    half = np.where(j % np.uint64(2) == 1, word >> np.uint64(16), word & np.uint64(0xFFFF))
    cut = round(p * 65536)
    return half >= cut, np.float32(65536 / (65536 - cut)) if cut < 65536 else np.float32(0)


def dropout(x, p, seed, offset, residual=None, first=0):
    """As the kernel rounds: a float32 product and sum, then the type.  The same bits."""
    keep, scale = kept(first, x.numel(), p, seed, offset)
    keep = torch.from_numpy(keep).to(x.device).view(x.shape)
    v = torch.where(keep, x.float() * float(scale), torch.zeros((), device=x.device))
    return (v if residual is None else residual.float() + v).to(x.dtype)


# ---- losses of sequences

def policy(nll, old, adv, lengths, ref, lo, hi, klw, reduction, grad):
    """dict of loss, stats, dnll and their bounds e_*; [S, L] tensors, adv [S, L]."""
    S, L = nll.shape
    n, live = frames(nll, lengths)
    zero = torch.zeros((), dtype=torch.float64, device=nll.device)
    nd, od, A = (torch.where(live, t.double(), zero) for t in (nll, old, adv))
    d = od - nd
    rho = torch.exp(d)
    s1, s2 = rho * A, rho.clamp(1 - lo, 1 + hi) * A
    held = live & (s1 > s2)
    loss = -torch.where(held, s2, s1)
    slope = torch.where(held, zero, s1)
    e = 8 * u * torch.where(held, s2.abs(), A.abs() * rho * (1 + d.abs()))
    es = 8 * u * A.abs() * rho * (1 + d.abs())
    k = torch.zeros_like(d)
    e_kl = zero
    if ref is not None:
        x = torch.where(live, nd - ref.double(), zero)
        k = torch.expm1(x) - x
        loss = loss + klw * k
        slope = slope + klw * torch.expm1(x)
        # next to 0 both are relative; elsewhere the exponential's rounding, and x's
        big = x.abs() >= 0.4
        ek = 8 * u * torch.where(big, torch.exp(x) * (1 + x.abs()) + x.abs(), k * 2)
        e = e + klw * ek
        es = es + klw * 8 * u * torch.where(big, torch.exp(x) * (1 + x.abs()), x.abs() * 2)
        e_kl = torch.where(live, ek, zero).sum()
    loss, slope, e, es = (torch.where(live, t, zero) for t in (loss, slope, e, es))
    tokens = n.sum().double()
    if reduction == "mean":
        w = (1 / tokens).expand(S, 1)
    elif reduction == "sequence_mean":
        w = (1 / (n.clamp(min=1) * (n > 0).sum()).double())[:, None]
    else:
        w = torch.ones(S, 1, dtype=torch.float64, device=nll.device)
    out = dict(stats=torch.stack([torch.where(live, k, zero).sum() / tokens, held.sum() / tokens]))
    out["e_stats"] = torch.stack([e_kl / tokens + 16 * u * out["stats"][0], 2 * u * out["stats"][1]])
    if reduction == "none":
        out.update(loss=loss, e_loss=e + 2 * u * loss.abs())
    else:
        out["loss"] = (loss * w).sum()
        out["e_loss"] = (e * w).sum() + 4 * u * out["loss"].abs()
    g = w * grad.double()
    out.update(dnll=torch.where(live, slope * g, zero), e_dnll=torch.where(live, (es + 6 * u * slope.abs()) * g.abs(), zero))
    return out


def preference(nll, chosen, rejected, lengths, ref, beta, margin, s, average, reduction, grad):
    B, N, L = nll.shape
    n, live = frames(nll.reshape(B * N, L), None if lengths is None else lengths.reshape(-1))
    n, live = n.view(B, N), live.view(B, N, L)
    zero = torch.zeros((), dtype=torch.float64, device=nll.device)
    f = torch.zeros_like(nll).double() if ref is None else ref.double()
    gain = torch.where(live, f - nll.double(), zero)
    scale = torch.where(live, f.abs() + nll.double().abs(), zero)
    per = n.clamp(min=1).double() if average else torch.ones(B, N, dtype=torch.float64, device=nll.device)
    R, size = gain.sum(2) / per, scale.sum(2) / per
    pair = (chosen >= 0) & (rejected >= 0) & (chosen < N) & (rejected < N)
    at = torch.arange(B, device=nll.device)
    c, r = (torch.where(pair, t, torch.zeros_like(t)).long() for t in (chosen, rejected))
    z = beta * (R[at, c] - R[at, r]) - margin
    # pairs of float32 lose the square of what float32 does, at each of L additions; beta, margin and s are float32
    e_z = 2 * u * (z.abs() + abs(margin) + beta * (R[at, c] - R[at, r]).abs()) \
        + beta * (size[at, c] + size[at, r]) * L * 2.0 ** -46
    sp, sn = torch.sigmoid(z), torch.sigmoid(-z)
    a, b = -torch.nn.functional.logsigmoid(z), -torch.nn.functional.logsigmoid(-z)
    loss = torch.where(pair, (1 - s) * a + s * b, zero)
    # the loss's slope in z is 1 at most; relative to z's error where it is small itself
    e_loss = torch.where(pair, e_z * ((1 - s) * sn + s * sp) * 2 + 12 * u * loss + 2 * u * (a * (s != 0) + b) * s, zero)
    pairs = pair.sum().double()
    g = grad.double() / (pairs if reduction == "mean" else 1)
    dz = torch.where(pair & (c != r), (s * sp - (1 - s) * sn) * g * beta, zero)
    # the two terms may cancel; each is right to a few units and to z's error, relative to itself
    e_dz = torch.where(pair & (c != r), (s * sp + (1 - s) * sn) * (e_z + 16 * u) * (g * beta).abs(), zero)
    coef = torch.zeros(B, N, dtype=torch.float64, device=nll.device)
    e = coef.clone()
    coef[at, c] -= dz
    coef[at, r] += dz
    e[at, c] += e_dz
    e[at, r] += e_dz
    coef, e = coef / per, e / per + 4 * u * (coef / per).abs()
    out = dict(margins=torch.where(pair, z, zero), e_margins=torch.where(pair, e_z, zero),
               dnll=torch.where(live, coef[..., None], zero), e_dnll=torch.where(live, e[..., None], zero))
    if reduction == "none":
        out.update(loss=loss, e_loss=e_loss)
    else:
        k = pairs if reduction == "mean" else 1
        out.update(loss=loss.sum() / k, e_loss=e_loss.sum() / k + 2 * u * (loss.sum() / k).abs())
    return out
