"""The label head's definitions in 64 bits, for the tests of its kernels."""
import torch

U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}  # unit roundoff
TINY = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24}  # least positive value


def logits(x, w, b):
    z = x.double() @ w.double().t()
    return z if b is None else z + b.double()


def logits_bound(x, w, b):
    """How far float32 sums of the exact products x w may be off: the rounding
    (or truncation) of H / 16 partial sums, each at most 2^-23 of the largest
    partial sum, which is at most sum |x w|; they add like a random walk, and
    8 sqrt(H) of them hold any that add up for H <= 8192.  The bias adds one."""
    s = x.double().abs() @ w.double().abs().t()
    s = torch.where(torch.isfinite(s), s, torch.zeros_like(s))
    e = 8.0 * x.shape[1] ** 0.5 * 2.0 ** -24 * s
    if b is not None:
        bb = torch.where(torch.isfinite(b.double()), b.double().abs(), torch.zeros_like(b.double()))
        e = e + 2.0 ** -24 * (s + bb)
    return e


def exp_log_bound(z, lse):
    """What exp2, the sums over V and log add to an lse: the exponent (z - m)
    log2(e) is rounded to 2^-24 of itself and matters while exp(z - m) does
    (|z - m| < 20), the sum of positive terms, the exponential and the log are
    good to a few units, lse itself is rounded."""
    return 40 * 2.0 ** -23 + 4 * 2.0 ** -24 * lse.abs()


def cross_entropy(x, w, b, t, ignore, reduction, grad):
    """(loss, lse, dx, dw, db, |d| |w|, |d|^T |x|): the gradients, and the sums
    that bound what rounding d to 16 bits changes."""
    V = w.shape[0]
    keep = (t != ignore) & (t >= 0) & (t < V)
    xk = torch.where(keep[:, None], x.double(), torch.zeros((), dtype=torch.float64, device=x.device))
    z = logits(xk, w, b)
    lse = torch.logsumexp(z, 1)
    at = torch.where(keep, t, torch.zeros_like(t)).long()[:, None]
    loss = torch.where(keep, lse - z.gather(1, at)[:, 0], torch.zeros_like(lse))
    n = int(keep.sum())
    g = grad.double()
    if reduction == "mean":
        g = g / max(n, 1)
    d = torch.exp(z - lse[:, None])
    d.scatter_add_(1, at, torch.full_like(at, -1, dtype=torch.float64))
    d = torch.where(keep[:, None], d * (g[:, None] if g.dim() else g), torch.zeros_like(d))
    total = loss if reduction == "none" else loss.sum() / (n if reduction == "mean" else 1) if n or reduction == "sum" \
        else torch.full((), float("nan"), dtype=torch.float64, device=x.device)
    return (total, torch.where(keep, lse, torch.zeros_like(lse)), d @ w.double(), d.t() @ xk, d.sum(0),
            d.abs() @ w.double().abs(), d.abs().t() @ xk.abs(), d.abs().sum(0))


def layer_norm(x, w, b, eps):
    x = x.double()
    var, mean = torch.var_mean(x, dim=1, correction=0, keepdim=True)
    r = 1.0 / torch.sqrt(var + eps)
    xh = (x - mean) * r
    y = xh if w is None else xh * w.double()
    y = y if b is None else y + b.double()
    return y, mean[:, 0], r[:, 0], xh


def layer_norm_backward(dy, x, w, eps):
    _, _, r, xh = layer_norm(x, None, None, eps)
    dy = dy.double()
    t = dy if w is None else dy * w.double()
    dx = r[:, None] * (t - t.mean(1, keepdim=True) - xh * (t * xh).mean(1, keepdim=True))
    return dx, (dy * xh).sum(0), dy.sum(0)
