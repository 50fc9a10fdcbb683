"""More of the label head's operators on their own: what each reads, what it has to return, and the sizes it meets.

What trains the model before the decoder, frame by frame and from the decoder's own N-best lists:

    gn   group norm with an activation over channels-last frames [B, T, C], each utterance with its length; with
         ``train`` also its backward pass (dx, dweight, dbias)
    do   dropout from a counter-based generator, with or without a residual, and its backward pass
    po   the clipped policy loss of N-best lists with a KL term: the loss, what it reports, and its gradient
    pr   the preference loss of a pair of hypotheses of each N-best list: the loss, the margins, and its gradient

The two losses read the tokens' negative log-probabilities, as cross entropy without a reduction gives them
[B, N, L], and the hypotheses' lengths [B, N]; their gradients are what its backward pass takes.

``run`` computes them from elementary operations, or, where ``own`` is true, by the calls a user makes of the package.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = 1e-5
CLIP_LOW, CLIP_HIGH = 0.2, 0.28
BETA = 0.1


def listed():
    return [
        # a 16-frame chunk of 128 streams through a convolutional block's norm: latency
        dict(name="gn chunk, 128 streams", op="gn", b=128, t=16, c=512, g=32, type="bf16", params="f32", act="silu",
             ragged=False, empty=False, train=False),
        # a 32-utterance offline batch of up to 500 frames, padded
        dict(name="gn offline, 32 utterances", op="gn", b=32, t=500, c=512, g=32, type="bf16", params="f32", act="silu",
             ragged=True, empty=False, train=False),
        # a training batch of 128 utterances of up to 500 frames
        dict(name="gn train, 128 utterances", op="gn", b=128, t=500, c=1024, g=32, type="bf16", params="bf16",
             act="silu", ragged=True, empty=False, train=True),
        # a small float32 model in training, a group's width that no vector load divides, an utterance without frames
        dict(name="gn train, odd width, f32", op="gn", b=7, t=429, c=771, g=3, type="f32", params="f32", act="relu",
             ragged=True, empty=True, train=True),
        # two long recordings: few utterances, many frames
        dict(name="gn long recordings, f16", op="gn", b=2, t=20000, c=512, g=8, type="f16", params="f16", act="silu",
             ragged=False, empty=False, train=False),
        # a tiny model's 50 frames: latency
        dict(name="do train, tiny", op="do", n=50, h=64, type="bf16", p=0.1, residual=False),
        # a training batch of 128 utterances of 500 frames, on the way into the residual stream
        dict(name="do train, 64000 frames, residual", op="do", n=64000, h=1024, type="bf16", p=0.1, residual=True),
        # a small float32 model in training, a width that no vector load divides
        dict(name="do train, odd width, f32", op="do", n=3001, h=769, type="f32", p=0.25, residual=False),
        # 10-best lists of 32 utterances, up to 40 tokens each
        dict(name="po 10-best lists", op="po", b=32, n=10, l=40, ragged=True, kl=0.05, per_token=False,
             reduction="mean"),
        # 16 samples of each of 256 inputs, up to 1024 tokens each, with an advantage for each token
        dict(name="po long sequences", op="po", b=256, n=16, l=1024, ragged=True, kl=0.01, per_token=True,
             reduction="sequence_mean"),
        # a pair of each of 32 10-best lists, up to 40 tokens
        dict(name="pr 10-best lists", op="pr", b=32, n=10, l=40, ragged=True, ref=True, average=False, smooth=0.0,
             margin=0.0, reduction="mean"),
        # 1024 pairs of long sequences, 2 of 4 samples each
        dict(name="pr long sequences", op="pr", b=1024, n=4, l=1000, ragged=True, ref=True, average=False, smooth=0.1,
             margin=0.0, reduction="mean"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["gn", "gn", "gn", "do", "do", "po", "pr"])
    if op == "gn":
        kind = rng.choice(["bf16", "bf16", "f16", "f32"])
        g = rng.choice([1, 2, 3, 4, 8, 16, 32, 32])
        d = _log(rng, 4, 2048 // g)
        if rng.random() < 0.6:
            d = max(4, d // 8 * 8)
        c = g * d
        most = 25000000 if kind == "f32" else 50000000
        t = _log(rng, -(-64 // d), min(20000, most // c))  # groups of 64 values or more
        b = _log(rng, 1, min(256, most // (t * c)))
        return dict(op="gn", b=b, t=t, c=c, g=g, type=kind, params=rng.choice([kind, "f32"]),
                    act=rng.choice(["silu", "silu", "relu", "none"]), ragged=rng.random() < 0.6, empty=rng.random() < 0.2,
                    train=rng.random() < 0.6)
    if op == "do":
        kind = rng.choice(["bf16", "bf16", "f16", "f32"])
        h = _log(rng, 16, 8192)
        if rng.random() < 0.6:
            h = h // 16 * 16
        return dict(op="do", n=_log(rng, 1, min(64000, (32000000 if kind == "f32" else 65000000) // h)), h=h, type=kind,
                    p=rng.choice([0.0, 0.05, 0.1, 0.2, 0.3, 0.5]), residual=rng.random() < 0.5)
    b = _log(rng, 1, 1024)
    n = rng.randint(2, 16)
    l = _log(rng, 1, min(2048, 4000000 // (b * n)))
    if op == "po":
        return dict(op="po", b=b, n=n, l=l, ragged=rng.random() < 0.8, kl=rng.choice([0.0, 0.01, 0.05]),
                    per_token=rng.random() < 0.4, reduction=rng.choice(["mean", "sequence_mean", "sum", "none"]))
    return dict(op="pr", b=b, n=n, l=l, ragged=rng.random() < 0.8, ref=rng.random() < 0.8, average=rng.random() < 0.3,
                smooth=rng.choice([0.0, 0.0, 0.1]), margin=rng.choice([0.0, 0.0, 0.5]),
                reduction=rng.choice(["mean", "mean", "sum", "none"]))


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 29)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device="cuda")

    if case["op"] == "gn":
        kind, params = TYPES[case["type"]], TYPES[case["params"]]
        b, t, c = case["b"], case["t"], case["c"]
        # a convolution's outputs: every channel with a level of its own, every utterance with a loudness
        x = (normal(b, t, c) * (0.5 + uniform(b, 1, 1)) + 0.5 * normal(1, 1, c)).to(kind)
        s = dict(case=case, x=x, weight=(1.0 + 0.2 * normal(c)).to(params), bias=(0.1 * normal(c)).to(params),
                 lengths=None)
        if case["ragged"] or case["empty"]:
            s["lengths"] = torch.randint(max(1, t // 2) if case["ragged"] else t, t + 1, (b,), generator=g, device="cuda",
                                         dtype=torch.int32)
            if case["empty"]:
                s["lengths"][-1:] = 0
            x *= (torch.arange(t, device="cuda") < s["lengths"][:, None])[..., None]  # a padded batch's zeros
        if case["train"]:
            s["dy"] = (normal(b, t, c) * 0.01).to(kind)
        return s
    if case["op"] == "do":
        kind = TYPES[case["type"]]
        n, h = case["n"], case["h"]
        s = dict(case=case, x=normal(n, h).to(kind), dy=(0.01 * normal(n, h)).to(kind), residual=None)
        if case["residual"]:
            s["residual"] = (2.0 * normal(n, h)).to(kind)
        # the generator's seed and the step's offset
        s["rng"] = torch.stack([torch.randint(-2 ** 62, 2 ** 62, (), generator=g, device="cuda"),
                                torch.randint(0, 2 ** 40, (), generator=g, device="cuda")])
        return s
    b, n, l = case["b"], case["n"], case["l"]
    s = dict(case=case, lengths=None)
    if case["ragged"]:
        s["lengths"] = torch.randint(l // 2, l + 1, (b, n), generator=g, device="cuda", dtype=torch.int32)
        s["lengths"][0, 0] = l  # not every hypothesis is empty
        live = torch.arange(l, device="cuda") < s["lengths"][..., None]
    else:
        live = torch.ones(b, n, l, dtype=torch.bool, device="cuda")
    # token scores of a trained model: most tokens are near certain, some are not; the model that is trained has
    # moved a little from the one that made the lists, and further from the one it is held near to
    old = -torch.log1p(-uniform(b, n, l).clamp(max=0.999)) * torch.where(uniform(b, n, l) < 0.6, 0.02, 1.5)
    nll = (old * torch.exp(0.1 * normal(b, n, l)) + 0.02 * normal(b, n, l).abs())
    ref = (old * torch.exp(0.2 * normal(b, n, l)) + 0.02 * normal(b, n, l).abs())
    zero = torch.zeros((), device="cuda")  # cross entropy gives 0 where a target is ignored
    s.update(nll=torch.where(live, nll, zero), old_nll=torch.where(live, old, zero), ref_nll=torch.where(live, ref, zero))
    s["grad"] = torch.full((), 1.0, device="cuda")
    if case["op"] == "po":
        if not case["kl"]:
            s["ref_nll"] = None
        # rewards of a list, less their mean, over their spread; or what is still to come at each token
        r = uniform(b, n)
        r = (r - r.mean(1, keepdim=True)) / (r.std(1, correction=0, keepdim=True) + 1e-4)
        s["advantages"] = (r[..., None] + 0.3 * normal(b, n, l)).contiguous() if case["per_token"] else r
        if case["reduction"] == "none":
            s["grad"] = uniform(b, n, l)
        return s
    if not case["ref"]:
        s["ref_nll"] = None
    del s["old_nll"]
    s["chosen"] = torch.randint(0, n, (b,), generator=g, device="cuda", dtype=torch.int32)
    s["rejected"] = (s["chosen"] + torch.randint(1, n, (b,), generator=g, device="cuda", dtype=torch.int32)) % n
    none = uniform(b) < 0.1  # lists whose hypotheses are all alike have no pair
    none[0] = False
    s["rejected"] = torch.where(none, torch.full_like(s["rejected"], -1), s["rejected"])
    if case["reduction"] == "none":
        s["grad"] = uniform(b)
    return s


# ---- the plain forms: elementary operations in 32 bits (in 64: long sums, those that cancel, and a ratio next to the
# clip's border), rounded once at the end

def _act(h, kind):
    return h / (1.0 + torch.exp(-h)) if kind == "silu" else h.clamp(min=0) if kind == "relu" else h


def _act_slope(h, kind):
    if kind == "silu":
        p = 1.0 / (1.0 + torch.exp(-h))
        return p * (1.0 + h * (1.0 - p))
    return (h > 0).float() if kind == "relu" else torch.ones_like(h)


def _plain_gn(s):
    c = s["case"]
    b, t, g = c["b"], c["t"], c["g"]
    d = c["c"] // g
    x = s["x"].float().view(b, t, g, d)
    w, beta = s["weight"].float().view(g, d), s["bias"].float().view(g, d)
    zero = torch.zeros((), device=x.device)
    if s["lengths"] is None:
        live = torch.ones(1, 1, 1, 1, dtype=torch.bool, device=x.device)
        count = torch.full((1, 1, 1, 1), float(t * d), device=x.device)
    else:
        live = (torch.arange(t, device=x.device) < s["lengths"][:, None])[:, :, None, None]
        count = (s["lengths"].float() * d).clamp(min=1.0)[:, None, None, None]
    x = torch.where(live, x, zero)
    mean = x.sum((1, 3), keepdim=True) / count
    xh = torch.where(live, x - mean, zero)
    del x
    rstd = torch.rsqrt((xh * xh).sum((1, 3), keepdim=True) / count + EPS)
    xh *= rstd
    h = xh * w + beta
    out = dict(y=torch.where(live, _act(h, c["act"]), zero).to(s["x"].dtype).view(b, t, c["c"]))
    if c["train"]:
        dh = torch.where(live, s["dy"].float().view(b, t, g, d) * _act_slope(h, c["act"]), zero)
        del h
        dw, db = (dh * xh).sum((0, 1)), dh.sum((0, 1))
        dh *= w
        m0, m1 = dh.sum((1, 3), keepdim=True) / count, (dh * xh).sum((1, 3), keepdim=True) / count
        dx = torch.where(live, rstd * (dh - m0 - xh * m1), zero)
        out.update(dx=dx.to(s["x"].dtype).view(b, t, c["c"]), dweight=dw.to(s["weight"].dtype).view(-1),
                   dbias=db.to(s["bias"].dtype).view(-1))
    return out


M32 = 0xFFFFFFFF


def _plain_uniform(n, rng):
    """n 16-bit numbers: Philox4x32 of 10 rounds, a block for every eight elements."""
    q = torch.arange((n + 7) // 8, device=rng.device)
    seed, offset = rng[0], rng[1]
    k0, k1 = seed & M32, (seed >> 32) & M32
    c0, c1, c2, c3 = q & M32, q >> 32, offset & M32, (offset >> 32) & M32
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57  # products of 32-bit numbers, their 64 bits in an int64
        c0, c1, c2, c3 = ((b >> 32) & M32) ^ c1 ^ k0, b & M32, ((a >> 32) & M32) ^ c3 ^ k1, a & M32
        k0, k1 = (k0 + 0x9E3779B9) & M32, (k1 + 0xBB67AE85) & M32
    return torch.stack([c0 & 0xFFFF, c0 >> 16, c1 & 0xFFFF, c1 >> 16, c2 & 0xFFFF, c2 >> 16, c3 & 0xFFFF, c3 >> 16],
                       1).view(-1)[:n]


def _plain_do(s):
    c = s["case"]
    cut = round(c["p"] * 65536)
    x, dy = s["x"], s["dy"]
    kept = (_plain_uniform(x.numel(), s["rng"]) >= cut).view(x.shape)
    scale = 65536.0 / (65536 - cut)
    zero = torch.zeros((), device=x.device)
    y = torch.where(kept, x.float() * scale, zero)
    if s["residual"] is not None:
        y += s["residual"].float()
    return dict(y=y.to(x.dtype), dx=torch.where(kept, dy.float() * scale, zero).to(dy.dtype))


def _live(s):
    c = s["case"]
    if s["lengths"] is None:
        return (torch.ones(c["b"], c["n"], c["l"], dtype=torch.bool, device=s["nll"].device),
                torch.full((c["b"], c["n"]), c["l"], device=s["nll"].device))
    return torch.arange(c["l"], device=s["nll"].device) < s["lengths"][..., None], s["lengths"]


def _plain_po(s):
    c = s["case"]
    nll, old, ref = s["nll"], s["old_nll"], s["ref_nll"]
    a = s["advantages"] if c["per_token"] else s["advantages"][..., None]
    live, lens = _live(s)
    tokens, zero = lens.sum(), torch.zeros((), device=nll.device)
    # in 64 bits: whether a ratio is past the border, and the loss, in which a list's advantages cancel
    ratio = torch.exp(old.double() - nll.double())
    cut = live & torch.where(a >= 0, (ratio > 1.0 + CLIP_HIGH) & (a > 0), ratio < 1.0 - CLIP_LOW)
    held = torch.where(a >= 0, 1.0 + CLIP_HIGH, 1.0 - CLIP_LOW)
    loss = -torch.where(cut, held.double(), ratio) * a
    slope = torch.where(cut, zero, ratio.float() * a)
    del ratio, held
    kl = zero.double()
    if ref is not None:
        u = nll.double() - ref.double()
        e = torch.expm1(u)
        k = e - u
        loss += c["kl"] * k
        slope += c["kl"] * e.float()
        kl = torch.where(live, k, zero.double()).sum()
        del u, e, k
    loss, slope = torch.where(live, loss, zero.double()), torch.where(live, slope, zero)
    stats = torch.stack([kl / tokens, cut.sum() / tokens.double()]).float()
    if c["reduction"] == "sequence_mean":
        w = (1.0 / (lens.clamp(min=1) * (lens > 0).sum()).double())[..., None]
    elif c["reduction"] == "mean":
        w = 1.0 / tokens.double()
    else:
        w = zero.double() + 1.0
    out = loss if c["reduction"] == "none" else (loss * w).sum()
    return dict(loss=out.float(), stats=stats, dnll=slope * (w * s["grad"]).float())


def _plain_pr(s):
    c = s["case"]
    nll, ref = s["nll"], s["ref_nll"]
    live, lens = _live(s)
    d = nll.double() if ref is None else nll.double() - ref.double()
    r = -torch.where(live, d, torch.zeros((), dtype=torch.float64, device=nll.device)).sum(2)
    if c["average"]:
        r = r / lens.clamp(min=1)
    pair = (s["chosen"] >= 0) & (s["rejected"] >= 0)
    at = torch.arange(c["b"], device=nll.device)
    i, j = s["chosen"].long().clamp(min=0), s["rejected"].long().clamp(min=0)
    z = (BETA * (r[at, i] - r[at, j]) - c["margin"]).float()
    e = torch.exp(-z.abs())
    tail = torch.log1p(e)
    up = torch.where(z >= 0, 1.0, e) / (1.0 + e)  # 1 / (1 + exp(-z))
    dn = torch.where(z >= 0, e, 1.0) / (1.0 + e)
    zero = torch.zeros((), device=nll.device)
    loss = torch.where(pair, (1.0 - c["smooth"]) * ((-z).clamp(min=0) + tail) + c["smooth"] * (z.clamp(min=0) + tail), zero)
    pairs = pair.sum()
    w = s["grad"] / pairs if c["reduction"] == "mean" else s["grad"]
    dz = torch.where(pair, (c["smooth"] * up - (1.0 - c["smooth"]) * dn) * w * BETA, zero)
    coef = torch.zeros(c["b"], c["n"], device=nll.device)
    coef[at, i] -= dz
    coef[at, j] += dz
    if c["average"]:
        coef = coef / lens.clamp(min=1)
    total = loss if c["reduction"] == "none" else loss.double().sum()
    return dict(loss=(total / pairs).float() if c["reduction"] == "mean" else total.float(),
                margins=torch.where(pair, z, zero), dnll=torch.where(live, coef[..., None], zero))


# ---- the package's calls

def _own(s):
    from ctc_prefix_beam_gb300 import head
    c = s["case"]
    if c["op"] == "gn":
        y, mean, rstd = head.group_norm(s["x"], c["g"], s["weight"], s["bias"], lengths=s["lengths"], eps=EPS,
                                        activation=c["act"])
        if not c["train"]:
            return dict(y=y)
        dx, dw, db = head.group_norm_backward(s["dy"], s["x"], c["g"], s["weight"], s["bias"], mean, rstd,
                                              lengths=s["lengths"], activation=c["act"])
        return dict(y=y, dx=dx, dweight=dw, dbias=db)
    if c["op"] == "do":
        y = head.dropout(s["x"], c["p"], s["rng"], residual=s["residual"])
        return dict(y=y, dx=head.dropout_backward(s["dy"], c["p"], s["rng"]))
    if c["op"] == "po":
        loss, stats, dnll = head.policy_loss(s["nll"], s["old_nll"], s["advantages"], lengths=s["lengths"],
                                             ref_nll=s["ref_nll"], clip_low=CLIP_LOW, clip_high=CLIP_HIGH,
                                             kl_weight=c["kl"], reduction=c["reduction"], grad=s["grad"])
        return dict(loss=loss, stats=stats, dnll=dnll)
    loss, margins, dnll = head.preference_loss(s["nll"], s["chosen"], s["rejected"], lengths=s["lengths"],
                                               ref_nll=s["ref_nll"], beta=BETA, margin=c["margin"],
                                               label_smoothing=c["smooth"], average=c["average"],
                                               reduction=c["reduction"], grad=s["grad"])
    return dict(loss=loss, margins=margins, dnll=dnll)


def run(state):
    if own:
        return _own(state)
    return {"gn": _plain_gn, "do": _plain_do, "po": _plain_po, "pr": _plain_pr}[state["case"]["op"]](state)


def work(case):
    if case["op"] == "gn":
        e, p = ({"bf16": 2, "f16": 2, "f32": 4}[case[k]] for k in ("type", "params"))
        full = case["b"] * case["t"] * case["c"]
        # a padded batch: frames past an utterance's end are a quarter, written and not read
        read = (0.75 if case["ragged"] else 1.0) * full
        if case["train"]:  # x in, y out; dy and x in, dx out
            return dict(bytes=(3 * read + 2 * full) * e + 6 * case["c"] * p, flops=40 * read)
        return dict(bytes=(read + full) * e + 2 * case["c"] * p, flops=15 * read)
    if case["op"] == "do":
        e, n = {"bf16": 2, "f16": 2, "f32": 4}[case["type"]], case["n"] * case["h"]
        return dict(bytes=(5 if case["residual"] else 4) * n * e, flops=16 * n)
    full = case["b"] * case["n"] * case["l"]
    part = 0.75 if case["ragged"] else 1.0
    if case["op"] == "po":
        reads = 2 + (1 if case["kl"] else 0) + (1 if case["per_token"] else 0)
        writes = 2 if case["reduction"] == "none" else 1
        return dict(bytes=4 * (reads * part + writes) * full, flops=25 * part * full)
    # two hypotheses of each list are read, the gradients of all are written
    return dict(bytes=4 * ((2 if case["ref"] else 1) * part * 2 * case["b"] * case["l"] + full),
                flops=4 * part * case["b"] * case["l"])


# ---- the definitions in 64 bits

def _exact_gn(case, s):
    grads = case["train"]
    w, beta = (s[k].double().requires_grad_(grads) for k in ("weight", "bias"))
    b, t, c, g = case["b"], case["t"], case["c"], case["g"]
    y = torch.zeros(b, t, c, dtype=torch.float64, device="cuda")
    dx = torch.zeros_like(y) if grads else None
    dw, db = torch.zeros_like(w), torch.zeros_like(beta)
    lens = [t] * b if s["lengths"] is None else s["lengths"].tolist()
    for i, n in enumerate(lens):
        if not n:
            continue
        x = s["x"][i, :n].double().requires_grad_(grads)
        by = x.view(n, g, c // g).transpose(0, 1).reshape(g, -1)
        var, mean = torch.var_mean(by, 1, correction=0, keepdim=True)
        h = ((by - mean) / torch.sqrt(var + EPS)).view(g, n, c // g).transpose(0, 1).reshape(n, c) * w + beta
        a = h * torch.sigmoid(h) if case["act"] == "silu" else torch.relu(h) if case["act"] == "relu" else h
        y[i, :n] = a.detach()
        if grads:
            gx, gw, gb = torch.autograd.grad(a, (x, w, beta), s["dy"][i, :n].double())
            dx[i, :n] = gx
            dw += gw
            db += gb
    return dict(y=y, dx=dx, dweight=dw.detach(), dbias=db.detach()) if grads else dict(y=y)


def _limbs_product(a, const):
    """(high, low) 32 bits of a 32-bit tensor times a 32-bit number, by 16-bit halves."""
    al, ah, bl, bh = a & 0xFFFF, a >> 16, const & 0xFFFF, const >> 16
    mid = (al * bl >> 16) + (ah * bl & 0xFFFF) + (al * bh & 0xFFFF)
    return (ah * bh + (ah * bl >> 16) + (al * bh >> 16) + (mid >> 16)), ((mid & 0xFFFF) << 16) | (al * bl & 0xFFFF)


def _exact_do(case, s):
    seed, offset = (int(v) % 2 ** 64 for v in s["rng"].tolist())
    n = case["n"] * case["h"]
    block = torch.arange(-(-n // 8), device="cuda")
    ctr = [block % 2 ** 32, block // 2 ** 32, torch.full_like(block, offset % 2 ** 32), torch.full_like(block, offset >> 32)]
    keys = [(((seed % 2 ** 32) + r * 0x9E3779B9) % 2 ** 32, ((seed >> 32) + r * 0xBB67AE85) % 2 ** 32) for r in range(10)]
    for k0, k1 in keys:
        h0, l0 = _limbs_product(ctr[0], 0xD2511F53)
        h1, l1 = _limbs_product(ctr[2], 0xCD9E8D57)
        ctr = [h1 ^ ctr[1] ^ k0, l1, h0 ^ ctr[3] ^ k1, l0]
    at = torch.arange(n, device="cuda")
    word = torch.stack(ctr)[at % 8 // 2, at // 8]
    half = torch.where(at % 2 == 1, word >> 16, word & 0xFFFF)
    cut = round(case["p"] * 65536)
    factor = ((half >= cut).double() * (65536.0 / (65536 - cut))).view(case["n"], case["h"])
    y = s["x"].double() * factor
    return dict(y=y if s["residual"] is None else y + s["residual"].double(), dx=s["dy"].double() * factor)


def _exact_po(case, s):
    b, n, l = case["b"], case["n"], case["l"]
    lens = torch.full((b * n,), l, device="cuda") if s["lengths"] is None else s["lengths"].reshape(-1).long()
    seq = torch.repeat_interleave(torch.arange(b * n, device="cuda"), lens)  # the sequence of each token
    start = torch.cumsum(lens, 0) - lens
    at = seq * l + torch.arange(seq.numel(), device="cuda") - start[seq]
    nll = s["nll"].reshape(-1)[at].double().requires_grad_()
    a = s["advantages"].double().reshape(-1)[at if case["per_token"] else seq]
    ratio = torch.exp(s["old_nll"].reshape(-1)[at].double() - nll)
    held = ratio.clamp(1.0 - CLIP_LOW, 1.0 + CLIP_HIGH)
    low = ratio * a > held * a
    loss = -torch.where(low, held * a, ratio * a)
    kl = torch.zeros((), dtype=torch.float64, device="cuda")
    if s["ref_nll"] is not None:
        u = nll - s["ref_nll"].reshape(-1)[at].double()
        k = torch.expm1(u) - u
        loss = loss + case["kl"] * k
        kl = k.detach().mean()
    if case["reduction"] == "none":
        total = torch.zeros(b * n * l, dtype=torch.float64, device="cuda").index_copy(0, at, loss)
        weighted = (total * s["grad"].double().reshape(-1)).sum()
        total = total.view(b, n, l)
    else:
        if case["reduction"] == "mean":
            total = loss.mean()
        elif case["reduction"] == "sum":
            total = loss.sum()
        else:
            total = (loss / lens[seq]).sum() / (lens > 0).sum()
        weighted = total * s["grad"].double()
    slope, = torch.autograd.grad(weighted, nll)
    dnll = torch.zeros(b * n * l, dtype=torch.float64, device="cuda").index_copy(0, at, slope)
    return dict(loss=total.detach(), stats=torch.stack([kl, low.double().mean()]), dnll=dnll.view(b, n, l))


def _exact_pr(case, s):
    b, n, l = case["b"], case["n"], case["l"]
    lens = torch.full((b, n), l, device="cuda") if s["lengths"] is None else s["lengths"].long()
    nll = s["nll"].double().requires_grad_()
    gain = -nll if s["ref_nll"] is None else s["ref_nll"].double() - nll
    cum = torch.cat([torch.zeros(b, n, 1, dtype=torch.float64, device="cuda"), gain.cumsum(2)], 2)
    score = cum.gather(2, lens[..., None])[..., 0]  # the sum up to the length
    if case["average"]:
        score = score / lens.clamp(min=1)
    keep = ((s["chosen"] >= 0) & (s["rejected"] >= 0)).nonzero()[:, 0]
    z = BETA * (score[keep, s["chosen"][keep].long()] - score[keep, s["rejected"][keep].long()]) - case["margin"]
    loss = -(1 - case["smooth"]) * torch.nn.functional.logsigmoid(z) - case["smooth"] * torch.nn.functional.logsigmoid(-z)
    if case["reduction"] == "none":
        total = torch.zeros(b, dtype=torch.float64, device="cuda").index_copy(0, keep, loss)
        weighted = (total * s["grad"].double()).sum()
    else:
        total = loss.mean() if case["reduction"] == "mean" else loss.sum()
        weighted = total * s["grad"].double()
    dnll, = torch.autograd.grad(weighted, nll)
    margins = torch.zeros(b, dtype=torch.float64, device="cuda").index_copy(0, keep, z.detach())
    return dict(loss=total.detach(), margins=margins, dnll=dnll)


def exact(case, seed):
    return {"gn": _exact_gn, "do": _exact_do, "po": _exact_po, "pr": _exact_pr}[case["op"]](case, prepare(case, seed))
