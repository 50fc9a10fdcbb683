"""The label head's operators on their own: what each reads, what it has to return, and the sizes it meets.

A CTC acoustic model ends in a layer norm and a linear head; the head's log-softmax is the decoder's
``log_prob``.  Training the head frame by frame (from an alignment), or scoring the tokens of N-best
hypotheses with a language model's head, is softmax cross entropy over the same product.  The operators:

    ln   layer norm; with ``train`` also its backward pass (dx, dweight, dbias)
    lp   the decoder's input: log-softmax(x w^T + b), float32
    ce   softmax cross entropy of x w^T + b; with ``train`` the mean loss and (dx, dw, db),
         without it every row's loss

``run`` computes them from elementary 32-bit operations, or, where ``own`` is true, by the calls a user
makes of the package.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = 1e-5
IGNORE = -1


def listed():
    return [
        # one frame of 128 concurrent streams through the final norm: latency only
        dict(name="ln one frame, 128 streams", op="ln", n=128, h=512, type="bf16", params="f32", train=False),
        # a small float32 model in training, a width that no vector load divides
        dict(name="ln train, odd width, f32", op="ln", n=3001, h=769, type="f32", params="f32", train=True),
        # a training batch of 128 utterances of 500 frames
        dict(name="ln train, 64000 frames", op="ln", n=64000, h=1024, type="bf16", params="bf16", train=True),
        # one frame of 128 concurrent streams: the streaming decoder's input for one step
        dict(name="lp one frame, 128 streams", op="lp", n=128, v=5000, h=512, type="bf16", params="f32"),
        # a 16-frame chunk of 128 streams: the streaming decoder's input for one chunk
        dict(name="lp chunk, 128 streams", op="lp", n=2048, v=5000, h=512, type="bf16", params="f32"),
        # a 32-utterance offline batch of 500 frames over 5000 word pieces
        dict(name="lp offline, word pieces", op="lp", n=16000, v=5000, h=512, type="bf16", params="bf16"),
        # a character model's offline batch: a vocabulary far narrower than any tile
        dict(name="lp offline, characters", op="lp", n=16000, v=29, h=256, type="f16", params="f16"),
        # a tiny model's training step, 50 frames: latency only
        dict(name="ce train, tiny", op="ce", n=50, v=32, h=64, type="bf16", params="f32", pad=False, train=True),
        # frame-wise training of the word-piece head; frames past an utterance's end are ignored
        dict(name="ce train, word pieces", op="ce", n=16000, v=5000, h=512, type="bf16", params="f32", pad=True,
             train=True),
        # odd everything, half precision
        dict(name="ce train, ragged, f16", op="ce", n=4099, v=10007, h=771, type="f16", params="f16", pad=True,
             train=True),
        # a language model's head in training over a large vocabulary
        dict(name="ce train, large vocabulary", op="ce", n=8192, v=65536, h=2048, type="bf16", params="bf16",
             pad=False, train=True),
        # rescoring: every token of 10-best lists of 32 utterances, 40 tokens each
        dict(name="ce score, 10-best lists", op="ce", n=12800, v=32000, h=1024, type="bf16", params="bf16",
             pad=False, train=False),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["ln", "lp", "lp", "ce", "ce", "ce"])
    kind = rng.choice(["bf16", "bf16", "f16"])
    if op == "ln":
        kind = rng.choice(["bf16", "f16", "f32"])
        h = _log(rng, 16, 8192)
        if rng.random() < 0.6:
            h = max(16, h // 16 * 16)
        n = _log(rng, 1, max(1, min(64000, 64000 * 1024 // h)))
        return dict(op="ln", n=n, h=h, type=kind, params=rng.choice([kind, "f32"]), train=rng.random() < 0.6)
    h = _log(rng, 64, 2048)
    if rng.random() < 0.7:
        h = h // 64 * 64
    if op == "lp":
        v = _log(rng, 29, 32768)
        n = _log(rng, 1, min(16000, 16000 * 5000 // v))
        return dict(op="lp", n=n, v=v, h=h, type=kind, params=rng.choice([kind, "f32"]))
    v = _log(rng, 29, 65536)
    n = _log(rng, 1, min(16000, int(3e11 // (v * h))))
    return dict(op="ce", n=n, v=v, h=h, type=kind, params=rng.choice([kind, "f32"]), pad=rng.random() < 0.5,
                train=rng.random() < 0.7)


def _labels(n, v, pad, g):
    """Frame labels of utterances of up to 500 frames: blank (0) for 0.7 of the frames, else any label;
    the frames past an utterance's end, drawn from half its length on, are ignored."""
    lab = torch.randint(1, v, (n,), generator=g, device="cuda")
    lab = torch.where(torch.rand(n, generator=g, device="cuda") < 0.7, torch.zeros_like(lab), lab)
    if pad:
        t = min(n, 500)
        ends = torch.randint(max(1, t // 2), t + 1, (-(-n // t),), generator=g, device="cuda")
        at = torch.arange(n, device="cuda")
        lab = torch.where(at % t < ends[at // t], lab, torch.full_like(lab, IGNORE))
    return lab.to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 17)
    kind, params = TYPES[case["type"]], TYPES[case["params"]]
    n, h = case["n"], case["h"]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    if case["op"] == "ln":
        # a residual stream: every frame with a level and a spread of its own
        x = normal(n, h) * (0.5 + 2.0 * torch.rand(n, 1, generator=g, device="cuda")) + 0.3 * normal(n, 1)
        s = dict(case=case, x=x.to(kind), weight=(1.0 + 0.2 * normal(h)).to(params), bias=(0.1 * normal(h)).to(params))
        if case["train"]:
            s["dy"] = (normal(n, h) * 0.01).to(kind)
        return s
    v = case["v"]
    w = normal(v, h) * (1.5 / math.sqrt(h))
    lab = _labels(n, v, case.get("pad", False), g)
    # a trained head's frames: noise, and towards the frame's label
    x = normal(n, h) + 3.0 * w[lab.long().clamp(min=0)]
    s = dict(case=case, x=x.to(kind), weight=w.to(kind), bias=(0.5 * normal(v)).to(params))
    if case["op"] == "ce":
        s["targets"] = lab
        if case["train"]:
            # the loss's own gradient: half precision is trained with a loss scale
            s["grad"] = torch.full((), 1024.0 if case["type"] == "f16" else 1.0, device="cuda")
    return s


# ---- the plain forms: 32-bit elementary operations, rounded once at the end

def _plain_ln(s):
    x, w, b = s["x"].float(), s["weight"].float(), s["bias"].float()
    d = x - x.mean(1, keepdim=True)
    r = torch.rsqrt((d * d).mean(1, keepdim=True) + EPS)
    xh = d * r
    out = dict(y=(xh * w + b).to(s["x"].dtype))
    if s["case"]["train"]:
        dy = s["dy"].float()
        t = dy * w
        dx = r * (t - t.mean(1, keepdim=True) - xh * (t * xh).mean(1, keepdim=True))
        out.update(dx=dx.to(s["x"].dtype), dweight=(dy * xh).sum(0).to(s["weight"].dtype),
                   dbias=dy.sum(0).to(s["bias"].dtype))
    return out


def _plain_logits(s):
    z = s["x"].float() @ s["weight"].float().t() + s["bias"].float()
    m = z.max(1, keepdim=True).values
    return z, m + torch.log(torch.exp(z - m).sum(1, keepdim=True))


def _plain_lp(s):
    z, lse = _plain_logits(s)
    return dict(log_prob=z - lse)


def _plain_ce(s):
    z, lse = _plain_logits(s)
    t = s["targets"].long()
    valid = t != IGNORE
    at = t.clamp(min=0)[:, None]
    loss = torch.where(valid, (lse - z.gather(1, at))[:, 0], torch.zeros_like(lse[:, 0]))
    if not s["case"]["train"]:
        return dict(loss=loss)
    scale = s["grad"] / valid.sum()
    d = torch.exp(z - lse)
    del z
    d.scatter_add_(1, at, torch.full_like(lse, -1.0))
    d *= valid[:, None] * scale
    return dict(loss=loss.sum() / valid.sum(), dx=(d @ s["weight"].float()).to(s["x"].dtype),
                dw=(d.t() @ s["x"].float()).to(s["weight"].dtype), db=d.sum(0).to(s["bias"].dtype))


# ---- the package's calls

def _own(s):
    from ctc_prefix_beam_gb300 import head
    c = s["case"]
    if c["op"] == "ln":
        y, mean, rstd = head.layer_norm(s["x"], s["weight"], s["bias"], eps=EPS)
        if not c["train"]:
            return dict(y=y)
        dx, dw, db = head.layer_norm_backward(s["dy"], s["x"], s["weight"], mean, rstd)
        return dict(y=y, dx=dx, dweight=dw, dbias=db)
    if c["op"] == "lp":
        return dict(log_prob=head.log_probs(s["x"], s["weight"], s["bias"]))
    loss, lse = head.cross_entropy(s["x"], s["weight"], s["targets"], s["bias"], ignore_index=IGNORE,
                                   reduction="mean" if c["train"] else "none")
    if not c["train"]:
        return dict(loss=loss)
    dx, dw, db = head.cross_entropy_backward(s["grad"], s["x"], s["weight"], s["targets"], lse, s["bias"],
                                             ignore_index=IGNORE, reduction="mean")
    return dict(loss=loss, dx=dx, dw=dw, db=db)


def run(state):
    if own:
        return _own(state)
    return {"ln": _plain_ln, "lp": _plain_lp, "ce": _plain_ce}[state["case"]["op"]](state)


def work(case):
    e = {"bf16": 2, "f16": 2, "f32": 4}[case["type"]]
    p = {"bf16": 2, "f16": 2, "f32": 4}[case["params"]]
    n, h = case["n"], case["h"]
    if case["op"] == "ln":
        # x in, y out; dy in, dx out; the parameters and their gradients
        return dict(bytes=(4 if case["train"] else 2) * n * h * e + (4 if case["train"] else 2) * h * p,
                    flops=(20 if case["train"] else 8) * n * h)
    v = case["v"]
    if case["op"] == "lp":
        return dict(bytes=(n + v) * h * e + v * p + 4 * n * v, flops=2 * n * v * h)
    # an ignored row needs no product: frames past the end are a quarter of a padded batch
    rows = 0.75 * n if case["pad"] else n
    if case["train"]:  # the logits, dx and dw
        return dict(bytes=2 * (n + v) * h * e + 2 * v * p + 4 * n, flops=6 * rows * v * h)
    return dict(bytes=(n + v) * h * e + v * p + 8 * n, flops=2 * rows * v * h)


# ---- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    x, w, b = (s[k].to(torch.float64) for k in ("x", "weight", "bias"))
    if case["op"] == "ln":
        var, mean = torch.var_mean(x, dim=1, correction=0, keepdim=True)
        inv = 1.0 / torch.sqrt(var + EPS)
        xh = (x - mean) * inv
        out = dict(y=torch.addcmul(b, xh, w))
        if case["train"]:
            dy = s["dy"].to(torch.float64)
            g = dy * w
            h = case["h"]
            out["dx"] = inv / h * (h * g - g.sum(1, keepdim=True) - xh * (g * xh).sum(1, keepdim=True))
            out["dweight"] = torch.einsum("nh,nh->h", dy, xh)
            out["dbias"] = dy.sum(0)
        return out
    z = torch.addmm(b, x, w.t())
    if case["op"] == "lp":
        return dict(log_prob=torch.log_softmax(z, 1))
    lab = s["targets"].long()
    keep = (lab != IGNORE).nonzero()[:, 0]
    lab = lab[keep]
    lp = torch.log_softmax(z if keep.numel() == case["n"] else z[keep], 1)
    del z
    nll = -lp[torch.arange(keep.numel(), device=lp.device), lab]
    if not case["train"]:
        return dict(loss=torch.zeros(case["n"], dtype=torch.float64, device=lp.device).index_copy(0, keep, nll))
    p = lp.exp_()
    p[torch.arange(keep.numel(), device=p.device), lab] -= 1.0
    p *= s["grad"].to(torch.float64) / keep.numel()
    dx = torch.zeros_like(x).index_copy(0, keep, p @ w)
    return dict(loss=nll.mean(), dx=dx, dw=p.t() @ x[keep], db=p.sum(0))
