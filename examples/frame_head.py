"""Train a label head frame by frame, then decode with it, offline and streaming.

    python examples/frame_head.py [--steps 80]

Synthetic utterances: every label is a direction in feature space, held for a
few frames, with blank frames between labels; frames past an utterance's end
are noise and carry no target.  The model is what stands before the decoder: a
layer norm and a linear head.

    y = layer_norm(x);  loss = cross_entropy(y, w, targets, b)      a training step
    log_prob = log_probs(layer_norm(x), w, b)                      the decoder's input
"""
import argparse
import os
import sys

import torch

if __package__ in (None, ""):
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from ctc_prefix_beam_gb300 import decoder as D  # noqa: E402
from ctc_prefix_beam_gb300 import head  # noqa: E402

BLANK = 0


def utterances(B, T, V, H, protos, g):
    """(x [B, T, H], frame targets [B, T] int32, lengths [B] int32, label sequences)."""
    targets = torch.full((B, T), -1, dtype=torch.int32)
    lens, seqs = [], []
    for b in range(B):
        end = int(torch.randint(T // 2, T + 1, (1,), generator=g))
        t, seq = 0, []
        while t < end:
            blanks = int(torch.randint(1, 5, (1,), generator=g))
            targets[b, t:min(t + blanks, end)] = BLANK
            t += blanks
            if t >= end:
                break
            lab, run = int(torch.randint(1, V, (1,), generator=g)), int(torch.randint(1, 4, (1,), generator=g))
            targets[b, t:min(t + run, end)] = lab
            seq.append(lab)
            t += run
        lens.append(end)
        seqs.append(seq)
    targets = targets.cuda()
    noise = torch.randn(B, T, H, generator=g).cuda()
    x = noise + 3.0 * protos[targets.clamp(min=0).long()] * (targets >= 0)[..., None]
    return x, targets, torch.tensor(lens, dtype=torch.int32, device="cuda"), seqs


def edit_distance(a, b):
    row = list(range(len(b) + 1))
    for i, x in enumerate(a, 1):
        last, row[0] = row[0], i
        for j, y in enumerate(b, 1):
            last, row[j] = row[j], min(row[j] + 1, row[j - 1] + 1, last + (x != y))
    return row[-1]


def label_error_rate(tokens, lengths, seqs):
    """Of the best hypotheses against the label sequences."""
    tokens, lengths = tokens[:, 0].cpu(), lengths[:, 0].cpu()
    wrong = sum(edit_distance(tokens[b, :lengths[b]].tolist(), s) for b, s in enumerate(seqs))
    return wrong / sum(len(s) for s in seqs)


def checked(workspace, what):
    """The status of the last call that used a workspace; it waits for the GPU."""
    status = D.read_status(workspace)
    if status:
        raise RuntimeError(f"{what}: " + ("a target is out of range" if status & head.DEV_TARGET else f"status {status:#x}"))


def main(steps=80, B=16, T=120, V=64, H=128, lr=2.0, seed=0, verbose=True):
    g = torch.Generator().manual_seed(seed)
    protos = torch.randn(V, H, generator=g).cuda() / H ** 0.5 * 2.0
    # float32 parameters; the head's product takes a 16-bit copy of its weight
    p = dict(gamma=torch.ones(H), beta=torch.zeros(H), w=torch.randn(V, H, generator=g) * 0.02, b=torch.zeros(V))
    p = {k: v.cuda() for k, v in p.items()}
    test = utterances(B, T, V, H, protos, g)
    one = torch.ones((), device="cuda")
    # workspaces of the calls, kept so that their statuses can be read
    n, dt = B * T, torch.bfloat16
    sizes = dict(lp=head.log_probs_workspace_size(dt, n, V, H),
                 ce=head.cross_entropy_workspace_size(dt, n, V, H, False),
                 grad=head.cross_entropy_workspace_size(dt, n, V, H, True))
    ws = {k: torch.empty(size, dtype=torch.uint8, device="cuda") for k, size in sizes.items()}

    def features(x):
        return head.layer_norm(x.to(torch.bfloat16), p["gamma"], p["beta"])

    def decode(x, lens):
        y, _, _ = features(x)
        log_prob = head.log_probs(y, p["w"].to(torch.bfloat16), p["b"], workspace=ws["lp"])
        checked(ws["lp"], "log-probabilities")
        return D.decode_offline(D.Config(beam=8, nbest=1), log_prob, lens)

    tokens, lengths, _ = decode(test[0], test[2])
    result = dict(error_before=label_error_rate(tokens, lengths, test[3]), losses=[])
    for step in range(steps):
        x, targets, _, _ = utterances(B, T, V, H, protos, g)
        x16, w16 = x.to(torch.bfloat16), p["w"].to(torch.bfloat16)
        y, mean, rstd = head.layer_norm(x16, p["gamma"], p["beta"])
        loss, lse = head.cross_entropy(y, w16, targets, p["b"], workspace=ws["ce"])
        dy, dw, db = head.cross_entropy_backward(one, y, w16, targets, lse, p["b"], workspace=ws["grad"])
        _, dgamma, dbeta = head.layer_norm_backward(dy, x16, p["gamma"], mean, rstd)
        for name, grad in (("gamma", dgamma), ("beta", dbeta), ("w", dw.float()), ("b", db)):
            p[name].sub_(grad, alpha=lr)
        result["losses"].append(loss.item())
        checked(ws["ce"], "loss")
        checked(ws["grad"], "gradients")
        if verbose and (step % 20 == 0 or step == steps - 1):
            print(f"step {step:3d}  loss {result['losses'][-1]:.4f}")

    x, _, lens, seqs = test
    tokens, lengths, scores = decode(x, lens)
    result["error_after"] = label_error_rate(tokens, lengths, seqs)

    # the same utterances as streams, 16 frames at a time
    st = D.StreamState(D.Config(beam=8, nbest=1, max_seq_len=T), B, V)
    w16 = p["w"].to(torch.bfloat16)
    for t in range(0, T, 16):
        y, _, _ = features(x[:, t:t + 16])
        st.step_chunk(head.log_probs(y, w16, p["b"]), n_frames=(lens - t).clamp(0, y.shape[1]).to(torch.int32))
    stok, slen, _ = st.read(out_len=T)
    result["error_streaming"] = label_error_rate(stok, slen, seqs)
    if verbose:
        print("label error rate: %.3f before training, %.3f after, %.3f streaming" %
              (result["error_before"], result["error_after"], result["error_streaming"]))
    return result


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=80)
    main(ap.parse_args().steps)
