"""Event streams over clustered instruments: which cluster does the next event hit?

The clustering gives every instrument soft loadings (rows of H) and a label. A
stream of events (the instrument that had a tail day, one after another) is a
sequence of instruments. This small model reads it with the library's sequence
operators:

    x_t    = scale * E[i_t]            api.embed, E starts as the unit rows of H
    gate_t = G[i_t]                    api.embed, how much of the past an event keeps
    h_t    = a_t h_{t-1} + (1 - a_t) x_t,  a_t = sigmoid(gate_t)    api.gated_scan
    ln p   = log softmax(h_t)[label(i_{t+1})]                       api.token_logprobs

so h holds one pressure per cluster, the log probabilities score the cluster of
the event that came, the entropy says how open the next one is and the
alternatives name the clusters next in line. Training follows the gradient
through the four operators (``token_logprobs_grad``, ``gated_scan_grad``, two
``embed_grad``) with the diagonal AdaGrad step of the fit. A live stream goes on
one event at a time from its state (``EventModel.step``).

Usage: python -m symmetric_nmf_clustering_amd.events [--n 256] [--k 4] [--steps 30]
"""
from __future__ import annotations

import argparse
import json
import sys

import numpy as np


def event_stream(labels: np.ndarray, streams: int, length: int, stay: float = 0.7, seed: int = 0):
    """Seeded synthetic events: ``streams`` sequences of ``length`` instruments.
    Each event hits a member of the stream's current group with probability
    ``stay`` (any instrument otherwise); after an event the current group moves
    to another one with probability 0.1. Returns int64 ids (streams x length)."""
    rng = np.random.default_rng(seed)
    labels = np.asarray(labels)
    groups = [np.flatnonzero(labels == g) for g in np.unique(labels)]
    ids = np.empty((streams, length), dtype=np.int64)
    for s in range(streams):
        g = rng.integers(len(groups))
        for t in range(length):
            inside = rng.random() < stay
            ids[s, t] = rng.choice(groups[g]) if inside else rng.integers(labels.size)
            if rng.random() < 0.1:
                g = rng.integers(len(groups))
    return ids


class EventModel:
    """Loadings table E and gate table G (n x k float32 device tensors)."""

    def __init__(self, H, scale: float = 4.0, gate: float = 1.0):
        import torch

        self.E = torch.nn.functional.normalize(H, dim=1)
        self.G = torch.full_like(self.E, gate)
        self.scale = scale
        self._sum = [torch.zeros_like(self.E), torch.zeros_like(self.E)]  # AdaGrad

    def _read(self, ids):
        from . import api

        return api.embed(self.E, ids, scale=self.scale), api.embed(self.G, ids)

    def score(self, ids, next_labels, lengths=None, top: int = 2):
        """TokenLogprobs of each next event's cluster, after the events so far
        (rows of streams x length; -1 in ``next_labels``: nothing to score)."""
        from . import api

        h, _ = api.gated_scan(*self._read(ids), lengths=lengths)
        return api.token_logprobs(h.view(-1, h.shape[2]), next_labels.reshape(-1), top=top)

    def gradients(self, ids, next_labels, lengths=None):
        """(mean -ln p, dE, dG) over the events that have a next one."""
        import torch

        from . import api

        x, gate = self._read(ids)
        h, _, states = api.gated_scan(x, gate, lengths=lengths, return_states=True)
        flat, tok = h.view(-1, h.shape[2]), next_labels.reshape(-1)
        r = api.token_logprobs(flat, tok)
        count = (tok >= 0).sum().clamp_min(1)
        w = (-1.0 / count).expand_as(r.logp)
        dh = api.token_logprobs_grad(flat, tok, r.lse, None, w).view_as(h)
        dx, dgate, _ = api.gated_scan_grad(x, gate, states, dh, lengths=lengths)
        n = self.E.shape[0]
        return (-(r.logp.double().sum() / count), api.embed_grad(dx, ids, n, scale=self.scale),
                api.embed_grad(dgate, ids, n))

    def train_step(self, ids, next_labels, lengths=None, lr: float = 0.01, eps: float = 1e-8):
        """One AdaGrad step on both tables; returns the loss before it."""
        loss, dE, dG = self.gradients(ids, next_labels, lengths)
        for table, acc, g in ((self.E, self._sum[0], dE), (self.G, self._sum[1], dG)):
            acc.addcmul_(g, g)
            table.addcdiv_(g, acc.sqrt().add_(eps), value=-lr)
        return loss

    def step(self, ids, state):
        """One live event per stream: (scores of the next one's clusters
        (streams x k), the new state)."""
        from . import api

        return api.gated_step(*self._read(ids), state)


def next_labels(ids, labels, lengths=None):
    """Cluster label of each event's successor (-1 after a stream's last one, and
    where the successor is an empty slot)."""
    import torch

    nxt = torch.full_like(ids, -1)
    after = ids[:, 1:]
    nxt[:, :-1] = torch.where(after < 0, -1, labels.to(ids.dtype)[after.clamp_min(0).long()])
    if lengths is not None:
        t = torch.arange(ids.shape[1], device=ids.device)[None, :]
        nxt[t >= lengths[:, None] - 1] = -1
    return nxt


def run(n: int = 256, k: int = 4, T: int = 96, streams: int = 64, length: int = 256,
        steps: int = 30, seed: int = 0) -> dict:
    """Cluster a synthetic window, then learn its event streams: the mean log
    probability of held-out events before and after, with the mean entropy and
    how often the cluster that came was among the two best."""
    import torch

    from . import api, synth

    w = synth.gaussian_blocks(n=n, k=k, T=T, seed=seed)
    S, _ = api.build_S(torch.from_numpy(w.X).cuda(), "abscorr")
    res = api.fit(S, k, solver="full", seed=seed, max_iters=200)
    lab = api.labels(res.H)
    train, test = (torch.from_numpy(event_stream(w.labels, streams, length, seed=s)).cuda()
                   for s in (seed + 1, seed + 2))
    model = EventModel(res.H)

    def measure():
        tok = next_labels(test, lab)
        r = model.score(test, tok, top=2)
        has = tok.reshape(-1) >= 0
        hit = (r.top_ids == tok.reshape(-1, 1)).any(1)
        return {"logp": r.logp[has].mean().item(), "entropy": r.entropy[has].mean().item(),
                "top2": hit[has].float().mean().item()}

    before = measure()
    tok = next_labels(train, lab)
    losses = [model.train_step(train, tok).item() for _ in range(steps)]
    after = measure()
    return {"n": n, "k": k, "streams": streams, "length": length, "steps": steps,
            "uniform_logp": -float(np.log(k)), "before": before, "after": after,
            "loss_first": losses[0] if losses else None, "loss_last": losses[-1] if losses else None}


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--n", type=int, default=256)
    ap.add_argument("--k", type=int, default=4)
    ap.add_argument("--streams", type=int, default=64)
    ap.add_argument("--length", type=int, default=256)
    ap.add_argument("--steps", type=int, default=30)
    ap.add_argument("--seed", type=int, default=0)
    args = ap.parse_args(argv)
    print(json.dumps(run(**vars(args))), flush=True)


if __name__ == "__main__":
    sys.exit(main())
