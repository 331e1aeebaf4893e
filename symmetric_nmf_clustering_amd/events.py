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


class HistoryModel:
    """Event streams with a memory of what followed what:

        x_t = scale E[i_t],  (q, k, v)_t = x_t W,  q and k turned by t
        o_t = linear attention of the heads, each with a decay of its own
        ln p = log softmax([x_t, o_t] U)[label(i_{t+1})]

    E (n x k) starts as the unit rows of H, W and U are seeded; all float32. Head h
    keeps 1 - 2^-(h + 2) of its memory a step. ``bits``: of the optimizer's states.
    """

    def __init__(self, H, classes: int, heads: int = 4, width: int = 16, scale: float = 4.0,
                 bits: int = 32, seed: int = 0):
        import torch

        from . import api

        if width % 2:
            raise ValueError("width must be even")
        g = torch.Generator(device=H.device).manual_seed(seed)
        k = H.shape[1]

        def drawn(*shape):
            return torch.randn(*shape, generator=g, device=H.device) * shape[0] ** -0.5

        self.E = torch.nn.functional.normalize(H, dim=1)
        self.W, self.U = drawn(k, 3 * heads * width), drawn(k + heads * width, classes)
        self.U[k:] /= 32  # sums over a memory of up to 2^(heads + 1) steps start small
        self.heads, self.width, self.scale = heads, width, scale
        self.freqs, self.amplitude = api.rotary_freqs(width, device=H.device)
        self.decay = torch.log1p(-(2.0 ** -(2 + torch.arange(heads, device=H.device).float())))
        self._moments = api.adamw_states(self.parameters(), bits)
        self._step = 0

    def parameters(self):
        return [self.E, self.W, self.U]

    def _turned(self, x, positions):
        """q, k, v (... x heads x width) of x, as views of one projection."""
        from . import api

        y = (x @ self.W).unflatten(-1, (3 * self.heads, self.width))
        qk = y[..., :2 * self.heads, :]
        api.rotary(qk, positions, self.freqs, amplitude=self.amplitude, out=qk)
        return y.split(self.heads, -2)

    def _read(self, ids, lengths):
        import torch

        from . import api

        x = api.embed(self.E, ids, scale=self.scale)
        pos = torch.arange(ids.shape[1], device=ids.device).expand(ids.shape)
        q, k, v = self._turned(x, pos)
        o, last = api.linear_attention(q, k, v, self.decay, lengths=lengths)
        return x, pos, q, k, v, torch.cat([x, o.flatten(2)], 2), last

    def score(self, ids, next_labels, lengths=None, top: int = 2):
        """As ``EventModel.score``."""
        from . import api

        xo = self._read(ids, lengths)[5]
        return api.token_logprobs((xo @ self.U).flatten(0, 1), next_labels.reshape(-1), top=top)

    def gradients(self, ids, next_labels, lengths=None):
        """(mean -ln p, [dE, dW, dU]) over the events that have a next one."""
        import torch

        from . import api

        x, pos, q, k, v, xo, _ = self._read(ids, lengths)
        z, tok = (xo @ self.U).flatten(0, 1), next_labels.reshape(-1)
        r = api.token_logprobs(z, tok)
        count = (tok >= 0).sum().clamp_min(1)
        w = (-1.0 / count).expand_as(r.logp)
        dz = api.token_logprobs_grad(z, tok, r.lse, None, w)
        dxo = (dz @ self.U.t()).view_as(xo)
        do = dxo[..., x.shape[2]:].unflatten(2, (self.heads, self.width))
        parts = api.linear_attention_grad(q, k, v, self.decay, do, lengths=lengths)[:3]
        dy = torch.cat(parts, 2)
        dqk = dy[..., :2 * self.heads, :]
        api.rotary(dqk, pos, self.freqs, amplitude=self.amplitude, inverse=True, out=dqk)
        dy = dy.flatten(2)
        dx = dxo[..., :x.shape[2]] + dy @ self.W.t()
        return (-(r.logp.double().sum() / count),
                [api.embed_grad(dx, ids, self.E.shape[0], scale=self.scale),
                 x.flatten(0, 1).t() @ dy.flatten(0, 1), xo.flatten(0, 1).t() @ dz])

    def train_step(self, ids, next_labels, lengths=None, lr: float = 0.001,
                   weight_decay: float = 0.01):
        """One AdamW step on the table and the projections; returns the loss before it. (AdamW's
        first steps move every element by lr: at 0.01 the loss more than doubles before it falls.)"""
        from . import api

        loss, grads = self.gradients(ids, next_labels, lengths)
        self._step += 1
        m, v, m_scale, v_scale = self._moments
        api.adamw_step(self.parameters(), grads, m, v, self._step, lr=lr, weight_decay=weight_decay,
                       m_scale=m_scale, v_scale=v_scale)
        return loss

    def start(self, streams: int):
        """The state of new streams: (memory, events so far)."""
        import torch

        return (torch.zeros(streams, self.heads, self.width, self.width, device=self.E.device),
                torch.zeros(streams, dtype=torch.int64, device=self.E.device))

    def step(self, ids, state):
        """One live event per stream: (scores of the next one's clusters (streams x
        classes), the new state)."""
        import torch

        from . import api

        memory, seen = state
        x = api.embed(self.E, ids, scale=self.scale)
        q, k, v = self._turned(x, seen)
        o, memory = api.linear_attention_step(q, k, v, self.decay, memory)
        return torch.cat([x, o.flatten(1)], 1) @ self.U, (memory, seen + 1)


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
        steps: int = 30, seed: int = 0, model: str = "scan", bits: int = 32) -> dict:
    """Cluster a synthetic window, then learn its event streams: the mean log
    probability of held-out events before and after, with the mean entropy and
    how often the cluster that came was among the two best. ``model``: "scan"
    (EventModel) or "history" (HistoryModel, optimizer states in ``bits``)."""
    import torch

    if model not in ("scan", "history"):
        raise ValueError(f'model must be "scan" or "history", not {model!r}')

    from . import api, synth

    w = synth.gaussian_blocks(n=n, k=k, T=T, seed=seed)
    S, _ = api.build_S(torch.from_numpy(w.X).cuda(), "abscorr")
    res = api.fit(S, k, solver="full", seed=seed, max_iters=200)
    lab = api.labels(res.H)
    train, test = (torch.from_numpy(event_stream(w.labels, streams, length, seed=s)).cuda()
                   for s in (seed + 1, seed + 2))
    learner = EventModel(res.H) if model == "scan" else HistoryModel(res.H, k, bits=bits, seed=seed)

    def measure():
        tok = next_labels(test, lab)
        r = learner.score(test, tok, top=2)
        has = tok.reshape(-1) >= 0
        hit = (r.top_ids == tok.reshape(-1, 1)).any(1)
        return {"logp": r.logp[has].mean().item(), "entropy": r.entropy[has].mean().item(),
                "top2": hit[has].float().mean().item()}

    before = measure()
    tok = next_labels(train, lab)
    losses = [learner.train_step(train, tok).item() for _ in range(steps)]
    after = measure()
    return {"n": n, "k": k, "streams": streams, "length": length, "steps": steps,
            "uniform_logp": -float(np.log(k)), "before": before, "after": after,
            "loss_first": losses[0] if losses else None, "loss_last": losses[-1] if losses else None}


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--model", choices=("scan", "history"), default="scan")
    ap.add_argument("--bits", type=int, choices=(8, 32), default=32)
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
