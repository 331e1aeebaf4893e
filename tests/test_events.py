"""The event-stream model: its generator (CPU), and its gradients, training and
live steps on the device."""
import numpy as np
import pytest

from oracle import sequence_oracle as so
from symmetric_nmf_clustering_amd import events


def test_event_stream_is_seeded_and_clustered():
    labels = np.repeat(np.arange(4), 25)
    a = events.event_stream(labels, 6, 400, seed=3)
    assert np.array_equal(a, events.event_stream(labels, 6, 400, seed=3))
    assert not np.array_equal(a, events.event_stream(labels, 6, 400, seed=4))
    assert a.min() >= 0 and a.max() < 100
    lab = labels[a]
    # two events in a row fall into one group far more often than 1 in 4
    assert (lab[:, 1:] == lab[:, :-1]).mean() > 0.4


def test_next_labels():
    import torch
    ids = torch.tensor([[0, 1, 2], [2, -1, -1]])
    lab = torch.tensor([5, 6, 7], dtype=torch.int32)
    assert events.next_labels(ids, lab).tolist()[0] == [6, 7, -1]
    lengths = torch.tensor([2, 1])
    assert events.next_labels(ids, lab, lengths).tolist() == [[6, -1, -1], [-1, -1, -1]]


def _model(torch, n, k, seed):
    rng = np.random.default_rng(seed)
    H = torch.from_numpy(rng.random((n, k)).astype(np.float32)).cuda()
    m = events.EventModel(H)
    m.G.copy_(torch.from_numpy(rng.standard_normal((n, k)).astype(np.float32)))
    return m, rng


@pytest.mark.gpu
def test_gradients_match_the_definitions():
    from tests.gpu_util import require_gpu
    torch = require_gpu()
    n, k, B, T = 50, 6, 5, 33
    m, rng = _model(torch, n, k, 1)
    ids = rng.integers(0, n, size=(B, T))
    lengths = np.array([33, 0, 1, 20, 33])
    for b in range(B):
        ids[b, lengths[b]:] = -1
    lab = rng.integers(0, k, size=n).astype(np.int32)
    tids, tlen = torch.from_numpy(ids).cuda(), torch.from_numpy(lengths).int().cuda()
    tok = events.next_labels(tids, torch.from_numpy(lab).cuda(), tlen)
    loss, dE, dG = m.gradients(tids, tok, tlen)
    E, G = m.E.double().cpu().numpy(), m.G.double().cpu().numpy()
    tk = tok.cpu().numpy().reshape(-1)
    x, g = so.embed(E, ids, m.scale), so.embed(G, ids, 1.0)
    h, _, _ = so.gated_scan(x, g, None, lengths)
    logp = so.token_logprobs(h.reshape(-1, k), tk, 0, 1.0)[0]
    count = (tk >= 0).sum()
    assert count == (np.maximum(lengths, 1) - 1).sum()
    w = np.full(tk.size, -1.0 / count)
    dh = so.token_logprobs_grad(h.reshape(-1, k), tk, w, None, 1.0).reshape(h.shape)
    dx, dg, _ = so.gated_scan_grad(x, g, dh, None, None, lengths)
    # float32 through four operators with values of order 1: relative 1e-5 of the
    # largest entry leaves two digits over their bounds
    for got, ref in ((dE, so.embed_grad(dx, ids, n, m.scale)), (dG, so.embed_grad(dg, ids, n, 1.0))):
        assert np.abs(got.double().cpu().numpy() - ref).max() <= 1e-5 * np.abs(ref).max()
    assert abs(loss.item() + logp.sum() / count) <= 1e-5 * abs(logp.sum() / count)


@pytest.mark.gpu
def test_live_steps_follow_the_sequence():
    from tests.gpu_util import require_gpu
    torch = require_gpu()
    from symmetric_nmf_clustering_amd import api
    m, rng = _model(torch, 40, 8, 2)
    ids = torch.from_numpy(rng.integers(0, 40, size=(7, 20))).cuda()
    h, last = api.gated_scan(*m._read(ids))
    s = torch.zeros(7, 8, device="cuda")
    for t in range(20):
        out, s = m.step(ids[:, t], s)
        # both are float32 evaluations of one convex combination of values below
        # 4 + 1: a few units of 2^-23 each per step
        assert (out - h[:, t]).abs().max() <= 20 * 5 * 2.0 ** -21
    assert (s - last).abs().max() <= 20 * 5 * 2.0 ** -21


@pytest.mark.gpu
def test_training_learns_the_streams():
    from tests.gpu_util import require_gpu
    require_gpu()
    r = events.run()
    assert r["loss_last"] < r["loss_first"]
    assert r["after"]["logp"] > r["before"]["logp"]
    assert r["after"]["logp"] > r["uniform_logp"] + 0.1   # better than no knowledge
    assert 0.0 < r["after"]["entropy"] < np.log(4)
    again = events.run()
    assert again == r                                   # the same bits on every run


def test_next_labels_of_empty_slots():
    """No label follows where the next slot is empty, with lengths and without."""
    import torch
    lab = torch.tensor([5, 6, 7], dtype=torch.int32)
    for dtype in (torch.int64, torch.int32):
        ids = torch.tensor([[0, 1, 2], [2, -1, -1], [1, -1, 0], [-1, 2, 1], [-1, -1, -1]], dtype=dtype)
        got = events.next_labels(ids, lab)
        assert got.dtype == dtype
        assert got.tolist() == [[6, 7, -1], [-1, -1, -1], [-1, 5, -1], [7, 6, -1], [-1, -1, -1]]
        lengths = torch.tensor([2, 1, 3, 3, 0])
        assert events.next_labels(ids, lab, lengths).tolist() == \
            [[6, -1, -1], [-1, -1, -1], [-1, 5, -1], [7, 6, -1], [-1, -1, -1]]
