"""The history model: its gradients, live steps and training on the device."""
import numpy as np
import pytest

from oracle import layers_oracle as lo
from oracle import sequence_oracle as so
from symmetric_nmf_clustering_amd import events

pytestmark = pytest.mark.gpu


def _model(torch, n, k, classes, seed, **kw):
    rng = np.random.default_rng(seed)
    H = torch.from_numpy(rng.random((n, k)).astype(np.float32)).cuda()
    return events.HistoryModel(H, classes, seed=seed, **kw), rng


def _scores(m, E, W, U, ids, lengths):
    """The model's scores in float64, from the definitions."""
    B, T = ids.shape
    x = so.embed(E, ids, m.scale)
    y = (x @ W).reshape(B, T, 3 * m.heads, m.width)
    pos = np.broadcast_to(np.arange(T), (B, T))
    qk = lo.rotary(y[:, :, :2 * m.heads], pos, m.freqs.cpu().numpy(), amplitude=m.amplitude)
    o, _ = lo.linear_attention(qk[:, :, :m.heads], qk[:, :, m.heads:], y[:, :, 2 * m.heads:],
                               m.decay.double().cpu().numpy(), None, lengths, m.width ** -0.5)
    return np.concatenate([x, o.reshape(B, T, -1)], 2) @ U


def test_gradients_against_differences_of_the_definitions():
    from tests.gpu_util import require_gpu
    torch = require_gpu()
    n, k, classes, B, T = 30, 6, 5, 4, 70
    m, rng = _model(torch, n, k, classes, 1, heads=3, width=8)
    ids = rng.integers(0, n, size=(B, T))
    lengths = np.array([70, 0, 1, 33])
    for b in range(B):
        ids[b, lengths[b]:] = -1
    lab = rng.integers(0, classes, size=n).astype(np.int32)
    tids, tlen = torch.from_numpy(ids).cuda(), torch.from_numpy(lengths).int().cuda()
    tok = events.next_labels(tids, torch.from_numpy(lab).cuda(), tlen)
    loss, grads = m.gradients(tids, tok, tlen)
    tk = tok.cpu().numpy().reshape(-1)
    count = (tk >= 0).sum()
    at = [p.double().cpu().numpy() for p in m.parameters()]

    def value(ps):
        z = _scores(m, *ps, ids, lengths).reshape(-1, classes)
        return -so.token_logprobs(z, tk, 0, 1.0)[0].sum() / count

    # float32 through the layers: six operators and three products, values of order 1 to 4
    assert abs(loss.item() - value(at)) <= 1e-5 * abs(value(at))
    for i, g in enumerate(grads):
        g = g.double().cpu().numpy()
        for _ in range(2):
            d = rng.standard_normal(at[i].shape)
            h = 1e-5
            hi, lo_ = list(at), list(at)
            hi[i], lo_[i] = at[i] + h * d, at[i] - h * d
            want = (value(hi) - value(lo_)) / (2 * h)
            # float32's 1e-5 of the terms' root mean square, and the differences' own h^2
            scale = np.sqrt((g ** 2).sum()) * np.sqrt((d ** 2).mean())
            assert abs((g * d).sum() - want) <= 1e-4 * scale


@pytest.mark.parametrize("B,T", [(7, 20), (1, 1)])
def test_live_steps_follow_the_sequence(B, T):
    from tests.gpu_util import require_gpu
    torch = require_gpu()
    m, rng = _model(torch, 40, 8, 6, 2)
    ids = torch.from_numpy(rng.integers(0, 40, size=(B, T))).cuda()
    z = m._read(ids, None)[5] @ m.U
    want = _scores(m, *(p.double().cpu().numpy() for p in m.parameters()), ids.cpu().numpy(), None)
    state = m.start(B)
    for t in range(T):
        out, state = m.step(ids[:, t], state)
        # both are float32 evaluations of sums of at most 100 terms of order 10
        for got in (out, z[:, t]):
            assert np.abs(got.double().cpu().numpy() - want[:, t]).max() <= 100 * 10 * 2.0 ** -21
    assert state[1].tolist() == [T] * B


@pytest.mark.parametrize("bits", [32, 8])
def test_training_runs(bits):
    from tests.gpu_util import require_gpu
    require_gpu()
    r = events.run(model="history", bits=bits, steps=6, length=128)
    assert np.isfinite(r["loss_first"]) and np.isfinite(r["loss_last"])
    assert r["loss_first"] != r["loss_last"]
    assert events.run(model="history", bits=bits, steps=6, length=128) == r  # the same bits on every run


def test_refusals():
    from tests.gpu_util import require_gpu
    torch = require_gpu()
    with pytest.raises(ValueError):
        events.HistoryModel(torch.ones(4, 3, device="cuda"), 2, width=5)
    with pytest.raises(ValueError):
        events.run(model="other")
