"""GPU tests of the sequence operators where values or sizes are extreme: what
stands beside masked steps, gates at their limits, logits far from zero,
expanded inputs, more streams and rows than one launch takes."""
import numpy as np
import pytest

from oracle import sequence_oracle as so
from tests import test_gpu_sequence as base
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")
KINDS = ["fp32", "bf16", "fp16"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("batch,steps,width", [(2, 6, 5), (3, 40, 300), (2, 200, 16), (2, 300, 7), (2, 2500, 16)])
def test_masked_steps_of_the_scan_gradient_are_zero_whatever_passes_them(batch, steps, width, kind):
    """The gradient at the last state and the state itself pass the masked steps;
    neither, infinite or NaN, may show in their dx and dgate. Other channels keep
    their bits."""
    torch = require_gpu()
    from symmetric_nmf_clustering_amd import api
    gen = torch.Generator(device="cuda").manual_seed(steps)
    x, g, dh = (torch.randn(batch, steps, width, generator=gen, device="cuda").to(base.types(torch)[kind])
                for _ in range(3))
    h0, dl = (torch.randn(batch, width, generator=gen, device="cuda") for _ in range(2))
    n = torch.arange(batch, device="cuda", dtype=torch.int32) * 3 + steps // 2
    n[0] = 0
    masked = torch.arange(steps, device="cuda")[None, :] >= n[:, None]

    def run(x, h0, dl):
        _, last, st = api.gated_scan(x, g, h0=h0, lengths=n, return_states=True)
        return api.gated_scan_grad(x, g, st, dh, dh_last=dl, lengths=n)
    want = run(x, h0, dl)
    px, ph, pl = x.clone(), h0.clone(), dl.clone()
    pl[:, 0], pl[:, 1], pl[:, 2] = INF, -INF, NAN
    ph[:, 3] = NAN
    px[1, n[1] - 1, 4] = NAN
    got = run(px, ph, pl)
    for a, b in zip(got[:2], want[:2]):
        assert not a[masked].any() and not torch.isnan(a[masked]).any()
        assert torch.equal(a[:, :, 5:], b[:, :, 5:])
        # dgate where the state is NaN; both where the gradient is not finite
        assert not torch.isfinite(a[1, :n[1], :3]).any()
    assert torch.isnan(got[1][1, :n[1], 3]).all()
    assert torch.equal(got[2][:, 5:], want[2][:, 5:])
    assert torch.equal(got[2][0], pl[0]) or torch.isnan(pl[0, 2])  # row 0 has no step
    assert torch.equal(got[2][0, [0, 1, 3]], pl[0, [0, 1, 3]]) and torch.isnan(got[2][0, 2])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("steps", [1, 5, 9, 200, 2500])
def test_a_gate_of_minus_infinity_drops_every_finite_state(steps, kind):
    torch = require_gpu()
    from symmetric_nmf_clustering_amd import api
    gen = torch.Generator(device="cuda").manual_seed(steps)
    x, dh = (torch.randn(2, steps, 12, generator=gen, device="cuda").to(base.types(torch)[kind]) for _ in range(2))
    big = torch.full((2, 12), 3e38, device="cuda")
    for gate in (torch.full_like(x, -INF), torch.full_like(x[0, 0], -INF).expand(2, steps, 12)):
        h, last, st = api.gated_scan(x, gate, h0=big, return_states=True)
        assert torch.equal(h, x) and torch.equal(last, x[:, -1].float())
        # and nothing of later steps' gradients reaches earlier ones
        dx, dgate, dh0 = api.gated_scan_grad(x, gate, st, dh, dh_last=big * 0)
        assert torch.equal(dx, dh) and not dgate.any() and not dh0.any()
        assert not torch.isnan(dgate).any()


def test_gates_over_their_whole_range():
    """a and c = 1 - a to (8 + 2 |g|) u each; below 2^-126 they may be 0."""
    torch = require_gpu()
    from symmetric_nmf_clustering_amd import api
    g = np.concatenate([np.linspace(-110, 110, 4401), [-3e38, 3e38, -1e4, 1e4, -88.8, 88.8, 0.0, -0.0]])
    t, gv = base.dev(torch, g)
    width = g.size
    one, none = torch.full((1, width), 2.0 ** 96, device="cuda"), torch.zeros(1, width, device="cuda")
    rel = (8 + 2 * np.minimum(np.abs(gv), 128)) * base.U  # the exponential's argument, and log2(e), to u each
    for steps in (1, 9):  # walked, and as a tile of which one step counts
        n = torch.ones(1, dtype=torch.int32, device="cuda")
        gate = t.expand(1, steps, width)
        ones = one.expand(1, steps, width)
        for x, h0, ref in ((none.expand(1, steps, width), one, so.sigmoid(gv)), (ones, none, so.sigmoid(-gv))):
            got = api.gated_scan(x, gate, h0=h0, lengths=n)[1][0].double().cpu().numpy() * 2.0 ** -96
            assert (np.abs(got - ref) <= rel * ref + 2.0 ** -126).all()
    # the gate's gradient falls off with a and c
    x, h0 = torch.zeros(1, 9, width, device="cuda"), torch.full((1, width), 2.0 ** 60, device="cuda")
    dh = torch.zeros(1, 9, width, device="cuda")
    dh[:, 0] = 2.0 ** 60
    gate = t.expand(1, 9, width)
    n = torch.ones(1, dtype=torch.int32, device="cuda")
    st = api.gated_scan(x, gate, h0=h0, lengths=n, return_states=True)[2]
    dg = api.gated_scan_grad(x, gate, st, dh, lengths=n)[1][0, 0].double().cpu().numpy() * 2.0 ** -120
    ref = so.sigmoid(gv) * so.sigmoid(-gv)
    assert (np.abs(dg - ref) <= (2 * rel + 4 * base.U) * ref + 2.0 ** -126 + 2.0 ** -149).all()


def check_grad_anywhere(zv, tok, w, q, scale, got, kind):
    """As check_grad, with an error of ln p that knows no lse: (|ln p| + 8) 4 u for
    its own rounding, at most 64 u where a small lse was rounded, and the sum's
    (logprob_bounds)."""
    lp, lse, h = so.log_softmax(zv, scale)
    p = np.exp(lp)
    wv, qv = w.double().cpu().numpy()[:, None], q.double().cpu().numpy()[:, None]
    core, bh = (b[:, None] for b in np.broadcast_arrays(*base.logprob_bounds(0 * np.ones(zv.shape), 1.0, np.zeros(len(zv)))))
    lp = np.where(np.isfinite(lp), lp, 0)
    ep = (np.abs(lp) + 8 + 64) * 4 * base.U + core
    bound = scale * (p * (np.abs(wv) + np.abs(qv) * (np.abs(lp) + h[:, None])) * (ep + 8 * base.U)
                     + np.abs(qv) * p * (ep + bh)
                     + 4 * base.U * np.abs(wv) * (np.arange(zv.shape[1])[None] == tok[:, None]))
    base.close(got, so.token_logprobs_grad(zv, tok, wv[:, 0], qv[:, 0], scale), bound, kind)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("count,vocab", [(5, 2), (70, 24), (9, 512), (6, 1003), (5, 2600), (5, 8200), (3, 20011)])
def test_logit_gradient_of_rows_far_from_zero(count, vocab, kind):
    """A common offset of the logits changes nothing, and neither does a mask of
    the type's lowest value (for a whole row: every column alike)."""
    torch = require_gpu()
    from symmetric_nmf_clustering_amd import api
    rng = np.random.default_rng(vocab)
    low = torch.finfo(base.types(torch)[kind]).min
    z = rng.standard_normal((count, vocab)) * 3
    z[::3, 1:][rng.random(z[::3, 1:].shape) < 0.5] = -np.inf
    at = np.broadcast_to(np.arange(vocab), z.shape)
    one, third = at == 1, at % 3 == 1
    rows = {"offset 50": z + 50, "offset 3000": z + 3000, "offset -30000": z - 30000,
            "confident": np.where(one, 3020.0, 3000.0),
            "lowest": np.full_like(z, low), "lowest but one": np.where(one, 0.0, low),
            "lowest and none": np.where(third, -np.inf, low),
            "highest": np.where(one, 0.0, -low)}
    tok = rng.integers(-1, vocab, size=count)
    dtok = torch.from_numpy(tok).cuda()
    w, q = (torch.from_numpy(rng.standard_normal(count).astype(np.float32)).cuda() for _ in range(2))
    for name, r in rows.items():
        t, zv = base.dev(torch, r, kind)
        for scale in (1.0, 0.7, 4.0):
            f = api.token_logprobs(t, dtok, scale=scale)
            d = api.token_logprobs_grad(t, dtok, f.lse, f.entropy, w, dentropy=q, scale=scale)
            check_grad_anywhere(zv, tok, w, q, np.float64(np.float32(scale)), d, kind)
            own = t.clone()
            api.token_logprobs_grad(own, dtok, f.lse, f.entropy, w, dentropy=q, scale=scale, out=own)
            assert torch.equal(own, d), name


def test_logit_gradient_takes_the_normaliser_it_is_given():
    """The columns in two parts, each with the whole row's lse and entropy."""
    torch = require_gpu()
    from symmetric_nmf_clustering_amd import api
    rng = np.random.default_rng(9)
    for offset in (0.0, 3000.0):
        for vocab in (40, 700, 12000):
            z, zv = base.dev(torch, rng.standard_normal((6, vocab)) + offset)
            tok = np.array([0, 1, vocab - 1, vocab // 2, -1, 5])
            dtok = torch.from_numpy(tok).cuda()
            w, q = (torch.from_numpy(rng.standard_normal(6).astype(np.float32)).cuda() for _ in range(2))
            f = api.token_logprobs(z, dtok)
            half = vocab // 2
            parts = []
            for lo, hi in ((0, half), (half, vocab)):
                at = torch.where((dtok >= lo) & (dtok < hi), dtok - lo, hi - lo - 1)
                here = ((dtok >= lo) & (dtok < hi)).float()
                d = api.token_logprobs_grad(z[:, lo:hi], at, f.lse, f.entropy, w, dentropy=q)
                # rows whose token lies in the other part: its one-hot put back
                fix = torch.zeros_like(d)
                fix[torch.arange(6, device="cuda"), at] = torch.where(dtok < 0, 0.0, 1.0) * w * (here - 1)
                fix[dtok < 0, at[dtok < 0]] = -w[dtok < 0]
                parts.append((d + fix, at))
            p = torch.softmax(z.double(), 1)
            ref = so.token_logprobs_grad(zv, np.maximum(tok, -1), w.double().cpu().numpy(), q.double().cpu().numpy(), 1.0)
            ref[4] -= (w[4].double() * p[4]).cpu().numpy()  # its parts were given a token
            got = torch.cat([a for a, _ in parts], 1).double().cpu().numpy()
            # p relative to 4 u (|lse| + |ln p| + 8), the one-hot's cancellation to 4 u
            lp = np.log(np.exp(zv - zv.max(1, keepdims=True)).sum(1)).max() + np.ptp(zv)
            ep = (offset + 2 * lp + 16) * 4 * base.U
            wq = (w.abs() + q.abs() * 40).double().cpu().numpy()[:, None]
            assert (np.abs(got - ref) <= wq * (p.cpu().numpy() * ep * 2 + 8 * base.U)).all()


@pytest.mark.parametrize("vocab", [24, 3001])
def test_excluded_columns_stay_without_gradient_under_large_weights(vocab):
    """p (ln p + H) is 0 at an excluded column for every finite weight."""
    torch = require_gpu()
    from symmetric_nmf_clustering_amd import api
    rng = np.random.default_rng(vocab)
    z = rng.standard_normal((6, vocab))
    z[:, ::2] = -np.inf
    t, zv = base.dev(torch, z)
    tok = torch.ones(6, dtype=torch.int64, device="cuda")
    f = api.token_logprobs(t, tok)
    w = torch.zeros(6, device="cuda")
    for weight in (1e9, -3e20, 1e34):
        d = api.token_logprobs_grad(t, tok, f.lse, f.entropy, w, dentropy=torch.full_like(w, weight))
        assert torch.isfinite(d).all() and not d[:, ::2].any()
        unit = api.token_logprobs_grad(t, tok, f.lse, f.entropy, w, dentropy=torch.ones_like(w))
        # one product more or less, each to u
        assert ((d / weight - unit).abs() <= 4 * base.U * unit.abs() + 1e-37).all()


@pytest.mark.parametrize("kind", KINDS)
def test_embedding_gradient_of_an_expanded_dout(kind):
    """What a sum or a mean over events sends back: one row, or one number, for all."""
    torch = require_gpu()
    from symmetric_nmf_clustering_amd import api
    rng = np.random.default_rng(8)
    for count, rows, width in ((1, 3, 5), (90, 20, 12), (9000, 70, 24)):
        ids = torch.from_numpy(rng.integers(-1, rows, size=(count,))).cuda()
        row, _ = base.dev(torch, rng.standard_normal(width), kind)
        num, _ = base.dev(torch, rng.standard_normal(1), kind)
        late, _ = base.dev(torch, rng.standard_normal(count + width), kind)
        for d in (row.expand(count, width), num.expand(count, width), late.as_strided((count, width), (1, 1)),
                  row[:1].expand(count, width)):
            assert torch.equal(api.embed_grad(d, ids, rows), api.embed_grad(d.contiguous(), ids, rows))
        two = ids.view(1, count).expand(2, count)
        d = row.expand(2, count, width)
        assert torch.equal(api.embed_grad(d, two, rows), api.embed_grad(d.contiguous(), two, rows))


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("steps", [1, 20])
def test_more_streams_than_a_call_of_the_library_takes(steps, kind):
    """One stream per instrument: batch rows past 65535, with every optional input."""
    torch = require_gpu()
    from symmetric_nmf_clustering_amd import api
    gen = torch.Generator(device="cuda").manual_seed(steps)
    batch, width = 65535 * 2 + 700, 6
    x, g, dh = (torch.randn(batch, steps, width, generator=gen, device="cuda").to(base.types(torch)[kind])
                for _ in range(3))
    h0, dl = (torch.randn(batch, width, generator=gen, device="cuda") for _ in range(2))
    n = torch.randint(0, steps + 1, (batch,), generator=gen, device="cuda").int()
    one = g[0, 0].expand(batch, steps, width)
    for gate in (g, one):
        h, last, st = api.gated_scan(x, gate, h0=h0, lengths=n, return_states=True)
        grads = api.gated_scan_grad(x, gate, st, dh, dh_last=dl, lengths=n)
        for lo in range(0, batch, 40000):  # the same rows in smaller batches
            s = slice(lo, min(lo + 40000, batch))
            a = api.gated_scan(x[s], gate[s], h0=h0[s], lengths=n[s], return_states=True)
            b = api.gated_scan_grad(x[s], gate[s], a[2], dh[s], dh_last=dl[s], lengths=n[s])
            for whole, part in zip((h, last, st, *grads), (*a, *b)):
                assert torch.equal(whole[s], part)
        assert torch.equal(api.gated_scan(x, gate)[0], torch.cat([api.gated_scan(x[i:i + 60000], gate[i:i + 60000])[0]
                                                                  for i in range(0, batch, 60000)]))
    out, state = api.gated_step(x[:, 0], g[:, 0], h0)
    for lo in range(0, batch, 40000):
        s = slice(lo, min(lo + 40000, batch))
        a, b = api.gated_step(x[s, 0], g[s, 0], h0[s])
        assert torch.equal(out[s], a) and torch.equal(state[s], b)
    with pytest.raises(ValueError):
        api.gated_step(x[:, 0], g[:, 0], h0[:-1])
    with pytest.raises(ValueError):
        api.gated_scan(x, g, lengths=n[:-1])


def test_embedding_of_more_rows_than_a_launch_takes():
    """2^24 and some rows of 513 columns, a workgroup each: 2^32 threads and more."""
    torch = require_gpu()
    from symmetric_nmf_clustering_amd import api
    rows, width, count = 1 << 10, 513, (1 << 24) + 1023
    table = torch.randn(rows, width, device="cuda")
    ids = torch.arange(count, device="cuda", dtype=torch.int32) % rows
    out = api.embed(table, ids, dtype=torch.bfloat16)
    want = table.bfloat16()
    for lo in range(0, count, 1 << 21):  # whole periods of the ids
        part = out[lo:lo + (1 << 21)]
        n = part.shape[0] // rows * rows
        assert (part[:n].view(-1, rows, width) == want).all()
        assert torch.equal(part[n:], want[:part.shape[0] - n])


def test_scan_of_more_channels_than_a_launch_takes():
    """Single steps of 2^32 channels of odd width, a thread each."""
    torch = require_gpu()
    from symmetric_nmf_clustering_amd import api
    batch, width = 65535, 65601
    x, g = (torch.randn(width, device="cuda").bfloat16() for _ in range(2))
    h, last = api.gated_scan(x.expand(batch, 1, width), g.expand(batch, 1, width))
    one, one_last = api.gated_scan(x.expand(1, 1, width), g.expand(1, 1, width))
    for lo in range(0, batch, 4096):
        assert (h[lo:lo + 4096] == one).all() and (last[lo:lo + 4096] == one_last).all()


def test_scan_of_more_tiles_than_a_launch_is_given():
    """2^20 workgroups and more, forward and backward: several launches."""
    torch = require_gpu()
    from symmetric_nmf_clustering_amd import api
    batch, steps, width = 65535, 9, 512 * 17
    x, g, d = (torch.randn(steps, width, device="cuda").bfloat16() for _ in range(3))
    n = (torch.arange(batch, device="cuda") % 10).int()
    big = [t.expand(batch, steps, width) for t in (x, g, d)]
    few = [t.expand(10, steps, width) for t in (x, g, d)]
    h, last, st = api.gated_scan(big[0], big[1], lengths=n, return_states=True)
    want = api.gated_scan(few[0], few[1], lengths=n[:10], return_states=True)

    def same(a, b):
        for lo in range(0, batch, 5000):
            part = a[lo:lo + 5000]
            assert (part.view(-1, 10, *part.shape[1:]) == b).all() if len(part) == 5000 else \
                torch.equal(part, b.repeat(-(-len(part) // 10), *[1] * (b.dim() - 1))[:len(part)])
    for a, b in zip((h, last, st), want):
        same(a, b)
    del h, last
    dx, dg, dh0 = api.gated_scan_grad(big[0], big[1], st, big[2], lengths=n)
    want = api.gated_scan_grad(few[0], few[1], want[2], few[2], lengths=n[:10])
    for a, b in zip((dx, dg, dh0), want):
        same(a, b)


@pytest.mark.parametrize("kind,vocab,count,top", [("bf16", 65, (1 << 26) + 2 * 999, 2), ("bf16", 1032, (1 << 22) + 2 * 999, 3),
                                                  ("bf16", 8200, (1 << 20) + 2 * 999, 2)])
def test_log_probabilities_of_more_rows_than_a_launch_is_given(kind, vocab, count, top):
    """Rows by the register kernel, by a wave and by a workgroup: several launches."""
    torch = require_gpu()
    from symmetric_nmf_clustering_amd import api
    period = 1 << 12
    z = torch.randn(period, vocab, device="cuda").to(base.types(torch)[kind])
    tok = torch.randint(-1, vocab, (period,), device="cuda").int()
    copies = -(-count // period)
    many = torch.empty(copies, period, vocab, dtype=z.dtype, device="cuda")
    many.copy_(z)
    r = api.token_logprobs(many.view(-1, vocab)[:count], tok.repeat(copies)[:count], top=top)
    want = api.token_logprobs(z, tok, top=top)
    whole = count // period * period
    for a, b in ((r.logp, want.logp), (r.entropy, want.entropy), (r.lse, want.lse), (r.top_ids, want.top_ids),
                 (r.top_logp, want.top_logp)):
        assert (a[:whole].view(-1, *b.shape) == b).all()
        assert torch.equal(a[whole:], b[:count - whole])


@pytest.mark.parametrize("rows,width", [(540001, 257), ((1 << 29) + 1000, 33)])
def test_embedding_gradient_clears_tables_of_many_rows(rows, width):
    """More rows without tokens than the launch has workgroups for, and more than a
    launch could have (2^24)."""
    torch = require_gpu()
    from symmetric_nmf_clustering_amd import api
    gen = torch.Generator(device="cuda").manual_seed(3)
    ids = torch.randint(0, rows, (9000,), generator=gen, device="cuda")
    ids[:3] = torch.tensor([0, rows - 1, 70])
    ids[100:200] = 70
    d = torch.randint(-8, 9, (9000, width), generator=gen, device="cuda").bfloat16()  # sums are exact
    out = torch.empty(rows, width, dtype=torch.bfloat16, device="cuda")
    out.view(torch.int16).fill_(0x7fc0)  # NaN
    api.embed_grad(d, ids, rows, out=out)
    named, at = torch.unique(ids, return_inverse=True)
    want = torch.zeros(len(named), width, device="cuda", dtype=torch.float64).index_add_(0, at, d.double())
    assert torch.equal(out[named].double(), want.bfloat16().double())
    out[named] = 0
    for lo in range(0, rows, 1 << 24):
        assert not out[lo:lo + (1 << 24)].view(torch.int16).any()


def test_embedding_gradient_of_the_widest_tables():
    """Short lists into rows of more column tiles than a grid's second dimension is said to take."""
    torch = require_gpu()
    from symmetric_nmf_clustering_amd import api
    width = 65535 * 128 + 300
    d = torch.randn(3, width, device="cuda").bfloat16()
    got = api.embed_grad(d, torch.tensor([1, 0, 1], device="cuda"), 3)
    assert torch.equal(got[0], d[1].float()) and torch.equal(got[1], d[0].float() + d[2].float())
    assert not got[2].any()
    more = torch.ones(3, width, device="cuda")
    api.embed_grad(d, torch.tensor([1, -1, 1], device="cuda"), 3, out=more, accumulate=True)
    assert (more[0] == 1).all() and torch.equal(more[1], 1 + (d[0].float() + d[2].float()))


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("batch,width", [(1, 64 * 127), (2, 64 * 64), (1, 64 * 191), (3, 64 * 64), (1, 64 * 255 - 1)])
def test_scan_where_cutting_time_begins(batch, width, kind):
    torch = require_gpu()
    from symmetric_nmf_clustering_amd import api
    rng = np.random.default_rng(width)
    steps = 530
    x, xv = base.dev(torch, rng.standard_normal((batch, steps, width)), kind)
    g, gv = base.dev(torch, rng.standard_normal((batch, steps, width)) + 2, kind)
    n = np.full(batch, 517)
    tn = torch.from_numpy(n).int().cuda()
    E, bx, bg, bm = base.scan_bounds(xv, gv, None, n, xv, None)
    h, last, st = api.gated_scan(x, g, lengths=tn, return_states=True)
    hr, lr, before = so.gated_scan(xv, gv, None, n)
    base.close(h, hr, E[:, 1:], kind)
    base.close(last, lr, E[:, -1])
    base.close(st, before[:, :-1:128], E[:, :-1:128])
    dx, dg, dh0 = api.gated_scan_grad(x, g, st, x, lengths=tn)
    rx, rg, r0 = so.gated_scan_grad(xv, gv, xv, None, None, n)
    base.close(dx, rx, bx, kind)
    base.close(dg, rg, bg, kind)
    base.close(dh0, r0, bm)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("vocab", [2, 24, 40, 130, 520, 1003, 2600])
def test_logit_gradient_of_near_and_far_rows_side_by_side(vocab, kind):
    """Rows that share a wave or a workgroup, every fourth far from zero, of the
    lowest value, empty or plain."""
    torch = require_gpu()
    from symmetric_nmf_clustering_amd import api
    rng = np.random.default_rng(vocab)
    count = 45
    z = rng.standard_normal((count, vocab)) * 3
    z[1::4] += 2000
    z[2::4] = torch.finfo(base.types(torch)[kind]).min
    z[3::4] = -np.inf
    t, zv = base.dev(torch, z, kind)
    tok = rng.integers(-1, vocab, size=count)
    dtok = torch.from_numpy(tok).cuda()
    w, q = (torch.from_numpy(rng.standard_normal(count).astype(np.float32)).cuda() for _ in range(2))
    f = api.token_logprobs(t, dtok)
    d = api.token_logprobs_grad(t, dtok, f.lse, f.entropy, w, dentropy=q)
    full = np.arange(count) % 4 != 3
    check_grad_anywhere(zv[full], tok[full], w[full], q[full], 1.0, d[full], kind)
    assert not d[3::4].any()
    wide = torch.zeros(count, vocab + 3, dtype=t.dtype, device="cuda")[:, 1:-2]  # rows at every alignment
    wide.copy_(t)
    api.token_logprobs_grad(wide, dtok, f.lse, f.entropy, w, dentropy=q, out=wide)
    check_grad_anywhere(zv[full], tok[full], w[full], q[full], 1.0, wide[full], kind)
