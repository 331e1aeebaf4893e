"""GPU tests of the layer operators against their float64 definitions.

Tolerances are per element, from float32 arithmetic (u = 2^-24), the roundings
that a type's kernel makes on the way (bfloat16: one of at most 2^-8 relative on
every term) and the one rounding of the output: see each ``bound``.
"""
import numpy as np
import pytest

from oracle import layers_oracle as lo
from tests.gpu_util import require_gpu
from tests.test_gpu_sequence import U, close, dev, types

pytestmark = pytest.mark.gpu


# ---- linear attention ---------------------------------------------------------

def attend_bound(kind, steps, dk, dv):
    """Relative to the sums of absolute values: a term meets at most dk + dv roundings of its
    dot product, 64 of its chunk, 3 a chunk of 32 steps on the state's way (each product and sum
    at most 2 u: the matrix cores may truncate), and in bfloat16 one rounding (P, or the state
    as an operand) of at most 2^-8."""
    return 2 * U * (dk + dv + 64 + 3 * (steps // 32 + 1) + 16) + (2.0 ** -8 if kind == "bf16" else 0.0)


def make(torch, kind, B, T, H, G, dk, dv, seed, lengths=None, decay=None):
    rng = np.random.default_rng(seed)
    t, x = {}, {}
    for name, shape in (("q", (B, T, H, dk)), ("k", (B, T, G, dk)), ("v", (B, T, G, dv)),
                        ("do", (B, T, H, dv))):
        t[name], x[name] = dev(torch, rng.standard_normal(shape), kind)
    for name in ("state", "dlast"):
        t[name], x[name] = dev(torch, rng.standard_normal((B, H, dk, dv)))
    t["decay"], x["decay"] = dev(torch, -np.exp(rng.uniform(-7, 0.5, H)) if decay is None else decay)
    t["lengths"] = x["lengths"] = None
    if lengths is not None:
        x["lengths"] = np.asarray(lengths)
        t["lengths"] = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    return t, x


def check_forward(got, x, kind, scale, state=True):
    B, T, H, dk = x["q"].shape
    dv = x["v"].shape[3]
    s = x["state"] if state else None
    ref = lo.linear_attention(x["q"], x["k"], x["v"], x["decay"], s, x["lengths"], scale)
    mag = lo.linear_attention(*(abs(x[n]) for n in "qkv"), x["decay"], None if s is None else abs(s),
                              x["lengths"], scale)
    c = attend_bound(kind, T, dk, dv)
    close(got[0], ref[0], c * mag[0], kind)
    close(got[1], ref[1], attend_bound("fp32", T, dk, dv) * mag[1])


def check_grad(got, x, kind, scale, state=True, dlast=True):
    B, T, H, dk = x["q"].shape
    dv = x["v"].shape[3]
    s, d = x["state"] if state else None, x["dlast"] if dlast else None
    ref = lo.linear_attention_grad(x["q"], x["k"], x["v"], x["decay"], x["do"], d, s, x["lengths"], scale)
    mag = lo.linear_attention_grad(*(abs(x[n]) for n in "qkv"), x["decay"], abs(x["do"]),
                                   None if d is None else abs(d), None if s is None else abs(s),
                                   x["lengths"], scale)
    # (a shared head's sum adds at most one u a term)
    c = attend_bound(kind, T, dk, dv) + 2 * U * H
    for i in range(3):
        close(got[i], ref[i], c * mag[i], kind)
    close(got[3], ref[3], attend_bound("fp32", T, dk, dv) * mag[3])


SIZES = [(1, 1, 1, 1, 1, 1), (2, 5, 3, 3, 8, 8), (3, 31, 2, 1, 24, 24), (1, 64, 4, 2, 64, 64),
         (2, 65, 2, 2, 33, 50), (1, 200, 6, 3, 128, 128), (2, 97, 2, 1, 80, 17), (1, 130, 1, 1, 256, 256),
         (1, 70, 2, 2, 16, 256), (1, 129, 2, 2, 200, 40), (1, 33, 3, 1, 32, 32), (2, 96, 1, 1, 7, 129)]


@pytest.mark.parametrize("kind", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("B,T,H,G,dk,dv", SIZES)
def test_linear_attention(kind, B, T, H, G, dk, dv):
    torch = require_gpu()
    from symmetric_nmf_clustering_amd import api
    t, x = make(torch, kind, B, T, H, G, dk, dv, T + dk)
    scale = dk ** -0.5
    got = api.linear_attention(t["q"], t["k"], t["v"], t["decay"], state=t["state"])
    check_forward(got, x, kind, scale)
    again = api.linear_attention(t["q"], t["k"], t["v"], t["decay"], state=t["state"])
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    got = api.linear_attention_grad(t["q"], t["k"], t["v"], t["decay"], t["do"], dlast=t["dlast"],
                                    state=t["state"])
    check_grad(got, x, kind, scale)
    again = api.linear_attention_grad(t["q"], t["k"], t["v"], t["decay"], t["do"], dlast=t["dlast"],
                                      state=t["state"])
    assert all(torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.parametrize("kind", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("T,lengths", [(70, [70, 0, 1, 64, 65]), (1100, [1100, 0, 500, 256, 1]),
                                       (512, [512, 511, 257, 600, -3]), (33, [32, 33, 31, 0, 2])])
def test_lengths(kind, T, lengths):
    """Padded batches: masked steps hold NaN, which nothing reads; some are cut in time."""
    torch = require_gpu()
    from symmetric_nmf_clustering_amd import api
    t, x = make(torch, kind, 5, T, 2, 1, 24, 40, T, lengths)
    for b, n in enumerate(lengths):
        for name in ("q", "k", "v", "do"):
            t[name][b, max(0, n):] = float("nan")
            x[name][b, max(0, n):] = 0.0
    for state in (True, False):
        s = t["state"] if state else None
        got = api.linear_attention(t["q"], t["k"], t["v"], t["decay"], state=s, lengths=t["lengths"], scale=0.3)
        check_forward(got, x, kind, 0.3, state)
        got = api.linear_attention_grad(t["q"], t["k"], t["v"], t["decay"], t["do"], state=s,
                                        dlast=t["dlast"] if state else None, lengths=t["lengths"], scale=0.3)
        check_grad(got, x, kind, 0.3, state, state)
        for i, b in ((0, 1), (0, 3)):
            n = min(max(lengths[b], 0), T)
            assert not got[i][b, n:].any()


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("B,T,H,dk,dv", [(1, 3000, 2, 64, 64), (1, 2049, 1, 128, 96), (2, 1500, 1, 24, 24)])
def test_long_histories_are_cut(kind, B, T, H, dk, dv):
    torch = require_gpu()
    from symmetric_nmf_clustering_amd import api
    t, x = make(torch, kind, B, T, H, H, dk, dv, 3)
    got = api.linear_attention(t["q"], t["k"], t["v"], t["decay"], state=t["state"], scale=0.2)
    check_forward(got, x, kind, 0.2)
    got = api.linear_attention_grad(t["q"], t["k"], t["v"], t["decay"], t["do"], dlast=t["dlast"],
                                    state=t["state"], scale=0.2)
    check_grad(got, x, kind, 0.2)


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
def test_decays_at_their_ends(kind):
    """Nothing kept (-inf, and far below), everything kept (0), and a growing memory."""
    torch = require_gpu()
    from symmetric_nmf_clustering_amd import api
    decay = [-np.inf, -1e30, -300.0, -90.0, -1e-6, 0.0, 0.01]
    t, x = make(torch, kind, 2, 150, 7, 7, 16, 20, 5, lengths=[150, 77], decay=decay)
    with np.errstate(invalid="ignore"):
        got = api.linear_attention(t["q"], t["k"], t["v"], t["decay"], state=t["state"], lengths=t["lengths"])
        check_forward(got, x, kind, 0.25)
        got = api.linear_attention_grad(t["q"], t["k"], t["v"], t["decay"], t["do"], dlast=t["dlast"],
                                        state=t["state"], lengths=t["lengths"])
        check_grad(got, x, kind, 0.25)
    t["decay"][0] = float("nan")
    o, last = api.linear_attention(t["q"], t["k"], t["v"], t["decay"], state=t["state"])
    assert torch.isnan(o[:, :, 0]).all() and torch.isnan(last[:, 0]).all()
    assert torch.isfinite(o[:, :, 1:]).all() and torch.isfinite(last[:, 1:]).all()


def test_strides_alignment_and_broadcast():
    torch = require_gpu()
    from symmetric_nmf_clustering_amd import api
    for kind in ("fp32", "bf16", "fp16"):
        rng = np.random.default_rng(7)
        B, T, H, G, dk, dv = 2, 67, 4, 2, 24, 33
        # one projection's columns: q heads, k heads, v heads next to one another, from an odd start
        wide, wv = dev(torch, rng.standard_normal((B, T, 1 + H * dk + G * dk + G * dv)), kind)
        t, x = make(torch, kind, B, T, H, G, dk, dv, 8)

        def heads(a, at, n, d):
            return a[:, :, at:at + n * d].unflatten(2, (n, d)) if hasattr(a, "unflatten") else \
                a[:, :, at:at + n * d].reshape(B, T, n, d)

        for name, at, n, d in (("q", 1, H, dk), ("k", 1 + H * dk, G, dk), ("v", 1 + (H + G) * dk, G, dv)):
            t[name], x[name] = heads(wide, at, n, d), heads(wv, at, n, d)
        t["do"] = t["do"].transpose(0, 1).contiguous().transpose(0, 1)  # steps first
        args = (t["q"], t["k"], t["v"], t["decay"])
        check_forward(api.linear_attention(*args, state=t["state"]), x, kind, dk ** -0.5)
        check_grad(api.linear_attention_grad(*args, t["do"], dlast=t["dlast"], state=t["state"]), x, kind,
                   dk ** -0.5)
        # one key row for the whole batch, one gradient row for all steps
        t["k"], x["k"] = t["k"][:1].expand(B, -1, -1, -1), np.broadcast_to(x["k"][:1], x["k"].shape)
        t["do"], x["do"] = t["do"][:, :1].expand(-1, T, -1, -1), np.broadcast_to(x["do"][:, :1], x["do"].shape)
        args = (t["q"], t["k"], t["v"], t["decay"])
        check_forward(api.linear_attention(*args, state=t["state"]), x, kind, dk ** -0.5)
        check_grad(api.linear_attention_grad(*args, t["do"], dlast=t["dlast"], state=t["state"]), x, kind,
                   dk ** -0.5)


def test_no_steps():
    torch = require_gpu()
    from symmetric_nmf_clustering_amd import api
    t, x = make(torch, "bf16", 2, 0, 4, 2, 24, 33, 9)
    o, last = api.linear_attention(t["q"], t["k"], t["v"], t["decay"], state=t["state"])
    assert o.shape == (2, 0, 4, 33) and torch.equal(last, t["state"])
    assert not api.linear_attention(t["q"], t["k"], t["v"], t["decay"])[1].any()
    dq, dk, dv, ds = api.linear_attention_grad(t["q"], t["k"], t["v"], t["decay"], t["do"], dlast=t["dlast"])
    assert dq.shape == (2, 0, 4, 24) and dk.shape == (2, 0, 2, 24) and dv.shape == (2, 0, 2, 33)
    assert torch.equal(ds, t["dlast"])


@pytest.mark.parametrize("kind", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("B,H,G,dk,dv", [(1, 1, 1, 1, 1), (64, 1, 1, 24, 24), (3, 4, 2, 128, 128), (2, 6, 2, 33, 50),
                                         (1, 2, 1, 256, 256), (5, 2, 2, 7, 65), (2, 2, 1, 255, 4)])
def test_step(kind, B, H, G, dk, dv):
    torch = require_gpu()
    from symmetric_nmf_clustering_amd import api
    t, x = make(torch, kind, B, 1, H, G, dk, dv, dk)
    ref = lo.linear_attention(x["q"], x["k"], x["v"], x["decay"], x["state"], None, 0.5)
    mag = lo.linear_attention(*(abs(x[n]) for n in "qkv"), x["decay"], abs(x["state"]), None, 0.5)
    q, k, v = (t[n][:, 0] for n in "qkv")
    state = t["state"].clone()
    o, new = api.linear_attention_step(q, k, v, t["decay"], state, scale=0.5)
    assert torch.equal(state, t["state"])
    # the state: decay, product, sum; o: dk products summed
    close(o, ref[0][:, 0], (dk + 5) * U * mag[0][:, 0], kind)
    close(new, ref[1], 4 * U * mag[1])
    o2, same = api.linear_attention_step(q, k, v, t["decay"], state, scale=0.5, out_state=state)
    assert same is state and torch.equal(o, o2) and torch.equal(state, new)


def test_steps_follow_the_sequence():
    """A history read at once, then single steps, then the sequence that holds both."""
    torch = require_gpu()
    from symmetric_nmf_clustering_amd import api
    t, x = make(torch, "fp32", 3, 90, 4, 2, 24, 24, 11)
    cut = 70
    _, s = api.linear_attention(*(t[n][:, :cut] for n in "qkv"), t["decay"], state=t["state"])
    out = []
    for i in range(cut, 90):
        o, s = api.linear_attention_step(*(t[n][:, i] for n in "qkv"), t["decay"], s)
        out.append(o)
    ref = lo.linear_attention(x["q"], x["k"], x["v"], x["decay"], x["state"], None, 24 ** -0.5)
    mag = lo.linear_attention(*(abs(x[n]) for n in "qkv"), x["decay"], abs(x["state"]), None, 24 ** -0.5)
    c = attend_bound("fp32", 90, 24, 24) + 20 * 4 * U
    close(torch.stack(out, 1), ref[0][:, cut:], c * mag[0][:, cut:])
    close(s, ref[1], c * mag[1])


def test_gradient_against_differences():
    """The outputs are linear in q, in k and state, in v and state: <do, f(x + d) - f(x)> is <dx, d>."""
    torch = require_gpu()
    from symmetric_nmf_clustering_amd import api
    t, x = make(torch, "fp32", 2, 300, 4, 2, 40, 24, 12, lengths=[300, 171])
    kw = dict(lengths=t["lengths"], scale=0.2)
    grads = api.linear_attention_grad(t["q"], t["k"], t["v"], t["decay"], t["do"], dlast=t["dlast"],
                                      state=t["state"], **kw)

    def loss(q, k, v, s):
        o, last = api.linear_attention(q, k, v, t["decay"], state=s, **kw)
        a, b = t["do"].double() * o.double(), t["dlast"].double() * last.double()
        return a.sum() + b.sum(), a.abs().sum() + b.abs().sum()

    g = torch.Generator(device="cuda").manual_seed(1)
    at = dict(q=t["q"], k=t["k"], v=t["v"], s=t["state"])
    for name, grad in zip("qkvs", grads):
        d = torch.randn(at[name].shape, generator=g, device="cuda")
        hi, lo_ = dict(at), dict(at)
        hi[name], lo_[name] = at[name] + d, at[name] - d
        (a, ma), (b, mb) = loss(**hi), loss(**lo_)
        want = (grad.double() * d.double()).sum()
        # the inputs' sums round by u each, the kernels by attend_bound of the terms' magnitudes,
        # which random signs make at most sqrt(dk T) ~ 100 times the terms seen here
        assert abs((a - b) / 2 - want) <= 100 * attend_bound("fp32", 300, 40, 24) * (ma + mb)


# ---- rotary --------------------------------------------------------------------

def rotary_bound(xv, half, interleaved, amp, far=0.0):
    """cos and sin to 8 u (the turn's rounding, 2 pi 2^-25, and the functions'), `far` on top,
    two products and a sum."""
    a = np.abs(xv)
    b = np.zeros_like(a)
    one, two = ((slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else
                (slice(0, half), slice(half, 2 * half)))
    b[..., one] = b[..., two] = (a[..., one] + a[..., two]) * (12 * U + far) * amp
    return b


@pytest.mark.parametrize("kind", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("heads,width,half", [(1, 2, 1), (3, 24, 12), (2, 128, 64), (5, 80, 20), (2, 33, 16),
                                              (1, 37, 3), (4, 96, 0), (20, 64, 30)])
def test_rotary(kind, layout, heads, width, half):
    torch = require_gpu()
    from symmetric_nmf_clustering_amd import api
    rng = np.random.default_rng(width + half)
    for n in (1, 77):
        x, xv = dev(torch, rng.standard_normal((n, heads, width)), kind)
        pos = rng.integers(-1000, 1 << 20, size=n)
        f = 10000.0 ** (-np.arange(half) / max(half, 1))
        tf = torch.from_numpy(f).cuda()
        for it in (torch.int32, torch.int64):
            tp = torch.from_numpy(pos).to(it).cuda()
            for inverse in (False, True):
                got = api.rotary(x, tp, tf, layout=layout, amplitude=1.25, inverse=inverse)
                ref = lo.rotary(xv, pos, f, layout == "interleaved", 1.25, inverse)
                close(got, ref, rotary_bound(xv, half, layout == "interleaved", 1.25), kind)
                if half * 2 < width:
                    assert torch.equal(got[..., 2 * half:], x[..., 2 * half:])
        mine = x.clone()
        assert api.rotary(mine, tp, tf, layout=layout, out=mine) is mine  # in place
        assert torch.equal(mine, api.rotary(x, tp, tf, layout=layout))
        if kind == "fp32":  # turned there and back: twice the bound, on values at most sqrt 2 larger
            back = api.rotary(mine, tp, tf, layout=layout, inverse=True)
            close(back, xv, 4 * rotary_bound(xv, half, layout == "interleaved", 1.0))


def test_rotary_strides_and_far_positions():
    torch = require_gpu()
    from symmetric_nmf_clustering_amd import api
    rng = np.random.default_rng(3)
    for kind in ("fp32", "bf16"):
        B, T, width, half = 2, 9, 24, 12
        wide, wv = dev(torch, rng.standard_normal((B, T, 1 + 5 * width)), kind)
        f = 10000.0 ** (-np.arange(half) / half)
        tf = torch.from_numpy(f).cuda()
        x, xv = wide[:, :, 1:].unflatten(2, (5, width)), wv[:, :, 1:].reshape(B, T, 5, width)
        # positions past 2^31 and 2^40, negative ones; one row for both batch rows
        pos = np.array([0, 1, -5, 2 ** 20, 2 ** 31 - 1, 2 ** 31 + 7, 2 ** 33, -2 ** 33, 123456789])
        tp = torch.from_numpy(pos).cuda().expand(B, T)
        # 2^33 radians in float64: their turns round by 3 2^-53 relative, 2^33 3 2^-53 / (2 pi) 2 pi = 2.9e-6
        bound = rotary_bound(xv, half, False, 1.0, far=3e-6)
        ref = lo.rotary(xv, np.broadcast_to(pos, (B, T)), f)
        close(api.rotary(x, tp, tf), ref, bound, kind)
        out = torch.zeros_like(wide)  # into strides of its own
        got = api.rotary(x, tp, tf, out=out[:, :, 1:].unflatten(2, (5, width)))
        close(got, ref, bound, kind)
        assert not out[:, :, 0].any()
        xt = x.transpose(0, 1)  # steps first
        close(api.rotary(xt, tp.t(), tf).transpose(0, 1), ref, bound, kind)
        part = x[:, :, 1:4]  # some heads, in place: the others stay
        mine = wide.clone()
        api.rotary(mine[:, :, 1:].unflatten(2, (5, width))[:, :, 1:4], tp, tf,
                   out=mine[:, :, 1:].unflatten(2, (5, width))[:, :, 1:4])
        close(mine[:, :, 1:].unflatten(2, (5, width))[:, :, 1:4], ref[:, :, 1:4], bound[:, :, 1:4], kind)
        assert torch.equal(mine[:, :, :1 + width], wide[:, :, :1 + width])
        assert torch.equal(mine[:, :, 1 + 4 * width:], wide[:, :, 1 + 4 * width:]) and part.shape[2] == 3
    for shape in ((0, 3, 24), (2, 0, 3, 24)):
        e = api.rotary(torch.empty(shape, device="cuda"),
                       torch.empty(shape[:-2], dtype=torch.int32, device="cuda"), tf)
        assert e.shape == shape


# ---- AdamW -----------------------------------------------------------------------

HYPER = dict(lr=0.01, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.1)


def adam_close(torch, got, x, kind, gs=1.0, step=3, hyper=HYPER):
    """p, m, v (float32 tensors or decoded) against the definition: m and v three operations each,
    the update about a dozen (root, quotient, product, the factors' own rounding)."""
    g = x["g"] * gs
    ref = lo.adamw(x["p"], g, x["m"], x["v"], step, **hyper)
    mm = np.abs(hyper["beta1"] * x["m"]) + np.abs((1 - hyper["beta1"]) * g)
    root = np.sqrt(ref[2] / (1 - hyper["beta2"] ** step)) + hyper["eps"]
    upd = hyper["lr"] * mm / (1 - hyper["beta1"] ** step) / root
    if "m" in got:
        close(got["m"], ref[1], 4 * U * mm)
        close(got["v"], ref[2], 6 * U * ref[2])
    bound = 3 * U * np.abs(x["p"]) + 20 * U * upd
    if "master" in got:
        close(got["master"], ref[0], bound)
    close(got["p"], ref[0], bound, kind)
    return ref


def adam_make(torch, shape, kind, gkind, seed):
    rng = np.random.default_rng(seed)
    t, x = {}, {}
    t["p"], x["p"] = dev(torch, rng.standard_normal(shape), kind)
    t["g"], x["g"] = dev(torch, rng.standard_normal(shape) * 10.0 ** rng.uniform(-3, 0, shape), gkind)
    t["m"], x["m"] = dev(torch, rng.standard_normal(shape) * 0.1)
    t["v"], x["v"] = dev(torch, rng.standard_normal(shape) ** 2 * 0.01)
    return t, x


@pytest.mark.parametrize("kind,gkind", [("fp32", "fp32"), ("bf16", "bf16"), ("fp16", "fp16"), ("fp32", "bf16"),
                                        ("bf16", "fp32"), ("fp16", "fp32"), ("fp32", "fp16"), ("bf16", "fp16"),
                                        ("fp16", "bf16")])
@pytest.mark.parametrize("master", [False, True])
def test_adamw_32(kind, gkind, master):
    torch = require_gpu()
    from symmetric_nmf_clustering_amd import api
    shapes = [(1,), (7,), (8,), (2048,), (2049,), (33, 100), (5, 3, 411)]
    made = [adam_make(torch, s, kind, gkind, i) for i, s in enumerate(shapes)]
    ts, xs = [m[0] for m in made], [m[1] for m in made]
    masters = None
    if master:  # the masters hold what the params have rounded away
        masters = []
        for t, x in made:
            mt, mv = dev(torch, x["p"] * (1 + 2.0 ** -12))
            masters.append(mt)
            x["p"] = mv
    before = [t["g"].clone() for t in ts]
    api.adamw_step([t["p"] for t in ts], [t["g"] for t in ts], [t["m"] for t in ts], [t["v"] for t in ts], 3,
                   masters=masters, grad_scale=0.5, **HYPER)
    for i, (t, x) in enumerate(zip(ts, xs)):
        assert torch.equal(t["g"], before[i])
        if master:
            t["master"] = masters[i]
        adam_close(torch, t, x, kind, gs=0.5)


def decode(torch, code, scale):
    n = code.numel()
    return code.float().reshape(-1).double() * scale.double().repeat_interleave(256)[:n]


@pytest.mark.parametrize("kind,gkind", [("fp32", "fp32"), ("bf16", "bf16"), ("fp16", "fp32")])
@pytest.mark.parametrize("master", [False, True])
def test_adamw_8(kind, gkind, master):
    torch = require_gpu()
    from symmetric_nmf_clustering_amd import api
    shapes = [(1,), (255,), (256,), (257,), (2048,), (4100,), (37, 111)]
    made = [adam_make(torch, s, kind, gkind, 50 + i) for i, s in enumerate(shapes)]
    params, grads = [t["p"] for t, _ in made], [t["g"] for t, _ in made]
    masters = [t["p"].float().clone() for t, _ in made] if master else None
    m, v, ms, vs = api.adamw_states(params, bits=8)
    for step in (1, 2, 3):
        olds = []
        for i, (t, x) in enumerate(made):
            olds.append(dict(p=(masters or params)[i].double().cpu().numpy(), g=x["g"],
                             m=decode(torch, m[i], ms[i]).cpu().numpy().reshape(x["g"].shape),
                             v=decode(torch, v[i], vs[i]).square().cpu().numpy().reshape(x["g"].shape)))
        api.adamw_step(params, grads, m, v, step, masters=masters, m_scale=ms, v_scale=vs, **HYPER)
        for i, x in enumerate(olds):
            got = dict(p=params[i])
            if master:
                got["master"] = masters[i]
            ref = adam_close(torch, got, x, kind, step=step)
            for code, scale, want in ((m[i], ms[i], ref[1]), (v[i], vs[i], np.sqrt(ref[2]))):
                want = want.reshape(-1)
                top = np.array([np.abs(want[j:j + 256]).max() for j in range(0, want.size, 256)])
                close(scale, top / 448, 8 * U * top / 448)
                each = np.repeat(scale.double().cpu().numpy(), 256)[:want.size]
                have = decode(torch, code, scale).cpu().numpy()
                # half a step of 4 significant bits, half a step (2^-9) below the normal range; a root
                # above zero that would be zero is one step: 2^-9
                assert (np.abs(have - want) <= np.abs(want) * (2.0 ** -4 + 2.0 ** -20) + each * 2.0 ** -9).all()
                if code is v[i]:
                    assert ((have > 0) == (want > 0)).all()
                assert not np.isnan(have).any()


def test_adamw_8_extremes():
    """Zeros, blocks of tiny and huge values, and what is not finite."""
    torch = require_gpu()
    from symmetric_nmf_clustering_amd import api
    n = 256 * 5
    p = torch.zeros(n, device="cuda")
    g = torch.zeros(n, device="cuda")
    g[256:512] = 1e-30                      # roots near 1e-31, moments near 1e-31
    g[512:768] = 1e15
    g[768:1024] = torch.logspace(-18, 0, 256, device="cuda")   # more than the codes span
    g[1024] = float("nan")
    g[1030] = float("inf")
    g[1031:] = 1.0
    m, v, ms, vs = api.adamw_states([p], bits=8)
    api.adamw_step([p], [g], m, v, 1, m_scale=ms, v_scale=vs, **HYPER)
    md, vd = decode(torch, m[0], ms[0]), decode(torch, v[0], vs[0])
    assert not md[:256].any() and not vd[:256].any() and not p[:256].any()
    assert torch.isfinite(ms[0]).all() and torch.isfinite(vs[0]).all()
    assert (vd[512:768] > 0).all() and (vd[768:1024] > 0).all()
    assert torch.isfinite(p[256:1024]).all()
    for x in (md, vd):
        assert torch.isnan(x[1024]) and torch.isnan(x[1030])
        assert torch.isfinite(x[1025:1030]).all() and torch.isfinite(x[1031:]).all()
    assert abs(md[1100].item() - 0.1) <= 0.1 * 2.0 ** -4 and abs(vd[1100].item() - 0.1) <= 0.1 * 2.0 ** -4
    # a second step without gradients moves nothing by more than the first could
    before = p.clone()
    api.adamw_step([p], [torch.zeros_like(g)], m, v, 2, m_scale=ms, v_scale=vs, **HYPER)
    assert ((p - before)[256:1024].abs() <= 20 * HYPER["lr"]).all()


def test_adamw_many_tensors_and_device_numbers():
    torch = require_gpu()
    from symmetric_nmf_clustering_amd import api
    rng = np.random.default_rng(2)
    made = [adam_make(torch, (int(n),), "fp32" if i % 3 else "bf16", "fp32" if i % 2 else "bf16", i)
            for i, n in enumerate(rng.integers(0, 3000, size=131))]
    cols = [[t[k] for t, _ in made] for k in "pgmv"]
    cols[1][5] = None  # no gradient: left alone
    keep = [made[5][0][k].clone() for k in "pmv"]
    step = torch.tensor(3, dtype=torch.int64, device="cuda")
    lr, gs = torch.tensor([0.01], device="cuda"), torch.tensor(0.5, device="cuda")
    hyper = {k: v for k, v in HYPER.items() if k != "lr"}
    api.adamw_step(*cols, step, lr=lr, grad_scale=gs, **hyper)
    for i, (t, x) in enumerate(made):
        if i == 5:
            assert all(torch.equal(a, t[k]) for a, k in zip(keep, "pmv"))
            continue
        # (the rate arrives as float32: u more on every update, decay's product u more)
        adam_close(torch, t, x, "fp32" if i % 3 else "bf16", gs=0.5)
    api.adamw_step([], [], [], [], 1)


# ---- streams, graphs, devices, refusals -------------------------------------------

def test_on_another_stream():
    torch = require_gpu()
    from symmetric_nmf_clustering_amd import api
    t, x = make(torch, "bf16", 1, 2000, 2, 2, 64, 64, 21)
    tf = torch.from_numpy(10000.0 ** (-np.arange(32) / 32)).cuda()
    pos = torch.arange(2000, device="cuda").expand(1, -1)
    want = api.linear_attention(api.rotary(t["q"], pos, tf), t["k"], t["v"], t["decay"])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = api.linear_attention(api.rotary(t["q"], pos, tf), t["k"], t["v"], t["decay"])
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_captured_step():
    """A training step of the layers as one graph, replayed between eager work; the optimizer's
    step, rate and scale change from replay to replay."""
    torch = require_gpu()
    from symmetric_nmf_clustering_amd import api
    t, x = make(torch, "fp32", 2, 700, 4, 2, 32, 24, 22, lengths=[700, 333])
    tf = torch.from_numpy(10000.0 ** (-np.arange(16) / 16)).cuda()
    pos = torch.arange(700, device="cuda").expand(2, -1)
    live = {n: t[n].clone() for n in "qkv"}
    states = {bits: api.adamw_states([live[n] for n in "qkv"], bits) for bits in (32, 8)}
    step = torch.ones((), dtype=torch.int64, device="cuda")
    lr = torch.full((), 0.01, device="cuda")

    def run(p, states):
        q = api.rotary(p["q"], pos, tf)
        o, last = api.linear_attention(q, p["k"], p["v"], t["decay"], lengths=t["lengths"])
        dq, dk, dv, _ = api.linear_attention_grad(q, p["k"], p["v"], t["decay"], o, dlast=last,
                                                  lengths=t["lengths"])
        g = [api.rotary(dq, pos, tf, inverse=True), dk, dv]
        for bits in (32, 8):
            m, v, ms, vs = states[bits]
            api.adamw_step([p[n] for n in "qkv"], g, m, v, step, lr=lr, m_scale=ms, v_scale=vs)
        return o, last

    def copies(p, states):
        return ({n: a.clone() for n, a in p.items()},
                {b: tuple(None if l is None else [a.clone() for a in l] for l in s) for b, s in states.items()})

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(*copies(live, states))
    torch.cuda.current_stream().wait_stream(side)
    eager, eager_states = copies(live, states)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run(live, states)
    for i in range(4):
        step.fill_(i + 1)
        lr.fill_(0.01 / (i + 1))
        graph.replay()
        torch.cuda.synchronize()
        want = run(eager, eager_states)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
        assert all(torch.equal(live[n], eager[n]) for n in "qkv")
        for b in (32, 8):
            for mine, theirs in zip(states[b], eager_states[b]):
                for p, q in zip(mine or [], theirs or []):
                    assert torch.equal(p.view(torch.uint8), q.view(torch.uint8))


def test_offsets_past_32_bits():
    torch = require_gpu()
    from symmetric_nmf_clustering_amd import api
    far = (1 << 32) + 40  # elements between two batch rows of one buffer
    buf = torch.zeros(far + 200 * 2 * 16, dtype=torch.bfloat16, device="cuda")
    t, x = make(torch, "bf16", 2, 200, 2, 2, 16, 16, 30)

    def spread(a):
        v = torch.as_strided(buf, a.shape, (far, 2 * 16, 16, 1))
        v.copy_(a)
        return v

    want = api.linear_attention(t["q"], t["k"], t["v"], t["decay"])
    got = api.linear_attention(spread(t["q"]), t["k"], t["v"], t["decay"])
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    tf = torch.ones(8, dtype=torch.float64, device="cuda")
    pos = torch.arange(200, device="cuda").expand(2, -1)
    want = api.rotary(t["q"], pos, tf)
    assert torch.equal(api.rotary(spread(t["q"]), pos, tf), want)
    mine = spread(t["q"])
    assert torch.equal(api.rotary(mine, pos, tf, out=mine), want)
    del buf, mine
    n = (1 << 31) + 5  # one tensor of more than 2^31 elements
    p = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g[-3:] = 1.0
    m, v, ms, vs = api.adamw_states([p], bits=8)
    api.adamw_step([p], [g], m, v, 1, m_scale=ms, v_scale=vs, lr=0.5, weight_decay=0.0)
    assert p[-3:].tolist() == [-0.5] * 3 and not p[:-3].any()
    assert abs(ms[0][-1].item() * 448 - 0.1) < 1e-6


def test_binding_refusals():
    torch = require_gpu()
    from symmetric_nmf_clustering_amd import api
    t, _ = make(torch, "fp32", 2, 5, 4, 2, 8, 6, 1)
    q, k, v, a, do = t["q"], t["k"], t["v"], t["decay"], t["do"]
    z = lambda *s, **kw: torch.zeros(*s, device="cuda", **kw)  # noqa: E731
    for args in ((q[0], k, v, a), (q, k[0], v, a), (q, k[:1], v, a), (q, k[..., :4], v, a), (q, k, v[:, :4], a),
                 (q, k, v[:, :, :1], a), (q.bfloat16(), k, v, a), (q, k, v, a[:3]), (q, k, v, a.double()),
                 (q, k, v, a.cpu()), (q[:, :, :3], k, v, a[:3]), (q, k, v, z(8)[::2]),
                 (q.transpose(2, 3), k, v, a), (z(2, 5, 4, 257), z(2, 5, 2, 257), v, a), (q[:0], k[:0], v[:0], a),
                 (z(2, 5, 4, 16)[..., ::2], k, v, a)):
        with pytest.raises(ValueError):
            api.linear_attention(*args)
        with pytest.raises(ValueError):
            api.linear_attention_grad(*args, do)
    for kw in (dict(state=z(2, 4, 8, 5)), dict(state=z(2, 4, 8, 6).double()), dict(state=z(2, 4, 6, 8).transpose(2, 3)),
               dict(lengths=z(3, dtype=torch.int32)), dict(lengths=z(2)), dict(scale=float("nan"))):
        with pytest.raises(ValueError):
            api.linear_attention(q, k, v, a, **kw)
        with pytest.raises(ValueError):
            api.linear_attention_grad(q, k, v, a, do, **kw)
    for d in (do[:, :4], do.bfloat16(), do[0], None):
        with pytest.raises(ValueError):
            api.linear_attention_grad(q, k, v, a, d)
    with pytest.raises(ValueError):
        api.linear_attention_grad(q, k, v, a, do, dlast=z(1, 4, 8, 6))
    s = z(2, 4, 8, 6)
    for args in ((q, k, v, a, s), (q[:, 0], k[:, 0], v[:, 0], a, None), (q[:, 0], k[:, 0], v[:, 0], a, s[:1]),
                 (q[:, 0], k, v, a, s)):
        with pytest.raises(ValueError):
            api.linear_attention_step(*args)
    with pytest.raises(ValueError):
        api.linear_attention_step(q[:, 0], k[:, 0], v[:, 0], a, s, out_state=s.bfloat16())
    pos, f = z(2, 5, dtype=torch.int32), z(4, dtype=torch.float64)
    for args, kw in (((q[0, 0], pos, f), {}), ((q, pos[:, :4], f), {}), ((q, pos.float(), f), {}),
                     ((q, pos, f.float()), {}), ((q, pos, z(5, dtype=torch.float64)), {}),
                     ((q, pos, z(8, dtype=torch.float64)[::2]), {}), ((q, pos, f), dict(layout="other")),
                     ((q, pos, f), dict(amplitude=float("inf"))), ((q, pos, f), dict(out=z(2, 5, 4, 7))),
                     ((q, pos, f), dict(out=q.bfloat16())), ((q, pos, f), dict(out=q[:1, :1].expand_as(q))),
                     ((q[:, :, :, ::2], pos, f[:2]), {})):
        with pytest.raises(ValueError):
            api.rotary(*args, **kw)
    p, g = z(300), z(300)
    m, v_, ms, vs = api.adamw_states([p], bits=8)
    m32, v32, _, _ = api.adamw_states([p])
    with pytest.raises(ValueError):
        api.adamw_states([p], bits=16)
    for args, kw in ((([p], [], m32, v32, 1), {}), (([p], [g[:9]], m32, v32, 1), {}), (([p], [g.double()], m32, v32, 1), {}),
                     (([p], [g], m, v_, 1), {}), (([p], [g], m, v_, 1), dict(m_scale=ms)),
                     (([p], [g], m, v_, 1), dict(m_scale=ms, v_scale=[z(1)])),
                     (([p], [g], m32, v32, 1), dict(m_scale=ms, v_scale=vs)),
                     (([p], [g], m32, m32, 1), {}), (([p, p], [g, g], m32 * 2, v32 * 2, 1), {}),
                     (([p], [g], m32, v32, 1), dict(masters=[p])), (([p], [g], m32, v32, 1), dict(masters=[z(299)])),
                     (([p[::2]], [g[::2]], [m32[0][:150]], [v32[0][:150]], 1), {}),
                     (([p], [g], m32, v32, torch.ones(1, device="cuda")), {}),
                     (([p], [g], m32, v32, 1), dict(lr=z(2)))):
        with pytest.raises(ValueError):
            api.adamw_step(*args, **kw)
    from symmetric_nmf_clustering_amd import _lib as L
    for kw in (dict(step=0), dict(lr=float("nan")), dict(beta1=1.0), dict(beta2=-0.1), dict(eps=-1.0)):
        with pytest.raises(L.SymNMFError):
            api.adamw_step([p], [g], m32, v32, **{**dict(step=1), **kw})


@pytest.mark.parametrize("far", [(1 << 23) - 8, 1 << 23, (1 << 23) + 8, (1 << 24) - 8, 1 << 24, (1 << 25) + 8])
def test_far_steps(far):
    """Steps far apart in memory, around where a walk's offsets change their arithmetic."""
    torch = require_gpu()
    from symmetric_nmf_clustering_amd import api
    T = 9
    t, x = make(torch, "bf16", 1, T, 2, 2, 16, 16, 31)
    buf = torch.zeros(4, far * (T - 1) + 32, dtype=torch.bfloat16, device="cuda")
    v = {}
    for i, name in enumerate(("q", "k", "v", "do")):
        v[name] = torch.as_strided(buf, (1, T, 2, 16), (far * T, far, 16, 1), i * buf.shape[1])
        v[name].copy_(t[name])
    got = api.linear_attention(v["q"], v["k"], v["v"], t["decay"], state=t["state"])
    want = api.linear_attention(t["q"], t["k"], t["v"], t["decay"], state=t["state"])
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    kw = dict(dlast=t["dlast"], state=t["state"])
    got = api.linear_attention_grad(v["q"], v["k"], v["v"], t["decay"], v["do"], **kw)
    want = api.linear_attention_grad(t["q"], t["k"], t["v"], t["decay"], t["do"], **kw)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
def test_lengths_over_many_heads(kind):
    """Padded batches large enough to be cut, with shared heads, more batch rows than XCDs and more
    workgroups than CUs: every row as when it is alone."""
    torch = require_gpu()
    from symmetric_nmf_clustering_amd import api
    B, T, H, G, d = 11, 520, 12, 4, 40
    lengths = [520, 0, 1, 130, 519, 256, 64, 300, 5, 520, 128]
    t, x = make(torch, kind, B, T, H, G, d, d, 41, lengths)
    kw = dict(state=t["state"], lengths=t["lengths"])
    got = api.linear_attention(t["q"], t["k"], t["v"], t["decay"], **kw)
    grad = api.linear_attention_grad(t["q"], t["k"], t["v"], t["decay"], t["do"], dlast=t["dlast"], **kw)
    check_forward(got, x, kind, d ** -0.5)
    check_grad(grad, x, kind, d ** -0.5)


def test_two_streams_at_once():
    torch = require_gpu()
    from symmetric_nmf_clustering_amd import api
    made = [make(torch, "bf16", 1, 3000, 2, 1, 64, 64, 50 + i)[0] for i in range(2)]
    want = [api.linear_attention(t["q"], t["k"], t["v"], t["decay"]) for t in made]
    streams = [torch.cuda.Stream() for _ in made]
    got = [[], []]
    torch.cuda.synchronize()
    for _ in range(5):
        for i, t in enumerate(made):
            with torch.cuda.stream(streams[i]):
                got[i].append(api.linear_attention(t["q"], t["k"], t["v"], t["decay"]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(a, b) for r in got[i] for a, b in zip(r, want[i]))


@pytest.mark.parametrize("kind", ["fp32", "bf16", "fp16"])
def test_many_rows(kind):
    """More batch rows than a grid's smaller dimensions take, and heads past a CU's: each row as
    when a few of them are alone."""
    torch = require_gpu()
    from symmetric_nmf_clustering_amd import api
    for B, T, H, G, d in ((70000, 2, 1, 1, 8), (3, 3, 600, 200, 16)):
        g = torch.Generator(device="cuda").manual_seed(B)
        dt = types(torch)[kind]
        q, k, v, do = (torch.randn(B, T, h, d, generator=g, device="cuda").to(dt) for h in (H, G, G, H))
        state, dlast = (torch.randn(B, H, d, d, generator=g, device="cuda") for _ in range(2))
        decay = -torch.rand(H, generator=g, device="cuda")
        lengths = torch.randint(0, T + 1, (B,), generator=g, device="cuda", dtype=torch.int32)

        def run(at):
            a = [x[at].contiguous() for x in (q, k, v)]
            o = api.linear_attention(*a, decay, state=state[at], lengths=lengths[at].contiguous())
            gr = api.linear_attention_grad(*a, decay, do[at], dlast=dlast[at], state=state[at],
                                           lengths=lengths[at].contiguous())
            st = api.linear_attention_step(*(x[:, 0] for x in a), decay, state[at])
            return *o, *gr, *st

        whole = run(slice(None))
        some = torch.tensor([0, B // 2, B - 1], device="cuda")
        for x, y in zip(whole, run(some)):
            assert torch.equal(x[some], y)


def test_overlapping_memory_is_refused():
    torch = require_gpu()
    from symmetric_nmf_clustering_amd import api
    buf = torch.zeros(4, 2, 8, 8, device="cuda")
    q = torch.ones(3, 2, 8, device="cuda")
    decay = torch.zeros(2, device="cuda")
    with pytest.raises(ValueError, match="overlaps"):
        api.linear_attention_step(q, q, q, decay, buf[:3], out_state=buf[1:])
    _, same = api.linear_attention_step(q, q, q, decay, buf[:3], out_state=buf[:3])
    assert same.data_ptr() == buf.data_ptr()
    flat = torch.zeros(100, device="cuda")
    for params in ([flat[:60], flat[50:]], [flat, flat[99:]], [flat[10:20], flat]):
        m, v, _, _ = api.adamw_states(params)
        with pytest.raises(ValueError, match="share memory"):
            api.adamw_step(params, [torch.ones_like(p) for p in params], m, v, 1)
    params = [flat[:50], flat[50:], flat[:0]]  # neighbours in one buffer are apart
    m, v, _, _ = api.adamw_states(params)
    api.adamw_step(params, [torch.ones_like(p) for p in params], m, v, 1, lr=0.5, eps=0.0, weight_decay=0.0)
    assert torch.allclose(flat, torch.full_like(flat, -0.5))


def test_two_streams_of_small_heads():
    """Calls whose segments' states are a few numbers have a workspace of their own too: many calls
    at once on two streams, and a replayed graph beside them."""
    torch = require_gpu()
    from symmetric_nmf_clustering_amd import api
    for d, T in ((4, 512), (1, 4096), (2, 1024)):
        made = [make(torch, "fp32", 1, T, 1, 1, d, d, 60 + i)[0] for i in range(3)]

        def run(t):
            return api.linear_attention(t["q"], t["k"], t["v"], t["decay"], state=t["state"])

        want = [run(t) for t in made]
        streams = [torch.cuda.Stream() for _ in range(2)]
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            replayed = run(made[2])
        got = [[], []]
        for _ in range(30):
            graph.replay()
            for i in range(2):
                with torch.cuda.stream(streams[i]):
                    got[i].append(run(made[i]))
        torch.cuda.synchronize()
        for i in range(2):
            assert all(torch.equal(a, b) for r in got[i] for a, b in zip(r, want[i]))
        assert all(torch.equal(a, b) for a, b in zip(replayed, want[2]))


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("T", [80, 128])
@pytest.mark.parametrize("d", [16, 128])
def test_pairs_that_do_not_count_may_overflow(kind, T, d):
    """Dot products past float32's range between steps that have no weight for one another (a later
    key, or a decay that keeps nothing) leave no trace: the definition is finite."""
    torch = require_gpu()
    from symmetric_nmf_clustering_amd import api
    t, x = make(torch, kind, 1, T, 3, 3, d, d, T + d, decay=[-0.01, -0.02, -np.inf])
    # one channel of a head for a pair of steps: 1e20 at each, 0 at all others
    pairs = [("q", 5, "k", 12, 0, 0), ("do", 5, "v", 12, 1, 1),  # later in the same 16 steps, either way
             ("q", 64, "k", 63, 2, 0), ("q", 16, "k", 15, 2, 1)]  # from one chunk to the next, either way
    for one, i, two, j, h, c in pairs:
        for name, at in ((one, i), (two, j)):
            for a in (t[name], x[name]):
                a[:, :, h, c] = 0.0
            t[name][:, at, h, c] = 1e20
            x[name][:, at, h, c] = t[name][0, at, h, c].item()
        for a in (t["state"], t["dlast"], x["state"], x["dlast"]):
            a[:, h, :, c] = 0.0
            a[:, h, c] = 0.0
    args = (t["q"], t["k"], t["v"], t["decay"])
    check_forward(api.linear_attention(*args, state=t["state"]), x, kind, d ** -0.5)
    check_grad(api.linear_attention_grad(*args, t["do"], dlast=t["dlast"], state=t["state"]), x, kind, d ** -0.5)


def test_rotary_into_shared_memory():
    torch = require_gpu()
    from symmetric_nmf_clustering_amd import api
    y = torch.randn(6, 9, 5, 24, device="cuda")
    pos = torch.arange(9, device="cuda").expand(6, 9)
    f = torch.ones(12, dtype=torch.float64, device="cuda")
    flat = torch.zeros(6 * 9 * 5 * 24, device="cuda")
    for x, out in ((y[:, :, :2], y[:, :, 1:3]), (y[:, :8], y[:, 1:]), (y[:5], y[1:]),
                   (y.transpose(0, 1)[:6, :6], y[:6, :6]),
                   (y, torch.as_strided(flat, y.shape, (24 * 9, 24, 12, 1))),
                   (y, torch.as_strided(flat, y.shape, (9 * 60, 60, 24, 1)))):
        with pytest.raises(ValueError, match="shares|overlapping"):
            api.rotary(x, pos[:1, :1].expand(x.shape[:2]), f, out=out)
    # other heads of the same rows, and other channels of the same heads, are memory apart
    want = api.rotary(y[:, :, :2], pos, f)
    mine = y.clone()
    api.rotary(mine[:, :, :2], pos, f, out=mine[:, :, 3:])
    assert torch.equal(mine[:, :, 3:], want) and torch.equal(mine[:, :, :3], y[:, :, :3])
    mine = y.clone()
    api.rotary(mine[..., :12], pos, f[:6], out=mine[..., 12:])
    assert torch.equal(mine[..., 12:], api.rotary(y[..., :12], pos, f[:6])) and torch.equal(mine[..., :12], y[..., :12])


def test_what_adamw_reads_is_apart_from_what_it_writes():
    torch = require_gpu()
    from symmetric_nmf_clustering_amd import api
    flat = torch.zeros(1000, device="cuda")
    p, rest = flat[:100], torch.ones(100, device="cuda")
    m, v, _, _ = api.adamw_states([p])
    for grad in (p, flat[60:160], m[0], v[0]):
        with pytest.raises(ValueError, match="shares memory"):
            api.adamw_step([p], [grad], m, v, 1)
    for kw in (dict(lr=p[7]), dict(grad_scale=m[0][:1])):
        with pytest.raises(ValueError, match="shares memory"):
            api.adamw_step([p], [rest], m, v, 1, **kw)
    assert not flat.any()  # refused before anything ran
    q = torch.zeros(100, device="cuda")
    m, v, _, _ = api.adamw_states([p, q])
    grad = flat[100:200].fill_(1.0)  # a neighbour, and one gradient for two parameters
    api.adamw_step([p, q], [grad, grad], m, v, 1, lr=0.5, eps=0.0, weight_decay=0.0)
    assert torch.allclose(p, torch.full_like(p, -0.5)) and torch.equal(p, q) and not flat[200:].any()


@pytest.mark.parametrize("low", [False, True])
def test_adamw_factors_are_not_rounded(low):
    """What a step keeps of m, v and p, averaged over many values: one of its own roundings is at
    most u and goes either way, the betas' and the decay's would all go one way (up to u / 2)."""
    torch = require_gpu()
    from symmetric_nmf_clustering_amd import api
    n = 1 << 20
    # factors half a step of float32 away from its numbers: each rounds by u / 2 or nearly
    beta1, beta2, lw = 1 - 2.0 ** -4 - 2.0 ** -25.1, 1 - 2.0 ** -12 + 2.0 ** -25.1, 2.0 ** -13 + 2.0 ** -25.1
    g = torch.Generator(device="cuda").manual_seed(5)

    def values():
        return torch.rand(n, generator=g, device="cuda") + 1.0

    p, m, v, zero = values(), values(), values(), torch.zeros(n, device="cuda")
    hyper = dict(lr=lw, beta1=beta1, beta2=beta2, weight_decay=1.0)
    before = [x.double() for x in (p, m, v)]
    if low:  # (held in 8 bits, the states show no more than 2^-4)
        api.adamw_step([p], [zero], *api.adamw_states([p], 8)[:2], 1, **hyper,
                       **dict(zip(("m_scale", "v_scale"), api.adamw_states([p], 8)[2:])))
        pairs = [(p, before[0], 1 - lw)]
    else:
        api.adamw_step([p], [zero], [zero.clone()], [zero.clone()], 1, **hyper)
        api.adamw_step([zero.clone()], [zero], [m], [v], 1, **hyper)
        pairs = list(zip((p, m, v), before, (1 - lw, beta1, beta2)))
    for got, was, factor in pairs:
        off = (got.double() / was - factor) / factor
        # p: one rounding; m, v: two, of which the first is of a number 2^-24 as large
        assert off.abs().max() <= 1.01 * U
        # the mean of n roundings uniform in +-u: u / sqrt(3 n), five times that
        assert abs(off.mean()) <= 5 * U / (3 * n) ** 0.5


def test_live_decay_is_not_rounded():
    """What a step keeps of the state, averaged over many values: the step's own rounding goes
    either way, the decay's would go one way (up to u / 2) at every step."""
    torch = require_gpu()
    from symmetric_nmf_clustering_amd import api
    g = -np.arange(1, 4000, dtype=np.float32) * np.float32(2.0 ** -14)
    a = np.exp(g.astype(np.float64))
    off = (a - a.astype(np.float32)) / a  # what float32 loses of each decay
    at = [int(off.argmax()), int(off.argmin())]
    decay = torch.from_numpy(g[at]).cuda()
    B, d = 16, 256
    gen = torch.Generator(device="cuda").manual_seed(6)
    q, k, v = (torch.zeros(B, 2, d, device="cuda") for _ in range(3))
    state = torch.rand(B, 2, d, d, generator=gen, device="cuda") + 1.0
    _, new = api.linear_attention_step(q, k, v, decay, state)
    for h in range(2):
        e = new[:, h].double() / state[:, h].double() / a[at[h]] - 1.0
        # one rounding (and one of a number 2^-24 as large); the mean of n, uniform in +-u
        assert e.abs().max() <= 1.01 * U
        assert abs(e.mean()) <= 5 * U / (3 * e.numel()) ** 0.5 < 0.1 * abs(off[at[h]])


def test_rotary_at_any_position():
    """Angles reduced in exact arithmetic: positions up to the ends of int64 are as precise as near ones."""
    from decimal import Decimal, getcontext
    torch = require_gpu()
    from symmetric_nmf_clustering_amd import api
    getcontext().prec = 90  # 2^63 radians have 19 digits before the point
    turn = Decimal("6.283185307179586476925286766559005768394338798750211641949889184615632812572417997256069650684")
    rng = np.random.default_rng(8)
    ends = [0, -1, 2047, 2048, -2048, 2 ** 53 + 1, -2 ** 53 - 1, 2 ** 63 - 1, -2 ** 63, 2 ** 63 - 1025]
    pos = np.array(ends + [int(x) * (-1) ** i for i, x in enumerate(2.0 ** rng.uniform(20, 63, 40))])
    f = np.concatenate([1000.0 ** (-np.arange(6) / 6), [np.pi, 0.1]])
    angle = np.array([[float(Decimal(int(p)) * Decimal(float(w)) % turn) for w in f] for p in pos])
    cos, sin = np.cos(angle)[:, None, :], np.sin(angle)[:, None, :]
    tp, tf = torch.from_numpy(pos).cuda(), torch.from_numpy(f).cuda()
    for kind in ("fp32", "bf16"):
        x, xv = dev(torch, rng.standard_normal((len(pos), 3, 16)), kind)
        a, b = xv[..., :8], xv[..., 8:]
        for inverse in (False, True):
            s = -sin if inverse else sin
            ref = np.concatenate([a * cos - b * s, b * cos + a * s], -1)
            got = api.rotary(x, tp, tf, inverse=inverse)
            close(got, ref, rotary_bound(xv, 8, False, 1.0), kind)


@pytest.mark.parametrize("B,T,H,G,dk,dv", [(2, 300, 2, 1, 128, 128), (1, 130, 2, 2, 64, 48), (1, 70, 1, 1, 256, 256),
                                           (20, 70, 16, 4, 128, 96), (1, 1500, 1, 1, 40, 33), (3, 64, 4, 2, 24, 24)])
def test_bf16_rounds_its_outputs_alone(B, T, H, G, dk, dv):
    """What is inside goes through two bfloat16 parts (2^-8 of 2^-8), not through one: besides the
    output's own rounding, 2^-16 of the terms and float32's share."""
    torch = require_gpu()
    from symmetric_nmf_clustering_amd import api
    t, x = make(torch, "bf16", B, T, H, G, dk, dv, 70 + dk)
    scale = dk ** -0.5
    args = [x[n] for n in "qkv"]
    mags = [abs(a) for a in args]
    c = attend_bound("fp32", T, dk, dv) + 2.0 ** -16
    got = api.linear_attention(t["q"], t["k"], t["v"], t["decay"], state=t["state"])
    ref = lo.linear_attention(*args, x["decay"], x["state"], None, scale)
    mag = lo.linear_attention(*mags, x["decay"], abs(x["state"]), None, scale)
    close(got[0], ref[0], c * mag[0], "bf16")
    got = api.linear_attention_grad(t["q"], t["k"], t["v"], t["decay"], t["do"], dlast=t["dlast"], state=t["state"])
    ref = lo.linear_attention_grad(*args, x["decay"], x["do"], x["dlast"], x["state"], None, scale)
    mag = lo.linear_attention_grad(*mags, x["decay"], abs(x["do"]), abs(x["dlast"]), abs(x["state"]), None, scale)
    for i in range(3):
        close(got[i], ref[i], (c + 2 * U * H) * mag[i], "bf16")


def test_adamw_8_keeps_tiny_roots():
    """Roots whose squares are among float32's smallest numbers survive a step without gradients."""
    torch = require_gpu()
    from symmetric_nmf_clustering_amd import api
    p = torch.zeros(512, device="cuda")
    g = torch.full_like(p, 1e-19)
    g[256:] = torch.logspace(-19, -17, 256, device="cuda")
    m, v, ms, vs = api.adamw_states([p], bits=8)
    hyper = {**HYPER, "beta2": 0.99, "eps": 1e-8}
    api.adamw_step([p], [g], m, v, 1, m_scale=ms, v_scale=vs, **hyper)
    first = decode(torch, v[0], vs[0])
    api.adamw_step([p], [torch.zeros_like(g)], m, v, 2, m_scale=ms, v_scale=vs, **hyper)
    second = decode(torch, v[0], vs[0])
    assert (first > 0).all() and (second > 0).all()
    # the code's half step, and 2^-149 on a square of at least 1e-40 or so
    want = first * 0.99 ** 0.5
    assert ((second - want).abs() <= want * (2.0 ** -4 + 1e-4) + vs[0].double().repeat_interleave(256) * 2.0 ** -9).all()


@pytest.mark.parametrize("kind", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_infinite_parameters_stay(kind, bits):
    """A parameter that holds a mask's infinities keeps them, with and without weight decay."""
    torch = require_gpu()
    from symmetric_nmf_clustering_amd import api
    for decay in (0.0, 0.1):
        p = torch.ones(300, device="cuda").to(types(torch)[kind])
        p[3::7], p[5::7], p[6::7] = float("-inf"), float("inf"), float("nan")
        keep = p.clone()
        m, v, ms, vs = api.adamw_states([p], bits)
        api.adamw_step([p], [torch.ones_like(p)], m, v, 1, lr=0.01, weight_decay=decay, m_scale=ms, v_scale=vs)
        odd = ~torch.isfinite(keep)
        assert torch.equal(torch.nan_to_num(p[odd].float(), nan=7.0), torch.nan_to_num(keep[odd].float(), nan=7.0))
        assert torch.isfinite(p[~odd]).all() and (p[~odd] < 1).all()


# ---- every walk: two column tiles a wave, cut and whole, with and without lengths ---------

def device_definition(torch, t, scale, gradient):
    """The definitions in float64 on the device (the oracle's loops, all batch rows at once)."""
    q, k, v, do = (t[n].double() for n in ("q", "k", "v", "do"))
    B, T, H, dk = q.shape
    shared = H // k.shape[2]
    k, v = (x.repeat_interleave(shared, 2) for x in (k, v))
    a = t["decay"].double().exp()[None, :, None, None]
    n = torch.full((B,), T, device="cuda") if t["lengths"] is None else t["lengths"].long().clamp(0, T)
    inside = (torch.arange(T, device="cuda")[:, None] < n)[:, :, None, None, None]
    S, o, dq = t["state"].double(), torch.zeros_like(do), torch.zeros_like(q)
    for i in range(T):
        new = a * S + k[:, i, :, :, None] * v[:, i, :, None, :]
        S = torch.where(inside[i], new, S)
        o[:, i] = torch.where(inside[i, ..., 0], scale * (q[:, i, :, :, None] * S).sum(2), 0.0)
        if gradient:
            dq[:, i] = torch.where(inside[i, ..., 0], scale * (S * do[:, i, :, None, :]).sum(3), 0.0)
    if not gradient:
        return o, S
    R, dk_, dv_ = t["dlast"].double(), torch.zeros_like(k), torch.zeros_like(v)
    for i in range(T - 1, -1, -1):
        new = R + scale * q[:, i, :, :, None] * do[:, i, :, None, :]
        dk_[:, i] = torch.where(inside[i, ..., 0], (new * v[:, i, :, None, :]).sum(3), 0.0)
        dv_[:, i] = torch.where(inside[i, ..., 0], (new * k[:, i, :, :, None]).sum(2), 0.0)
        R = torch.where(inside[i], a * new, R)
    dk_, dv_ = (x.unflatten(2, (-1, shared)).sum(3) for x in (dk_, dv_))
    return dq, dk_, dv_, R


def check_on_device(torch, t, clean, kind, gradient):
    """The library's outputs on t against the definition on the same tensors, ``clean`` of masked NaN."""
    from symmetric_nmf_clustering_amd import api
    B, T, H, dk = t["q"].shape
    dv = t["v"].shape[3]
    scale = dk ** -0.5
    kw = dict(state=t["state"], lengths=t["lengths"])
    if gradient:
        got = api.linear_attention_grad(t["q"], t["k"], t["v"], t["decay"], t["do"], dlast=t["dlast"], **kw)
    else:
        got = api.linear_attention(t["q"], t["k"], t["v"], t["decay"], **kw)
    ref = device_definition(torch, clean, scale, gradient)
    sizes = {n: x if x is None or n in ("decay", "lengths") else x.abs() for n, x in clean.items()}
    mag = device_definition(torch, sizes, scale, gradient)
    inner = attend_bound("fp32", T, dk, dv) + (2 * U * H if gradient else 0.0)
    for i, (g, r, m) in enumerate(zip(got, ref, mag)):
        state = i == len(got) - 1
        c = inner + (0.0 if state or kind == "fp32" else 2.0 ** -16)
        close(g, r.cpu().numpy(), (c * m).cpu().numpy(), "fp32" if state else kind)


@pytest.mark.parametrize("kind", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("ragged", [False, True])
@pytest.mark.parametrize("B,T,H,G,dk,dv", [
    (1, 1100, 64, 16, 128, 128),  # cut in six, more than 256 workgroups' worth of heads
    (1, 700, 32, 8, 128, 128),    # its gradient cut in four, likewise
    (1, 601, 96, 96, 88, 96),     # cut in five, heads of 96
    (20, 70, 16, 4, 128, 128),    # whole
    (24, 75, 12, 3, 104, 72),     # whole, columns missing from the last tile
    (6, 33, 48, 48, 96, 96),      # whole, heads of 96
    (1, 700, 3, 1, 256, 256),     # a cut history of wide heads
    (2, 520, 3, 3, 256, 64), (2, 520, 3, 3, 40, 256), (1, 650, 2, 2, 255, 130),
])
def test_every_walk(kind, ragged, B, T, H, G, dk, dv):
    torch = require_gpu()
    lengths = None
    if ragged:
        lengths = [(T - 1, T, T // 2, 0, 1, 64, T // 3)[(b + (0 if B > 1 else 2)) % 7] for b in range(B)]
    t, _ = make(torch, kind, B, T, H, G, dk, dv, B + T, lengths)
    clean = dict(t)
    for name in ("q", "k", "v", "do") if ragged else ():
        clean[name] = t[name].clone()
        for b, n in enumerate(lengths):
            t[name][b, n:] = float("nan")
            clean[name][b, n:] = 0.0
    for gradient in (False, True):
        check_on_device(torch, t, clean, kind, gradient)


@pytest.mark.parametrize("ragged", [False, True])
def test_definition_on_the_device(ragged):
    """The device's float64 definition is the oracle's."""
    torch = require_gpu()
    t, x = make(torch, "fp32", 3, 20, 4, 2, 5, 7, 90, [20, 0, 11] if ragged else None)
    args = [x[n] for n in "qkv"]
    for got, want in ((device_definition(torch, t, 0.3, False),
                       lo.linear_attention(*args, x["decay"], x["state"], x["lengths"], 0.3)),
                      (device_definition(torch, t, 0.3, True),
                       lo.linear_attention_grad(*args, x["decay"], x["do"], x["dlast"], x["state"],
                                                x["lengths"], 0.3))):
        for a, b in zip(got, want):
            assert np.abs(a.cpu().numpy() - b).max() <= 1e-12 * np.abs(b).max()


def test_gradient_along_itself():
    """The outputs are linear in each of q, k, v and the state, so differences of any size are exact
    but for rounding. Along the gradient itself (of one head, too) they are far above what rounding
    can make: a gradient that is scaled, turned or 0 fails."""
    torch = require_gpu()
    from symmetric_nmf_clustering_amd import api
    t, _ = make(torch, "fp32", 2, 300, 4, 2, 40, 24, 13, lengths=[300, 171])
    kw = dict(lengths=t["lengths"], scale=0.2)
    grads = api.linear_attention_grad(t["q"], t["k"], t["v"], t["decay"], t["do"], dlast=t["dlast"],
                                      state=t["state"], **kw)

    def value(at):
        o, last = api.linear_attention(at["q"], at["k"], at["v"], t["decay"], state=at["state"], **kw)
        return ((t["do"].double() * o.double()).sum() + (t["dlast"].double() * last.double()).sum()).item()

    def terms(at):
        o, last = device_definition(torch, {n: x if n in ("decay", "lengths") else x.abs() for n, x in at.items()},
                                    0.2, False)
        return ((t["do"].double().abs() * o).sum() + (t["dlast"].double().abs() * last).sum()).item()

    for name, grad in zip(("q", "k", "v", "state"), grads):
        head = torch.zeros_like(grad)
        if name == "state":
            head[:, 1] = grad[:, 1]
        else:
            head[:, :, 1] = grad[:, :, 1]
        for along in (grad, head):
            d = along * (30.0 / along.square().mean().sqrt())
            hi, lo_ = ({**t, name: t[name] + sign * d} for sign in (1, -1))
            want = (grad.double() * d.double()).sum().item()
            # the kernels' share of the terms, the inputs' sums and the gradient's own rounding
            limit = (attend_bound("fp32", 300, 40, 24) + 2 * U) * (terms(hi) + terms(lo_))
            assert limit < 0.05 * want
            assert abs((value(hi) - value(lo_)) / 2 - want) <= limit
