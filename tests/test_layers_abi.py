"""Refusals and workspace sizes of the layer operators (no device work)."""
import ctypes
import os

import pytest

from symmetric_nmf_clustering_amd import _lib as L

pytestmark = pytest.mark.skipif(not os.path.exists(L.LIB_PATH),
                                reason="libsymnmf.so not built (run __graft_entry__.build())")
P = ctypes.c_void_p(0x10000)  # never dereferenced: every call below is refused
ODD = ctypes.c_void_p(0x10001)
Z = 1 << 40


def desc(**change):
    d = dict(type=0, heads=4, kv_heads=2, dk=8, dv=6, scale=0.5, batch=2, steps=5,
             q_stride=(160, 32, 8), k_stride=(80, 16, 8), v_stride=(60, 12, 6), do_stride=(120, 24, 6))
    d.update(change)
    return ctypes.byref(L.AttendDesc(**d))


BAD = [dict(type=3), dict(heads=0), dict(heads=3), dict(heads=65537), dict(kv_heads=0), dict(kv_heads=8),
       dict(dk=0), dict(dk=257), dict(dv=0), dict(dv=257), dict(scale=float("nan")),
       dict(scale=float("inf")), dict(batch=0), dict(steps=-1), dict(steps=1 << 31),
       dict(batch=1 << 29), dict(q_stride=(-1, 0, 0)), dict(k_stride=(0, -1, 0)),
       dict(v_stride=(0, 0, -1)), dict(do_stride=(0, -1, 0))]


def test_workspace_sizes():
    f = L.load().symnmf_linear_attention_ws_bytes
    for bad in BAD:
        assert f(desc(**bad), 0) == 0 and f(desc(**bad), 1) == 0, bad
    assert f(None, 0) == 0 and f(desc(), 2) == 0
    assert f(desc(), 0) == 256 and f(desc(steps=0), 1) > 0
    # shared key heads: their gradients for each query head in float32 first
    assert f(desc(), 1) >= 2 * 5 * 4 * (8 + 6) * 4
    assert f(desc(kv_heads=4), 1) == 256
    # few heads: time is cut, a state for each segment
    long = dict(batch=1, heads=1, kv_heads=1, steps=1 << 16, dk=128, dv=128)
    assert f(desc(**long), 0) > 2 * 128 * 128 * 4


@pytest.mark.parametrize("heads,d,steps", [(1, 4, 512), (2, 2, 1024), (1, 1, 4096), (1, 1, 512), (2, 3, 700)])
def test_a_used_workspace_is_never_the_least(heads, d, steps):
    """256 bytes stand for "not touched", and the binding's calls share them: a call that is cut in
    time asks for more, however small its segments' states."""
    f = L.load().symnmf_linear_attention_ws_bytes
    small = dict(batch=1, heads=heads, kv_heads=heads, dk=d, dv=d)
    assert f(desc(steps=steps, **small), 0) > 256 and f(desc(steps=steps, **small), 1) > 256
    assert f(desc(steps=300, **small), 0) == 256 and f(desc(steps=300, **small), 1) == 256


def test_linear_attention_refusals():
    f = L.load().symnmf_linear_attention
    good = [desc(), P, P, P, P, None, None, P, None, P, Z, None]
    for i, bad in [(0, desc(**b)) for b in BAD] + [
            (0, None), (1, None), (1, ODD), (2, None), (3, ODD), (4, None), (4, ODD), (5, ODD), (6, ODD),
            (7, None), (7, ODD), (8, ODD)]:
        a = list(good)
        a[i] = bad
        assert f(*a) == L.E_INVALID, (i, bad)
    for i, bad in ((9, None), (9, ctypes.c_void_p(0x10010)), (10, 64)):
        a = list(good)
        a[i] = bad
        assert f(*a) == L.E_WORKSPACE, (i, bad)


def test_linear_attention_grad_refusals():
    f = L.load().symnmf_linear_attention_grad
    good = [desc(), P, P, P, P, None, None, P, None, P, P, P, None, P, Z, None]
    for i, bad in [(0, desc(**b)) for b in BAD] + [
            (0, None), (1, None), (2, ODD), (3, None), (4, None), (5, ODD), (6, ODD), (7, None), (7, ODD),
            (8, ODD), (9, None), (10, ODD), (11, None), (12, ODD)]:
        a = list(good)
        a[i] = bad
        assert f(*a) == L.E_INVALID, (i, bad)
    for i, bad in ((13, None), (13, ctypes.c_void_p(0x10010)), (14, 64)):
        a = list(good)
        a[i] = bad
        assert f(*a) == L.E_WORKSPACE, (i, bad)


def test_linear_attention_step_refusals():
    f = L.load().symnmf_linear_attention_step
    good = [desc(steps=1), P, P, P, P, P, P, P, None]
    for i, bad in [(0, desc(**{**dict(steps=1), **b})) for b in BAD] + [
            (0, None), (0, desc(steps=2)), (0, desc(steps=0))] + [(i, x) for i in range(1, 8) for x in (None, ODD)]:
        a = list(good)
        a[i] = bad
        assert f(*a) == L.E_INVALID, (i, bad)


def test_rotary_refusals():
    f = L.load().symnmf_rotary
    good = [0, 2, 5, 4, 8, 6, 0, 0, 1.0, P, 160, 32, 8, P, 0, 5, 1, P, P, 160, 32, 8, None]
    for i, bad in ((0, 3), (1, -1), (2, -1), (3, 0), (4, 0), (5, 7), (5, 10), (5, -2), (6, 2), (7, 2),
                   (8, float("nan")), (9, None), (9, ODD), (10, -1), (11, -1), (12, -1), (13, None),
                   (13, ODD), (14, 2), (15, -1), (16, -1), (17, None), (17, ODD), (18, None), (18, ODD),
                   (19, -1), (20, -1), (21, -1)):
        a = list(good)
        a[i] = bad
        assert f(*a) == L.E_INVALID, (i, bad)
    for i in (1, 2):
        a = list(good)
        a[i] = 0
        assert f(*a) == L.OK  # nothing to turn


def tensors(n=4, **change):
    t = dict(param=0x10000, grad=0x20000, m=0x30000, v=0x40000, m_scale=0x50000, v_scale=0x60000,
             master=None, n=n)
    t.update(change)
    return (L.AdamwTensor * 1)(L.AdamwTensor(**t))


def test_adamw_refusals():
    f = L.load().symnmf_adamw
    good = [0, 0, 8, tensors(), 1, 1e-3, 0.9, 0.999, 1e-8, 0.0, 1, 1.0, None, None, None, None]
    nan, inf = float("nan"), float("inf")
    for i, bad in ((0, 3), (1, -1), (2, 16), (3, None), (4, -1), (5, nan), (5, inf), (6, 1.0), (6, -0.1),
                   (6, nan), (7, 1.0), (7, nan), (8, -1e-8), (8, inf), (9, nan), (10, 0), (10, -3), (11, nan),
                   (12, ctypes.c_void_p(0x10004)), (13, ODD), (14, ODD)):
        a = list(good)
        a[i] = bad
        assert f(*a) == L.E_INVALID, (i, bad)
    for change in (dict(param=None), dict(param=0x10001), dict(grad=None), dict(m=None), dict(v=None),
                   dict(m_scale=None), dict(v_scale=0x60002), dict(master=0x10002), dict(n=-1)):
        a = list(good)
        a[3] = tensors(**change)
        assert f(*a) == L.E_INVALID, change
    a = list(good)
    a[2], a[3] = 32, tensors(m=0x30001)
    assert f(*a) == L.E_INVALID
    for a in (good[:4] + [0] + good[5:], good[:3] + [tensors(n=0, param=None)] + good[4:]):
        assert f(*a) == L.OK  # nothing to update


def test_binding_refuses_host_tensors():
    import torch

    from symmetric_nmf_clustering_amd import api
    t = torch.zeros(2, 3, 4, 5)
    for call in (lambda: api.linear_attention(t, t, t, t[0, 0, :, 0]),
                 lambda: api.linear_attention_grad(t, t, t, t[0, 0, :, 0], t),
                 lambda: api.linear_attention_step(t[0], t[0], t[0], t[0, 0, :, 0], t),
                 lambda: api.rotary(t, torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2).double()),
                 lambda: api.adamw_step([t], [t], [t], [t], 1)):
        with pytest.raises(ValueError, match="device tensor"):
            call()


def test_rotary_freqs():
    import math

    import torch

    from symmetric_nmf_clustering_amd import api
    f, amp = api.rotary_freqs(8, 100.0, device="cpu")
    assert amp == 1.0 and f.dtype == torch.float64
    assert torch.allclose(f, torch.tensor([1.0, 100.0 ** -0.25, 0.1, 100.0 ** -0.75]).double())
    g, amp = api.rotary_freqs(8, 100.0, scaling="linear", factor=4.0, device="cpu")
    assert amp == 1.0 and torch.allclose(g, f / 4)
    g, amp = api.rotary_freqs(8, 100.0, scaling="base", factor=4.0, device="cpu")
    assert amp == 1.0 and torch.allclose(g[0], f[0]) and torch.allclose(g[3], f[3] / 4)
    g, amp = api.rotary_freqs(64, scaling="parts", factor=8.0, original=4096, device="cpu")
    f, _ = api.rotary_freqs(64, device="cpu")
    turns = 4096 * f / (2 * math.pi)
    assert torch.allclose(g[turns >= 32], f[turns >= 32]) and torch.allclose(g[turns <= 1], f[turns <= 1] / 8)
    mid = (turns > 1) & (turns < 32)
    assert mid.any() and (g[mid] < f[mid]).all() and (g[mid] > f[mid] / 8).all()
    assert abs(amp - 1 - 0.1 * math.log(8.0)) < 1e-15
    for bad in (dict(dims=7), dict(dims=0), dict(dims=8, base=0.0), dict(dims=8, factor=0.0),
                dict(dims=2, scaling="base"), dict(dims=8, scaling="other"),
                dict(dims=8, scaling="parts", fast=1.0, slow=1.0)):
        with pytest.raises(ValueError):
            api.rotary_freqs(device="cpu", **bad)


def test_shared_elements_of_views():
    """The overlap checks against the sets of addresses, over random views of one buffer."""
    import random

    import torch

    from symmetric_nmf_clustering_amd import api
    buf = torch.zeros(400)
    rng = random.Random(3)

    def view():
        while True:
            shape = tuple(rng.choice((1, 2, 3, 5)) for _ in range(rng.choice((3, 4))))
            strides = tuple(rng.choice((0, 1, 2, 3, 4, 8, 12, 24, 25, 48)) for _ in shape[:-1]) + (1,)
            at = rng.randrange(60)
            if at + sum((n - 1) * s for n, s in zip(shape, strides)) < 400:
                return torch.as_strided(buf, shape, strides, at)

    def cells(v):
        a = torch.as_strided(torch.arange(400), v.shape, v.stride(), v.storage_offset())
        return a.reshape(-1).tolist()

    seen = set()
    for _ in range(3000):
        a, b = view(), view()
        ca, cb = cells(a), cells(b)
        assert api._elements_apart(a.shape, a.stride()) == (len(set(ca)) == len(ca)), (a.shape, a.stride())
        assert api._share(a, b) == bool(set(ca) & set(cb)), (a.shape, a.stride(), b.shape, b.stride())
        seen.add((api._share(a, b), max(ca) >= min(cb) and max(cb) >= min(ca)))
    assert seen == {(True, True), (False, True), (False, False)}
    wide = torch.zeros(64, 7 * 128).unflatten(1, (7, 128))  # heads of one projection
    assert not api._share(wide[:, :3], wide[:, 3:6]) and api._share(wide[:, :3], wide[:, 2:5])
    assert api._elements_apart(wide.shape, wide.stride()) and not api._share(wide[:0], wide[:0])


def test_ranges_that_meet_are_refused():
    from symmetric_nmf_clustering_amd import api
    apart = [(100, 140), (140, 180), (300, 301)]
    for read in ([], [(60, 40), (180, 120), (301, 9)], [(200, 8), (200, 8)]):
        api._check_apart(apart[::-1], read)
    for written in ([(100, 140), (139, 180)], [(0, 50), (10, 20), (60, 70)], [(5, 9), (5, 9)]):
        with pytest.raises(ValueError, match="share memory"):
            api._check_apart(written, [])
    for read in ((99, 2), (100, 40), (179, 1), (0, 1000), (290, 11), (120, 4), (150, 100)):
        with pytest.raises(ValueError, match="shares memory"):
            api._check_apart(list(apart), [(0, 10), read])
