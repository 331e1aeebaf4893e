"""Refusals and workspace sizes of the sequence operators (no device work)."""
import ctypes
import os

import pytest

from symmetric_nmf_clustering_amd import _lib as L

pytestmark = pytest.mark.skipif(not os.path.exists(L.LIB_PATH),
                                reason="libsymnmf.so not built (run __graft_entry__.build())")
P = ctypes.c_void_p(0x10000)  # never dereferenced: every call below is refused
ODD = ctypes.c_void_p(0x10001)
Z = 1 << 40


def test_workspace_sizes():
    wb = L.load().symnmf_workspace_bytes
    # sorted tokens and their chunks' partial rows, a flag per table row
    assert 0 < wb(L.OP_EMBED_GRAD, 100000, 1024, 32768, None) < 32768 * 16 + 100000 + \
        2 * 1024 * 1024 * 4 + 2 ** 20
    assert wb(L.OP_EMBED_GRAD, 5, 3, 0, None) > 0
    assert 0 < wb(L.OP_GATED_SCAN, 1024, 2, 32768, None) < 2 ** 21
    assert wb(L.OP_GATED_SCAN, 1024, 2, 0, None) > 0
    assert wb(L.OP_TOKEN_LOGPROBS, 24, 3, 100000, None) > 0
    assert wb(L.OP_TOKEN_LOGPROBS, 100000, 32, 0, None) > 0
    for op, n, k, T in ((L.OP_EMBED_GRAD, 0, 4, 4), (L.OP_EMBED_GRAD, 4, 0, 4),
                        (L.OP_EMBED_GRAD, 4, 4, -1), (L.OP_GATED_SCAN, 4, 65536, 4),
                        (L.OP_GATED_SCAN, 4, 0, 4), (L.OP_GATED_SCAN, 4, 1, -1),
                        (L.OP_TOKEN_LOGPROBS, 4, 33, 4), (L.OP_TOKEN_LOGPROBS, 0, 1, 4),
                        (L.OP_TOKEN_LOGPROBS, 4, -1, 4), (L.OP_TOKEN_LOGPROBS, 4, 1, -1)):
        assert wb(op, n, k, T, None) == 0, (op, n, k, T)


def test_embed_refusals():
    f = L.load().symnmf_embed
    good = [P, 0, 10, 8, 8, P, 0, 4, 1.0, P, 0, 8, None]
    for i, bad in ((0, None), (0, ODD), (1, 3), (2, 0), (3, 0), (4, 7), (5, None), (5, ODD),
                   (6, 2), (7, -1), (9, None), (9, ODD), (10, 9), (11, 7)):
        a = list(good)
        a[i] = bad
        assert f(*a) == L.E_INVALID, (i, bad)
    good[7] = 0
    assert f(*good) == L.OK  # nothing to look up


def test_embed_grad_refusals():
    f = L.load().symnmf_embed_grad
    good = [P, 0, 4, 8, 8, P, 0, 1.0, 0, P, 0, 10, 8, P, Z, None]
    for i, bad in ((0, None), (0, ODD), (1, 3), (2, -1), (3, 0), (4, 7), (5, None), (6, 2),
                   (8, 2), (9, None), (9, ODD), (10, -1), (11, 0), (12, 7)):
        a = list(good)
        a[i] = bad
        assert f(*a) == L.E_INVALID, (i, bad)
    for i, bad in ((13, None), (13, ctypes.c_void_p(0x10010)), (14, 64)):
        a = list(good)
        a[i] = bad
        assert f(*a) == L.E_WORKSPACE, (i, bad)


def test_gated_scan_refusals():
    f = L.load().symnmf_gated_scan
    good = [0, 2, 5, 8, P, 40, 8, P, 40, 8, None, None, P, None, None, P, Z, None]
    for i, bad in ((0, 3), (1, 0), (1, 65536), (2, -1), (3, 0), (4, None), (4, ODD), (5, -1),
                   (6, -8), (7, None), (7, ODD), (8, -1), (9, -8), (10, ODD), (11, ODD),
                   (12, None), (12, ODD), (13, ODD), (14, ODD)):
        a = list(good)
        a[i] = bad
        assert f(*a) == L.E_INVALID, (i, bad)
    for i, bad in ((15, None), (15, ctypes.c_void_p(0x10010)), (16, 64)):
        a = list(good)
        a[i] = bad
        assert f(*a) == L.E_WORKSPACE, (i, bad)


def test_gated_scan_grad_refusals():
    f = L.load().symnmf_gated_scan_grad
    good = [0, 2, 5, 8, P, 40, 8, P, 40, 8, None, P, P, 40, 8, None, P, P, None, P, Z, None]
    for i, bad in ((0, 3), (1, 0), (2, -1), (3, 0), (4, None), (5, -1), (6, -8), (7, None),
                   (8, -1), (9, -8), (10, ODD), (11, None), (11, ODD), (12, None), (13, -1),
                   (14, -1), (15, ODD), (16, None), (16, ODD), (17, None), (18, ODD)):
        a = list(good)
        a[i] = bad
        assert f(*a) == L.E_INVALID, (i, bad)
    for i, bad in ((19, None), (19, ctypes.c_void_p(0x10010)), (20, 64)):
        a = list(good)
        a[i] = bad
        assert f(*a) == L.E_WORKSPACE, (i, bad)


def test_token_logprobs_refusals():
    f = L.load().symnmf_token_logprobs
    good = [P, 0, 4, 1000, 1000, P, 0, 1.0, P, None, None, 2, P, P, P, Z, None]
    for i, bad in ((0, None), (0, ODD), (1, 3), (2, -1), (3, 0), (4, 999), (5, None), (5, ODD),
                   (6, 2), (7, 0.0), (7, -1.0), (7, float("nan")), (7, float("inf")), (8, None),
                   (9, ODD), (10, ODD), (11, -1), (11, 33), (12, None), (13, None)):
        a = list(good)
        a[i] = bad
        assert f(*a) == L.E_INVALID, (i, bad)
    for i, bad in ((14, None), (14, ctypes.c_void_p(0x10010)), (15, 8)):
        a = list(good)
        a[i] = bad
        assert f(*a) == L.E_WORKSPACE, (i, bad)
    good[2] = 0
    assert f(*good) == L.OK  # no rows


def test_token_logprobs_grad_refusals():
    f = L.load().symnmf_token_logprobs_grad
    good = [P, 0, 4, 1000, 1000, P, 0, 1.0, P, P, P, P, P, 1000, None]
    for i, bad in ((0, None), (0, ODD), (1, 3), (2, -1), (3, 0), (4, 999), (5, None), (6, 2),
                   (7, 0.0), (7, float("nan")), (8, None), (9, None), (9, ODD), (10, None),
                   (11, ODD), (12, None), (12, ODD), (13, 999)):
        a = list(good)
        a[i] = bad
        assert f(*a) == L.E_INVALID, (i, bad)
    good[2] = 0
    assert f(*good) == L.OK


def test_binding_refuses_host_tensors():
    import torch

    from symmetric_nmf_clustering_amd import api
    t, i = torch.zeros(4, 3), torch.zeros(2, dtype=torch.int32)
    for call in (lambda: api.embed(t, i), lambda: api.embed_grad(t, i, 4),
                 lambda: api.gated_scan(t[None], t[None]),
                 lambda: api.gated_scan_grad(t[None], t[None], t[None], t[None]),
                 lambda: api.token_logprobs(t, i),
                 lambda: api.token_logprobs_grad(t, i, t[:, 0], None, t[:, 0])):
        with pytest.raises(ValueError, match="device tensor"):
            call()
