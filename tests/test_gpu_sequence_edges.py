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
