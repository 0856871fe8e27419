"""The training entry points on the GPU where they could go wrong at the edges of what they document: rounding of
the gradients' largest entries, logits that are not finite, values below the normal range, steps and streams."""

import numpy as np
import pytest
import torch

from oracle import xent
from test_gpu_xent import IGNORE, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dg():
    from discrete_diffusion_decoding_b200 import build
    build.build()
    import discrete_diffusion_decoding_b200 as m
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return m


def half_sure(n, V, d, kept, seed):
    """Positions whose target has about half the probability, among rows of W that are otherwise small."""
    g = torch.Generator().manual_seed(seed)
    y = torch.randperm(V, generator=g)[:n]
    W = torch.randn(V, d, generator=g) * 2.0 ** -9
    W[y] = torch.randn(n, d, generator=g) * 0.25
    W = W.bfloat16()
    to = W[y].float()
    h = (torch.log(torch.tensor(float(V))) * to / (to * to).sum(1, keepdim=True)).bfloat16()
    y[torch.randperm(n, generator=g)[:n - kept]] = IGNORE
    return h, W, y.int(), torch.rand(n, generator=g) + 0.5


@pytest.mark.parametrize("n,V,d,kept,scratch", [(1, 200, 64, 1, 0), (5, 700, 72, 5, 0), (31, 600, 136, 31, 0),
                                                (32, 600, 64, 32, 1), (33, 600, 64, 33, 0), (300, 1500, 96, 32, 1),
                                                (300, 1500, 96, 33, 0), (300, 1500, 96, 200, 0)])
def test_the_targets_entry_of_g_is_not_rounded_away(dg, n, V, d, kept, scratch):
    """The target's entry of G reaches dh, and dW of at most 32 positions, with more than bf16's digits."""
    h, W, y, dl = half_sure(n, V, d, kept, n + kept)
    got = run(dg, h, W, y, dl, dw=torch.zeros(V, d, device="cuda"), scratch_bytes=scratch)
    h64, W64, dn = h.double().numpy(), W.double().numpy(), np.where(y == IGNORE, 0.0, dl.double().numpy())
    loss, lse, dh, dW, G = xent.cross_entropy(h64, W64, y.numpy(), 1.0, IGNORE, dn)
    dz = xent.bounds(h64, W64, y.numpy(), 1.0, G, loss, lse)[0].max()
    T = np.zeros_like(G)
    rows = np.flatnonzero(y != IGNORE)
    T[rows, y[rows]] = np.abs(G)[rows, y[rows]]
    rest = np.abs(G) - T
    # every entry: the logits' error three times over (z, lse and the exponential), the weights' and the fp32
    # factors' roundings 2^-20, the sums' steps; the other entries are rounded to bf16, and of the target's what
    # that leaves out is rounded once more: 2^-8 of 2^-8
    each = 3 * dz + 2.0 ** -20
    aw, ah = np.abs(W64), np.where((y != IGNORE).numpy()[:, None], np.abs(h64), 0)
    tol_h = (each + 2.0 ** -16 + (V / 16 + 64) * 2.0 ** -23) * (np.abs(G) @ aw) + 2.0 ** -8 * (rest @ aw)
    tol_w = (each + 2.0 ** -16 + (n / 16 + 4) * 2.0 ** -23) * (np.abs(G).T @ ah) + 2.0 ** -8 * (rest.T @ ah)
    tol_h = tol_h * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(dh)
    tol_w = tol_w + 2.0 ** -24 * np.abs(dW) + (2.0 ** -8 * (T.T @ ah) if kept > 32 else 0)
    assert np.all(np.abs(got[2] - dh) <= tol_h) and np.all(np.abs(got[3] - dW) <= tol_w)
    # the same with the entry rounded is outside
    B = torch.from_numpy(G).bfloat16().double().numpy()
    assert np.any(np.abs(torch.from_numpy(B @ W64).bfloat16().double().numpy() - dh) > tol_h)
    assert kept > 32 or np.any(np.abs(B.T @ h64 - dW) > tol_w)


# ------------------------------------------------------------------ logits that are not finite
@pytest.mark.parametrize("n", [4, 40])
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), "overflow"])
def test_a_target_whose_logit_is_not_finite_gives_nan(dg, n, value):
    """A diverged row of the head reports no perfect loss: NaN in loss, lse, dh and dW, not 0."""
    V, d = 600, 64
    g = torch.Generator().manual_seed(n)
    W = (torch.randn(V, d, generator=g) * 0.05).bfloat16()
    h = torch.randn(n, d, generator=g).bfloat16()
    y = torch.randint(0, V, (n,), generator=g).int()
    y[y == 17] = 18
    y[2] = 17
    keep = np.arange(n) != 2
    if value == "overflow":               # only position 2 has this product
        W[:, 5], h[:, 5] = 0, 0
        W[17, 5], h[2, 5] = 1e30, 1e30
    else:                                 # every position sees the infinity; it is the target's at position 2
        W[17, 6], h[:, 6] = value, 1.0
    loss, lse, dh, dW = run(dg, h, W, y, torch.ones(n))
    assert np.isnan(loss[2]) and np.isnan(lse[2]) and np.isnan(dh[2]).all() and np.isnan(dW).all()
    if value == "overflow":
        assert np.isfinite(loss[keep]).all() and np.isfinite(dh[keep]).all()
    elif value == float("inf"):
        assert np.isnan(loss).all() and np.isnan(dh).all()
    elif value == float("-inf"):
        # elsewhere the column has no share: the loss is that of the head without it
        h64, W64 = h.double().numpy()[keep], np.delete(W.double().numpy(), 17, 0)
        y0 = np.where(y.numpy() > 17, y.numpy() - 1, y.numpy())[keep]
        want, want_lse = xent.cross_entropy(h64, W64, y0)
        dz = xent.bounds(h64, W64, y0, 1.0, np.zeros((n - 1, V - 1)), want, want_lse)[0]
        assert np.all(np.abs(loss[keep] - want) <= 2 * dz + 2.0 ** -20 * want)
