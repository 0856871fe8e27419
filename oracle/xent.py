"""Cross entropy of the vocabulary head and its gradients in float64, from the formulas.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).  The pages describe inference only; the
definitions are those of the softmax cross entropy: z = h W^T / T, lse_i = ln sum_v e^{z_iv},
loss_i = lse_i - z_{i,y_i}, and for sum_i g_i loss_i the gradients dz = g (softmax(z) - onehot(y)),
dh = dz W / T, dW = dz^T h / T.

`bounds` gives how far fp32 sums of the same products and a bf16 G may be off, element by element.
"""

import numpy as np


def cross_entropy(h, W, y, T=1.0, ignore=-100, dloss=None):
    """float64 loss, lse (0 at ignored positions) and, with dloss, (dh, dW, G) of the positions."""
    h, W = np.asarray(h, np.float64), np.asarray(W, np.float64)
    y = np.asarray(y, np.int64)
    n = len(y)
    loss, lse = np.zeros(n), np.zeros(n)
    keep = np.flatnonzero(y != ignore)
    G = np.zeros((n, W.shape[0]))
    if len(keep):
        z = h[keep] @ W.T / T
        yt = y[keep]
        k = np.arange(len(keep))
        zt = z[k, yt].copy()
        others = z.copy()
        others[k, yt] = -np.inf
        top = others.max(1)
        top = np.where(np.isfinite(top), top, 0.0)
        with np.errstate(divide="ignore"):
            x = top + np.log(np.exp(others - top[:, None]).sum(1))
        loss[keep] = np.logaddexp(0.0, x - zt)
        lse[keep] = zt + loss[keep]
        if dloss is not None:
            P = np.exp(z - lse[keep][:, None])
            P[k, yt] = np.expm1(-loss[keep])
            G[keep] = P * (np.asarray(dloss, np.float64)[keep] / T)[:, None]
    if dloss is None:
        return loss, lse
    G[np.asarray(dloss) == 0] = 0.0
    live = np.where((G != 0).any(1)[:, None], h, 0.0)
    return loss, lse, G @ W, G.T @ live, G


def bounds(h, W, y, T, G, loss, lse, ignore=-100):
    """(per-position bound of |z|'s error, and elementwise bounds of dh and dW before their own rounding).

    A sum of d exact products in fp32 whose every step may drop up to one unit in the last place of the
    running sum (2^-23, no more than the sum of the magnitudes) is off by at most d 2^-23 sum |h W|; the
    tensor core adds 16 products a step, so d / 16 + 4 steps count.  z in log2 units, the exponential
    (2^-21 with its argument's rounding at |z| <= 64) and lse's own error come on top; G's rounding to bf16
    is 2^-8 of each entry.
    """
    y = np.asarray(y, np.int64)
    ah = np.where((y != ignore)[:, None], np.abs(np.nan_to_num(np.asarray(h, np.float64), posinf=0, neginf=0)), 0.0)
    aW = np.abs(np.asarray(W, np.float64))
    d, n = ah.shape[1], len(y)
    mag = (ah @ aW.T).max(1) / T
    dz = (d / 16 + 4) * 2.0 ** -23 * mag + 2.0 ** -22 * (1 + np.abs(lse))
    rel = 2.0 ** -8 + 3 * dz.max(initial=0) + 2.0 ** -20
    aG = np.abs(G)
    dh = (rel + (W.shape[0] / 16 + 64) * 2.0 ** -23) * (aG @ aW)
    dW = (rel + (n / 16 + 4) * 2.0 ** -23) * (aG.T @ ah)
    return dz, dh, dW
