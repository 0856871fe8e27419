"""AdamW with decoupled weight decay, states in fp32 or as E4M3 codes in blocks of 256.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).  Loshchilov and Hutter, "Decoupled Weight Decay
Regularization" (ICLR 2019), algorithm 2, with Kingma and Ba's bias corrections.  `step` is float64;
`moments` and `encode` repeat what is stored in the fp32 roundings that the library's header states (each
product and sum rounded by itself), so that codes, exponents and fp32 states can be compared bit by bit.
"""

import numpy as np

from . import fp8, philox

BLOCK = 256
TAG_STATE, TAG_PARAM = 5, 6


def step(p, g, m, v, t, lr, b1, b2, eps, wd, grad_scale=1.0):
    """One float64 step: new (p, m, v)."""
    p, g, m, v = (np.asarray(x, np.float64) for x in (p, g, m, v))
    g = g * grad_scale
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    p = p - lr * wd * p - lr * (m / (1 - b1 ** t)) / (np.sqrt(v / (1 - b2 ** t)) + eps)
    return p, m, v


def moments(g, m, v, b1, b2, grad_scale=1.0):
    """The fp32 moments, each operation rounded."""
    f = np.float32
    g = np.asarray(g, f) * f(grad_scale)
    m = np.asarray(m, f) * f(b1) + g * f(1.0 - b1)
    v = np.asarray(v, f) * f(b2) + (g * g) * f(1.0 - b2)
    return m, v


def exponent(x):
    """Per block of 256: the smallest e with max |x| 2^-e <= 448, 0 for zeros, at least -100 (finite values)."""
    n = len(x)
    pad = np.zeros(-(-n // BLOCK) * BLOCK)
    pad[:n] = np.where(np.isfinite(x), np.abs(np.asarray(x, np.float64)), 0.0)
    out = []
    for peak in pad.reshape(-1, BLOCK).max(1):
        e = -100
        while peak * 2.0 ** -e > 448:
            e += 1
        out.append(0 if peak == 0 else e)
    return np.array(out, np.int64)


def random_halves(seed, n, t, tensor):
    """16 random bits for each element: (for m, for sqrt(v))."""
    i = np.arange(n)
    w = philox.words(seed, i // 4, t, tensor, TAG_STATE)[np.arange(n), i % 4].astype(np.int64)
    return w & 0xFFFF, w >> 16


def random_param(seed, n, t, tensor):
    i = np.arange(n)
    w = philox.words(seed, i // 8, t, tensor, TAG_PARAM)[np.arange(n), (i % 8) // 2].astype(np.int64)
    return np.where(i % 2, w >> 16, w & 0xFFFF)


def encode(x, u, root=False):
    """(codes, exponents) of x with 16 random bits u an element."""
    x = np.asarray(x, np.float32)
    e = exponent(x)
    y = np.abs(x.astype(np.float64)) * 2.0 ** -np.repeat(e, BLOCK)[:len(x)].astype(np.float64)
    fin = np.isfinite(y)
    y = np.where(fin, y, 0.0)
    # below the smallest normal the library adds 2^-6 in fp32 before it cuts
    small = y < 2.0 ** -6
    y = np.where(small, (y + 2.0 ** -6).astype(np.float32).astype(np.float64) - 2.0 ** -6, y)
    k = np.floor(np.log2(np.maximum(y, 2.0 ** -6)))
    spacing = 2.0 ** (k - 3)
    q = np.floor(y / spacing + u / 65536) * spacing
    if root:
        q = np.where((x > 0) & (q == 0), 2.0 ** -9, q)
    codes = np.array([_code(v) for v in q], np.uint8)
    codes = np.where(fin, codes, 0x7F).astype(np.uint8)
    return codes | np.where(np.signbit(x) & (x != 0), 0x80, 0).astype(np.uint8), e


_TABLE = {float(v): c for c, v in enumerate(fp8.decode(np.arange(127, dtype=np.uint8)))}


def _code(v):
    return _TABLE[float(v)]


def decode(codes, e):
    n = len(codes)
    return fp8.decode(np.asarray(codes, np.uint8)) * 2.0 ** np.repeat(np.asarray(e, np.float64), BLOCK)[:n]


def round_bf16_random(p, u):
    """fp32 values cut to bf16 after u is added to their low 16 bits."""
    bits = np.asarray(p, np.float32).view(np.uint32).astype(np.int64) + u
    return ((bits >> 16) << 16).astype(np.uint32).view(np.float32)
