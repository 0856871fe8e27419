"""Training the head, without a GPU: the float64 oracles against independent forms and differences, and the
refusals of the bindings and of the C entry points that need no device."""

import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

from oracle import adamw, fp8, philox, xent

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def dg():
    from discrete_diffusion_decoding_b200 import build
    build.build()
    import discrete_diffusion_decoding_b200 as m
    return m


# ------------------------------------------------------------------ cross entropy oracle
@pytest.mark.parametrize("n,V,d,T", [(1, 1, 8, 1.0), (5, 7, 8, 0.5), (40, 33, 16, 1.3)])
def test_oracle_matches_autograd(n, V, d, T):
    g = torch.Generator().manual_seed(n)
    h = torch.randn(n, d, generator=g, dtype=torch.float64, requires_grad=True)
    W = torch.randn(V, d, generator=g, dtype=torch.float64, requires_grad=True)
    y = torch.randint(0, V, (n,), generator=g)
    y[::4] = -100
    w = torch.rand(n, generator=g, dtype=torch.float64)
    z = h @ W.T / T
    loss = torch.nn.functional.cross_entropy(z, y, reduction="none", ignore_index=-100)
    (loss * w).sum().backward()
    got = xent.cross_entropy(h.detach().numpy(), W.detach().numpy(), y.numpy(), T, -100, w.numpy())
    kept = (y != -100).numpy()
    assert np.allclose(got[0], loss.detach().numpy(), rtol=1e-12, atol=1e-13)
    assert np.allclose(got[1][kept], torch.logsumexp(z, 1).detach().numpy()[kept], rtol=1e-12)
    assert np.allclose(got[2], h.grad.numpy(), rtol=1e-10, atol=1e-13)
    assert np.allclose(got[3], W.grad.numpy(), rtol=1e-10, atol=1e-13)


def test_oracle_gradient_against_differences():
    rng = np.random.default_rng(0)
    h, W, y, w = rng.normal(size=(6, 5)), rng.normal(size=(9, 5)), rng.integers(0, 9, 6), rng.random(6)
    _, _, dh, dW, _ = xent.cross_entropy(h, W, y, 0.7, -100, w)

    def total(h, W):
        return (xent.cross_entropy(h, W, y, 0.7)[0] * w).sum()

    e = 1e-5
    for x, grad, of in ((h, dh, lambda q: total(q, W)), (W, dW, lambda q: total(h, q))):
        for i in np.ndindex(x.shape):
            up, down = x.copy(), x.copy()
            up[i] += e
            down[i] -= e
            assert abs((of(up) - of(down)) / (2 * e) - grad[i]) < 1e-8


def test_oracle_keeps_the_digits_of_small_losses():
    """One competitor at distance x: loss = ln(1 + e^-x)."""
    for x in (1.0, 10.0, 40.0, 300.0):
        loss, lse = xent.cross_entropy(np.array([[x]]), np.array([[1.0], [0.0]]), [0])
        assert loss[0] == pytest.approx(np.log1p(np.exp(-x)), rel=1e-14) and lse[0] == pytest.approx(x + loss[0])


def test_oracle_catches_planted_mistakes():
    rng = np.random.default_rng(1)
    h, W, y, w = rng.normal(size=(6, 5)), rng.normal(size=(9, 5)), rng.integers(0, 9, 6), rng.random(6) + 0.5
    loss, lse, dh, dW, G = xent.cross_entropy(h, W, y, 0.7, -100, w)
    _, tol_h, tol_w = xent.bounds(h, W, y, 0.7, G, loss, lse)
    for wrong in (G + 0.01 * np.eye(6, 9), G * 0.7, np.where(G < 0, 0, G)):
        assert np.any(np.abs(wrong @ W - dh) > tol_h) and np.any(np.abs(wrong.T @ h - dW) > tol_w)


# ------------------------------------------------------------------ AdamW oracle
def test_adamw_oracle_matches_torch():
    g = torch.Generator().manual_seed(0)
    p = torch.randn(50, generator=g, dtype=torch.float64, requires_grad=True)
    opt = torch.optim.AdamW([p], lr=1e-2, betas=(0.8, 0.99), eps=1e-6, weight_decay=0.1)
    q, m, v = p.detach().numpy().copy(), np.zeros(50), np.zeros(50)
    for t in range(1, 8):
        p.grad = torch.randn(50, generator=g, dtype=torch.float64)
        q, m, v = adamw.step(q, p.grad.numpy(), m, v, t, 1e-2, 0.8, 0.99, 1e-6, 0.1)
        opt.step()
        assert np.allclose(q, p.detach().numpy(), rtol=1e-12, atol=1e-14)


def test_block_exponents():
    x = np.zeros(256 * 5, np.float32)
    x[256] = 448.0
    x[512] = np.nextafter(np.float32(448), np.float32(1000))
    x[768] = 1e-38
    x[1024] = -3.0
    assert adamw.exponent(x).tolist() == [0, 0, 1, -100, -7]


def test_codes_round_between_their_neighbours_and_on_average_to_the_value():
    rng = np.random.default_rng(0)
    x = (rng.normal(size=4096) * np.exp(rng.normal(size=4096) * 3)).astype(np.float32)
    _, e = adamw.encode(x, np.zeros(4096, np.int64))
    total = np.zeros(4096)
    lo = adamw.decode(adamw.encode(x, np.zeros(4096, np.int64))[0], e)
    hi = adamw.decode(adamw.encode(x, np.full(4096, 65535))[0], e)
    assert np.all(np.abs(lo) <= np.abs(x)) and np.all(np.abs(hi) >= np.abs(lo))
    reps = 512
    for k in range(reps):
        u = (np.arange(4096) * 0 + (k * 65536 + 32768) // reps)
        total += adamw.decode(adamw.encode(x, u)[0], e)
    step = np.abs(hi - lo)
    # evenly spaced u: the mean is off by at most one of the reps, and by 2^-16 of the step
    assert np.all(np.abs(total / reps - x) <= step * (1 / reps + 2.0 ** -15) + 1e-30)


def test_positive_roots_are_never_stored_as_zero():
    x = np.array([0.0, 1e-30, 1.0, 0.0], np.float32)
    codes, e = adamw.encode(x, np.zeros(4, np.int64), root=True)
    assert codes.tolist()[0] == 0 and codes.tolist()[1] == 1 and codes.tolist()[3] == 0
    assert adamw.decode(codes, e)[2] == 1.0


def test_random_streams_of_states_and_parameters_differ():
    a, b = adamw.random_halves(7, 512, 3, 2)
    c = adamw.random_param(7, 512, 3, 2)
    for x, y in ((a, b), (a, c), (b, c), (a, adamw.random_halves(7, 512, 4, 2)[0]), (a, adamw.random_halves(7, 512, 3, 1)[0]),
                 (a, adamw.random_halves(8, 512, 3, 2)[0])):
        assert np.mean(x == y) < 0.02
    w = philox.words(7, np.arange(128), 3, 2, adamw.TAG_STATE)
    assert np.array_equal(a, (w & 0xFFFF).reshape(-1)) and np.array_equal(b, (w >> 16).reshape(-1))
    assert fp8.decode(np.uint8(0x7E)) == 448.0


# ------------------------------------------------------------------ refusals
def test_bindings_refuse_host_tensors(dg):
    h, W, y = torch.zeros(4, 8).bfloat16(), torch.zeros(9, 8).bfloat16(), torch.zeros(4, dtype=torch.int64)
    with pytest.raises(dg.DgError):
        dg.head_cross_entropy(h, W, y)
    with pytest.raises(dg.DgError):
        dg.head_cross_entropy(h[:3], W, y)
    with pytest.raises(dg.DgError):
        dg.head_cross_entropy(h, W[:, :4], y)
    with pytest.raises(dg.DgError):
        dg.XentWorkspace(dg.xent_params(4, 9, 8), device="cpu")
    T = dg.AdamWTensors([torch.zeros(5)], [torch.zeros(5)], [torch.zeros(5)], [torch.zeros(5)])
    with pytest.raises(dg.DgError):
        dg.dg_adamw_step(dg.adamw_params(), T)
    with pytest.raises(KeyError):
        dg.adamw_params(momentum=0.9)
    with pytest.raises(KeyError):
        dg.xent_params(4, 9, 8, smoothing=0.1)
    for bad in (dict(state_bits=4), dict(weight_decay=[0.1, 0.2])):
        with pytest.raises(dg.DgError):
            dg.AdamW([torch.zeros(5)], **bad)
    with pytest.raises(dg.DgError):
        dg.AdamW([torch.zeros(5, dtype=torch.float16)])
    with pytest.raises(dg.DgError):
        dg.adamw_params(step_dev=torch.zeros(1))
    with pytest.raises(dg.DgError):
        dg.HeadTrainer(torch.zeros(5))


def test_lists_refuse_overlaps_and_mixtures(dg):
    def z(n, dtype=torch.float32):
        return torch.zeros(n, dtype=dtype)

    buf = z(100)
    for args, kw in ((([buf[:60], buf[40:]], [z(60)] * 2, [z(60), z(60)], [z(60), z(60)]), {}),
                     (([z(5)], [z(5)], [buf[:5]], [buf[:5]]), {}),
                     (([z(5), z(5, torch.bfloat16)], [z(5)] * 2, [z(5), z(5)], [z(5), z(5)]), {}),
                     (([z(5)], [z(5), z(5)], [z(5)], [z(5)]), {}),
                     (([z(5)], [z(5)], [z(5)], [z(5)]), dict(m_exp=[z(1, torch.int8)])),
                     (([z(5)], [z(5)], [z(5)], [z(5)]), dict(weight_decay=[0.1, 0.1])),
                     (([z(5)], [z(5)], [z(5, torch.uint8)], [z(5, torch.uint8)]), {}),
                     (([z(10)[::2]], [z(5)], [z(5)], [z(5)]), {})):
        with pytest.raises(dg.DgError):
            dg.AdamWTensors(*args, **kw)


def test_c_entry_points_refuse_bad_arguments_without_a_device(dg):
    from discrete_diffusion_decoding_b200._abi import DG_EINVAL, DG_EUNSUPPORTED, lib
    L = lib()
    a = 1 << 20                          # never dereferenced
    p = dg.xent_params(4, 9, 8)
    for field, value, want in (("n", -1, DG_EINVAL), ("vocab", 0, DG_EINVAL), ("hidden", 0, DG_EINVAL),
                               ("temperature", 0.0, DG_EINVAL), ("temperature", float("inf"), DG_EINVAL),
                               ("temperature", 1e-42, DG_EINVAL),
                               ("target_type", 2, DG_EINVAL), ("dw_type", 5, DG_EINVAL), ("dw_accumulate", -1, DG_EINVAL),
                               ("h_stride", 7, DG_EINVAL), ("hidden", 12, DG_EUNSUPPORTED),
                               ("hidden", 65544, DG_EUNSUPPORTED), ("n", (1 << 22) + 1, DG_EUNSUPPORTED),
                               ("vocab", (1 << 28) + 1, DG_EUNSUPPORTED)):
        q = type(p).from_buffer_copy(p)
        setattr(q, field, value)
        assert L.dg_xent_forward(ctypes.byref(q), a, a, a, a, a, a, 1 << 40, None) == want, field
        assert L.dg_xent_backward(ctypes.byref(q), a, a, a, a, a, a, a, a, a, 1 << 40, None) == want, field
        assert L.dg_xent_workspace_size(ctypes.byref(q), 1) == 0
    assert L.dg_xent_forward(None, a, a, a, a, a, a, 1 << 40, None) == DG_EINVAL
    hp = dg.adamw_params()
    one = (dg.AdamWTensors([torch.zeros(5)], [torch.zeros(5)], [torch.zeros(5)], [torch.zeros(5)])).table
    hp.param_type = hp.grad_type = 0
    for field, value in (("lr", -1.0), ("beta1", 1.0), ("beta2", float("nan")), ("eps", -1.0), ("step", 0),
                         ("state_bits", 16), ("param_type", 2), ("grad_type", -1), ("stochastic", 1)):
        q = type(hp).from_buffer_copy(hp)
        setattr(q, field, value)
        assert L.dg_adamw_step(ctypes.byref(q), one, 1, None) == DG_EINVAL, field
    assert L.dg_adamw_step(ctypes.byref(hp), None, 1, None) == DG_EINVAL
    assert L.dg_adamw_step(ctypes.byref(hp), one, -1, None) == DG_EINVAL
    for field, value in (("n", -1), ("n", 1 << 34), ("m", None), ("param", a + 1), ("weight_decay", float("nan")),
                         ("master", a)):
        row = type(one[0]).from_buffer_copy(one[0])
        setattr(row, field, value)
        assert L.dg_adamw_step(ctypes.byref(hp), (type(row) * 1)(row), 1, None) == DG_EINVAL, field


def test_struct_layouts_match_the_header(dg, tmp_path):
    from discrete_diffusion_decoding_b200 import _abi
    cc = shutil.which("gcc")
    if cc is None:
        pytest.skip("no host compiler")
    names = {"dg_xent_params": _abi.DgXentParams, "dg_adamw_params": _abi.DgAdamWParams,
             "dg_adamw_tensor": _abi.DgAdamWTensor}
    body = "".join(f'printf("{n} %zu\\n", sizeof({n}));' + "".join(
        f'printf("{n}.{f} %zu\\n", offsetof({n}, {f}));' for f, _ in s._fields_) for n, s in names.items())
    src = tmp_path / "layout.c"
    src.write_text(f'#include <stdio.h>\n#include "{ROOT}/include/dg.h"\nint main(void) {{ {body} return 0; }}\n')
    subprocess.run([cc, "-o", str(tmp_path / "layout"), str(src)], check=True, timeout=60)
    out = subprocess.run([str(tmp_path / "layout")], capture_output=True, text=True, check=True, timeout=60).stdout
    got = dict(line.split() for line in out.splitlines())
    for n, s in names.items():
        assert int(got[n]) == ctypes.sizeof(s)
        for f, _ in s._fields_:
            assert int(got[f"{n}.{f}"]) == getattr(s, f).offset, f"{n}.{f}"


def test_the_products_and_the_update_keep_to_registers(tmp_path):
    """ptxas reports no spills in the kernels that stream the head (accumulators are held in registers there)."""
    import re
    nvcc = next((c for c in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc"))
                 if c and os.path.exists(c)), None)
    if nvcc is None:
        pytest.skip("nvcc not available")
    src = os.path.join(ROOT, "discrete_diffusion_decoding_b200", "csrc", "dg_xent.cu")
    out = subprocess.run([nvcc, "-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-std=c++17", "-Xptxas", "-v", "-c",
                          "-o", str(tmp_path / "k.o"), src], capture_output=True, text=True, timeout=600)
    assert out.returncode == 0, out.stderr[-2000:]
    spills = [tuple(map(int, m)) for m in re.findall(r"(\d+) bytes spill stores, (\d+) bytes spill loads", out.stderr)]
    assert len(spills) >= 6 and all(s == (0, 0) for s in spills), spills
