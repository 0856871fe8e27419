"""The training entry points on the GPU where they could go wrong at the edges of what they document: rounding of
the gradients' largest entries, logits that are not finite, values below the normal range, steps and streams."""

import gc
import time
import weakref

import numpy as np
import pytest
import torch

from oracle import adamw, xent
from test_gpu_adamw import check_roots
from test_gpu_xent import IGNORE, check, inputs, run

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
    """The target's entry of G reaches dh and dW with more than bf16's digits."""
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
    # that leaves out may be rounded once more: 2^-8 of 2^-8
    each = 3 * dz + 2.0 ** -20
    aw, ah = np.abs(W64), np.where((y != IGNORE).numpy()[:, None], np.abs(h64), 0)
    tol_h = (each + 2.0 ** -16 + (V / 16 + 64) * 2.0 ** -23) * (np.abs(G) @ aw) + 2.0 ** -8 * (rest @ aw)
    tol_w = (each + 2.0 ** -16 + (n / 16 + 4) * 2.0 ** -23) * (np.abs(G).T @ ah) + 2.0 ** -8 * (rest.T @ ah)
    tol_h = tol_h * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(dh)
    tol_w = tol_w + 2.0 ** -24 * np.abs(dW)
    assert np.all(np.abs(got[2] - dh) <= tol_h) and np.all(np.abs(got[3] - dW) <= tol_w)
    # the same with the entry rounded is outside
    B = torch.from_numpy(G).bfloat16().double().numpy()
    assert np.any(np.abs(torch.from_numpy(B @ W64).bfloat16().double().numpy() - dh) > tol_h)
    assert np.any(np.abs(B.T @ h64 - dW) > tol_w)


@pytest.mark.parametrize("n,V,d,dtype", [(300, 40, 64, torch.float32), (3000, 700, 72, torch.bfloat16),
                                         (2500, 5, 2104, torch.float32), (9000, 300, 8, torch.bfloat16),
                                         (20, 6, 2104, torch.bfloat16), (10000, 30, 520, torch.float32)])
@pytest.mark.parametrize("add", [0, 1])
def test_many_positions_of_one_target(dg, n, V, d, dtype, add):
    """Half of the positions have one target, more than the last launch holds of one at a time; equal calls give equal
    bits, and rows that are added to keep what was there."""
    h, W, y, dl = inputs(n, V, d, seed=n, ignored=0.1)
    y[(torch.arange(n) % 2 == 0) & (y != IGNORE)] = 3
    base = torch.randn(V, d, generator=torch.Generator().manual_seed(1)).to(dtype)
    got = run(dg, h, W, y, dl, dw=base.cuda(), dw_accumulate=add)
    h64, W64, dn = h.double().numpy(), W.double().numpy(), np.where(y == IGNORE, 0.0, dl.double().numpy())
    loss, lse, dh, dW, G = xent.cross_entropy(h64, W64, y.numpy(), 1.0, IGNORE, dn)
    _, tol_h, tol_w = xent.bounds(h64, W64, y.numpy(), 1.0, G, loss, lse)
    want, eps = dW + add * base.double().numpy(), torch.finfo(dtype).eps / 2
    assert np.all(np.abs(got[3] - want) <= tol_w * (1 + eps) + (eps + 2.0 ** -24) * np.abs(want) + 1e-38)
    assert np.all(np.abs(got[2] - dh) <= tol_h * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(dh) + 1e-38)
    again = run(dg, h, W, y, dl, dw=base.cuda(), dw_accumulate=add)
    assert all(np.array_equal(a, b) for a, b in zip(got, again))


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


# ------------------------------------------------------------------ values below the normal range
@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("eps", [0.0, 1e-8])
def test_roots_of_subnormal_second_moments(dg, bits, eps):
    """Gradients of 1e-19: v is positive but below the normal range.  Its root is normal, and is what the step
    divides by and what an 8-bit state holds."""
    n = 512
    g = torch.linspace(1.5e-19, 1e-18, n)
    g[300:] = 1e-3
    g[0] = 0
    p = torch.zeros(n)
    p[0] = 1.0
    dev = {k: torch.zeros(n, dtype=torch.uint8 if bits == 8 else torch.float32, device="cuda") for k in "mv"}
    ex = {k: torch.zeros(2, dtype=torch.int8, device="cuda") for k in "mv"}
    pd = p.cuda()
    # element 0 has no moments: with eps 0 the definition divides 0 by 0
    T = dg.AdamWTensors([pd], [g.cuda()], [dev["m"]], [dev["v"]], m_exp=[ex["m"]] if bits == 8 else None,
                        v_exp=[ex["v"]] if bits == 8 else None)
    dg.dg_adamw_step(dg.adamw_params(lr=1e-2, beta1=0.9, beta2=0.99, eps=eps, step=1, seed=4), T)
    m, v = adamw.moments(g.numpy(), np.zeros(n), np.zeros(n), 0.9, 0.99)
    assert 0 < v[1] < 2.0 ** -126 and v[299] < 2.0 ** -126 < v[300]
    with np.errstate(invalid="ignore"):
        want = -1e-2 * (m.astype(np.float64) / (1 - 0.9)) / (np.sqrt(v.astype(np.float64) / (1 - 0.99)) + eps)
    got = pd.cpu().double().numpy()
    assert np.isnan(got[0]) if eps == 0 else got[0] == 1
    # root 3 u, its product and the sum 3 u, the rate and the numerator 3 u, the quotient 4 u, the sum u
    assert np.all(np.abs(got - want)[1:] <= 16 * 2.0 ** -24 * np.abs(want[1:]))
    if bits == 32:
        assert np.array_equal(dev["m"].cpu().numpy(), m) and np.array_equal(dev["v"].cpu().numpy(), v)
        return
    um, uv = adamw.random_halves(4, n, 1, 0)
    cm, em = adamw.encode(m, um)
    assert np.array_equal(dev["m"].cpu().numpy(), cm) and np.array_equal(ex["m"].cpu().numpy(), em)
    check_roots(dev["v"], ex["v"], v, uv)
    root = adamw.decode(dev["v"].cpu().numpy(), ex["v"].cpu().numpy())
    assert np.all(np.abs(root[1:256] / np.sqrt(v[1:256].astype(np.float64)) - 1) <= 0.125)


# ------------------------------------------------------------------ the trainer's weights
@pytest.mark.parametrize("junk", [float("inf"), float("nan"), -float("inf")])
def test_weights_of_ignored_positions_may_hold_anything(dg, junk):
    V, d, n = 300, 64, 50
    h, W, y, w = inputs(n, V, d, seed=1, ignored=0.4)
    bad = torch.where(y == IGNORE, torch.tensor(junk), w)
    out = []
    for weight in (torch.where(y == IGNORE, 0.0, w), bad):
        tr = dg.HeadTrainer(W.cuda().clone())
        loss, dh = tr.accumulate(h.cuda(), y.cuda(), weight.cuda())
        out.append((loss, dh, tr.dW))
    for a, b in zip(*out):
        assert torch.isfinite(b).all() and torch.equal(a, b)


def test_weights_of_either_sign(dg):
    """The loss is sum w loss / sum w also where the weights' sum is negative; without any weight it is 0."""
    V, d, n = 300, 64, 50
    h, W, y, w = inputs(n, V, d, seed=2, ignored=0.2)
    out = []
    for weight in (w, -w, w * 0):
        tr = dg.HeadTrainer(W.cuda().clone())
        loss, dh = tr.accumulate(h.cuda(), y.cuda(), weight.cuda())
        out.append((loss, dh, tr.dW))
    for a, b, c in zip(*out):
        assert torch.equal(a, b) and (c == 0).all()


# ------------------------------------------------------------------ autograd and the optimizer
@pytest.mark.parametrize("update", ["AdamW", "HeadTrainer", "dg_adamw_step"])
def test_a_backward_after_the_weights_changed_is_refused(dg, update):
    W = torch.randn(100, 64, device="cuda").bfloat16().requires_grad_()
    h = torch.randn(5, 64, device="cuda").bfloat16().requires_grad_()
    y = torch.arange(5, device="cuda")
    loss = dg.head_cross_entropy(h, W, y).sum()
    if update == "AdamW":
        dg.AdamW([W]).step([torch.ones_like(W)])
    elif update == "HeadTrainer":
        dg.HeadTrainer(W).step(h.detach(), y)
    else:
        m, v = torch.zeros(100, 64, device="cuda"), torch.zeros(100, 64, device="cuda")
        dg.dg_adamw_step(dg.adamw_params(), dg.AdamWTensors([W], [torch.ones_like(W)], [m], [v]))
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_tensors_that_the_entry_points_write_count_it(dg):
    h, W, y, dl = (x.cuda() for x in inputs(20, 300, 64))
    p = dg.xent_params(20, 300, 64)
    ws = dg.XentWorkspace(p)
    loss, lse = torch.zeros(20, device="cuda"), torch.zeros(20, device="cuda")
    dh, dW = torch.zeros_like(h), torch.zeros_like(W)
    seen = [x._version for x in (loss, lse, dh, dW)]
    dg.dg_xent_forward(p, h, W, y, loss, lse, ws)
    dg.dg_xent_backward(p, h, W, y, loss, lse, dl, dh, dW, ws)
    assert all(x._version > v for x, v in zip((loss, lse, dh, dW), seen))
    assert h._version == 0 and W._version == 0
    # a parameter without a gradient is not written
    q = [torch.zeros(5, device="cuda"), torch.zeros(5, device="cuda")]
    dg.AdamW(q, state_bits=32).step([torch.ones(5, device="cuda"), None])
    assert q[0]._version == 1 and q[1]._version == 0
    with torch.inference_mode():
        r = torch.zeros(5, device="cuda")
    dg.AdamW([r], state_bits=32).step([torch.ones(5, device="cuda")])
    assert (r < 0).all()


def test_zero_grad_frees_the_gradients(dg):
    p = torch.nn.Parameter(torch.zeros(1000, device="cuda"))
    opt = dg.AdamW([p])
    p.grad = torch.ones(1000, device="cuda")
    held = weakref.ref(p.grad)
    opt.step()
    opt.zero_grad()
    gc.collect()
    assert held() is None
    with pytest.raises(dg.DgError, match="gradients"):
        dg.dg_adamw_step(dg.adamw_params(), opt.groups[0][1])


def test_gradients_outlive_a_step_on_another_stream(dg):
    """Gradients dropped after a step that still waits on its stream are not handed out again before it ran."""
    n = 1 << 20
    p = torch.zeros(n, device="cuda")
    opt, side = dg.AdamW([p], lr=1.0, eps=0.0, state_bits=32), torch.cuda.Stream()
    g = torch.ones(n, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)        # 0.1 s
    opt.step([g], stream=side)
    del g
    opt.zero_grad()
    other = [torch.full((n,), -1.0, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    # one step of a gradient of 1: m / (1 - b1) over the root of v / (1 - b2), each within 2^-20
    assert ((p + 1).abs() <= 2.0 ** -19).all() and len(other) == 4


def test_a_first_gradient_that_comes_late_counts_from_one(dg):
    """Bias corrections, random bits and states of each parameter follow its own steps, also through a state_dict."""
    for bits, dtype in ((32, torch.float32), (8, torch.float32), (8, torch.bfloat16)):
        g = torch.Generator().manual_seed(bits)
        base = [torch.randn(n, generator=g).to(dtype) for n in (700, 300, 40)]
        grads = [[torch.randn(x.shape, generator=g).to(dtype).cuda() for x in base] for _ in range(6)]
        ps = [x.cuda() for x in base]
        opt = dg.AdamW(ps, lr=1e-2, betas=(0.9, 0.99), state_bits=bits, seed=9)
        for t in range(6):
            if t == 3:
                state, ps = opt.state_dict(), [x.clone() for x in ps]
                opt = dg.AdamW(ps, lr=1e-2, betas=(0.9, 0.99), state_bits=bits, seed=9)
                opt.load_state_dict(state)
            opt.step([grads[t][0], grads[t][1] if t >= 2 else None, grads[t][2] if t % 2 else None])
        assert opt.steps == 6
        # each alone, at its place in the list, stepped only when it has a gradient
        for i, when in enumerate((range(6), range(2, 6), (1, 3, 5))):
            x = [b.cuda() for b in base]
            kind = torch.uint8 if bits == 8 else torch.float32
            s = [[torch.zeros(b.shape, dtype=kind, device="cuda") for b in base] for _ in range(2)]
            e = [[torch.zeros(-(-b.numel() // 256), dtype=torch.int8, device="cuda") for b in base] for _ in range(2)]
            T = dg.AdamWTensors(x, [None] * 3, *s, m_exp=e[0] if bits == 8 else None, v_exp=e[1] if bits == 8 else None)
            for k, t in enumerate(when):
                T.set_grads([grads[t][j] if j == i else None for j in range(3)])
                dg.dg_adamw_step(dg.adamw_params(lr=1e-2, beta1=0.9, beta2=0.99, step=k + 1, seed=9,
                                                 stochastic=int(dtype == torch.bfloat16)), T)
            assert torch.equal(x[i], ps[i])


def test_many_batches_are_accumulated_without_losing_any(dg):
    """64 batches at the default type: the sum of their gradients, where a bf16 sum would drop what is below half a
    step of it."""
    V, d, n, k = 300, 64, 40, 64
    h, W, y, w = inputs(n, V, d, seed=3)
    tr = dg.HeadTrainer(W.cuda())
    one = dg.HeadTrainer(W.cuda().clone(), grad_dtype=torch.float32)
    hd, yd, wd = h.cuda(), y.cuda(), w.cuda()
    one.accumulate(hd, yd, wd)
    for _ in range(2):                        # the first steps to accumulate, and the ones after it
        for _ in range(k):
            tr.accumulate(hd, yd, wd)
        want = k * one.dW.double()
        # each of the k - 1 fp32 sums is off by 2^-24 of itself, the first batch by bf16's half step
        assert ((tr.dW.double() - want).abs() <= (k * 2.0 ** -24 + 2.0 ** -8 / k) * want.abs() + 1e-38).all()
        tr.batches = 0
    tr.batches = k
    before = tr.W.clone()
    tr.update()
    assert tr.optimizer.steps == 1 and not torch.equal(tr.W, before)


# ------------------------------------------------------------------ overlaps, captures, streams
def test_no_positions_do_not_clear_the_head(dg):
    """dW on top of W is refused whatever the number of positions."""
    W = torch.randn(300, 64).bfloat16().cuda()
    before = W.clone()
    h = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    y, f = torch.empty(0, dtype=torch.int32, device="cuda"), torch.empty(0, device="cuda")
    p = dg.xent_params(0, 300, 64)
    with pytest.raises(dg.DgError):
        dg.dg_xent_backward(p, h, W, y, f, f, f, None, W, dg.XentWorkspace(p))
    assert torch.equal(W, before)


def test_a_step_on_a_stream_under_capture_is_refused(dg):
    """Also where that stream is not the current one."""
    W = torch.ones(64, 8, dtype=torch.bfloat16, device="cuda")
    opt, x, g = dg.AdamW([W]), torch.zeros(4, device="cuda"), torch.cuda.CUDAGraph()
    grad, side, other = torch.ones_like(W), torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=side):
        x.add_(1)
        with torch.cuda.stream(other):
            with pytest.raises(dg.DgError, match="captured"):
                opt.step([grad], stream=side)
    assert opt.steps == 0


def test_a_trainer_moved_between_streams_keeps_its_workspace(dg):
    """A larger batch on another stream renews the workspace: the old one is not handed out while it is in use."""
    V, d = 20000, 512
    h, W, y, w = inputs(300, V, d, seed=5)
    hd, yd = h.cuda(), y.cuda()
    want = dg.HeadTrainer(W.cuda()).accumulate(hd[:20], yd[:20])[1]
    tr = dg.HeadTrainer(W.cuda())
    tr.accumulate(hd[:20], yd[:20])
    size, main, side = tr._ws.nbytes, torch.cuda.current_stream(), torch.cuda.Stream()
    side.wait_stream(main)
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)
        tr.batches = 0
        got = tr.accumulate(hd[:20], yd[:20])[1]
        tr.accumulate(hd, yd)
    junk = torch.zeros(size, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    assert torch.equal(got, want) and (junk == 0).all()

# ------------------------------------------------------------------ waits that run out, and the largest hidden size
@pytest.mark.parametrize("n", [3, 40])
def test_waits_that_run_out(dg, n):
    """With a limit that the long sums of the largest hidden size exceed, the kernels leave on their own and at once:
    NaN in loss, lse and both gradients, 0 at ignored positions.  The next calls with the same workspace are right."""
    V, d = 700, 65536
    g = torch.Generator().manual_seed(n)
    W = (torch.randn(V, d, generator=g) / 64).bfloat16()
    h = (torch.randn(n, d, generator=g) / 4).bfloat16()
    y, dl = torch.randint(0, V, (n,), generator=g).int(), torch.rand(n, generator=g) + 0.5
    y[1] = IGNORE
    p = dg.xent_params(n, V, d)
    ws = dg.XentWorkspace(p)
    want = run(dg, h, W, y, dl, ws=ws)
    check(h, W, y, dl, 1.0, want)
    hd, Wd, yd, dld = h.cuda(), W.cuda(), y.cuda(), dl.cuda()
    loss, lse = (torch.from_numpy(x).float().cuda() for x in want[:2])
    bad, bad_lse, dh, dW = (torch.zeros_like(x) for x in (loss, lse, hd, Wd))
    torch.cuda.synchronize()
    start = time.time()
    try:
        dg.dg_debug_set_counter_wait_limit(1)          # 1 ns: a wait not satisfied at once runs out
        dg.dg_xent_forward(p, hd, Wd, yd, bad, bad_lse, ws)
        dg.dg_xent_backward(p, hd, Wd, yd, loss, lse, dld, dh, dW, ws)
        torch.cuda.synchronize()
    finally:
        dg.dg_debug_set_counter_wait_limit(0)
    # well under the 2 s limit of a drain: every drain ended on the loads and products in flight
    assert time.time() - start < 1.0
    kept = yd != IGNORE
    assert torch.isnan(bad[kept]).all() and torch.isnan(bad_lse[kept]).all() and bad[1] == 0 and bad_lse[1] == 0
    assert torch.isnan(dh[kept]).all() and torch.isnan(dW).all() and (dh[1] == 0).all()
    for a, b in zip(run(dg, h, W, y, dl, ws=ws), want):
        assert np.array_equal(a, b)


# ------------------------------------------------------------------ the limits that the header states
@pytest.mark.parametrize("n,V,d,scratch", [
    (63, 5000, 64, 0), (64, 5000, 64, 0), (65, 5000, 64, 0),       # around one stage of positions
    (255, 3000, 72, 0), (256, 2999, 72, 0), (257, 3001, 72, 0),    # around one tile
    (40, 768, 16, 0), (40, 769, 16, 0), (40, 40000, 16, 0),        # dh in one part, in two, in 70
    (256, 147 * 256, 8, 0), (256, 148 * 256, 8, 0), (256, 149 * 256 + 1, 8, 0),   # one tile an item, two
    (300, 74 * 256, 264, 0), (300, 75 * 256, 520, 0),
    (300, 5000, 264, 2 * 2 * 512 * 256), (300, 5000, 264, 2 * 2 * 512 * 256 * 10 - 1),    # pieces of one tile, of nine
])
def test_around_the_limits_of_tiles_items_and_pieces(dg, n, V, d, scratch):
    h, W, y, dl = inputs(n, V, d, seed=n + V)
    check(h, W, y, dl, 1.0, run(dg, h, W, y, dl, scratch_bytes=scratch))


def test_the_most_positions(dg):
    """2^22 positions, against float64 on the device, some thousands at a time."""
    n, V, d = 1 << 22, 300, 8
    g = torch.Generator(device="cuda").manual_seed(0)
    W = (torch.randn(V, d, device="cuda", generator=g) * 0.5).bfloat16()
    h = torch.randn(n, d, device="cuda", generator=g).bfloat16()
    y = torch.randint(0, V, (n,), device="cuda", generator=g).int()
    y[torch.rand(n, device="cuda", generator=g) < 0.2] = IGNORE
    dl = torch.rand(n, device="cuda", generator=g) + 0.5
    p = dg.xent_params(n, V, d)
    ws = dg.XentWorkspace(p)
    loss, lse = torch.full((n,), 7.0, device="cuda"), torch.full((n,), 7.0, device="cuda")
    dg.dg_xent_forward(p, h, W, y, loss, lse, ws)
    dh, dW = torch.full_like(h, 7.0), torch.full((V, d), 7.0, device="cuda")
    dg.dg_xent_backward(p, h, W, y, loss, lse, dl, dh, dW, ws)
    W64 = W.double()
    sums, sizes = torch.zeros_like(W64), torch.zeros_like(W64)
    # 8 products and fp32 factors: every logit is within 2^-19 of its magnitude (8 x 0.5 x 4 x 4 at most 64) and lse
    # near 6 within 2^-21 of it
    dz = 2.0 ** -13
    step = 1 << 18
    for a in range(0, n, step):
        at = slice(a, a + step)
        kept = y[at] != IGNORE
        yy = torch.where(kept, y[at], 0).long()
        h64 = torch.where(kept[:, None], h[at].double(), 0)
        z = h64 @ W64.T
        want_lse = torch.logsumexp(z, 1)
        want = want_lse - z.gather(1, yy[:, None])[:, 0]
        assert ((loss[at] - torch.where(kept, want, 0)).abs() <= 2 * dz * kept).all()
        assert ((lse[at] - torch.where(kept, want_lse, 0)).abs() <= 2 * dz * kept).all()
        G = torch.exp(z - want_lse[:, None])
        G[torch.arange(len(yy), device="cuda"), yy] -= 1
        G *= torch.where(kept, dl[at].double(), 0)[:, None]
        off, tol = (dh[at] - G @ W64).abs(), (2.0 ** -8 + 3 * dz) * (G.abs() @ W64.abs())
        assert (off <= tol + 2.0 ** -8 * (G @ W64).abs() + 1e-38).all()
        sums += G.T @ h64
        sizes += G.abs().T @ h64.abs()
    assert ((dW - sums).abs() <= (2.0 ** -8 + 3 * dz + (n / 16) * 2.0 ** -23) * sizes).all()


@pytest.mark.parametrize("n", [3, 40])
def test_the_largest_vocabulary(dg, n):
    """2^28 rows, against float64 on the device, a part of the vocabulary at a time; targets at both ends."""
    V, d = 1 << 28, 8
    g = torch.Generator(device="cuda").manual_seed(n)
    W = torch.empty(V, d, dtype=torch.bfloat16, device="cuda").normal_(0.0, 0.25, generator=g)
    y = torch.randint(0, V, (n,), device="cuda", generator=g).int()
    y[0], y[1], y[2] = V - 1, 0, (1 << 27) + 1
    # half of the probability at the target of two positions, far less at the others
    h = torch.randn(n, d, device="cuda", generator=g)
    h[:2] = W[y[:2].long()].float() * (20 / (W[y[:2].long()].float() ** 2).sum(1, keepdim=True))
    h, dl = h.bfloat16(), torch.rand(n, device="cuda", generator=g) + 0.5
    p = dg.xent_params(n, V, d)
    ws = dg.XentWorkspace(p)
    loss, lse = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    dg.dg_xent_forward(p, h, W, y, loss, lse, ws)
    dh, dW = torch.empty_like(h), torch.empty_like(W)
    dg.dg_xent_backward(p, h, W, y, loss, lse, dl, dh, dW, ws)
    h64, step = h.double(), 1 << 22
    total = torch.full((n,), -float("inf"), dtype=torch.float64, device="cuda")
    most = 0.0
    for a in range(0, V, step):
        W64 = W[a:a + step].double()
        total = torch.logaddexp(total, torch.logsumexp(h64 @ W64.T, 1))
        most = max(most, float((h64.abs() @ W64.abs().T).max()))
    zt = (h64 * W[y.long()].double()).sum(1)
    # a logit is a few sums of fp32; the sum over the vocabulary has at most 2^14 + 2^11 steps in one thread, each
    # rounded twice where two sums are joined
    dz = 2.0 ** -19 * most
    sums = (2 ** 14 + 2 ** 11) * 2.0 ** -23
    assert ((lse - total).abs() <= dz + sums).all() and ((loss - (total - zt)).abs() <= 2 * dz + sums).all()
    want_h, size_h = torch.zeros_like(h64), torch.zeros_like(h64)
    rel = 2.0 ** -8 + 3 * dz + sums
    for a in range(0, V, step):
        W64 = W[a:a + step].double()
        G = torch.exp(h64 @ W64.T - total[:, None])
        for i in range(n):
            if a <= int(y[i]) < a + step:
                G[i, int(y[i]) - a] -= 1
        G *= dl.double()[:, None]
        want_h += G @ W64
        size_h += G.abs() @ W64.abs()
        want, size = G.T @ h64, G.abs().T @ h64.abs()
        assert ((dW[a:a + step] - want).abs() <= rel * (1 + 2.0 ** -8) * size + 2.0 ** -8 * want.abs() + 1e-38).all()
    # dh: 74 parts of a piece of 409600 columns, 656 pieces: 346 sums of 16 products, 656 and 74 sums of those
    assert ((dh - want_h).abs() <= (rel + 1100 * 2.0 ** -23) * size_h + 2.0 ** -8 * want_h.abs()).all()


# ------------------------------------------------------------------ truncated sums
@pytest.mark.parametrize("n", [1, 17, 32])
def test_long_sums_of_few_positions_are_cut_into_parts(dg, n):
    """Products of one sign, whose running sum the tensor core cuts off at every 16: with the sum in eight parts the
    logits are off by an eighth of that."""
    V, d = 1000, 4096
    g = torch.Generator().manual_seed(n)
    W = ((0.5 + torch.rand(V, d, generator=g)) / 128).bfloat16()
    h = (0.5 + torch.rand(n, d, generator=g)).bfloat16()
    y = torch.randint(0, V, (n,), generator=g).int()
    p = dg.xent_params(n, V, d)
    loss, lse = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    dg.dg_xent_forward(p, h.cuda(), W.cuda(), y.cuda(), loss, lse, dg.XentWorkspace(p, backward=False))
    want, want_lse = xent.cross_entropy(h.double().numpy(), W.double().numpy(), y.numpy())
    z = (h.double() @ W.double().T).max()
    # a part has 32 steps of 16 products and loses at most 2^-23 of its running sum at each, half of its sum on
    # average as all products have one sign; the parts' sum has 8 roundings.  The exponentials and their sum in log2
    # units: 2^-20; lse's own rounding
    tol = float((32 / 2 + 8) * 2.0 ** -23 * z + 2.0 ** -20 + 2.0 ** -23 * want_lse.max())
    assert np.all(np.abs(lse.cpu().double().numpy() - want_lse) <= tol)
    assert np.all(np.abs(loss.cpu().double().numpy() - want) <= 2 * tol)


@pytest.mark.parametrize("n", [17, 40])
def test_gradients_use_the_losses_own_logits(dg, n):
    """The largest hidden size with products of one sign: what is cut off the logits is the same in both directions, so
    that the backward's softmax adds up to 1 and the common part of W's rows cancels."""
    V, d = 700, 65536
    g = torch.Generator().manual_seed(n)
    W = ((0.5 + torch.rand(V, d, generator=g)) / 2048).bfloat16()
    h = (0.5 + torch.rand(n, d, generator=g)).bfloat16()
    y, dl = torch.randint(0, V, (n,), generator=g).int(), torch.rand(n, generator=g) + 0.5
    got = run(dg, h, W, y, dl)
    W64 = W.double().numpy()
    *_, dh, _, G = xent.cross_entropy(h.double().numpy(), W64, y.numpy(), 1.0, IGNORE, dl.double().numpy())
    T = np.zeros_like(G)
    T[np.arange(n), y] = np.abs(G)[np.arange(n), y]
    # the logits lie within 1 % of 32 and lose at most 4096 / 2 x 2^-23 of that, 7.8e-3, nearly the same in each: the
    # difference and the rest of the fp32 errors are within 2^-12.  The other entries are rounded to bf16, and dh is
    tol = 2.0 ** -12 * (np.abs(G) @ W64) + 2.0 ** -8 * ((np.abs(G) - T) @ W64) + 2.0 ** -8 * np.abs(dh)
    assert np.all(np.abs(got[2] - dh) <= tol * (1 + 2.0 ** -8))
