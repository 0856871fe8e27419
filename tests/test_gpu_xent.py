"""The head's cross entropy and its gradients on the GPU against the float64 oracle, over sizes, masks, strides,
types and ways of calling.  Tolerances are the elementwise bounds of oracle.xent.bounds, and half a bf16 step
for outputs in bf16."""

import numpy as np
import pytest
import torch

from oracle import xent

pytestmark = pytest.mark.gpu
IGNORE = -100


@pytest.fixture(scope="module")
def dg():
    from discrete_diffusion_decoding_b200 import build
    build.build()
    import discrete_diffusion_decoding_b200 as m
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return m


def inputs(n, V, d, seed=0, ignored=0.0, index=torch.int32, lean=8.0):
    g = torch.Generator().manual_seed(seed)
    W = (torch.randn(V, d, generator=g) * 0.05).bfloat16()
    y = torch.randint(0, V, (n,), generator=g)
    h = (torch.randn(n, d, generator=g) + lean * torch.rand(n, 1, generator=g) / (0.0025 * d) * W[y].float()).bfloat16()
    drop = torch.randperm(n, generator=g)[:int(n * ignored)]
    y[drop] = IGNORE
    dl = torch.rand(n, generator=g) + 0.5
    return h, W, y.to(index), dl


def run(dg, h, W, y, dl, T=1.0, want=("dh", "dW"), dw=None, ws=None, **params):
    """Forward and backward on the device; host float64 results."""
    n, d = h.shape
    p = dg.xent_params(n, W.shape[0], d, temperature=T, **params)
    ws = ws or dg.XentWorkspace(p)
    hd, Wd, yd, dld = h.cuda() if not h.is_cuda else h, W.cuda(), y.cuda(), dl.cuda()
    loss = torch.full((n,), 7.0, device="cuda")
    lse = torch.full((n,), 7.0, device="cuda")
    dg.dg_xent_forward(p, hd, Wd, yd, loss, lse, ws)
    dh = torch.full((n, d), 7.0, dtype=torch.bfloat16, device="cuda") if "dh" in want else None
    if dw is None:
        dw = torch.full(W.shape, 7.0, dtype=torch.bfloat16, device="cuda") if "dW" in want else None
    dg.dg_xent_backward(p, hd, Wd, yd, loss, lse, dld, dh, dw, ws)
    torch.cuda.synchronize()
    return tuple(None if x is None else x.cpu().double().numpy() for x in (loss, lse, dh, dw))


def near(name, got, want, tol):
    off = np.abs(got - want)
    assert np.all(off <= tol), f"{name}: off by {off.max():.3g}, at most {np.max(off / np.maximum(tol, 1e-300)):.3g} of the bound"


def check(h, W, y, dl, T, got, dw_eps=2.0 ** -8):
    h64, W64 = h.double().numpy(), W.double().numpy()
    yn, dn = y.numpy(), dl.double().numpy()
    loss, lse, dh, dW, G = xent.cross_entropy(h64, W64, yn, T, IGNORE, dn)
    dz, tol_h, tol_w = xent.bounds(h64, W64, yn, T, G, loss, lse)
    # both logits of the gap move by dz, and the loss by (1 - e^-loss) <= min(1, loss) of that
    near("loss", got[0], loss, 2.0 * dz * np.minimum(1.0, loss) * (1 + 4 * dz) + 2.0 ** -20 * loss + 1e-30)
    near("lse", got[1], lse, 2 * dz + 2.0 ** -22 * np.abs(lse))
    if got[2] is not None:
        near("dh", got[2], dh, tol_h * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(dh) + 1e-38)
    if got[3] is not None:
        near("dW", got[3], dW, tol_w * (1 + dw_eps) + dw_eps * np.abs(dW) + 1e-38)
    return loss, lse, dh, dW


@pytest.mark.parametrize("n,V,d,ignored,T,index", [
    (1, 1, 8, 0.0, 1.0, torch.int32),
    (1, 7, 8, 0.0, 0.5, torch.int64),
    (3, 256, 64, 0.0, 1.0, torch.int32),
    (16, 40000, 72, 0.3, 1.0, torch.int64),
    (17, 129, 1000, 0.0, 0.7, torch.int32),
    (32, 38000, 64, 0.1, 1.0, torch.int32),
    (33, 20011, 64, 0.0, 1.0, torch.int32),
    (5, 300, 72, 0.4, 1.0, torch.int64),
    (128, 257, 128, 0.0, 0.8, torch.int32),
    (129, 511, 136, 0.5, 1.0, torch.int32),
    (256, 1024, 256, 0.0, 1.0, torch.int32),
    (257, 1000, 264, 0.01, 0.4, torch.int64),
    (300, 4096, 128, 0.9, 1.0, torch.int32),
    (700, 2049, 520, 0.3, 1.0, torch.int32),
])
def test_loss_and_gradients(dg, n, V, d, ignored, T, index):
    h, W, y, dl = inputs(n, V, d, seed=n + V, ignored=ignored, index=index)
    check(h, W, y, dl, T, run(dg, h, W, y, dl, T))


@pytest.mark.parametrize("n,V,d,scratch,pieces", [
    (40, 40000, 64, 0, 1),
    (40, 4000, 64, 1, 16),                      # a tile of columns at a time
    (300, 5000, 136, 2 * 2 * 512 * 1024, 5),
    (1030, 18001, 96, 2 * 2 * 1280 * 7000, 3),
    (257, 1281, 72, 2 * 512 * 1280, 3),         # one column more than fits at once
    (257, 1280, 72, 2 * 512 * 1280, 1),
])
def test_pieces_of_the_vocabulary(dg, n, V, d, scratch, pieces):
    h, W, y, dl = inputs(n, V, d, seed=3, ignored=0.2)
    got = run(dg, h, W, y, dl, scratch_bytes=scratch)
    assert dg.last_launch_count() == 3 + pieces
    check(h, W, y, dl, 1.0, got)


@pytest.mark.parametrize("n,V,d,ignored,scratch", [
    (7, 80000, 72, 0.0, 0), (1, 76000, 8, 0.0, 0), (65, 20100, 1000, 0.2, 0), (256, 30001, 520, 0.0, 0),
    (257, 30001, 520, 0.0, 0), (128, 40000, 264, 0.0, 2 * 2 * 256 * 9000), (200, 20001, 776, 1.0, 0),
])
def test_few_positions_and_a_large_head(dg, n, V, d, ignored, scratch):
    """dW by the kernel that keeps the positions' hidden states, just under and over its limits; both types,
    stored and added."""
    h, W, y, dl = inputs(n, V, d, seed=n, ignored=ignored)
    got = run(dg, h, W, y, dl, scratch_bytes=scratch)
    if ignored < 1:
        check(h, W, y, dl, 1.0, got)
    assert ignored < 1 or all((x == 0).all() for x in got)
    full = run(dg, h, W, y, dl, dw=torch.full(W.shape, 7.0, device="cuda"), scratch_bytes=scratch)[3]
    assert np.array_equal(torch.from_numpy(full).float().bfloat16().double().numpy(), got[3])
    added = run(dg, h, W, y, dl, dw=torch.ones(W.shape, device="cuda"), scratch_bytes=scratch, dw_accumulate=1)[3]
    assert np.array_equal(added, (torch.from_numpy(full).float() + 1).double().numpy())
    half = run(dg, h, W, y, dl, dw=torch.ones(W.shape, dtype=torch.bfloat16, device="cuda"), scratch_bytes=scratch,
               dw_accumulate=1)[3]
    assert np.array_equal(half, (torch.from_numpy(full).float() + 1).bfloat16().double().numpy())


@pytest.mark.parametrize("n", [16384, 16385, 70001])
def test_many_positions(dg, n):
    """Past the sizes from which a CTA of the gather looks at more rows than 8."""
    h, W, y, dl = inputs(n, 300, 16, seed=4, ignored=0.37)
    check(h, W, y, dl, 1.0, run(dg, h, W, y, dl))


def test_confident_positions_keep_their_digits(dg):
    """Losses down to 1e-10: the loss and the gradient's dominant term keep their relative precision."""
    h, W, y, dl = inputs(64, 512, 256, seed=5, lean=60.0)
    got = run(dg, h, W, y, dl)
    loss, *_ = check(h, W, y, dl, 1.0, got)
    assert loss.min() < 1e-8 and (got[0] > 0).all()


@pytest.mark.parametrize("n", [1, 200, 300])
def test_every_position_ignored(dg, n):
    h, W, y, dl = inputs(n, 600, 64, ignored=0.0)
    y.fill_(IGNORE)
    h.fill_(float("nan"))
    got = run(dg, h, W, y, dl)
    for x in got:
        assert (x == 0).all()


def test_masked_positions_may_hold_anything(dg):
    """NaN and infinities at ignored positions and at positions of zero weight reach nothing."""
    h, W, y, dl = inputs(200, 600, 64, seed=2, ignored=0.3)
    clean = h.clone()
    clean[y == IGNORE] = 0
    junk = h.clone()
    junk[y == IGNORE] = float("nan")
    a, b = run(dg, clean, W, y, dl), run(dg, junk, W, y, dl)
    for u, v in zip(a, b):
        assert np.array_equal(u, v)
    # zero weight: the loss is the position's own, its gradients are 0
    dl0, k = dl.clone(), int(torch.nonzero(y != IGNORE)[0])
    dl0[k] = 0
    h0 = clean.clone()
    h0[k] = float("inf")
    got = run(dg, h0, W, y, dl0)
    assert np.isnan(got[0][k]) and (got[2][k] == 0).all() and np.isfinite(got[3]).all()


def test_rows_behind_the_last_kept_position_are_left_out(dg):
    """The workspace of a larger batch holds older rows; a smaller batch does not see them."""
    p = dg.xent_params(600, 700, 64)
    ws = dg.XentWorkspace(p)
    ws.buf.fill_(0xFF)                       # NaN everywhere
    h, W, y, dl = inputs(600, 700, 64, seed=1)
    check(h, W, y, dl, 1.0, run(dg, h, W, y, dl, ws=ws))
    ws.buf.fill_(0xFF)
    y2 = y.clone()
    y2[5:] = IGNORE
    check(h, W, y2, dl, 1.0, run(dg, h, W, y2, dl, ws=ws))


@pytest.mark.parametrize("bad", [-1, 600, -2 ** 31])
def test_target_outside_the_vocabulary_is_nan(dg, bad):
    h, W, y, dl = inputs(40, 600, 64)
    y[7] = bad
    loss, lse, dh, dW = run(dg, h, W, y, dl)
    assert np.isnan(loss[7]) and np.isnan(lse[7]) and np.isnan(dh[7]).all() and np.isnan(dW).all()
    others = np.arange(40) != 7
    assert np.isfinite(loss[others]).all() and np.isfinite(dh[others]).all()


def test_int64_targets_beyond_32_bits(dg):
    h, W, y, dl = inputs(10, 600, 64, index=torch.int64)
    y[3] = 2 ** 32 + 5
    loss, *_ = run(dg, h, W, y, dl)
    assert np.isnan(loss[3]) and np.isfinite(np.delete(loss, 3)).all()


def test_other_ignore_index(dg):
    h, W, y, dl = inputs(50, 600, 64)
    y[::3] = 17
    got = run(dg, h, W, y, dl, ignore_index=17)
    assert (got[0][::3] == 0).all()
    z = y.clone()
    z[y == 17] = IGNORE
    check(h, W, z, dl, 1.0, got)


@pytest.mark.parametrize("pad,shift", [(8, 0), (8, 8), (1, 0), (0, 3)])
def test_strided_and_misaligned_hidden_states(dg, pad, shift):
    h, W, y, dl = inputs(70, 600, 72)
    flat = torch.full((70 * (72 + pad) + shift,), float("nan"), dtype=torch.bfloat16, device="cuda")
    view = flat[shift:].as_strided((70, 72), (72 + pad, 1), shift)
    view.copy_(h)
    p = dg.xent_params(70, 600, 72)
    ws = dg.XentWorkspace(p)
    yd, Wd, dld = y.cuda(), W.cuda(), dl.cuda()
    loss, lse = torch.empty(70, device="cuda"), torch.empty(70, device="cuda")
    dg.dg_xent_forward(p, view, Wd, yd, loss, lse, ws)
    dh, dW = torch.empty(70, 72, dtype=torch.bfloat16, device="cuda"), torch.empty_like(Wd)
    dg.dg_xent_backward(p, view, Wd, yd, loss, lse, dld, dh, dW, ws)
    want = run(dg, h, W, y, dl)
    for a, b in zip((loss, lse, dh, dW), want):
        assert np.array_equal(a.cpu().double().numpy(), b)


def test_one_gradient_at_a_time(dg):
    h, W, y, dl = inputs(300, 700, 136, ignored=0.2)
    both = run(dg, h, W, y, dl)
    assert np.array_equal(run(dg, h, W, y, dl, want=("dh",))[2], both[2])
    assert np.array_equal(run(dg, h, W, y, dl, want=("dW",))[3], both[3])


@pytest.mark.parametrize("dtype,eps", [(torch.float32, 2.0 ** -24), (torch.bfloat16, 2.0 ** -8)])
def test_gradients_of_the_head_in_both_types_and_added(dg, dtype, eps):
    h, W, y, dl = inputs(300, 700, 136)
    first = torch.full(W.shape, 7.0, dtype=dtype, device="cuda")
    check(h, W, y, dl, 1.0, run(dg, h, W, y, dl, dw=first), dw_eps=eps)
    base = torch.randn(W.shape, generator=torch.Generator().manual_seed(1)).to(dtype)
    got = run(dg, h, W, y, dl, dw=base.cuda(), dw_accumulate=1)[3]
    h64, W64 = h.double().numpy(), W.double().numpy()
    loss, lse, _, dW, G = xent.cross_entropy(h64, W64, y.numpy(), 1.0, IGNORE, dl.double().numpy())
    tol = xent.bounds(h64, W64, y.numpy(), 1.0, G, loss, lse)[2]
    want = base.double().numpy() + dW
    near("dW", got, want, tol * (1 + eps) + (eps + 2.0 ** -24) * np.abs(want) + 1e-38)


def test_no_positions(dg):
    W = torch.randn(600, 64).bfloat16().cuda()
    h = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    y = torch.empty(0, dtype=torch.int32, device="cuda")
    f = torch.empty(0, device="cuda")
    p = dg.xent_params(0, 600, 64)
    ws = dg.XentWorkspace(p)
    dg.dg_xent_forward(p, h, W, y, f, f.clone(), ws)
    assert dg.last_launch_count() == 0
    dW = torch.ones_like(W)
    dg.dg_xent_backward(p, h, W, y, f, f, f, h.clone(), dW, ws)
    assert (dW == 0).all()
    p.dw_accumulate = 1
    dW.fill_(1)
    dg.dg_xent_backward(p, h, W, y, f, f, f, h.clone(), dW, ws)
    assert (dW == 1).all()


def test_equal_calls_give_equal_bits(dg):
    h, W, y, dl = inputs(700, 9000, 200, ignored=0.3)
    a = run(dg, h, W, y, dl)
    for _ in range(5):
        for u, v in zip(a, run(dg, h, W, y, dl)):
            assert np.array_equal(u, v)


def test_two_streams_at_once(dg):
    cases = [inputs(300, 6000, 128, seed=k, ignored=0.1 * k) for k in range(2)]
    want = [run(dg, *c) for c in cases]
    state = []
    for h, W, y, dl in cases:
        p = dg.xent_params(300, 6000, 128)
        state.append((p, h.cuda(), W.cuda(), y.cuda(), dl.cuda(), dg.XentWorkspace(p), torch.empty(300, device="cuda"),
                      torch.empty(300, device="cuda"), torch.empty(300, 128, dtype=torch.bfloat16, device="cuda"),
                      torch.empty(6000, 128, dtype=torch.bfloat16, device="cuda"), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(5):
        for p, h, W, y, dl, ws, loss, lse, dh, dW, s in state:
            dg.dg_xent_forward(p, h, W, y, loss, lse, ws, s)
            dg.dg_xent_backward(p, h, W, y, loss, lse, dl, dh, dW, ws, s)
    torch.cuda.synchronize()
    for w, st in zip(want, state):
        for a, b in zip(w, st[6:10]):
            assert np.array_equal(a, b.cpu().double().numpy())


def test_captured_and_replayed_with_new_inputs(dg):
    """A replay sees the inputs, and the number of positions kept, that its buffers then hold."""
    h, W, y, dl = inputs(300, 3000, 128, seed=1)
    p = dg.xent_params(300, 3000, 128)
    hd, Wd, yd, dld, ws = h.cuda(), W.cuda(), y.cuda(), dl.cuda(), dg.XentWorkspace(p)
    loss, lse = torch.empty(300, device="cuda"), torch.empty(300, device="cuda")
    dh, dW = torch.empty_like(hd), torch.empty_like(Wd)

    dlsrc = dld.clone()

    def calls():
        dld.copy_(dlsrc)                 # a copy node before the first kernel
        dg.dg_xent_forward(p, hd, Wd, yd, loss, lse, ws)
        dg.dg_xent_backward(p, hd, Wd, yd, loss, lse, dld, dh, dW, ws)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        calls()
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        calls()
    for seed, ignored in ((1, 0.0), (2, 0.6), (3, 1.0), (4, 0.1)):
        h, W, y, dl = inputs(300, 3000, 128, seed=seed, ignored=ignored)
        want = run(dg, h, W, y, dl)
        for a, b in ((hd, h), (Wd, W), (yd, y), (dlsrc, dl)):
            a.copy_(b)
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip((loss, lse, dh, dW), want):
            assert np.array_equal(a.cpu().double().numpy(), b)


def test_autograd(dg):
    """Shapes beyond two, a weighted sum and a mean (a broadcast gradient), one leaf or both."""
    h, W, y, dl = inputs(60, 700, 64, ignored=0.2, index=torch.int64)
    want = run(dg, h, W, y, dl, T=0.8)
    hd, Wd = h.cuda().view(3, 20, 64).requires_grad_(), W.cuda().requires_grad_()
    loss = dg.head_cross_entropy(hd, Wd, y.cuda().view(3, 20), temperature=0.8)
    assert loss.shape == (3, 20)
    (loss * dl.cuda().view(3, 20)).sum().backward()
    for a, b in ((loss, want[0]), (hd.grad, want[2]), (Wd.grad, want[3])):
        assert np.array_equal(a.detach().cpu().double().numpy().reshape(b.shape), b)
    one = run(dg, h, W, y, torch.ones(60), T=0.8)
    hd2 = h.cuda().requires_grad_()
    dg.head_cross_entropy(hd2, W.cuda(), y.cuda(), temperature=0.8).sum().backward()
    assert np.array_equal(hd2.grad.cpu().double().numpy(), one[2])
    # hidden states that are broadcast: one row for every target
    row = h[:1].cuda().requires_grad_()
    dg.head_cross_entropy(row.expand(60, 64), W.cuda(), y.cuda(), temperature=0.8).sum().backward()
    full = run(dg, h[:1].expand(60, 64).contiguous(), W, y, torch.ones(60), T=0.8)[2].sum(0)
    # autograd adds the 60 rows itself, in bf16 at worst: half a step for each partial sum
    assert np.all(np.abs(row.grad.cpu().double().numpy()[0] - full) <= 60 * 2.0 ** -8 * np.abs(
        run(dg, h[:1].expand(60, 64).contiguous(), W, y, torch.ones(60), T=0.8)[2]).sum(0) + 1e-30)


def test_gradients_against_differences_of_the_kernels_loss(dg):
    """The loss along a direction in h and in W that bf16 holds exactly, against the gradients' products."""
    n, V, d = 40, 300, 64
    g = torch.Generator().manual_seed(9)
    h = (torch.randint(-64, 65, (n, d), generator=g) / 32).bfloat16()
    W = (torch.randint(-64, 65, (V, d), generator=g) / 256).bfloat16()
    y = torch.randint(0, V, (n,), generator=g).int()
    dl = torch.rand(n, generator=g) + 0.5
    _, _, dh, dW = run(dg, h, W, y, dl)

    def total(h, W):
        return float((run(dg, h, W, y, dl)[0] * dl.double().numpy()).sum())

    for which, x, grad, e in (("h", h, dh, 2.0 ** -5), ("W", W, dW, 2.0 ** -8)):
        sign = torch.randint(0, 2, x.shape, generator=g) * 2 - 1
        up, down = (x.float() + e * sign).bfloat16(), (x.float() - e * sign).bfloat16()
        assert torch.equal(up.float() - x.float(), e * sign.float())
        a = total(up, W) if which == "h" else total(h, up)
        b = total(down, W) if which == "h" else total(h, down)
        slope = (a - b) / (2 * e)
        want = float((grad * sign.numpy()).sum())
        # Third derivative of a log-sum-exp along the direction: at most 2 max|dz|^3 a position, dz the logits'
        # slope; the error of the central difference is e^2 / 6 of that.  fp32 losses add 2^-19 of themselves
        # over 2 e, the gradients' bf16 2^-7 of each product.
        other = (W if which == "h" else h).double().numpy()
        dz = np.abs(sign.double().numpy() @ other.T).max() if which == "h" else np.abs(
            other @ sign.double().numpy().T).max()
        tol = (e * e / 6 * 2 * dz ** 3 * dl.sum().item() + 2.0 ** -19 * (abs(a) + abs(b)) / (2 * e)
               + 2.0 ** -7 * np.abs(grad).sum())
        assert abs(slope - want) <= tol and tol < 0.5 * np.abs(grad).sum()


def test_refusals_on_the_device(dg):
    h, W, y, dl = inputs(20, 600, 64)
    p = dg.xent_params(20, 600, 64)
    ws = dg.XentWorkspace(p)
    hd, Wd, yd, dld = h.cuda(), W.cuda(), y.cuda(), dl.cuda()
    loss, lse = torch.empty(20, device="cuda"), torch.empty(20, device="cuda")
    for args in ((h, Wd, yd, loss, lse), (hd.float(), Wd, yd, loss, lse), (hd[:19], Wd, yd, loss, lse),
                 (hd, Wd.float(), yd, loss, lse), (hd, Wd.t().contiguous().t(), yd, loss, lse),
                 (hd, Wd, yd.float(), loss, lse), (hd, Wd, yd[:19], loss, lse), (hd, Wd, yd, loss.double(), lse),
                 (hd, Wd, yd, loss[:10], lse), (hd, Wd, yd, loss, lse.cpu()), (hd[:1].expand(20, 64), Wd, yd, loss, lse),
                 (hd.t().contiguous().t(), Wd, yd, loss, lse)):
        with pytest.raises(dg.DgError):
            dg.dg_xent_forward(p, *args, ws)
    small = dg.XentWorkspace(dg.xent_params(20, 600, 64), backward=False)
    dh, dW = torch.empty_like(hd), torch.empty_like(Wd)
    dg.dg_xent_forward(p, hd, Wd, yd, loss, lse, small)
    with pytest.raises(dg.DgError) as e:
        dg.dg_xent_backward(p, hd, Wd, yd, loss, lse, dld, dh, dW, small)
    assert e.value.status == -5
    for grads in ((None, None), (hd, dW), (dh, Wd), (Wd[:20], dW), (dh.float(), dW), (dh, dW.half())):
        with pytest.raises(dg.DgError):
            dg.dg_xent_backward(p, hd, Wd, yd, loss, lse, dld, *grads, ws)
    flat = torch.empty(600 * 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(dg.DgError):      # dh inside dW
        dg.dg_xent_backward(p, hd, Wd, yd, loss, lse, dld, flat[64:21 * 64].view(20, 64), flat.view(600, 64), ws)
    for k, v in (("temperature", 0.0), ("temperature", float("nan")), ("temperature", 1e-42), ("dw_accumulate", 2), ("hidden", 60), ("scratch_bytes", -1)):
        q = dg.xent_params(20, 600, 64)
        setattr(q, k, v)
        with pytest.raises(dg.DgError):
            dg.XentWorkspace(q)


def test_a_call_clears_the_error_word_of_an_earlier_one(dg):
    """A raised error word (a wait that ran out) in a workspace does not reach the next call with it."""
    h, W, y, dl = inputs(20, 600, 64)
    p = dg.xent_params(20, 600, 64)
    ws = dg.XentWorkspace(p)
    ws.buf[:4] = 1
    check(h, W, y, dl, 1.0, run(dg, h, W, y, dl, ws=ws))
