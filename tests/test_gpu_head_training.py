"""The head's training as it is used: loss, gradients, AdamW and the decode that reads the trained head."""

import threading

import numpy as np
import pytest
import torch

from oracle import adamw, stage, xent

import synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dg():
    from discrete_diffusion_decoding_b200 import build
    build.build()
    import discrete_diffusion_decoding_b200 as m
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return m


def batch(n, V, d, seed, ignored=0.2):
    g = torch.Generator().manual_seed(seed)
    h = torch.randn(n, d, generator=g).bfloat16()
    y = torch.randint(0, V, (n,), generator=g).int()
    y[torch.rand(n, generator=g) < ignored] = -100
    return h, y, torch.rand(n, generator=g) + 0.5


def mean_gradient(W, h, y, w, T=1.0):
    """float64 (loss, dh, dW and their bounds) of the weighted mean over the kept positions."""
    keep = y.numpy() != -100
    dl = np.where(keep, w.double().numpy(), 0.0)
    dl /= dl.sum()
    h64, W64 = h.double().numpy(), W.double().numpy()
    loss, lse, dh, dW, G = xent.cross_entropy(h64, W64, y.numpy(), T, -100, dl)
    dz, th, tw = xent.bounds(h64, W64, y.numpy(), T, G, loss, lse)
    # the weights themselves are fp32: each off by at most 4 steps (two products, the sum, the quotient)
    th, tw = th + 2.0 ** -22 * (np.abs(G) @ np.abs(W64)), tw + 2.0 ** -22 * (np.abs(G).T @ np.abs(h64))
    return (dl * loss).sum(), dh, dW, 2 * dz.max() + 2.0 ** -18 * np.abs(loss).max(), th, tw


@pytest.mark.parametrize("n,V,d", [(1, 257, 72), (300, 1000, 136)])
def test_steps_of_the_trainer(dg, n, V, d):
    """Each batch's loss and gradients against the oracle at the head of that moment, each update against the
    oracle's step from the gradient that the kernels left."""
    W = (torch.randn(V, d, generator=torch.Generator().manual_seed(0)) * 0.05).bfloat16().cuda()
    tr = dg.HeadTrainer(W, lr=1e-2, betas=(0.9, 0.99), weight_decay=0.1, state_bits=32, master=True,
                        grad_dtype=torch.float32)
    master, m, v = W.double().cpu().numpy(), np.zeros((V, d)), np.zeros((V, d))
    for t in range(1, 4):
        now = W.cpu()
        sums = np.zeros((V, d))
        for k in range(2):              # two batches a step
            h, y, w = batch(n, V, d, 10 * t + k, 0.2 if n > 1 else 0.0)
            loss, dh = tr.accumulate(h.cuda(), y.cuda(), w.cuda())
            want, dh64, dW64, tol, th, tw = mean_gradient(now, h, y, w)
            assert abs(float(loss) - want) <= tol
            assert np.all(np.abs(dh.cpu().double().numpy() - dh64) <= th * 1.01 + 2.0 ** -8 * np.abs(dh64) + 1e-38)
            sums += dW64
            off = np.abs(tr.dW.cpu().double().numpy() - sums)
            # the earlier batch's bound is of the same size: twice this one's largest element covers both
            assert np.all(off <= 2.0 ** -22 * np.abs(sums) + 2 * max(tw.max(), 1e-38))
        g = tr.dW.cpu().numpy()
        tr.update()
        want, m, v = adamw.step(master, g, m, v, t, 1e-2, 0.9, 0.99, 1e-8, 0.1, 0.5)
        got = tr.optimizer._states()[-1].cpu().double().numpy()
        assert np.all(np.abs(got - want) <= 64 * 2.0 ** -24 * (np.abs(want) + 1e-2))
        assert torch.equal(W.cpu(), torch.from_numpy(got).float().bfloat16())
        master = got


def test_eight_bit_trainer_runs_and_updates_every_row(dg):
    """bf16 alone with 8-bit states: the update is the one that the entry points make from the same tensors."""
    V, d, n = 600, 64, 200
    W = (torch.randn(V, d, generator=torch.Generator().manual_seed(0)) * 0.05).bfloat16().cuda()
    W2 = W.clone()
    tr = dg.HeadTrainer(W, lr=1e-3, seed=5)
    blocks = V * d // 256
    st = [torch.zeros(V, d, dtype=torch.uint8, device="cuda") for _ in range(2)]
    ex = [torch.zeros(blocks, dtype=torch.int8, device="cuda") for _ in range(2)]
    T = dg.AdamWTensors([W2], [torch.empty_like(W2)], [st[0]], [st[1]], m_exp=[ex[0]], v_exp=[ex[1]])
    for t in range(1, 4):
        h, y, w = (x.cuda() for x in batch(n, V, d, t))
        assert torch.equal(W, W2)
        tr.accumulate(h, y, w)
        T.set_grads([tr.dW.clone()])
        dg.dg_adamw_step(dg.adamw_params(lr=1e-3, step=t, seed=5, stochastic=1), T)
        tr.update()
        assert torch.equal(W, W2) and tr.batches == 0
    with pytest.raises(dg.DgError):
        tr.update()
    with pytest.raises(dg.DgError):
        dg.HeadTrainer(W.float())


def test_a_trained_head_decodes_in_every_serving_form(dg):
    """Train, then one denoising step with the head as rows, as tiles (the same bits) and against the oracle."""
    V, d = 4096, 128
    W = synth.weights(V, d).cuda()
    tr = dg.HeadTrainer(W, lr=1e-3, temperature=0.8)
    for t in range(3):
        h, y, w = (x.cuda() for x in batch(256, V, d, t))
        tr.step(h, y, w)
    host = W.cpu()
    h, _ = synth.spiked_hidden(host, 256, gain_lo=0.5, gain_hi=20.0)
    seeds = torch.zeros(1, dtype=torch.int64, device="cuda")
    out = []
    for form, layout in (("rows", 0), ("tiles", 1)):
        p = dg.params(1, V, d, head_layout=layout)
        ws, b = dg.Workspace(p), dg.StepBuffers(p)
        E = tr.serving(form)
        dg.dg_canvas_init(p, seeds, b.tokens, ws)
        b.h.copy_(h.cuda())
        dg.dg_denoise_step(p, 1, b.h, E, E, seeds, b.tokens, b.entropy, b.argmax, b.accept, b.lse, b.selfcond, ws)
        dg.dg_stop_check(p, ws)
        out.append((b.entropy.cpu().numpy(), b.argmax.cpu().numpy(), b.tokens.cpu().numpy(), b.selfcond.cpu().numpy()))
    for a, b in zip(*out):
        assert np.array_equal(a, b)
    Wb = synth.bf16_bits(host)
    r = stage.step_rows(synth.bf16_bits(h), Wb, Wb, dg.temperature(dg.params(1, V, d), 1), 0.1, 0, 1, 0, np.arange(256), V)
    assert np.abs(out[0][0] - r["H"]).max() <= 1e-3
    codes, e = tr.serving("e4m3")
    assert codes.dtype == torch.uint8 and codes.shape == W.shape and isinstance(e, int)
    # the loss that the trainer reports is the decode's own softmax: lse of the same head at the same temperature
    p = dg.xent_params(256, V, d, temperature=dg.temperature(dg.params(1, V, d), 1))
    loss, lse = torch.empty(256, device="cuda"), torch.empty(256, device="cuda")
    dg.dg_xent_forward(p, h.cuda(), W, torch.zeros(256, dtype=torch.int32, device="cuda"), loss, lse,
                       dg.XentWorkspace(p, backward=False))
    assert np.abs(lse.cpu().numpy() - r["lse"]).max() <= 1e-3 * np.abs(r["lse"]).max()
    with pytest.raises(ValueError):
        tr.serving("int8")


def test_batches_of_growing_and_shrinking_size(dg):
    """One trainer over batches of many sizes gives what a new one gives for each."""
    V, d = 700, 64
    W = (torch.randn(V, d, generator=torch.Generator().manual_seed(0)) * 0.05).bfloat16().cuda()
    tr = dg.HeadTrainer(W.clone(), lr=0.0)
    for t, n in enumerate((5, 300, 1, 40, 0, 520)):
        h, y, w = (x.cuda() for x in batch(n, V, d, t))
        a, da = tr.accumulate(h, y, w)
        other = dg.HeadTrainer(W.clone(), lr=0.0)
        b, db = other.accumulate(h, y, w)
        assert torch.equal(a, b) and torch.equal(da, db) and torch.equal(tr.dW, other.dW)
        tr.batches = 0


def test_captured_autograd_step(dg):
    """Forward and backward of head_cross_entropy in one graph, replayed on new inputs."""
    V, d, n = 700, 64, 100
    W = (torch.randn(V, d, generator=torch.Generator().manual_seed(0)) * 0.05).bfloat16().cuda().requires_grad_()
    h = torch.zeros(n, d, dtype=torch.bfloat16, device="cuda", requires_grad=True)
    y = torch.zeros(n, dtype=torch.int64, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        dg.head_cross_entropy(h, W, y).mean().backward()
    torch.cuda.current_stream().wait_stream(side)
    h.grad = W.grad = None
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        loss = dg.head_cross_entropy(h, W, y)
        loss.mean().backward()
    for seed in (1, 2):
        hb, yb, _ = batch(n, V, d, seed, 0.3)
        with torch.no_grad():
            h.copy_(hb)
        y.copy_(yb)
        g.replay()
        torch.cuda.synchronize()
        a, b = hb.cuda().requires_grad_(), W.detach().clone().requires_grad_()
        eager = dg.head_cross_entropy(a, b, yb.cuda().long())
        eager.mean().backward()
        assert torch.equal(loss, eager) and torch.equal(h.grad, a.grad) and torch.equal(W.grad, b.grad)


def test_optimizer_notices_moved_parameters(dg):
    p = torch.nn.Parameter(torch.zeros(10, device="cuda"))
    opt = dg.AdamW([p], state_bits=32)
    p.grad = torch.ones(10, device="cuda")
    opt.step()
    p.data = torch.zeros(10, device="cuda")
    with pytest.raises(dg.DgError):
        opt.step()
    assert opt.steps == 1
    q = torch.nn.Parameter(torch.zeros(300, dtype=torch.bfloat16, device="cuda"))
    opt = dg.AdamW([q], lr=0.0, master=True)
    with torch.no_grad():
        q.fill_(3.0)
    opt.refresh_master()
    opt.step([torch.ones_like(q)])
    assert (q == 3.0).all()


def test_steps_that_count_on_the_host_are_not_captured(dg):
    """A graph would repeat the bias correction, the random bits and the choice to add to dW of its capture."""
    W = torch.ones(64, 8, dtype=torch.bfloat16, device="cuda")
    tr, opt = dg.HeadTrainer(W.clone()), dg.AdamW([W])
    h, y = torch.ones(3, 8, dtype=torch.bfloat16, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    x = torch.zeros(4, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        x.add_(1)
        for call in (lambda: tr.step(h, y), lambda: tr.accumulate(h, y), lambda: opt.step([W.clone()])):
            with pytest.raises(dg.DgError, match="captured"):
                call()
    assert tr.batches == 0 and opt.steps == 0
    tr.step(h, y)
    assert tr.optimizer.steps == 1


def test_params_shared_by_lists_of_two_types(dg):
    """The types of a call are its tensors', also while another thread steps with the same params."""
    p = dg.adamw_params(lr=0.5, step=1)
    before = bytes(p)
    sets = []
    for dtype in (torch.float32, torch.bfloat16):
        w = torch.zeros(5000, dtype=dtype, device="cuda")
        m, v = (torch.zeros(5000, device="cuda") for _ in range(2))
        sets.append((w, dg.AdamWTensors([w], [torch.ones_like(w)], [m], [v])))
    threads = [threading.Thread(target=lambda t=t: [dg.dg_adamw_step(p, t) for _ in range(200)]) for _, t in sets]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert bytes(p) == before
    for w, t in sets:
        one = torch.zeros_like(w)
        alone = dg.AdamWTensors([one], [torch.ones_like(w)], [torch.zeros(5000, device="cuda")],
                                [torch.zeros(5000, device="cuda")])
        for _ in range(200):
            dg.dg_adamw_step(p, alone)
        assert torch.equal(w, one)
