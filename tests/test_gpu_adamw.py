"""AdamW on the GPU against the float64 oracle: fp32 states and 8-bit codes bit by bit, parameters within their
type's rounding, ragged and misaligned tensors, long lists, streams, graphs, refusals."""

import numpy as np
import pytest
import torch

from oracle import adamw

pytestmark = pytest.mark.gpu
LR, B1, B2, EPS = 1e-2, 0.9, 0.99, 1e-8


@pytest.fixture(scope="module")
def dg():
    from discrete_diffusion_decoding_b200 import build
    build.build()
    import discrete_diffusion_decoding_b200 as m
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return m


def at(x, shift):
    """x on the device, `shift` elements behind an aligned address."""
    buf = torch.empty(x.numel() + shift, dtype=x.dtype, device="cuda")
    buf[shift:].copy_(x.view(-1))
    return buf[shift:]


def make(sizes, param, grad, bits, master, seed=0, shift=0):
    g = torch.Generator().manual_seed(seed)
    S = dict(p=[], g=[], m=[], v=[], m_exp=[], v_exp=[], master=[])
    for n in sizes:
        p = torch.randn(n, generator=g) * 0.05
        S["p"].append(at(p.to(param), shift))
        S["master"].append(at(p, shift))
        S["g"].append(at((torch.randn(n, generator=g) * 1e-2 * torch.exp(torch.randn(n, generator=g))).to(grad), shift))
        m, r = torch.randn(n, generator=g) * 3e-3, torch.randn(n, generator=g).abs() * 1e-2
        m[torch.rand(n, generator=g) < 0.05] = 0
        r[torch.rand(n, generator=g) < 0.05] = 0
        if bits == 32:
            S["m"].append(at(m, shift))
            S["v"].append(at(r * r, shift))
        else:
            half = np.full(n, 32768)
            for k, x in (("m", m), ("v", r)):
                c, e = adamw.encode(x.numpy(), half, k == "v")
                S[k].append(at(torch.from_numpy(c), shift))
                S[k + "_exp"].append(torch.from_numpy(e.astype(np.int8)).cuda())
    if bits == 32:
        S["m_exp"] = S["v_exp"] = None
    if not master:
        S["master"] = None
    return S


def tensors(dg, S, decay=0.1):
    return dg.AdamWTensors(S["p"], S["g"], S["m"], S["v"], m_exp=S["m_exp"], v_exp=S["v_exp"], master=S["master"],
                           weight_decay=decay)


def copy(S):
    return {k: None if x is None else [t.cpu().clone() for t in x] for k, x in S.items()}


def check_roots(codes, exps, v, u):
    """Exponents are those of the correctly rounded roots.  The roots that are rounded to codes come from the SFU,
    off by at most 2^-23 of themselves: a code is one of those of the roots 2^-22 below and above."""
    r = np.sqrt(v)
    _, e = adamw.encode(r, u, root=True)
    assert np.array_equal(exps.cpu().numpy(), e)
    scale = 2.0 ** -np.repeat(e, 256)[:len(v)].astype(np.float64)
    y, got = r.astype(np.float64) * scale, adamw.decode(codes.cpu().numpy(), np.zeros_like(e))

    def cut(y):
        y = np.where(y < 2.0 ** -6, (y + 2.0 ** -6).astype(np.float32) - 2.0 ** -6, y)
        step = 2.0 ** (np.floor(np.log2(np.maximum(y, 2.0 ** -6))) - 3)
        return np.where(r > 0, np.maximum(np.floor(y / step + u / 65536) * step, 2.0 ** -9), 0)

    lo, hi = cut(y * (1 - 2.0 ** -22)), cut(np.minimum(y * (1 + 2.0 ** -22), 448))
    fin = np.isfinite(y)
    assert np.all(((got >= lo) & (got <= hi))[fin]) and np.isnan(got[~fin]).all()
    assert len(v) < 1000 or np.mean(lo == hi) > 0.999


def check(before, S, t, seed, decay, bits, stochastic, grad_scale=1.0, lr=LR):
    """What the call left in S, against the oracle's step from `before`."""
    for i, p0 in enumerate(before["p"]):
        n = p0.numel()
        wd = decay[i] if hasattr(decay, "__len__") else decay
        g = before["g"][i].float().numpy()
        if bits == 32:
            m0, v0 = before["m"][i].numpy(), before["v"][i].numpy()
        else:
            m0 = adamw.decode(before["m"][i].numpy(), before["m_exp"][i].numpy()).astype(np.float32)
            r0 = adamw.decode(before["v"][i].numpy(), before["v_exp"][i].numpy()).astype(np.float32)
            v0 = r0 * r0
        src = before["p"][i].float() if before["master"] is None else before["master"][i]
        m, v = adamw.moments(g, m0, v0, B1, B2, grad_scale)
        want, _, _ = adamw.step(src.numpy(), g, m0, v0, t, lr, B1, B2, EPS, wd, grad_scale)
        # fp32, in units u = 2^-24: m = b1 m0 + (1 - b1) g' has each constant, product and the sum rounded, so it is
        # off by at most 4 u (|b1 m0| + |(1 - b1) g'|), which is more than u |m| where the two cancel; v's terms
        # have one sign, so the root is off by 3 u of itself, its product with the bias correction by 5 u, the
        # denominator by 6 u; lr / (1 - b1^t) and the numerator's product add 2 u, the quotient 4 u (2 units in
        # the last place): 12 u of the update in all.  The kept share 1 - lr wd and the final sum add u |p0| and
        # u |p|.
        gs = np.abs(g.astype(np.float64) * grad_scale)
        den = np.sqrt(v.astype(np.float64) / (1 - B2 ** t)) + EPS
        scale = lr / (1 - B1 ** t) / den
        tol = 2.0 ** -24 * (scale * (4 * (B1 * np.abs(m0) + (1 - B1) * gs) + 12 * np.abs(m)) + np.abs(src.double().numpy())
                            + 2 * np.abs(want))
        if bits == 32:
            assert np.array_equal(S["m"][i].cpu().numpy(), m) and np.array_equal(S["v"][i].cpu().numpy(), v)
        else:
            um, uv = adamw.random_halves(seed, n, t, i)
            cm, em = adamw.encode(m, um)
            assert np.array_equal(S["m_exp"][i].cpu().numpy(), em) and np.array_equal(S["m"][i].cpu().numpy(), cm)
            check_roots(S["v"][i], S["v_exp"][i], v, uv)
        got = S["p"][i].cpu()
        if before["master"] is not None:
            mast = S["master"][i].cpu()
            assert np.all(np.abs(mast.double().numpy() - want) <= tol)
            assert torch.equal(got, mast.to(got.dtype))
        elif got.dtype == torch.float32:
            assert np.all(np.abs(got.double().numpy() - want) <= tol)
        elif stochastic:
            # the oracle's cut of its own value; a value within tol of a border may fall on the other side
            u = adamw.random_param(seed, n, t, i)
            lo = adamw.round_bf16_random((want - np.sign(want) * tol).astype(np.float32), u)
            hi = adamw.round_bf16_random((want + np.sign(want) * tol).astype(np.float32), u)
            x = got.float().numpy()
            assert np.all((np.abs(x) >= np.abs(lo)) & (np.abs(x) <= np.abs(hi)))
            assert n < 1000 or np.mean(lo == hi) > 0.99
        else:
            assert np.all(np.abs(got.double().numpy() - want) <= tol + 2.0 ** -8 * np.abs(want))


TYPES = [(torch.float32, torch.float32, False), (torch.float32, torch.bfloat16, False),
         (torch.bfloat16, torch.bfloat16, False), (torch.bfloat16, torch.float32, False),
         (torch.bfloat16, torch.bfloat16, True), (torch.bfloat16, torch.float32, True)]


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("param,grad,master", TYPES)
@pytest.mark.parametrize("shift", [0, 1])
def test_types_and_ragged_sizes(dg, param, grad, master, bits, shift):
    sizes = [1, 7, 8, 255, 256, 257, 0, 2816, 5000, 33]
    S = make(sizes, param, grad, bits, master, shift=shift)
    T = tensors(dg, S)
    plain = param == torch.bfloat16 and not master
    for t in (1, 2, 50):
        before = copy(S)
        dg.dg_adamw_step(dg.adamw_params(lr=LR, beta1=B1, beta2=B2, eps=EPS, step=t, seed=11 + (5 << 40),
                                         stochastic=int(plain)), T)
        assert dg.last_launch_count() == 1
        check(before, S, t, 11 + (5 << 40), 0.1, bits, plain)


def test_bf16_parameters_to_nearest(dg):
    S = make([3000], torch.bfloat16, torch.bfloat16, 32, False)
    before = copy(S)
    dg.dg_adamw_step(dg.adamw_params(lr=LR, beta1=B1, beta2=B2, eps=EPS, step=3), tensors(dg, S))
    check(before, S, 3, 0, 0.1, 32, False)


@pytest.mark.parametrize("count", [24, 25, 400, 401, 1000])
def test_long_lists(dg, count):
    sizes = [(7 * k) % 700 for k in range(count)]
    S = make(sizes, torch.float32, torch.float32, 8, False, seed=1)
    decay = [0.1 * (k % 3) for k in range(count)]
    before = copy(S)
    dg.dg_adamw_step(dg.adamw_params(lr=LR, beta1=B1, beta2=B2, eps=EPS, step=4, seed=5), tensors(dg, S, decay))
    # one launch for each 400 tensors of which any holds an element: of 401 the last is empty (2800 % 700)
    assert dg.last_launch_count() == sum(any(sizes[i:i + 400]) for i in range(0, count, 400))
    check(before, S, 4, 5, decay, 8, False)


def test_a_large_tensor_among_small_ones(dg):
    """Over the size from which a warp takes several blocks."""
    sizes = [100, 20_000_003, 9]
    g = torch.Generator(device="cuda").manual_seed(0)
    p = [torch.randn(n, generator=g, device="cuda") for n in sizes]
    gr = [torch.randn(n, generator=g, device="cuda") for n in sizes]
    m, v = [torch.zeros_like(x) for x in p], [torch.zeros_like(x) for x in p]
    p0 = [x.clone() for x in p]
    dg.dg_adamw_step(dg.adamw_params(lr=LR, beta1=B1, beta2=B2, eps=EPS, step=1), dg.AdamWTensors(p, gr, m, v))
    for a, b, c, e, w in zip(p, p0, gr, m, v):
        assert torch.equal(e, c * torch.tensor(1 - B1, device="cuda")) and torch.equal(w, c * c * torch.tensor(1 - B2, device="cuda"))
        want = b.double() - LR * c.double() / (c.double().abs() + EPS)
        assert ((a.double() - want).abs() <= 2.0 ** -23 * b.double().abs() + 2.0 ** -20 * LR).all()


def test_zero_gradients_and_states(dg):
    """Nothing moves but the decay; codes and exponents stay 0."""
    for bits in (8, 32):
        S = make([600], torch.float32, torch.float32, bits, False)
        for k in ("g", "m", "v", "m_exp", "v_exp"):
            for t in S[k] or []:
                t.zero_()
        p0 = S["p"][0].clone()
        dg.dg_adamw_step(dg.adamw_params(lr=LR, step=1), tensors(dg, S, 0.0))
        assert torch.equal(S["p"][0], p0) and (S["m"][0] == 0).all() and (S["v"][0] == 0).all()
        if bits == 8:
            assert (S["m_exp"][0] == 0).all() and (S["v_exp"][0] == 0).all()


def test_extreme_gradients(dg):
    """Blocks of tiny, huge and non-finite gradients: exponents stay in range, NaN stays where it came from."""
    n = 1024
    g = torch.zeros(n)
    g[:256] = torch.linspace(1e-38, 1e-36, 256)
    g[256:512] = torch.linspace(1e17, 1.8e19, 256)
    g[600] = float("nan")
    g[700] = float("inf")
    g[512:768:2] += 1.0
    S = make([n], torch.float32, torch.float32, 8, False)
    S["g"][0].copy_(g)
    for k in ("m", "v", "m_exp", "v_exp"):
        S[k][0].zero_()
    before = copy(S)
    dg.dg_adamw_step(dg.adamw_params(lr=LR, beta1=B1, beta2=B2, eps=EPS, step=1, seed=3), tensors(dg, S, 0.0))
    with np.errstate(all="ignore"):
        m, v = adamw.moments(g.numpy(), np.zeros(n), np.zeros(n), B1, B2)
        um, uv = adamw.random_halves(3, n, 1, 0)
        cm, em = adamw.encode(m, um)
        check_roots(S["v"][0], S["v_exp"][0], v, uv)
    assert np.array_equal(S["m_exp"][0].cpu().numpy(), em)
    assert np.array_equal(S["m"][0].cpu().numpy() & 0x7F, cm & 0x7F)
    moved = S["p"][0].cpu().numpy()
    odd = ~np.isfinite(moved)
    assert set(np.flatnonzero(odd)) <= {600, 700} and odd[600]
    assert before["p"][0].numel() == n


def test_scalars_on_the_device(dg):
    """lr, step and gradient scale read when the kernel runs give what the host values give."""
    for bits in (8, 32):
        a, b = (make([5000], torch.bfloat16, torch.float32, bits, False, seed=4) for _ in range(2))
        dg.dg_adamw_step(dg.adamw_params(lr=float(np.float32(LR)), beta1=B1, beta2=B2, eps=EPS, step=7, seed=9,
                                         grad_scale=0.25, stochastic=1), tensors(dg, a))
        hp = dg.adamw_params(lr=123.0, beta1=B1, beta2=B2, eps=EPS, step=0, seed=9, grad_scale=0.5, stochastic=1,
                             lr_dev=torch.tensor([LR], device="cuda"),
                             step_dev=torch.tensor([7], dtype=torch.int32, device="cuda"),
                             grad_scale_dev=torch.tensor([0.5], device="cuda"))
        dg.dg_adamw_step(hp, tensors(dg, b))
        for k in ("m", "v"):
            assert torch.equal(a[k][0], b[k][0])
        # bias corrections through expm1 and log instead of pow: a unit in the last place of the update
        assert (a["p"][0].float() - b["p"][0].float()).abs().max() <= 2.0 ** -7 * a["p"][0].float().abs().max()
        assert torch.mean((a["p"][0] != b["p"][0]).float()) < 0.01


def test_captured_and_replayed(dg):
    """A graph of the step with its count and rate on the device, replayed, equals eager steps."""
    a, b = (make([3000, 77], torch.float32, torch.float32, 8, False, seed=6) for _ in range(2))
    step = torch.zeros(1, dtype=torch.int32, device="cuda")
    rate = torch.zeros(1, device="cuda")
    hp = dg.adamw_params(beta1=B1, beta2=B2, eps=EPS, seed=2, lr_dev=rate, step_dev=step)
    T = tensors(dg, a)
    g = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=side):
        step.add_(1)
        dg.dg_adamw_step(hp, T)
    step.zero_()
    hp2 = dg.adamw_params(beta1=B1, beta2=B2, eps=EPS, seed=2, lr_dev=rate, step_dev=step)
    U = tensors(dg, b)
    for k in range(4):
        rate.fill_(LR / (k + 1))
        g.replay()
    step.zero_()
    for k in range(4):
        rate.fill_(LR / (k + 1))
        step.add_(1)
        dg.dg_adamw_step(hp2, U)
    for k in ("p", "m", "v", "m_exp", "v_exp"):
        for x, y in zip(a[k], b[k]):
            assert torch.equal(x, y)


def test_nothing_to_do(dg):
    """Empty tensors and missing gradients launch nothing and change nothing."""
    p = [torch.ones(300, device="cuda"), torch.ones(0, device="cuda")]
    T = dg.AdamWTensors(p, [None, torch.ones(0, device="cuda")], [torch.zeros_like(x) for x in p],
                        [torch.zeros_like(x) for x in p])
    dg.dg_adamw_step(dg.adamw_params(), T)
    assert dg.last_launch_count() == 0 and (p[0] == 1).all()
    T.set_grads([torch.ones(300, device="cuda"), None])
    dg.dg_adamw_step(dg.adamw_params(), T)
    assert dg.last_launch_count() == 1 and (p[0] < 1).all()


def test_two_lists_on_two_streams(dg):
    sets = [make([40000, 300], torch.bfloat16, torch.bfloat16, 8, False, seed=k) for k in range(2)]
    same = [make([40000, 300], torch.bfloat16, torch.bfloat16, 8, False, seed=k) for k in range(2)]
    hp = [dg.adamw_params(lr=LR, step=1, seed=k, stochastic=1) for k in range(2)]
    for S, p in zip(same, hp):
        dg.dg_adamw_step(p, tensors(dg, S))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for S, p, s in zip(sets, hp, streams):
        dg.dg_adamw_step(p, tensors(dg, S), s)
    torch.cuda.synchronize()
    for A, B in zip(sets, same):
        for k in ("p", "m", "v"):
            for x, y in zip(A[k], B[k]):
                assert torch.equal(x, y)


def test_slow_drift_is_kept_on_average(dg):
    """sqrt(v) moves by far less than half a code step each time; rounded at random it follows all the same."""
    n, steps, b2 = 1 << 16, 400, 0.999
    p = [torch.zeros(n, device="cuda")]
    g = [torch.full((n,), 1e-2, device="cuda")]
    m, v = [torch.zeros(n, dtype=torch.uint8, device="cuda")], [torch.zeros(n, dtype=torch.uint8, device="cuda")]
    e = [[torch.zeros(n // 256, dtype=torch.int8, device="cuda")] for _ in range(2)]
    T = dg.AdamWTensors(p, g, m, v, m_exp=e[0], v_exp=e[1])
    for t in range(1, steps + 1):
        dg.dg_adamw_step(dg.adamw_params(lr=0.0, beta2=b2, step=t, seed=1), T)
    root = adamw.decode(v[0].cpu().numpy(), e[1][0].cpu().numpy())
    want = 1e-2 * np.sqrt(1 - b2 ** steps)
    # sqrt is concave and the codes are spread by at most 1/8 around it: the mean lies within 5 percent
    assert abs(root.mean() / want - 1) < 0.05


def test_optimizer_object(dg):
    """AdamW over mixed types against the oracle's float64 path; parameters without gradients stay; states round
    trip through state_dict."""
    g = torch.Generator().manual_seed(0)
    base = [torch.randn(50, 40, generator=g), torch.randn(300, generator=g), torch.randn(10, generator=g)]

    def fresh():
        return [base[0].cuda(), base[1].bfloat16().cuda(), base[2].cuda()]

    ps = fresh()
    opt = dg.AdamW(ps, lr=LR, betas=(B1, B2), weight_decay=[0.1, 0.0, 0.1], state_bits=32, master=True)
    want = [b.double().numpy() for b in (base[0], base[1].bfloat16().float())]
    M, V = [np.zeros_like(w) for w in want], [np.zeros_like(w) for w in want]
    for t in range(1, 6):
        gr = [torch.randn(b.shape, generator=g) for b in base]
        opt.step([gr[0].cuda(), gr[1].bfloat16().cuda(), None])
        for i, wd in ((0, 0.1), (1, 0.0)):
            x = gr[i] if i == 0 else gr[i].bfloat16().float()
            want[i], M[i], V[i] = adamw.step(want[i], x.numpy(), M[i], V[i], t, LR, B1, B2, EPS, wd)
    assert np.abs(ps[0].cpu().double().numpy() - want[0]).max() <= 5 * 2.0 ** -22 * np.abs(want[0]).max()
    assert np.abs(ps[1].cpu().double().numpy() - want[1]).max() <= 2.0 ** -8 * np.abs(want[1]).max() * 1.01
    assert torch.equal(ps[2].cpu(), base[2])
    # resumed from a state_dict: the same bits as going on
    for bits in (8, 32):
        a, b = fresh(), fresh()
        one = dg.AdamW(a, lr=LR, state_bits=bits, seed=3)
        grads = [[torch.randn(x.shape, generator=g).to(x.dtype).cuda() for x in a] for _ in range(4)]
        for k in range(2):
            one.step(grads[k])
        two = dg.AdamW(b, lr=LR, state_bits=bits, seed=3)
        two.load_state_dict(one.state_dict())
        for x, y in zip(a, b):
            y.copy_(x)
        for k in range(2, 4):
            one.step(grads[k])
            two.step(grads[k])
        for x, y in zip(a, b):
            assert torch.equal(x, y)


def test_refusals_on_the_device(dg):
    def t(n, dtype=torch.float32):
        return torch.zeros(n, dtype=dtype, device="cuda")

    ok = ([t(300)], [t(300)], [t(300)], [t(300)])
    for bad in (([], [], [], []), ([t(300)], [t(299)], [t(300)], [t(300)]), ([t(300)], [t(300)], [t(299)], [t(300)]),
                ([t(300, torch.float16)], *ok[1:]), ([t(300)], [t(300, torch.float16)], *ok[2:]),
                ([torch.zeros(300)], *ok[1:]), (ok[0], [t(300).cpu()], *ok[2:]), ([t((20, 30)).t()], [t(600)], [t(600)], [t(600)])):
        with pytest.raises(dg.DgError):
            dg.AdamWTensors(*bad)
    x = t(300)
    with pytest.raises(dg.DgError):
        dg.AdamWTensors([x], [t(300)], [x], [t(300)])
    with pytest.raises(dg.DgError):
        dg.AdamWTensors([x[:200], x[100:]], [t(200)] * 2, [t(200), t(200)], [t(200), t(200)])
    with pytest.raises(dg.DgError):
        dg.AdamWTensors(*ok, m_exp=[t(2, torch.int8)])
    with pytest.raises(dg.DgError):
        dg.AdamWTensors([t(300)], [t(300)], [t(300, torch.uint8)], [t(300, torch.uint8)], m_exp=[t(1, torch.int8)],
                        v_exp=[t(2, torch.int8)])
    T = dg.AdamWTensors(*ok)
    for bad in (dict(lr=-1.0), dict(lr=float("nan")), dict(beta1=1.0), dict(beta2=-0.1), dict(eps=-1.0), dict(step=0),
                dict(stochastic=1), dict(stochastic=2)):
        with pytest.raises(dg.DgError):
            dg.dg_adamw_step(dg.adamw_params(**bad), T)
    with pytest.raises(dg.DgError):          # a master beside fp32 parameters
        dg.dg_adamw_step(dg.adamw_params(), dg.AdamWTensors(*ok[:2], [t(300)], [t(300)], master=[t(300)]))
