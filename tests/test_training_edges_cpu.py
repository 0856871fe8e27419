"""Refusals of the training entry points at the edges of what they document, without a GPU."""

import ctypes
import os
import re
import shutil
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def dg():
    from discrete_diffusion_decoding_b200 import build
    build.build()
    import discrete_diffusion_decoding_b200 as m
    return m


@pytest.mark.parametrize("order", [(0, 1), (1, 0)])
@pytest.mark.parametrize("count", [2, 30, 500])
def test_a_master_of_an_empty_tensor_asks_for_the_others(dg, order, count):
    """An empty tensor's master among tensors without one: refused like the mixture of tensors with elements, before
    the device is looked at."""
    from discrete_diffusion_decoding_b200._abi import DG_EINVAL, DgAdamWTensor, lib
    a = 1 << 20                               # never dereferenced
    p = dg.adamw_params(param_type=1, grad_type=1)
    empty = dict(param=a, grad=a, m=a, v=a, master=a, n=0)
    plain = dict(param=a, grad=a, m=a, v=a, n=8)
    table = (DgAdamWTensor * count)(*[DgAdamWTensor(**plain)] * count)
    for place, at in zip((empty, plain), (0, count - 1) if order == (0, 1) else (count - 1, 0)):
        table[at] = DgAdamWTensor(**place)
    assert lib().dg_adamw_step(ctypes.byref(p), table, count, None) == DG_EINVAL


def test_scalars_of_another_device_are_refused(dg):
    """The kernel reads them, so they lie where the tensors do."""
    z = [torch.zeros(5) for _ in range(4)]
    T = dg.AdamWTensors(z[:1], z[1:2], z[2:3], z[3:])
    T.device = torch.device("cuda", 0)
    p = dg.adamw_params()
    p.held = [torch.zeros(1, device="meta")]          # stands for a second CUDA device's
    with pytest.raises(dg.DgError, match="lr_dev, step_dev and grad_scale_dev"):
        dg.dg_adamw_step(p, T)


def test_gradients_and_states_have_their_parameters_shape(dg):
    """A [6, 4] gradient of a [4, 6] parameter is another parameter's; flat ones are read in its order."""
    def z(*shape):
        return torch.zeros(shape)

    for grad in (z(6, 4), z(24, 1), z(1, 4, 6)):
        with pytest.raises(dg.DgError):
            dg.AdamWTensors([z(4, 6)], [grad], [z(4, 6)], [z(4, 6)])
        T = dg.AdamWTensors([z(4, 6)], [None], [z(4, 6)], [z(24)])
        with pytest.raises(dg.DgError):
            T.set_grads([grad])
        assert T.table[0].n == 0
    opt = dg.AdamW([z(4, 6), z(6, 4)], state_bits=32)
    with pytest.raises(dg.DgError):
        opt.step([z(6, 4), z(4, 6)])
    assert opt.steps == 0
    with pytest.raises(dg.DgError):
        dg.AdamWTensors([z(4, 6)], [z(4, 6)], [z(6, 4)], [z(4, 6)])
    assert dg.AdamWTensors([z(4, 6)], [z(24)], [z(24)], [z(24)]).table[0].n == 24


def test_a_step_is_whole_or_not_at_all(dg, monkeypatch):
    """What one list's launch would refuse is refused before another list's launch."""
    from types import SimpleNamespace
    from discrete_diffusion_decoding_b200 import training
    launched = []
    real = training.lib()
    fake = SimpleNamespace(dg_adamw_step=lambda *a: launched.append(a) or 0,
                           dg_adamw_params_default=real.dg_adamw_params_default)
    monkeypatch.setattr(training, "lib", lambda: fake)
    monkeypatch.setattr(training, "_current_stream", lambda i: 0)
    monkeypatch.setattr(training, "_current_device", lambda: 0)
    monkeypatch.setattr(training, "_refuse_capture", lambda *a: None)
    ps = [torch.zeros(5), torch.zeros(5, dtype=torch.bfloat16)]

    def step(devices, stream=None):
        opt = dg.AdamW(ps)
        for (_, tensors), d in zip(opt.groups, devices):
            monkeypatch.setattr(tensors, "set_grads", lambda g, t=tensors: (
                setattr(t, "grads", g), setattr(t, "live", [0]), setattr(t, "updated", [])))
            tensors.device = torch.device(d)
        opt.step([torch.ones_like(p) for p in ps], stream=stream)
        return opt

    assert step(["cuda:0", "cuda:0"]).steps == 1 and len(launched) == 2
    launched.clear()
    with pytest.raises(dg.DgError):
        step(["cuda:0", "cpu"])
    with pytest.raises(dg.DgError):
        step(["cuda:0", "cuda:1"], SimpleNamespace(device=torch.device("cuda:0"), cuda_stream=0))
    assert not launched
    for decay in (float("nan"), float("inf"), 1e39, [0.0, -float("inf")]):
        with pytest.raises(dg.DgError):
            dg.AdamW(ps, weight_decay=decay)


def test_the_update_keeps_to_registers_but_for_a_few_words(tmp_path):
    """ptxas reports spills of the AdamW kernels only for bf16 parameters with 8-bit states, and at most 24 bytes."""
    nvcc = next((c for c in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc"))
                 if c and os.path.exists(c)), None)
    if nvcc is None:
        pytest.skip("nvcc not available")
    src = os.path.join(ROOT, "discrete_diffusion_decoding_b200", "csrc", "dg_adamw.cu")
    out = subprocess.run([nvcc, "-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-std=c++17", "-Xptxas", "-v", "-c",
                          "-o", str(tmp_path / "k.o"), src], capture_output=True, text=True, timeout=600)
    assert out.returncode == 0, out.stderr[-2000:]
    found = re.findall(r"Compiling entry function '(\S+)'.*?(\d+) bytes spill stores, (\d+) bytes spill loads",
                       out.stderr, re.S)
    assert len(found) == 24
    for name, *spills in found:
        # <parameter, gradient, 8-bit states, ...> as the name holds them: the parameter's type, then the first flag
        of_bf16 = "kernelI13__nv_bfloat16" in name
        state8 = name.split("Lb")[1][0] == "1"
        assert max(map(int, spills)) <= (24 if of_bf16 and state8 else 0), name


@pytest.mark.parametrize("eps", [1e-46, 1e-40, 2.0 ** -127])
def test_an_eps_below_the_normal_range_is_refused(dg, eps):
    """The quotient takes a subnormal denominator for 0: an element without moments would become 0 / 0."""
    from discrete_diffusion_decoding_b200._abi import DG_EINVAL, lib
    z = [torch.zeros(5) for _ in range(4)]
    p = dg.adamw_params(eps=eps, param_type=0, grad_type=0)
    T = dg.AdamWTensors(z[:1], z[1:2], z[2:3], z[3:])
    assert lib().dg_adamw_step(ctypes.byref(p), T.table, 1, None) == DG_EINVAL


def test_states_saved_without_counts(dg):
    """A state_dict from before each parameter had a count takes the step count for all; another number of counts is
    another optimizer's."""
    ps = [torch.zeros(5), torch.zeros(7, dtype=torch.bfloat16)]
    opt = dg.AdamW(ps)
    state = opt.state_dict()
    state["steps"] = 7
    saved = dict(state)
    del saved["counts"]
    opt.load_state_dict(saved)
    assert opt.steps == 7 and opt.counts == [7, 7]
    opt.load_state_dict(dict(state, counts=[7, 3]))
    assert opt.counts == [7, 3]
    with pytest.raises(dg.DgError):
        opt.load_state_dict(dict(state, counts=[7]))
