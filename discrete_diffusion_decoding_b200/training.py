"""Training the vocabulary head: its cross entropy with gradients, AdamW, and the loop that joins them.

Bindings over the training entry points of ``include/dg.h`` (``dg_xent_*``, ``dg_adamw_step``), which hold
the definitions.  Tensors are checked here (device, type, layout, size) and refused with :class:`DgError`;
every step runs in the library's sm_100a kernels, on the tensors' device and on ``stream`` or that device's
current stream.
"""

import ctypes
import math

import torch

from . import _abi
from ._abi import DgAdamWParams, DgAdamWTensor, DgError, DgXentParams, check, lib

# what the public forms of these do with a few microseconds of checks and objects around it: the handle of a device's
# current stream, the current device, and a count of a write in each of a list of tensors
_current_stream = torch._C._cuda_getCurrentRawStream
_current_device = getattr(torch._C, "_cuda_getDevice", None)
_count_writes = torch._C._increment_version

_TYPES = {torch.float32: _abi.DG_FP32, torch.bfloat16: _abi.DG_BF16}
_INDEX = {torch.int32: _abi.DG_INT32, torch.int64: _abi.DG_INT64}
BLOCK = 256       # elements of an 8-bit state that share an exponent


def _refuse(fn, why):
    raise DgError(fn, _abi.DG_EINVAL, why)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _tensor(fn, name, t, dtypes, shape, device):
    """Check one dense CUDA tensor of an entry point."""
    if not isinstance(t, torch.Tensor):
        _refuse(fn, f"{name} is not a tensor")
    if t.device != device or t.dtype not in dtypes or t.shape != shape or not t.is_contiguous():
        _refuse(fn, f"{name} is {'' if t.is_contiguous() else 'not contiguous, '}{t.dtype} {tuple(t.shape)} on {t.device}, "
                    f"expected dense {' or '.join(str(d) for d in dtypes)} {tuple(shape)} on {device}")


def _refuse_capture(fn, instead, stream=None):
    """Calls that count on the host: a graph would repeat the counts of its capture."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return _refuse_capture(fn, instead)
    if torch.cuda.is_available() and torch.cuda.is_current_stream_capturing():
        _refuse(fn, f"the stream is being captured; capture {instead}")


def _check_place(fn, device, stream):
    if device.index is None:      # host and meta tensors have none
        _refuse(fn, f"tensors are on {device}, expected a CUDA device")
    if stream is not None and stream.device != device:
        _refuse(fn, f"the stream is on {stream.device}, the tensors on {device}")


def _call(fn, device, stream, written, *args):
    """The library's entry point `fn` on `stream`, or the device's current stream, with the device made current.

    The tensors `written` count a write as torch's own in-place operations do, so that a backward which saved one
    of them refuses (a replay of a captured call is not counted).
    """
    index = device.index
    _check_place(fn, device, stream)
    handle = _current_stream(index) if stream is None else stream.cuda_stream
    if _current_device() == index:
        check(fn, getattr(lib(), fn)(*args, handle))
    else:
        with torch.cuda.device(device):
            check(fn, getattr(lib(), fn)(*args, handle))
    _count_writes(written)


_DEFAULTS = {}


def _params(struct, init, overrides):
    """A params struct with the library's defaults (init fills them, once a process) and the overrides."""
    if struct not in _DEFAULTS:
        p = struct()
        init(ctypes.byref(p))
        _DEFAULTS[struct] = p
    p = struct.from_buffer_copy(_DEFAULTS[struct])
    names = struct.NAMES
    for k, v in overrides.items():
        if k not in names:
            raise KeyError(k)
        setattr(p, k, v)
    return p


# ------------------------------------------------------------------ cross entropy
def xent_params(n, vocab, hidden, **overrides):
    """dg_xent_params for n positions of a [vocab, hidden] head (temperature 1, ignore_index -100).

    The types of targets and dW and the row stride of h are taken from the tensors of each call.
    """
    return _params(DgXentParams, lambda p: lib().dg_xent_params_default(p, 0, 1, 8),
                   dict(overrides, n=int(n), vocab=int(vocab), hidden=int(hidden)))


def xent_workspace_size(p, backward=True):
    size = lib().dg_xent_workspace_size(ctypes.byref(p), int(bool(backward)))
    if size == 0:
        raise DgError("dg_xent_workspace_size", _abi.DG_EINVAL, "invalid or unsupported params")
    return size


class XentWorkspace:
    """Device workspace of dg_xent_forward, and with `backward` of dg_xent_backward too."""

    def __init__(self, p, device="cuda", backward=True):
        device = torch.device(device)
        if device.type != "cuda":
            _refuse("XentWorkspace", f"{device} is not a CUDA device")
        with torch.cuda.device(device):
            self.nbytes = xent_workspace_size(p, backward)
            self.buf = torch.empty(self.nbytes, dtype=torch.uint8, device=device)


def _xent_inputs(fn, p, h, W, targets, ws):
    """A copy of p with the tensors' types and stride, after checking them."""
    if not isinstance(h, torch.Tensor) or h.device.type != "cuda":
        _refuse(fn, "h is not a CUDA tensor")
    dev = h.device
    if h.dtype != torch.bfloat16 or h.shape != (p.n, p.hidden):
        _refuse(fn, f"h is {h.dtype} {tuple(h.shape)}, expected torch.bfloat16 {(p.n, p.hidden)}")
    stride = h.stride(0) if p.n > 1 else p.hidden
    if (p.hidden > 1 and h.stride(1) != 1 and p.n > 0) or stride < p.hidden:
        _refuse(fn, f"h has strides {h.stride()}: rows must be dense and must not overlap")
    _tensor(fn, "W", W, (torch.bfloat16,), (p.vocab, p.hidden), dev)
    _tensor(fn, "targets", targets, (torch.int32, torch.int64), (p.n,), dev)
    if ws.buf.device != dev:
        _refuse(fn, f"the workspace is on {ws.buf.device}, the tensors on {dev}")
    q = DgXentParams.from_buffer_copy(p)
    q.h_stride = stride
    q.target_type = _INDEX[targets.dtype]
    return q, dev


def dg_xent_forward(p, h, W, targets, loss, lse, ws, stream=None):
    """Per-position cross entropy and log-sum-exp into loss and lse (float32 [n]; lse may be None)."""
    fn = "dg_xent_forward"
    q, dev = _xent_inputs(fn, p, h, W, targets, ws)
    _tensor(fn, "loss", loss, (torch.float32,), (p.n,), dev)
    if lse is not None:
        _tensor(fn, "lse", lse, (torch.float32,), (p.n,), dev)
    _call(fn, dev, stream, (loss,) if lse is None else (loss, lse), ctypes.byref(q), _ptr(h), _ptr(W), _ptr(targets),
          _ptr(loss), _ptr(lse), _ptr(ws.buf), ws.nbytes)


def dg_xent_backward(p, h, W, targets, loss, lse, dloss, dh, dW, ws, stream=None):
    """Gradients for dloss (float32 [n]): dh (bf16 like h, or None) and dW (bf16 or float32 like W, or None).

    loss and lse are the forward's.  p.dw_accumulate = 1 adds to dW instead of overwriting it.
    """
    fn = "dg_xent_backward"
    q, dev = _xent_inputs(fn, p, h, W, targets, ws)
    for name, t in (("loss", loss), ("lse", lse), ("dloss", dloss)):
        _tensor(fn, name, t, (torch.float32,), (p.n,), dev)
    if dh is not None:
        _tensor(fn, "dh", dh, (torch.bfloat16,), (p.n, p.hidden), dev)
    if dW is not None:
        _tensor(fn, "dW", dW, (torch.bfloat16, torch.float32), (p.vocab, p.hidden), dev)
        q.dw_type = _TYPES[dW.dtype]
    _call(fn, dev, stream, [t for t in (dh, dW) if t is not None], ctypes.byref(q), _ptr(h), _ptr(W), _ptr(targets),
          _ptr(loss), _ptr(lse), _ptr(dloss), _ptr(dh), _ptr(dW), _ptr(ws.buf), ws.nbytes)


class _HeadCrossEntropy(torch.autograd.Function):
    @staticmethod
    def forward(ctx, h, W, targets, temperature, ignore_index):
        p = xent_params(h.shape[0], W.shape[0], h.shape[1], temperature=temperature, ignore_index=ignore_index)
        loss = torch.empty(p.n, dtype=torch.float32, device=h.device)
        lse = torch.empty_like(loss)
        dg_xent_forward(p, h, W, targets, loss, lse, XentWorkspace(p, h.device, backward=False))
        ctx.save_for_backward(h, W, targets, loss, lse)
        ctx.params = p
        return loss

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dloss):
        h, W, targets, loss, lse = ctx.saved_tensors
        dh = torch.empty(h.shape, dtype=h.dtype, device=h.device) if ctx.needs_input_grad[0] else None
        dW = torch.empty_like(W) if ctx.needs_input_grad[1] else None
        dg_xent_backward(ctx.params, h, W, targets, loss, lse, dloss.contiguous(), dh, dW,
                         XentWorkspace(ctx.params, h.device, backward=True))
        return dh, dW, None, None, None


def head_cross_entropy(h, W, targets, temperature=1.0, ignore_index=-100):
    """Cross entropy of softmax(h W^T / temperature) at `targets`, per position, differentiable in h and W.

    h [..., d] bf16, W [V, d] bf16, targets [...] int32 or int64.  Returns float32 [...]: 0 where the target
    is ignore_index.  No logits are stored; weight or average the result as the objective asks.  dh and dW are
    bf16.  Both directions can be captured into a CUDA graph as any autograd function can: after a warm-up on
    the capturing stream, with no eager graph of the same leaves alive.
    """
    fn = "head_cross_entropy"
    if h.dim() < 1 or W.dim() != 2 or tuple(h.shape[:-1]) != tuple(targets.shape) or h.shape[-1] != W.shape[1]:
        _refuse(fn, f"shapes h {tuple(h.shape)}, W {tuple(W.shape)}, targets {tuple(targets.shape)}")
    rows = h.reshape(-1, h.shape[-1])
    if rows.stride(-1) != 1 or rows.stride(0) < rows.shape[1]:
        rows = rows.contiguous()          # broadcast or transposed hidden states
    loss = _HeadCrossEntropy.apply(rows, W, targets.reshape(-1).contiguous(), float(temperature), int(ignore_index))
    return loss.view(targets.shape)


# ------------------------------------------------------------------ AdamW
_SCALARS = (("lr_dev", torch.float32), ("step_dev", torch.int32), ("grad_scale_dev", torch.float32))


def adamw_params(**overrides):
    """dg_adamw_params (lr 1e-3, betas 0.9 / 0.999, eps 1e-8, step 1, rounding to nearest).

    lr_dev and grad_scale_dev (float32) and step_dev (int32) take one-element CUDA tensors that the kernel
    reads when it runs.  The types and state_bits are taken from the tensors of each call.
    """
    held = []
    for name, dtype in _SCALARS:
        t = overrides.get(name)
        if t is not None:
            if t.dtype != dtype or t.numel() != 1 or t.device.type != "cuda":
                _refuse("adamw_params", f"{name} must be a one-element {dtype} CUDA tensor")
            held.append(t)
            overrides[name] = t.data_ptr()
    p = _params(DgAdamWParams, lambda p: lib().dg_adamw_params_default(p), overrides)
    p.held = held         # the scalars' memory lives as long as p
    return p


class AdamWTensors:
    """The list of tensors of dg_adamw_step: parameters, gradients, states, and optionally 32-bit masters.

    m and v are float32 like the parameters, or uint8 codes beside m_exp and v_exp (int8, one for every 256
    elements); gradients and states have their parameter's shape or are flat.  `grads` may hold None for a tensor
    to leave out; set_grads renews them.  The tensors are held by this list; memory that is written must not
    overlap.
    """

    def __init__(self, params, grads, m, v, m_exp=None, v_exp=None, master=None, weight_decay=0.0):
        fn = "AdamWTensors"
        params = list(params)
        k = len(params)
        if k == 0:
            _refuse(fn, "no tensors")
        self.device = params[0].device
        self.n_tensors = k
        ptype = params[0].dtype
        bits8 = m_exp is not None
        if ptype not in _TYPES:
            _refuse(fn, f"parameters are {ptype}, expected float32 or bfloat16")
        if (v_exp is not None) != bits8:
            _refuse(fn, "m_exp and v_exp go together")
        lists = {"m": m, "v": v, "m_exp": m_exp, "v_exp": v_exp, "master": master}
        lists = {name: list(x) for name, x in lists.items() if x is not None}
        decay = [float(weight_decay)] * k if not hasattr(weight_decay, "__len__") else [float(x) for x in weight_decay]
        if any(len(x) != k for x in lists.values()) or len(decay) != k:
            _refuse(fn, "the lists differ in length")
        state = torch.uint8 if bits8 else torch.float32
        self.param_type, self.state_bits = _TYPES[ptype], 8 if bits8 else 32
        self.params, self.master = params, lists.get("master")
        self.held = [params] + list(lists.values())
        self.table = (DgAdamWTensor * k)()
        self.rows = list(self.table)          # views of it
        self.shapes, self.sizes = [p.shape for p in params], [p.numel() for p in params]
        self.at = [p.data_ptr() for p in params]
        spans = []
        for i, p in enumerate(params):
            _tensor(fn, f"parameter {i}", p, (ptype,), p.shape, self.device)
            n = self.sizes[i]
            row = self.rows[i]
            row.param, row.n, row.weight_decay = _ptr(p), n, decay[i]
            if not math.isfinite(row.weight_decay):          # as float32
                _refuse(fn, f"weight_decay {decay[i]} is not finite")
            spans.append((p.data_ptr(), n * p.element_size()))
            for name, x in lists.items():
                t = x[i]
                if name in ("m_exp", "v_exp"):
                    _tensor(fn, f"{name} {i}", t, (torch.int8,), (-(-n // BLOCK),), self.device)
                else:
                    dtype = torch.float32 if name == "master" else state
                    # as the parameter, or flat
                    _tensor(fn, f"{name} {i}", t, (dtype,), t.shape if t.shape == (n,) else p.shape, self.device)
                setattr(row, name, _ptr(t))
                spans.append((t.data_ptr(), t.numel() * t.element_size()))
        spans = sorted(s for s in spans if s[1])
        if any(a + size > b for (a, size), (b, _) in zip(spans, spans[1:])):
            _refuse(fn, "tensors that are written overlap")
        self.set_grads(grads)

    def set_grads(self, grads):
        """The gradients of the next steps (dense, of one type; None leaves its tensor as it is)."""
        fn = "AdamWTensors"
        grads = list(grads)
        if len(grads) != self.n_tensors:
            _refuse(fn, "the lists differ in length")
        gtype = None
        live = []                             # the places that a step takes
        for k, g in enumerate(grads):
            if g is None:
                continue
            if gtype is None:
                gtype = g.dtype
                if gtype not in _TYPES:
                    _refuse(fn, f"gradients are {gtype}, expected float32 or bfloat16")
            shape = g.shape
            if (g.dtype != gtype or g.device != self.device or not g.is_contiguous() or
                    shape != self.shapes[k] and shape != (self.sizes[k],)):
                _refuse(fn, f"gradient {g.dtype} {tuple(shape)} on {g.device} of a parameter {tuple(self.shapes[k])}: "
                            "expected dense gradients of one type, in their parameters' shapes or flat, on their "
                            "device")
            live.append(k)
        for row, g, n in zip(self.rows, grads, self.sizes):
            if g is None:
                row.grad, row.n = None, 0
            else:
                row.grad, row.n = g.data_ptr(), n
        self.grad_type = _TYPES[gtype or torch.float32]
        self.grads = grads
        self.live = live
        self._count_live()

    def select(self, places):
        """Let the next steps take these places alone, among those with a gradient, until set_grads."""
        for k in self.live:
            self.rows[k].n = 0
        for k in places:
            self.rows[k].n = self.sizes[k]
        self.live = places
        self._count_live()

    def _count_live(self):
        # what a step writes and autograd may have saved
        if len(self.live) == self.n_tensors:
            self.updated = self.params + (self.master or [])
        else:
            self.updated = [part[k] for part in (self.params, self.master) if part for k in self.live]


    def release_grads(self):
        """Drop the gradients; the next step needs set_grads first."""
        self.grads = None


def dg_adamw_step(p, tensors, stream=None):
    """One AdamW step of every tensor of an AdamWTensors list; p from adamw_params (p.step counts from 1)."""
    if tensors.grads is None:
        _refuse("dg_adamw_step", "the list's gradients were released: call set_grads first")
    for t in getattr(p, "held", ()):
        if t.device != tensors.device:
            _refuse("dg_adamw_step", f"lr_dev, step_dev and grad_scale_dev lie where the tensors do, on "
                                     f"{tensors.device}, not on {t.device}")
    q = DgAdamWParams.from_buffer_copy(p)     # p may be another thread's too, beside tensors of other types
    q.param_type, q.grad_type, q.state_bits = tensors.param_type, tensors.grad_type, tensors.state_bits
    _call("dg_adamw_step", tensors.device, stream, tensors.updated, ctypes.byref(q), tensors.table, tensors.n_tensors)


class AdamW:
    """AdamW over a list of dense float32 and bf16 tensors, states in 8 or 32 bits, one launch a step, type and count.

    bf16 parameters keep a 32-bit master copy (`master`) or are rounded at random without one; `weight_decay`
    is one value or one for each parameter.  Steps take the parameters' .grad, or the list given to step();
    a parameter without a gradient is left as it is, and its bias corrections count the steps that had one.  No
    gradient is held after the step.  The step counts live on the host, so a step is not captured into a graph:
    graphs take dg_adamw_step with step_dev and lr_dev.
    """

    def __init__(self, params, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.0, state_bits=8, master=False,
                 seed=0):
        self.params = list(params)
        if state_bits not in (8, 32):
            _refuse("AdamW", "state_bits must be 8 or 32")
        if hasattr(weight_decay, "__len__"):
            if len(weight_decay) != len(self.params):
                _refuse("AdamW", "weight_decay has another length than params")
            decay = list(weight_decay)
        else:
            decay = [weight_decay] * len(self.params)
        self.lr, self.betas, self.eps, self.seed, self.steps = lr, betas, eps, int(seed), 0
        self.counts = [0] * len(self.params)          # the steps that each parameter had a gradient in
        self.groups = []          # one for each parameter type: (places in params, list)
        for dtype in (torch.float32, torch.bfloat16):
            at = [i for i, p in enumerate(self.params) if p.dtype == dtype]
            if not at:
                continue
            ps = [self.params[i].detach() for i in at]

            def zeros(of, like=lambda p: p.shape):
                return [torch.zeros(like(p), dtype=of, device=p.device) for p in ps]

            bits8 = state_bits == 8
            blocks = lambda p: (-(-p.numel() // BLOCK),)     # noqa: E731
            self.groups.append((at, AdamWTensors(
                ps, [None] * len(ps), zeros(torch.uint8 if bits8 else torch.float32),
                zeros(torch.uint8 if bits8 else torch.float32), zeros(torch.int8, blocks) if bits8 else None,
                zeros(torch.int8, blocks) if bits8 else None,
                [p.float() for p in ps] if master and dtype == torch.bfloat16 else None, [decay[i] for i in at])))
        if sum(len(at) for at, _ in self.groups) != len(self.params):
            _refuse("AdamW", "parameters must be float32 or bfloat16")

    def step(self, grads=None, grad_scale=1.0, stream=None):
        _refuse_capture("AdamW.step", "dg_adamw_step with step_dev", stream)
        grads = [p.grad for p in self.params] if grads is None else list(grads)
        if len(grads) != len(self.params):
            _refuse("AdamW.step", "grads has another length than params")
        for at, tensors in self.groups:
            for i, where in zip(at, tensors.at):
                if self.params[i].data_ptr() != where:
                    _refuse("AdamW.step", f"parameter {i} lies elsewhere than when the optimizer was made")
        # a step is whole or not at all: what one list would refuse is refused before another one's launch
        for _, tensors in self.groups:
            _check_place("AdamW.step", tensors.device, stream)
        try:
            for at, tensors in self.groups:
                tensors.set_grads([grads[i] for i in at])
            for k, (at, tensors) in enumerate(self.groups):
                plain_bf16 = tensors.param_type == _abi.DG_BF16 and not tensors.table[0].master
                of = {}                               # count: the places in the list that it is of
                for j in tensors.live:
                    of.setdefault(self.counts[at[j]], []).append(j)
                for count, now in of.items():
                    if len(of) > 1:
                        tensors.select(now)
                    # a key of its own for each list, whose tensors count from 0
                    p = adamw_params(lr=self.lr, beta1=self.betas[0], beta2=self.betas[1], eps=self.eps,
                                     step=count + 1, grad_scale=grad_scale,
                                     seed=(self.seed + (k << 63)) & (1 << 64) - 1, stochastic=int(plain_bf16))
                    dg_adamw_step(p, tensors, stream)
                    for j in now:
                        self.counts[at[j]] = count + 1
        finally:
            for _, tensors in self.groups:
                tensors.release_grads()
        if stream is not None:
            # the caller may drop them too, while this stream still waits to read them
            for g in grads:
                if g is not None:
                    g.record_stream(stream)
        self.steps += 1

    def refresh_master(self):
        """Take the 32-bit master copies from the parameters again (after they were loaded or changed)."""
        for at, tensors in self.groups:
            for i, m in zip(at, tensors.master or ()):
                m.copy_(self.params[i].detach())

    def zero_grad(self):
        for p in self.params:
            p.grad = None

    def _states(self):
        return [x for _, t in self.groups for part in t.held[1:] for x in part]

    def state_dict(self):
        """The step counts and every state tensor (codes and exponents, or values, and masters)."""
        return {"steps": self.steps, "counts": list(self.counts), "states": [t.clone() for t in self._states()]}

    def load_state_dict(self, state):
        mine = self._states()
        counts = state.get("counts", [state["steps"]] * len(self.params))
        if (len(counts) != len(self.params) or len(mine) != len(state["states"]) or
                any(a.shape != b.shape or a.dtype != b.dtype for a, b in zip(mine, state["states"]))):
            _refuse("AdamW.load_state_dict", "the states are of other parameters or of another format")
        for a, b in zip(mine, state["states"]):
            a.copy_(b)
        self.steps, self.counts = int(state["steps"]), [int(c) for c in counts]


# ------------------------------------------------------------------ the head's training loop
class HeadTrainer:
    """Trains a vocabulary head W [V, d] (bf16) in place: cross entropy, its gradients, AdamW.

    accumulate(h, targets) adds the gradients of one batch and returns (loss, dh): the weighted mean loss as
    a device scalar and the hidden states' gradient, for a denoiser to go on with; update() applies AdamW;
    step() does both.  They count batches and steps on the host and are not captured into graphs (capture
    dg_xent_forward, dg_xent_backward and dg_adamw_step).  serving() gives the head in the layout that
    dg_denoise_step reads.

    The head's gradient dW is held in bf16 while a step is one batch, and in float32 from the first step that
    accumulates more: a bf16 sum drops what is below half a step of it.  grad_dtype fixes the type.
    """

    def __init__(self, W, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.0, state_bits=8, master=False,
                 grad_dtype=None, temperature=1.0, ignore_index=-100, seed=0):
        if W.dim() != 2 or W.dtype != torch.bfloat16 or not W.is_contiguous():
            _refuse("HeadTrainer", f"W is {W.dtype} {tuple(W.shape)}, expected a dense torch.bfloat16 [V, d]")
        if grad_dtype is not None and grad_dtype not in _TYPES:
            _refuse("HeadTrainer", f"grad_dtype is {grad_dtype}, expected bfloat16 or float32")
        self.W = W.detach()
        self.optimizer = AdamW([self.W], lr, betas, eps, weight_decay, state_bits, master, seed)
        self.dW = torch.empty(W.shape, dtype=grad_dtype or torch.bfloat16, device=W.device)
        self.widens = grad_dtype is None
        self.temperature, self.ignore_index = temperature, ignore_index
        self.batches = 0          # batches whose gradients dW holds
        self._ws = None           # the workspace of the largest batch so far

    def accumulate(self, h, targets, weight=None):
        """h [n, d] bf16, targets [n]; weight float32 [n] (1 where None): the loss is sum w loss / sum w over the
        positions whose target counts; elsewhere the weight may hold anything."""
        _refuse_capture("HeadTrainer.accumulate", "dg_xent_forward and dg_xent_backward")
        p = xent_params(targets.numel(), self.W.shape[0], self.W.shape[1], temperature=self.temperature,
                        ignore_index=self.ignore_index, dw_accumulate=int(self.batches > 0))
        with torch.cuda.device(self.W.device):
            size = xent_workspace_size(p)
        if self._ws is None or self._ws.nbytes < size:
            self._ws = XentWorkspace(p, self.W.device)
        # a larger batch renews it, and a second one dW, perhaps while another stream than their own works in them
        here = torch.cuda.current_stream(self.W.device)
        self._ws.buf.record_stream(here)
        self.dW.record_stream(here)
        loss = torch.empty(p.n, dtype=torch.float32, device=self.W.device)
        lse = torch.empty_like(loss)
        dg_xent_forward(p, h, self.W, targets, loss, lse, self._ws)
        kept = targets != self.ignore_index
        w = kept.float() if weight is None else torch.where(kept, weight, 0.0).float()
        dloss = torch.where(w != 0, w / w.sum(), 0)         # 0 also where nothing counts
        dh = torch.empty((p.n, p.hidden), dtype=torch.bfloat16, device=self.W.device)
        if self.batches > 0 and self.widens and self.dW.dtype != torch.float32:
            self.dW = self.dW.float()
        dg_xent_backward(p, h, self.W, targets, loss, lse, dloss, dh, self.dW, self._ws)
        self.batches += 1
        return torch.where(dloss != 0, dloss * loss, 0).sum(), dh

    def update(self):
        """AdamW on the mean of the accumulated batches' gradients."""
        if self.batches == 0:
            _refuse("HeadTrainer.update", "no gradients: call accumulate first")
        self.optimizer.step([self.dW], grad_scale=1.0 / self.batches)
        self.batches = 0

    def step(self, h, targets, weight=None):
        loss, dh = self.accumulate(h, targets, weight)
        self.update()
        return loss, dh

    def serving(self, form="rows"):
        """The head as the decode takes it: "rows" (W itself), "tiles" (params(head_layout=1)) or "e4m3"
        (codes and exponent of params(logits_format=1))."""
        from . import quantize_head_e4m3, tile_head
        if form == "rows":
            return self.W
        if form == "tiles":
            return tile_head(self.W)
        if form == "e4m3":
            return quantize_head_e4m3(self.W)
        raise ValueError(f"form must be rows, tiles or e4m3, not {form!r}")
