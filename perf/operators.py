"""The training operators' measured cases: the vocabulary head's cross entropy with its gradients, and the
AdamW step over many tensors.

`run` computes a case either with the library's kernels (`own` true) or in a plain form from elementary torch
operations (`own` false); `exact` gives the same outputs from the definitions in 64 bits.

Cross entropy of a head W [V, d] at positions with hidden states h [N, d] and target tokens y [N]:

    z[i, v] = (h_i . W_v) / T      lse_i = ln sum_v exp z[i, v]      loss_i = lse_i - z[i, y_i]
    G[i, v] = dloss_i / T (exp(z[i, v] - lse_i) - [v = y_i])         dh = G W        dW = G^T h

The sum over v is taken without the target's term, x_i = ln sum_{v != y_i} exp z[i, v], so that loss_i =
ln(1 + exp(x_i - z[i, y_i])) and G[i, y_i] = dloss_i / T (exp(-loss_i) - 1) keep their digits at positions that
the head is sure of.  A position whose target is the ignored index has loss 0, lse 0 and no part in the gradients, whatever its
hidden state holds.

AdamW with decoupled weight decay, step t, gradient g:

    m <- b1 m + (1 - b1) g     v <- b2 v + (1 - b2) g^2
    p <- p (1 - lr wd) - lr (m / (1 - b1^t)) / (sqrt(v / (1 - b2^t)) + eps)

States in 8 bits hold m and sqrt(v) of each tensor in blocks of 256 values as E4M3 codes times a power of two
per block: the exponent e is the smallest with max |x| 2^-e <= 448 (0 for a block of zeros, at least -100), and
x 2^-e is rounded between its two neighbouring E4M3 values at random, up with the probability of its distance
from the lower one (16 random bits); a positive sqrt(v) is never stored as 0.  bf16 parameters without a 32-bit
master copy round the same way.  The random words are Philox4x32-10 of (key: seed; counter: element / 4, step,
tensor, 5) for the states, low half for m and high half for sqrt(v), and (element / 8, step, tensor, 6) for the
parameters, where word j holds elements 2 j (low half) and 2 j + 1 (high half).
"""

import math

import torch

own = False

IGNORE = -100
BLOCK = 256
BETA1, BETA2, EPS, LR, DECAY = 0.9, 0.99, 1e-8, 1e-3, 0.1


def listed():
    return [
        # the loss of one token of the full head: scoring a single position, where the head's bytes count
        {"name": "loss 1 position", "op": "loss", "n": 1, "vocab": 262144, "hidden": 2816, "ignored": 0.0,
         "junk": False, "temperature": 1.0, "index": "int64"},
        # the evaluation loss of one canvas of 256 positions
        {"name": "loss canvas", "op": "loss", "n": 256, "vocab": 262144, "hidden": 2816, "ignored": 0.0,
         "junk": False, "temperature": 1.0, "index": "int32"},
        # the evaluation loss of a batch of eight canvases, where the products count
        {"name": "loss batch", "op": "loss", "n": 2048, "vocab": 262144, "hidden": 2816, "ignored": 0.0,
         "junk": False, "temperature": 0.8, "index": "int32"},
        # loss and gradients on a small head: launches and latency count
        {"name": "train small", "op": "train", "n": 256, "vocab": 4096, "hidden": 128, "ignored": 0.0,
         "junk": False, "temperature": 1.0, "index": "int32"},
        # a ragged batch on a head of odd size, a third of its positions padding with anything in it
        {"name": "train ragged", "op": "train", "n": 777, "vocab": 50021, "hidden": 1000, "ignored": 0.3,
         "junk": True, "temperature": 0.8, "index": "int64"},
        # one canvas on the full head: the head's gradient is written once
        {"name": "train canvas", "op": "train", "n": 256, "vocab": 262144, "hidden": 2816, "ignored": 0.0,
         "junk": False, "temperature": 1.0, "index": "int32"},
        # a training batch of 16 canvases on the full head
        {"name": "train batch", "op": "train", "n": 4096, "vocab": 262144, "hidden": 2816, "ignored": 0.0,
         "junk": False, "temperature": 1.0, "index": "int64"},
        # norms and biases alone: one small launch
        {"name": "adamw vectors", "op": "adamw", "tensors": 13, "largest": 2816, "param": "float32",
         "grad": "float32", "master": False, "bits": 32},
        # a 65536-token head in bf16 with a 32-bit copy and 32-bit states
        {"name": "adamw head 32", "op": "adamw", "tensors": 1, "largest": 65536 * 2816, "param": "bfloat16",
         "grad": "bfloat16", "master": True, "bits": 32},
        # the full head in bf16 alone with 8-bit states
        {"name": "adamw head 8", "op": "adamw", "tensors": 1, "largest": 262144 * 2816, "param": "bfloat16",
         "grad": "bfloat16", "master": False, "bits": 8},
        # a network's many tensors, small ones among them, in one call
        {"name": "adamw many 8", "op": "adamw", "tensors": 301, "largest": 512 * 2816, "param": "float32",
         "grad": "float32", "master": False, "bits": 8},
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["loss", "train", "train", "adamw", "adamw"])
    if op == "adamw":
        param = rng.choice(["float32", "bfloat16"])
        tensors = _log_uniform(rng, 1, 300)
        return {"op": op, "tensors": tensors, "largest": _log_uniform(rng, 100, 400_000_000 // tensors),
                "param": param, "grad": rng.choice(["float32", "bfloat16"]),
                "master": param == "bfloat16" and rng.random() < 0.5, "bits": rng.choice([8, 32])}
    vocab = _log_uniform(rng, 256, 262144)
    hidden = 8 * _log_uniform(rng, 8, 352)
    n = _log_uniform(rng, 1, min(16384, 4096 * 262144 // vocab))
    ignored = rng.choice([0.0, rng.uniform(0.05, 0.95)])
    return {"op": op, "n": n, "vocab": vocab, "hidden": hidden, "ignored": round(ignored, 3), "junk": ignored > 0,
            "temperature": rng.choice([1.0, 0.8, 0.4]), "index": rng.choice(["int32", "int64"])}


def work(case):
    if case["op"] == "adamw":
        n = sum(_sizes(case))
        size = {"float32": 4, "bfloat16": 2}
        param = 2 * size[case["param"]] + (8 if case["master"] else 0)
        if case["master"]:
            param -= size[case["param"]]          # the bf16 copy is only written
        state = 16 if case["bits"] == 32 else 4 + 4 / BLOCK
        return {"bytes": n * (param + size[case["grad"]] + state), "flops": 16 * n}
    n, v, d = case["n"], case["vocab"], case["hidden"]
    kept = n - int(n * case["ignored"])
    index = 4 if case["index"] == "int32" else 8
    read = 2 * v * d + 2 * kept * d + index * n
    if case["op"] == "loss":
        return {"bytes": read + 8 * n, "flops": 2 * kept * v * d}
    # the products of the loss, of the logits once more (they are not kept) and of the two gradients
    return {"bytes": read + 4 * n + 8 * n + 2 * n * d + 2 * v * d, "flops": 8 * kept * v * d}


def _sizes(case):
    """Element counts of the tensors: the largest first, then smaller and odd ones."""
    most, count = case["largest"], case["tensors"]
    out = [most]
    for k in range(1, count):
        out.append(max(1, [most // 2 + k % 7, most // 37 + k % 5, 1 + most // 1021, most - k % 3][k % 4]))
    return out


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] == "adamw":
        return _prepare_adamw(case, g, seed)
    n, v, d = case["n"], case["vocab"], case["hidden"]
    W = torch.empty((v, d), device="cuda", dtype=torch.bfloat16).normal_(0.0, 0.02, generator=g)
    target = torch.randint(0, v, (n,), device="cuda", generator=g)
    # hidden states that lean toward their target by different amounts: from a loss of ln V to a small one
    lean = torch.rand((n, 1), device="cuda", generator=g) * (14.0 / (4e-4 * d))
    h = torch.randn((n, d), device="cuda", generator=g) + lean * W[target].float()
    drop = int(n * case["ignored"])
    at = torch.randperm(n, device="cuda", generator=g)[:drop]
    target[at] = IGNORE
    if case["junk"]:
        h[at[0::3]] = math.nan
        h[at[1::3]] = math.inf
    # the gradient of a weighted mean over the positions kept
    dloss = (0.5 + torch.rand((n,), device="cuda", generator=g)) / max(1, n - drop)
    return {"case": dict(case), "h": h.to(torch.bfloat16), "W": W,
            "target": target.to(getattr(torch, case["index"])), "dloss": dloss}


def _prepare_adamw(case, g, seed):
    """Every tensor starts at a multiple of BLOCK in one flat buffer of its kind; what lies between is 0."""
    sizes = _sizes(case)
    blocks = [-(-n // BLOCK) for n in sizes]
    first = [0]
    for b in blocks:
        first.append(first[-1] + b)
    total = first[-1] * BLOCK
    block_first = torch.tensor(first[:-1], device="cuda")
    tensor = torch.repeat_interleave(torch.arange(len(sizes), device="cuda"), torch.tensor(blocks, device="cuda"))
    left = (torch.tensor(sizes, device="cuda")[tensor] -
            (torch.arange(first[-1], device="cuda") - block_first[tensor]) * BLOCK)
    live = torch.arange(BLOCK, device="cuda")[None, :] < left[:, None]

    def normal(std):
        return torch.empty((first[-1], BLOCK), device="cuda").normal_(0.0, std, generator=g)

    # blocks of different scale, as the gradients of common and rare tokens are
    spread = torch.exp(torch.empty((first[-1], 1), device="cuda").normal_(0.0, 1.0, generator=g))
    s = {"case": dict(case), "sizes": sizes, "first": first, "tensor": tensor, "block_first": block_first,
         "seed": seed, "t": 9,
         # matrices decay, vectors do not
         "decay": [DECAY if n > 4096 else 0.0 for n in sizes]}
    s["block_decay"] = torch.tensor(s["decay"], device="cuda")[tensor][:, None]
    p = normal(0.02).mul_(live)
    s["p"] = p.to(getattr(torch, case["param"])).view(total)
    if case["master"]:
        s["master"] = p.clone().view(total)
    del p
    s["g"] = normal(1e-3).mul_(spread).mul_(live).to(getattr(torch, case["grad"])).view(total)
    m = normal(2.5e-4).mul_(spread).mul_(live)
    root = normal(1e-3).abs_().add_(2e-4).mul_(spread).mul_(live)
    if case["bits"] == 32:
        s["m"], s["v"] = m.view(total), root.square_().view(total)
    else:
        for k, x in (("m", m), ("v", root)):
            e = _block_exponent(x)
            s[k + "_exp"] = e.view(-1).to(torch.int8)
            s[k] = (x * torch.exp2(-e.float())).to(torch.float8_e4m3fn).view(torch.uint8).view(total)
    return s


def run(state):
    op = state["case"]["op"]
    if own:
        return _own_adamw(state) if op == "adamw" else _own_head(state, op == "train")
    return _plain_adamw(state) if op == "adamw" else _plain_head(state, op == "train")


# ------------------------------------------------------------------ with the library's kernels
def _own_head(s, train):
    import discrete_diffusion_decoding_b200 as dg

    if "ws" not in s:      # kept from pass to pass, as a training loop keeps it
        n, d = s["h"].shape
        s["params"] = dg.xent_params(n, s["W"].shape[0], d, ignore_index=IGNORE,
                                     temperature=s["case"]["temperature"])
        s["ws"] = dg.XentWorkspace(s["params"], s["h"].device, backward=train)
    loss = torch.empty_like(s["dloss"])
    lse = torch.empty_like(s["dloss"])
    dg.dg_xent_forward(s["params"], s["h"], s["W"], s["target"], loss, lse, s["ws"])
    if not train:
        return {"loss": loss, "lse": lse}
    dh, dW = torch.empty_like(s["h"]), torch.empty_like(s["W"])
    dg.dg_xent_backward(s["params"], s["h"], s["W"], s["target"], loss, lse, s["dloss"], dh, dW, s["ws"])
    return {"loss": loss, "lse": lse, "dh": dh, "dW": dW}


def _own_adamw(s):
    import discrete_diffusion_decoding_b200 as dg

    if "table" not in s:   # the list of tensors, as an optimizer keeps it
        def views(key, per_block=False):
            if key not in s:
                return None
            if per_block:
                return [s[key][a:b] for a, b in zip(s["first"], s["first"][1:])]
            return [s[key][a * BLOCK:a * BLOCK + n] for a, n in zip(s["first"], s["sizes"])]

        s["table"] = dg.AdamWTensors(views("p"), views("g"), views("m"), views("v"),
                                     m_exp=views("m_exp", True), v_exp=views("v_exp", True),
                                     master=views("master"), weight_decay=s["decay"])
    s["t"] += 1
    dg.dg_adamw_step(dg.adamw_params(lr=LR, beta1=BETA1, beta2=BETA2, eps=EPS, step=s["t"], seed=s["seed"],
                                     stochastic=s["case"]["param"] == "bfloat16" and not s["case"]["master"]),
                     s["table"])
    return _adamw_outputs(s)


def _adamw_outputs(s):
    if s["case"]["bits"] == 32:
        return {k: s[k] for k in ("p", "m", "v", "master") if k in s}
    out = {k: s[k] for k in ("p", "master", "m_exp", "v_exp") if k in s}
    out["m"] = s["m"].view(torch.float8_e4m3fn)       # in units of the block's power of two
    out["v"] = s["v"].view(torch.float8_e4m3fn)
    return out


# ------------------------------------------------------------------ plain forms
def _plain_head(s, train):
    T = s["case"]["temperature"]
    kept = s["target"] != IGNORE
    y = torch.where(kept, s["target"], 0).long()
    h = torch.where(kept[:, None], s["h"], 0).float()
    W = s["W"].float()
    z = (h @ W.T) / T
    row = torch.arange(len(y), device=y.device)
    picked = z[row, y]
    z[row, y] = -math.inf
    top = z.amax(1)
    others = top + torch.log(torch.exp(z - top[:, None]).sum(1))
    gap = others - picked
    loss = gap.clamp(min=0) + torch.log1p(torch.exp(-gap.abs()))
    lse = picked + loss
    out = {"loss": torch.where(kept, loss, 0), "lse": torch.where(kept, lse, 0)}
    if train:
        G = torch.exp(z - lse[:, None])
        G[row, y] = torch.expm1(-loss)
        G *= (torch.where(kept, s["dloss"], 0) / T)[:, None]
        out["dh"] = (G @ W).to(s["h"].dtype)
        out["dW"] = (G.T @ h).to(s["W"].dtype)
    return out


def _block_exponent(x):
    """The smallest e with max |x| 2^-e <= 448, for each row of x; 0 for a row of zeros, at least -100."""
    f, k = torch.frexp(x.abs().amax(1, keepdim=True))       # f in [1/2, 1), 448 = 0.875 2^9
    e = (k - 9 + (f > 0.875)).clamp_(min=-100)
    return torch.where(f == 0, 0, e)


def _philox(counter, seed):
    """The four words of Philox4x32-10 (Salmon et al., SC'11) for counter words given as int64 tensors."""
    low = 0xFFFFFFFF
    k0, k1 = seed & low, seed >> 32 & low
    a, b, c, d = counter
    for _ in range(10):
        p0, p1 = a * 0xD2511F53, c * 0xCD9E8D57
        a, b, c, d = (p1 >> 32 & low) ^ b ^ k0, p1 & low, (p0 >> 32 & low) ^ d ^ k1, p0 & low
        k0, k1 = k0 + 0x9E3779B9 & low, k1 + 0xBB67AE85 & low
    return a, b, c, d


def _random_halves(s, per, tag):
    """[blocks, BLOCK / per, 4] random words: one counter for each `per` elements."""
    count = BLOCK // per
    block = torch.arange(len(s["tensor"]), device="cuda") - s["block_first"][s["tensor"]]
    q = block[:, None] * count + torch.arange(count, device="cuda")
    words = _philox((q, torch.full_like(q, s["t"]), s["tensor"][:, None].expand_as(q), torch.full_like(q, tag)),
                    s["seed"])
    return torch.stack(words, -1)


def _round_e4m3(y, u):
    """E4M3 codes of y in [0, 448], rounded up where the discarded part exceeds what the 16 bits u say."""
    small = y < 2.0 ** -6
    bits = torch.where(small, y + 2.0 ** -6, y).view(torch.int32) + (u << 4)
    return (bits >> 20) - torch.where(small, 968, 960)


def _plain_adamw(s):
    s["t"] += 1
    t, case = s["t"], s["case"]
    rows = (-1, BLOCK)
    g = s["g"].view(rows).float()
    if case["bits"] == 32:
        m, v = s["m"].view(rows), s["v"].view(rows)
    else:
        scale = {k: torch.exp2(s[k + "_exp"].float())[:, None] for k in ("m", "v")}
        m = s["m"].view(torch.float8_e4m3fn).view(rows).float() * scale["m"]
        v = (s["v"].view(torch.float8_e4m3fn).view(rows).float() * scale["v"]).square()
    m = m * BETA1 + g * (1 - BETA1)
    v = v * BETA2 + g * g * (1 - BETA2)
    p = s["master" if case["master"] else "p"].view(rows).float()
    step = m * (LR / (1 - BETA1 ** t)) / (v.sqrt() * (1 / math.sqrt(1 - BETA2 ** t)) + EPS)
    p = p * (1 - LR * s["block_decay"]) - step
    del step, g
    if case["master"]:
        s["master"].copy_(p.view(-1))
    if case["param"] == "bfloat16" and not case["master"]:
        words = _random_halves(s, 8, 6)
        u = torch.stack((words & 0xFFFF, words >> 16), -1).view(rows).to(torch.int32)
        del words
        p = ((p.view(torch.int32) + u) >> 16 << 16).view(torch.float32)
        del u
    s["p"].copy_(p.view(-1))
    del p
    if case["bits"] == 32:
        s["m"].copy_(m.view(-1))
        s["v"].copy_(v.view(-1))
        return _adamw_outputs(s)
    words = _random_halves(s, 4, 5).view(rows)
    e = _block_exponent(m)
    code = _round_e4m3(m.abs() * torch.exp2(-e.float()), (words & 0xFFFF).to(torch.int32))
    s["m"].copy_((code | (m < 0).to(torch.int32) << 7).view(-1))
    s["m_exp"].copy_(e.view(-1))
    root = v.sqrt_()
    e = _block_exponent(root)
    code = _round_e4m3(root * torch.exp2(-e.float()), (words >> 16).to(torch.int32))
    s["v"].copy_(torch.where(root > 0, code.clamp_(min=1), code).view(-1))
    s["v_exp"].copy_(e.view(-1))
    return _adamw_outputs(s)


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return _exact_adamw(s) if case["op"] == "adamw" else _exact_head(s, case["op"] == "train")


def _exact_head(s, train):
    keep = torch.nonzero(s["target"] != IGNORE)[:, 0]
    y = s["target"][keep].to(torch.int64)
    h = s["h"][keep].double()
    W = s["W"].double()
    T = s["case"]["temperature"]
    n = s["h"].shape[0]
    z = torch.addmm(torch.zeros((), dtype=torch.float64, device=h.device), h, W.T, alpha=1.0 / T)
    at = (torch.arange(len(y), device=y.device), y)
    picked = z[at]
    z[at] = -math.inf
    others = torch.logsumexp(z, 1)
    loss = torch.logaddexp(others - picked, torch.zeros_like(picked))
    lse = picked + loss

    def spread(x):
        full = torch.zeros((n,) + x.shape[1:], dtype=torch.float64, device=x.device)
        full[keep] = x
        return full

    out = {"loss": spread(loss), "lse": spread(lse)}
    if not train:
        return out
    weight = s["dloss"][keep].double() / T
    z.sub_(lse[:, None]).exp_()
    z[at] = torch.expm1(-loss)
    z.mul_((s["dloss"][keep].double() / T)[:, None])
    dh, dW = z @ W, z.T @ h
    out["dh"], out["dW"] = spread(dh), dW
    return out


def _exact_adamw(s):
    """Tensor by tensor, in pieces of whole blocks."""
    case, t = s["case"], s["t"] + 1
    out = {k: torch.zeros_like(s[k], dtype=torch.float64) for k in ("p", "m", "v")}
    if case["master"]:
        out["master"] = torch.zeros_like(s["master"], dtype=torch.float64)
    if case["bits"] == 8:
        out["m_exp"] = out["v_exp"] = None
    piece = 1 << 17
    for a in range(0, len(s["tensor"]), piece):
        b = min(len(s["tensor"]), a + piece)
        at = slice(a * BLOCK, b * BLOCK)
        owner = s["tensor"][a:b]
        inside = (torch.arange(a, b, device="cuda") - s["block_first"][owner])[:, None] * BLOCK
        element = inside + torch.arange(BLOCK, device="cuda")
        g = s["g"][at].double()
        if case["bits"] == 32:
            m, v = s["m"][at].double(), s["v"][at].double()
        else:
            def decoded(k):
                x = s[k][at].view(torch.float8_e4m3fn).double().view(-1, BLOCK)
                return torch.ldexp(x, s[k + "_exp"][a:b, None].to(torch.int32)).view(-1)
            m, v = decoded("m"), decoded("v") ** 2
        m = BETA1 * m + (1 - BETA1) * g
        v = BETA2 * v + (1 - BETA2) * g * g
        p = s["master" if case["master"] else "p"][at].double()
        decay = s["block_decay"][a:b].double().expand(-1, BLOCK).reshape(-1)
        p = p - LR * decay * p - LR * (m / (1 - BETA1 ** t)) / ((v / (1 - BETA2 ** t)).sqrt() + EPS)
        if case["master"]:
            out["master"][at] = p
        if case["param"] == "bfloat16" and not case["master"]:
            u = _exact_random(s, owner, element, 8, 6, t)
            step = torch.ldexp(torch.ones_like(p), torch.frexp(p)[1] - 8)     # spacing of the 8-bit significands
            p = torch.sign(p) * torch.floor(p.abs() / step + u / 65536) * step
        out["p"][at] = p
        if case["bits"] == 32:
            out["m"][at], out["v"][at] = m, v
            continue
        for k, x, high in (("m", m, False), ("v", v.sqrt(), True)):
            x = x.view(-1, BLOCK)
            peak = x.abs().amax(1, keepdim=True)
            e = torch.where(peak > 0, torch.ceil(torch.log2(peak / 448)).clamp(min=-100), 0.0)
            y = x.abs() / torch.exp2(e)
            step = torch.exp2(torch.floor(torch.log2(y.clamp(min=2.0 ** -6))) - 3)
            u = _exact_random(s, owner, element, 4, 5, t, high).view(-1, BLOCK)
            q = torch.floor(y / step + u / 65536) * step
            if k == "v":
                q = torch.where(x > 0, q.clamp(min=2.0 ** -9), q)
            out[k][at] = (torch.sign(x) * q).view(-1)
    return out


def _exact_random(s, owner, element, per, tag, t, high=False):
    """The 16 random bits of each element, one counter for one element at a time."""
    lane = element % per
    words = _philox((element // per, torch.full_like(element, t), owner[:, None].expand_as(element),
                     torch.full_like(element, tag)), s["seed"])
    words = torch.stack(words, -1)
    word = words.gather(-1, (lane if per == 4 else lane // 2)[..., None])[..., 0]
    upper = torch.full_like(lane, int(high)) if per == 4 else lane % 2
    return (word >> 16 * upper & 0xFFFF).view(-1).double()
