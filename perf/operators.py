"""The vocabulary head's operators: what is measured, and their plain form.

Three operators, the life of a language model's vocabulary head: the softmax
cross entropy of the head's logits with its gradient (training), the AdamW step
(training), and the product in 8-bit integers with scales for each token and
each channel (serving).  `listed()` gives the cases, `prepare` a user's data,
`run` one pass (the plain form in elementary torch operations in 32 bits, or
the framework's kernels where `own` is true), `exact` the same values from the
definitions in 64 bits.
"""
import math

import torch

own = False

IGNORE = -100          # label of a position that carries no loss
BLOCK = 256            # elements that share one scale of an 8-bit AdamW state
LR, BETA1, BETA2, EPS, DECAY, STEP = 1e-3, 0.9, 0.95, 1e-8, 0.1, 100
TYPES = {"bfloat16": torch.bfloat16, "float16": torch.float16, "float32": torch.float32}
SIZE = {"bfloat16": 2, "float16": 2, "float32": 4}


def listed():
    return [
        # the log-probability of one token: the head's weights are read once
        {"name": "score_one_token", "op": "xent", "n": 1, "k": 1024, "v": 32000, "dtype": "bfloat16", "masked": 0.0, "train": False},
        # a few hundred tokens scored, no size a multiple of a tile
        {"name": "score_odd", "op": "xent", "n": 333, "k": 1000, "v": 50021, "dtype": "float16", "masked": 0.0, "train": False},
        # a small model's training step: latency counts
        {"name": "train_small", "op": "xent", "n": 256, "k": 512, "v": 8192, "dtype": "bfloat16", "masked": 0.0, "train": True},
        # instruction tuning: two fifths of the positions are prompt and carry no loss
        {"name": "train_masked", "op": "xent", "n": 2047, "k": 1536, "v": 32003, "dtype": "float16", "masked": 0.4, "train": True},
        # a training step's whole micro-batch
        {"name": "train_large", "op": "xent", "n": 4096, "k": 4096, "v": 65536, "dtype": "bfloat16", "masked": 0.0, "train": True},
        # decoding one token through a projection
        {"name": "i8_token", "op": "i8", "m": 1, "k": 4096, "n": 4096, "dtype": "bfloat16", "out": "bfloat16", "bias": False},
        # a dozen streams decoded at once through the head
        {"name": "i8_streams", "op": "i8", "m": 12, "k": 2048, "n": 32000, "dtype": "float16", "out": "float32", "bias": False},
        # a short prompt, odd sizes, a bias
        {"name": "i8_prompt_odd", "op": "i8", "m": 205, "k": 1777, "n": 5003, "dtype": "float32", "out": "float32", "bias": True},
        # prefill of a long batch
        {"name": "i8_prefill", "op": "i8", "m": 8192, "k": 4096, "n": 16384, "dtype": "bfloat16", "out": "bfloat16", "bias": False},
        # an adapter's parameters: many small tensors
        {"name": "adamw_small", "op": "adamw", "tensors": 24, "numel": 300001, "bits": 32, "param": "float32", "grad": "float32"},
        # a head and its trunk in 32-bit states, gradients in bfloat16
        {"name": "adamw_large", "op": "adamw", "tensors": 60, "numel": 268435457, "bits": 32, "param": "float32", "grad": "bfloat16"},
        # the same with 8-bit states and bfloat16 parameters
        {"name": "adamw_8bit", "op": "adamw", "tensors": 37, "numel": 150000001, "bits": 8, "param": "bfloat16", "grad": "bfloat16"},
    ]


def _between(rng, lo, hi):
    """A whole number, its logarithm uniform in [log lo, log hi]."""
    size = max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))
    return size - (size == 3072)


def _width(rng, hi):
    """An inner size: most are 4, 5 or 7 times a power of two, as models have them, the others any."""
    if rng.random() < 0.4:
        return _between(rng, 64, hi)
    return min(hi, rng.choice((4, 5, 7)) << rng.randint(4, 10))


def draw(rng):
    op = rng.choice(("xent", "xent", "i8", "i8", "adamw"))
    if op == "xent":
        c = {"op": op, "n": _between(rng, 1, 4096), "k": _width(rng, 4096), "v": _between(rng, 500, 65536),
             "dtype": rng.choice(("bfloat16", "float16")), "masked": rng.choice((0.0, 0.25, 0.6)), "train": rng.random() < 0.6}
        return c
    if op == "i8":
        c = {"op": op, "m": _between(rng, 1, 8192), "k": _width(rng, 8192), "n": _between(rng, 64, 16384),
             "dtype": rng.choice(("bfloat16", "float16", "float32")), "out": rng.choice(("bfloat16", "float16", "float32")),
             "bias": rng.random() < 0.5}
        while c["m"] * c["k"] * c["n"] > 8192 * 4096 * 16384:
            c["m"] = c["m"] // 2 + 1
        return c
    return {"op": op, "tensors": _between(rng, 1, 200), "numel": _between(rng, 20000, 150000000), "bits": rng.choice((8, 32)),
            "param": rng.choice(("float32", "bfloat16")), "grad": rng.choice(("float32", "bfloat16"))}


def _sizes(case):
    """The tensors' sizes: every other one a short vector, the rest share what is left unevenly."""
    t, left, sizes = case["tensors"], case["numel"], []
    for i in range(t):
        vector = i % 2 == 1
        n = min(1000 + 37 * i, left // (2 * t) + 1) if vector else left // max(1, (t - i + 1) // 2)
        n = max(1, min(n, left - (t - i - 1))) if i < t - 1 else left
        sizes.append(n)
        left -= n
    return sizes


def _spread(g, *shape):
    """Normal values whose columns differ in size, a few of them by much, as activations do."""
    x = torch.randn(*shape, generator=g, device="cuda")
    size = torch.exp(0.5 * torch.randn(shape[-1], generator=g, device="cuda"))
    size[torch.rand(shape[-1], generator=g, device="cuda") < 0.01] *= 8
    return x.mul_(size)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case)
    if case["op"] == "xent":
        n, k, v, dt = case["n"], case["k"], case["v"], TYPES[case["dtype"]]
        s["h"] = torch.randn(n, k, generator=g, device="cuda").to(dt)
        s["w"] = torch.randn(v, k, generator=g, device="cuda").mul_(2.0 / math.sqrt(k)).to(dt)
        # labels: low numbers are frequent words
        s["labels"] = (v ** torch.rand(n, generator=g, device="cuda", dtype=torch.float64)).long().clamp_(max=v - 1)
        masked = torch.rand(n, generator=g, device="cuda") < case["masked"]
        s["labels"][masked] = IGNORE
        valid = s["labels"] != IGNORE
        # the gradient of the mean over the positions that count
        s["grad"] = valid.float() / valid.sum().clamp(min=1)
    elif case["op"] == "i8":
        m, k, n = case["m"], case["k"], case["n"]
        s["x"] = _spread(g, m, k).to(TYPES[case["dtype"]])
        w = torch.randn(n, k, generator=g, device="cuda").mul_(1.0 / math.sqrt(k))
        s["w_scale"] = w.abs().amax(1) / torch.full((n,), 127.0, device="cuda")
        s["w"] = torch.round(w / s["w_scale"][:, None]).to(torch.int8)
        s["b"] = torch.randn(n, generator=g, device="cuda") if case["bias"] else None
    else:
        sizes = _sizes(case)
        starts, total = [], 0
        for n in sizes:  # every tensor starts on a block of its own in storage that they share
            starts.append(total)
            total += -(-n // BLOCK) * BLOCK
        keep = torch.zeros(total, dtype=torch.bool, device="cuda")
        for a, n in zip(starts, sizes):
            keep[a:a + n] = True
        rand = lambda scale: torch.randn(total, generator=g, device="cuda").mul_(scale).mul_(keep)  # noqa: E731
        s["p"] = rand(0.02).to(TYPES[case["param"]])
        # rows of a gradient differ in size by orders of magnitude
        size = torch.exp(2.0 * torch.randn(total // BLOCK, generator=g, device="cuda")).repeat_interleave(BLOCK)
        s["g"] = rand(1e-3).mul_(size).to(TYPES[case["grad"]])
        m, v = rand(3e-4).mul_(size), rand(1e-3).mul_(size).square_().add_(1e-12 * keep)
        if case["bits"] == 32:
            s["m"], s["v"] = m, v
        else:
            s["m"], s["m_scale"], s["v"], s["v_scale"] = _encode(m, v)
        views = lambda x: [x[a:a + n] for a, n in zip(starts, sizes)]  # noqa: E731
        s["params"], s["grads"], s["ms"], s["vs"] = views(s["p"]), views(s["g"]), views(s["m"]), views(s["v"])
        if case["bits"] == 8:
            blocks = lambda x: [x[a // BLOCK:a // BLOCK - (-n // BLOCK)] for a, n in zip(starts, sizes)]  # noqa: E731
            s["m_scales"], s["v_scales"] = blocks(s["m_scale"]), blocks(s["v_scale"])
    return s


def _encode(m, v):
    """The 8-bit states of moments m and v: codes, and the largest magnitude of each block."""
    m, v = m.view(-1, BLOCK), v.view(-1, BLOCK)
    am, av = m.abs().amax(1), v.amax(1)
    dm, dv = torch.where(am > 0, am, 1.0)[:, None], torch.where(av > 0, av, 1.0)[:, None]
    cm = torch.round(torch.sqrt(m.abs() / dm) * 127.0) * torch.sign(m)
    cv = torch.round(torch.sqrt(torch.sqrt(v / dv)) * 255.0)
    cv = torch.where(v > 0, cv.clamp(min=1.0), cv)
    return cm.to(torch.int8).view(-1), am, cv.to(torch.uint8).view(-1), av


def _decode(cm, am, cv, av):
    a, b = cm.view(-1, BLOCK).float() * (1.0 / 127.0), cv.view(-1, BLOCK).float() * (1.0 / 255.0)
    b = b * b
    return (am[:, None] * (a * a.abs())).view(-1), (av[:, None] * (b * b)).view(-1)


def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import rns_emulated_fp64_gb300 as os2
    if s["op"] == "xent":
        loss, lse = os2.xent(s["h"], s["w"], s["labels"], ignore_index=IGNORE)
        if not s["train"]:
            return {"loss": loss, "lse": lse}
        dh, dw = os2.xent_backward(s["h"], s["w"], s["labels"], lse, s["grad"], ignore_index=IGNORE)
        return {"loss": loss, "lse": lse, "dh": dh, "dw": dw}
    if s["op"] == "i8":
        return {"y": os2.i8linear(s["x"], s["w"], s["w_scale"], bias=s["b"], out_dtype=TYPES[s["out"]])}
    scales = {} if s["bits"] == 32 else {"exp_avg_scales": s["m_scales"], "exp_avg_sq_scales": s["v_scales"]}
    os2.adamw(s["params"], s["grads"], s["ms"], s["vs"], step=STEP, lr=LR, beta1=BETA1, beta2=BETA2, eps=EPS,
              weight_decay=DECAY, **scales)
    if s["bits"] == 32:
        return {"p": s["p"], "m": s["m"], "v": s["v"]}
    m, v = os2.adamw_moments(s["m"], s["m_scale"], s["v"], s["v_scale"])
    return {"p": s["p"], "m": m, "v": v}


def _run_plain(s):
    if s["op"] == "xent":
        h, w, y = s["h"].float(), s["w"].float(), s["labels"]
        z = h @ w.t()
        top = z.amax(1, keepdim=True)
        lse = torch.log(torch.exp(z - top).sum(1)) + top[:, 0]
        valid = y != IGNORE
        at = torch.where(valid, y, 0)[:, None]
        loss = torch.where(valid, lse - z.gather(1, at)[:, 0], 0.0)
        lse = torch.where(valid, lse, 0.0)
        if not s["train"]:
            return {"loss": loss, "lse": lse}
        d = torch.exp(z - lse[:, None])
        d.scatter_add_(1, at, torch.full_like(d[:, :1], -1.0))
        d = torch.where(valid[:, None], d * s["grad"][:, None], 0.0)
        return {"loss": loss, "lse": lse, "dh": (d @ w).to(s["h"].dtype), "dw": (d.t() @ h).to(s["w"].dtype)}
    if s["op"] == "i8":
        x = s["x"].float()
        top = x.abs().amax(1)
        scale = top / torch.full_like(top, 127.0)
        q = torch.round(x / torch.where(scale > 0, scale, 1.0)[:, None]).clamp(-127.0, 127.0)
        y = (q @ s["w"].float().t()) * scale[:, None] * s["w_scale"][None, :]
        if s["b"] is not None:
            y = y + s["b"]
        return {"y": y.to(TYPES[s["out"]])}
    p, g = s["p"].float(), s["g"].float()
    m, v = (s["m"], s["v"]) if s["bits"] == 32 else _decode(s["m"], s["m_scale"], s["v"], s["v_scale"])
    m = m * BETA1 + g * (1.0 - BETA1)
    v = v * BETA2 + (g * g) * (1.0 - BETA2)
    c1, c2 = 1.0 / (1.0 - BETA1 ** STEP), 1.0 / (1.0 - BETA2 ** STEP)
    p = p * (1.0 - LR * DECAY) - (m * (LR * c1)) / (torch.sqrt(v * c2) + EPS)
    s["p"].copy_(p)
    if s["bits"] == 32:
        s["m"].copy_(m)
        s["v"].copy_(v)
        return {"p": s["p"], "m": s["m"], "v": s["v"]}
    cm, am, cv, av = _encode(m, v)
    s["m"].copy_(cm)
    s["m_scale"].copy_(am)
    s["v"].copy_(cv)
    s["v_scale"].copy_(av)
    m, v = _decode(s["m"], s["m_scale"], s["v"], s["v_scale"])
    return {"p": s["p"], "m": m, "v": v}


def work(case):
    """Inputs read once, outputs written once; the products that the definitions have.

    The gradient needs the logits' product once more or the logits kept, so the
    three products of a training step are counted once each.  Positions without
    a loss need no products.
    """
    if case["op"] == "xent":
        n, k, v, e = case["n"], case["k"], case["v"], SIZE[case["dtype"]]
        rows = n * (1.0 - case["masked"])
        b = e * (rows * k + v * k) + 8 * n + 8 * n
        if case["train"]:
            return {"bytes": b + e * (n * k + v * k) + 4 * n, "flops": 6.0 * rows * v * k}
        return {"bytes": b, "flops": 2.0 * rows * v * k}
    if case["op"] == "i8":
        m, k, n = case["m"], case["k"], case["n"]
        b = SIZE[case["dtype"]] * m * k + n * k + 4 * n + SIZE[case["out"]] * m * n + (4 * n if case["bias"] else 0)
        return {"bytes": b, "flops": 2.0 * m * k * n}
    n, p, g = case["numel"], SIZE[case["param"]], SIZE[case["grad"]]
    if case["bits"] == 32:
        return {"bytes": n * (2 * p + g + 16), "flops": 15.0 * n}
    # 8-bit states read and written, and the moments returned as values
    return {"bytes": n * (2 * p + g + 4 + 8) + n / BLOCK * 16, "flops": 40.0 * n}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "xent":
        rows = (s["labels"] >= 0).nonzero()[:, 0]
        out = {key: torch.zeros(case["n"], dtype=torch.float64, device="cuda") for key in ("loss", "lse")}
        w = s["w"].double()
        if case["train"]:
            out["dh"] = torch.zeros(case["n"], case["k"], dtype=torch.float64, device="cuda")
            out["dw"] = torch.zeros_like(w)
        for part in rows.split(1024):
            h, y = s["h"][part].double(), s["labels"][part]
            z = torch.matmul(h, w.T)
            lse = torch.logsumexp(z, dim=1)
            out["lse"][part] = lse
            out["loss"][part] = lse - z[torch.arange(len(part), device="cuda"), y]
            if case["train"]:
                z = z.sub_(lse[:, None]).exp_()
                z[torch.arange(len(part), device="cuda"), y] -= 1.0
                z *= s["grad"][part].double()[:, None]
                out["dh"][part] = torch.matmul(z, w)
                out["dw"].addmm_(z.T, h)
        return out
    if case["op"] == "i8":
        x, w = s["x"].double(), s["w"].double()
        scale = x.abs().max(dim=1).values / 127.0
        q = torch.round(x / torch.where(scale == 0, 1.0, scale)[:, None])
        y = torch.matmul(q, w.T) * (scale[:, None] * s["w_scale"].double())
        return {"y": y if s["b"] is None else y + s["b"].double()}
    p, g = s["p"].double(), s["g"].double()
    if case["bits"] == 32:
        m, v = s["m"].double(), s["v"].double()
    else:
        a, b = s["m"].double().view(-1, BLOCK) / 127, s["v"].double().view(-1, BLOCK) / 255
        m = (s["m_scale"].double()[:, None] * a * a.abs()).flatten()
        v = (s["v_scale"].double()[:, None] * b ** 4).flatten()
    m = torch.lerp(g, m, BETA1)
    v = torch.lerp(g ** 2, v, BETA2)
    p = p - LR * (m / (1 - BETA1 ** STEP) / ((v / (1 - BETA2 ** STEP)).sqrt() + EPS) + DECAY * p)
    if case["bits"] == 8:
        m, v = m.view(-1, BLOCK), v.view(-1, BLOCK)
        am, av = m.abs().max(1, keepdim=True).values, v.max(1, keepdim=True).values
        cm = torch.round(127 * (m.abs() / am.clamp(min=1e-300)) ** 0.5)
        cv = torch.round(255 * (v / av.clamp(min=1e-300)) ** 0.25)
        cv = torch.where(v > 0, cv.clamp(min=1), cv)
        m, v = (m.sign() * am * (cm / 127) ** 2).flatten(), (av * (cv / 255) ** 4).flatten()
    return {"p": p, "m": m, "v": v}
