"""The cases on which the operators beside the sketched layer are measured.

Three operators train what a sketch does not: the vocabulary head's loss (a
linear layer and its softmax cross entropy, with the gradient that feeds the
head's sketch), layer norms with their weights' gradients, and an AdamW step
for the tensors that keep a dense gradient (norm gains, biases, embeddings).

`own` false: each operator in elementary torch operations, in 32 bits, rounded
once at the end. `own` true: the calls of rank_randomized_gradient_amd.
"""
import math

import torch

own = False

BLOCK = 128  # elements of an 8-bit state that share a scale
FP8 = torch.float8_e4m3fn
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # scoring one short answer against a small vocabulary: launch latency counts
        {"name": "loss 24x8000x512", "op": "loss", "T": 24, "V": 8000, "k": 512, "r": 16},
        # a microbatch's loss at the default layer's width: 4096 tokens, a large vocabulary
        {"name": "loss 4096x131072x4096", "op": "loss", "T": 4096, "V": 131072, "k": 4096, "r": 128},
        # a frozen head (no sketch) behind a trained body: an odd token count and an odd vocabulary
        {"name": "grad 1001x50001x2048 frozen", "op": "grad", "T": 1001, "V": 50001, "k": 2048, "r": 0},
        # a half microbatch of a 2048-wide model, rank 64
        {"name": "grad 2048x32768x2048 r64", "op": "grad", "T": 2048, "V": 32768, "k": 2048, "r": 64},
        # the whole microbatch of 4096 tokens at width 4096, rank 128
        {"name": "grad 4096x131072x4096 r128", "op": "grad", "T": 4096, "V": 131072, "k": 4096, "r": 128},
        # one token through a norm, as a rollout takes it
        {"name": "norm 1x4096 forward", "op": "norm", "rows": 1, "width": 4096, "kind": "layer", "x": "bf16", "w": "bf16",
         "train": False},
        # one microbatch through a root-mean-square norm, forward and backward
        {"name": "norm 4096x4096 rms", "op": "norm", "rows": 4096, "width": 4096, "kind": "rms", "x": "bf16", "w": "fp32",
         "train": True},
        # a whole step's tokens through a layer norm at once
        {"name": "norm 32768x4096 layer", "op": "norm", "rows": 32768, "width": 4096, "kind": "layer", "x": "bf16",
         "w": "bf16", "train": True},
        # an odd width in fp32, whose rows start at odd addresses
        {"name": "norm 5000x1003 fp32", "op": "norm", "rows": 5000, "width": 1003, "kind": "layer", "x": "fp32", "w": "fp32",
         "train": True},
        # the gains of every norm of a 36-layer model: many small tensors, 8-bit states
        {"name": "adamw 145x4096 8-bit", "op": "adamw", "n": 145, "numel": 4096, "spread": 0, "p": "bf16", "g": "bf16",
         "bits": 8},
        # one embedding of 32768 x 4096 in bf16 with 8-bit states
        {"name": "adamw 134M 8-bit", "op": "adamw", "n": 1, "numel": 134217728, "spread": 0, "p": "bf16", "g": "bf16",
         "bits": 8},
        # ragged fp32 tensors (biases, gains, small matrices) with fp32 states
        {"name": "adamw 60 ragged fp32", "op": "adamw", "n": 60, "numel": 1000003, "spread": 17477, "p": "fp32", "g": "fp32",
         "bits": 32},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["loss", "grad", "norm", "adamw"])
    if op in ("loss", "grad"):
        k = 8 * _log(rng, 32, 512)
        r = rng.choice([0, 4, 16, 64, 128])
        V = _log(rng, 1000, 131072)
        if r and op == "grad":
            V = 8 * (V // 8)  # a head whose gradient is sketched has a multiple of 8 rows
        return {"op": op, "T": _log(rng, 1, 4096), "V": V, "k": k, "r": r}
    if op == "norm":
        return {"op": op, "rows": _log(rng, 1, 32768), "width": _log(rng, 64, 4096),
                "kind": rng.choice(["layer", "rms"]), "x": rng.choice(["bf16", "bf16", "fp32"]),
                "w": rng.choice(["bf16", "fp32"]), "train": rng.random() < 0.75}
    n = _log(rng, 1, 200)
    numel = _log(rng, 64, 20000000 // n)
    return {"op": op, "n": n, "numel": numel, "spread": numel // (n + 1) if rng.random() < 0.5 else 0,
            "p": rng.choice(["bf16", "fp32"]), "g": rng.choice(["bf16", "fp32"]), "bits": rng.choice([8, 32])}


def _sizes(case):
    return [case["numel"] - i * case["spread"] for i in range(case["n"])]


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=gen, device=dev) * std).to(dtype)

    if case["op"] in ("loss", "grad"):
        T, V, k, r = case["T"], case["V"], case["k"], case["r"]
        s = {"case": case, "X": normal(T, k), "W": normal(V, k, std=0.02)}
        targets = torch.randint(0, V, (T,), generator=gen, device=dev)
        # prompt and padding tokens carry no loss
        s["targets"] = torch.where(torch.rand(T, generator=gen, device=dev) < 0.1, -100, targets)
        if case["op"] == "loss":
            s["P"] = normal(k, r) if r else None
            return s
        # the gradient of each token's loss: an advantage over the token count
        s["grad"] = normal(T, dtype=torch.float32) / T
        s["XP"] = normal(T, r, std=math.sqrt(k)) if r else None
        s["C"] = torch.zeros(V, r, device=dev) if r else None
        return s
    if case["op"] == "norm":
        rows, width, x, w = case["rows"], case["width"], DTYPES[case["x"]], DTYPES[case["w"]]
        # a residual stream: every row with its own mean and size
        size = torch.exp(torch.randn(rows, 1, generator=gen, device=dev) * 0.5)
        mean = torch.randn(rows, 1, generator=gen, device=dev) * 0.5
        X = ((torch.randn(rows, width, generator=gen, device=dev) + mean) * size).to(x)
        s = {"case": case, "X": X, "weight": 1 + normal(width, std=0.1, dtype=torch.float32)}
        s["weight"] = s["weight"].to(w)
        s["bias"] = normal(width, std=0.1, dtype=w) if case["kind"] == "layer" else None
        s["dY"] = normal(rows, width, std=1e-3, dtype=x) if case["train"] else None
        return s
    # the tensors lie in flat buffers, one of each kind, each at a multiple of 16 elements
    eight = case["bits"] == 8
    s = {"case": case, "seed": seed, "step": 100, "P": [], "G": [], "M": [], "V": []}
    s["grad_scale"] = 0.5 + 0.5 * torch.rand(1, generator=gen, device=dev)  # a clipping coefficient, on the device
    s["Ms"], s["Vs"] = ([], []) if eight else (None, None)
    sizes = _sizes(case)
    total = sum((n + 15) // 16 * 16 for n in sizes)
    flat = s["flat"] = {"P": normal(total, std=0.02 if case["n"] == 1 else 1.0, dtype=DTYPES[case["p"]])}
    grads = normal(total, std=1e-2, dtype=DTYPES[case["g"]])
    if eight:
        flat["M"] = (torch.randn(total, generator=gen, device=dev) * 40).clamp(-240, 240).to(FP8)
        flat["V"] = (torch.rand(total, generator=gen, device=dev) * 200 + 8).to(FP8)
        # block scales are powers of two: momenta near 2^-10, root second moments near 2^-7
        blocks = sum((n + BLOCK - 1) // BLOCK for n in sizes)
        e = torch.randint(-16, -13, (2, blocks), generator=gen, device=dev).float()
        flat["Ms"], flat["Vs"] = torch.exp2(e[0] - 1), torch.exp2(e[1])
    else:
        flat["M"] = normal(total, std=1e-3, dtype=torch.float32)
        flat["V"] = normal(total, std=1e-2, dtype=torch.float32).square()
    at = block = 0
    for n in sizes:
        s["G"].append(grads[at:at + n])
        for name in "PMV":
            s[name].append(flat[name][at:at + n])
        at += (n + 15) // 16 * 16
        for name in ("Ms", "Vs") if eight else ():
            s[name].append(flat[name][block:block + (n + BLOCK - 1) // BLOCK])
        block += (n + BLOCK - 1) // BLOCK
    return s


LR, BETA1, BETA2, EPS, DECAY, NORM_EPS = 1e-3, 0.9, 0.999, 1e-8, 0.01, 1e-5


def run(state):
    op = state["case"]["op"]
    if own:
        return {"loss": _own_loss, "grad": _own_grad, "norm": _own_norm, "adamw": _own_adamw}[op](state)
    return {"loss": _loss, "grad": _grad, "norm": _norm, "adamw": _adamw}[op](state)


# ---- the framework's calls ---------------------------------------------------

def _own_loss(s):
    from rank_randomized_gradient_amd import rgc

    loss, lse, XP = rgc.rgc_linear_cross_entropy_forward(s["X"], s["W"], s["targets"], s["P"])
    return {"loss": loss, "lse": lse, "XP": XP}


def _own_grad(s):
    from rank_randomized_gradient_amd import rgc

    loss, lse, _ = rgc.rgc_linear_cross_entropy_forward(s["X"], s["W"], s["targets"])
    dX = rgc.rgc_linear_cross_entropy_backward(s["X"], s["W"], s["targets"], lse, s["grad"], s["XP"], s["C"])
    return {"loss": loss, "dX": dX, "C": s["C"]}


def _own_norm(s):
    from rank_randomized_gradient_amd import rgc

    kind = s["case"]["kind"]
    Y, mean, rstd = rgc.rgc_layer_norm_forward(s["X"], s["weight"], s["bias"], eps=NORM_EPS, kind=kind)
    if s["dY"] is None:
        return {"Y": Y}
    dX, dweight, dbias = rgc.rgc_layer_norm_backward(s["dY"], s["X"], s["weight"], mean, rstd,
                                                     bias=s["bias"] is not None, kind=kind)
    return {"Y": Y, "dX": dX, "dweight": dweight, "dbias": dbias}


def _own_adamw(s):
    from rank_randomized_gradient_amd import rgc

    rgc.rgc_adamw_batch(s["P"], s["G"], s["M"], s["V"], LR, s["step"], seed=s["seed"], beta1=BETA1, beta2=BETA2, eps=EPS,
                        weight_decay=DECAY, M_scales=s["Ms"], V_scales=s["Vs"], grad_scale=s["grad_scale"])
    return s["flat"]


# ---- the plain forms ---------------------------------------------------------

def _logits(s):
    targets = s["targets"]
    V = s["W"].shape[0]
    z = s["X"].float() @ s["W"].float().T
    kept = (targets >= 0) & (targets < V)
    at = torch.where(kept, targets, 0)
    top = z.amax(1)
    lse = top + torch.log(torch.exp(z - top[:, None]).sum(1))
    loss = torch.where(kept, lse - z.gather(1, at[:, None])[:, 0], 0.0)
    return z, kept, at, lse, loss


def _loss(s):
    _, _, _, lse, loss = _logits(s)
    XP = (s["X"].float() @ s["P"].float()).to(torch.bfloat16) if s["P"] is not None else None
    return {"loss": loss, "lse": lse, "XP": XP}


def _grad(s):
    z, kept, at, lse, loss = _logits(s)
    D = torch.exp(z - lse[:, None])
    rows = torch.arange(len(at), device=at.device)
    D[rows, at] -= 1.0
    D = torch.where(kept[:, None], D * s["grad"][:, None], 0.0)
    dX = (D @ s["W"].float()).to(torch.bfloat16)
    if s["C"] is not None:
        s["C"] += D.T @ s["XP"].float()
    return {"loss": loss, "dX": dX, "C": s["C"]}


def _norm(s):
    x = s["X"].float()
    centre = s["case"]["kind"] == "layer"
    c = x - x.mean(1, keepdim=True) if centre else x
    rstd = 1.0 / torch.sqrt(c.square().mean(1, keepdim=True) + NORM_EPS)
    xhat = c * rstd
    w = s["weight"].float()
    y = xhat * w
    if s["bias"] is not None:
        y = y + s["bias"].float()
    y = y.to(s["X"].dtype)
    if s["dY"] is None:
        return {"Y": y}
    dy = s["dY"].float()
    h = dy * w
    dx = h - xhat * (h * xhat).mean(1, keepdim=True)
    if centre:
        dx = dx - h.mean(1, keepdim=True)
    dx = (dx * rstd).to(s["X"].dtype)
    dweight = (dy * xhat).sum(0).to(s["weight"].dtype)
    dbias = dy.sum(0).to(s["bias"].dtype) if s["bias"] is not None else None
    return {"Y": y, "dX": dx, "dweight": dweight, "dbias": dbias}


def _random16(n, tensor, seed, dev):
    """Two arrays of n 16-bit numbers, for the parameters and for the second moments of one tensor:
    Philox4x32-10 of the counter (group low, group high, 4, tensor) under the key `seed`, a group being
    eight elements; element j of a group takes half j % 2 of word j / 2 for its parameter and the other
    half for its second moment."""
    group = torch.arange((n + 7) // 8, device=dev, dtype=torch.int64)
    m = 0xFFFFFFFF
    c0, c1 = group & m, group >> 32
    c2, c3 = torch.full_like(group, 4), torch.full_like(group, tensor)
    k0, k1 = seed & m, (seed >> 32) & m
    for _ in range(10):
        p0, p1 = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = ((p1 >> 32) & m) ^ c1 ^ k0, p1 & m, ((p0 >> 32) & m) ^ c3 ^ k1, p0 & m
        k0, k1 = (k0 + 0x9E3779B9) & m, (k1 + 0xBB67AE85) & m
    words = torch.stack([c0, c1, c2, c3], 1)
    low, high = words & 0xFFFF, words >> 16
    p = torch.stack([low, high], 2).reshape(-1)[:n].to(torch.int32)
    v = torch.stack([high, low], 2).reshape(-1)[:n].to(torch.int32)
    return p, v


def _blocks(x):
    n = x.numel()
    padded = x.new_zeros((n + BLOCK - 1) // BLOCK * BLOCK)
    padded[:n] = x
    return padded.view(-1, BLOCK)


def _scale(x):
    """Powers of two that bring each block's largest finite magnitude into 128 .. 256."""
    top = torch.where(torch.isfinite(x), x.abs(), 0.0).amax(1)
    return ((top.view(torch.int32) >> 23) - 7).clamp(min=1).bitwise_left_shift(23).view(torch.float32)


def _adamw(s):
    c2 = 1.0 / math.sqrt(1.0 - BETA2 ** s["step"])
    size = LR / (1.0 - BETA1 ** s["step"])
    for i, (P, G, M, V) in enumerate(zip(s["P"], s["G"], s["M"], s["V"])):
        n = P.numel()
        g = G.float() * s["grad_scale"]
        if s["Ms"] is None:
            m, v = M, V
        else:
            m = (_blocks(M.float()) * s["Ms"][i][:, None]).view(-1)[:n]
            v = (_blocks(V.float()) * s["Vs"][i][:, None]).view(-1)[:n].square()
        m = m * BETA1 + g * (1 - BETA1)
        v = v * BETA2 + g * g * (1 - BETA2)
        root = torch.sqrt(v)
        p = P.float() * (1 - LR * DECAY) - size * (m / (root * c2 + EPS))
        rp, rv = _random16(n, i, s["seed"], P.device) if s["Ms"] is not None or P.dtype == torch.bfloat16 else (None, None)
        if P.dtype == torch.bfloat16:
            p = ((p.view(torch.int32) + rp) & -65536).view(torch.float32)
        P.copy_(p)
        if s["Ms"] is None:
            M.copy_(m)
            V.copy_(v)
            continue
        m, root, rv = _blocks(m), _blocks(root), _blocks(rv)
        s["Ms"][i].copy_(_scale(m))
        s["Vs"][i].copy_(_scale(root))
        M.copy_((m / s["Ms"][i][:, None]).to(FP8).view(-1)[:n])
        x = root / s["Vs"][i][:, None]
        # stochastic rounding to three bits of mantissa: below 2^-6 the step is 2^-9, the step of
        # numbers from 2^-6 on; what is not zero never rounds to zero
        lift = torch.where(x < 2.0 ** -6, 2.0 ** -6, 0.0)
        y = (((x + lift).view(torch.int32) + (rv << 4)) & -1048576).view(torch.float32) - lift
        y = torch.where(x > 0, y.clamp(min=2.0 ** -9), 0.0)
        V.copy_(y.to(FP8).view(-1)[:n])
    return s["flat"]


# ---- the definitions in 64 bits ----------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"loss": _exact_ce, "grad": _exact_ce, "norm": _exact_norm, "adamw": _exact_adamw}[case["op"]](s)


def _exact_ce(s):
    X, W, t = s["X"].double(), s["W"].double(), s["targets"]
    logp = torch.mm(X, W.t())
    lse = torch.logsumexp(logp, 1)
    logp -= lse[:, None]
    live = t.ge(0) & t.lt(W.shape[0])
    y = t.clamp(0, W.shape[0] - 1).unsqueeze(1)
    loss = -logp.gather(1, y).squeeze(1) * live
    if s["case"]["op"] == "loss":
        return {"loss": loss, "lse": lse, "XP": X.mm(s["P"].double()) if s["P"] is not None else None}
    g = s["grad"].double() * live
    prob = logp.exp_().mul_(g[:, None])
    prob.scatter_add_(1, y, -g[:, None])
    C = prob.t().mm(s["XP"].double()) if s["C"] is not None else None
    return {"loss": loss, "dX": prob.mm(W), "C": C}


def _exact_norm(s):
    x, w = s["X"].double(), s["weight"].double()
    mu = x.mean(1, keepdim=True) if s["case"]["kind"] == "layer" else torch.zeros_like(x[:, :1])
    sigma = ((x - mu).pow(2).mean(1, keepdim=True) + NORM_EPS).sqrt()
    u = (x - mu) / sigma
    y = u * w + (s["bias"].double() if s["bias"] is not None else 0.0)
    if s["dY"] is None:
        return {"Y": y}
    dy = s["dY"].double()
    a = dy * w
    along = (a * u).sum(1, keepdim=True) / x.shape[1]
    flat = a.mean(1, keepdim=True) if s["case"]["kind"] == "layer" else 0.0
    return {"Y": y, "dX": (a - flat - u * along) / sigma, "dweight": torch.sum(dy * u, 0),
            "dbias": torch.sum(dy, 0) if s["bias"] is not None else None}


def _exact_adamw(s):
    """Parameters and 32-bit states in 64 bits, before any rounding, and the blocks' scales; an 8-bit
    state is given before its rounding too, in units of its block's scale."""
    t = s["step"]
    out = {name: x.clone() if name in ("Ms", "Vs") else x.double() for name, x in s["flat"].items()}
    at = block = 0
    for i, P in enumerate(s["P"]):
        n = P.numel()
        here, blocks = slice(at, at + n), slice(block, block + (n + BLOCK - 1) // BLOCK)
        at, block = at + (n + 15) // 16 * 16, blocks.stop
        g = s["G"][i].double() * s["grad_scale"].double()
        m, v = s["M"][i].double(), s["V"][i].double()
        if s["Ms"] is not None:
            m = m * torch.repeat_interleave(s["Ms"][i].double(), BLOCK)[:n]
            v = (v * torch.repeat_interleave(s["Vs"][i].double(), BLOCK)[:n]) ** 2
        m = BETA1 * m + (1 - BETA1) * g
        v = BETA2 * v + (1 - BETA2) * g ** 2
        step = (m / (1 - BETA1 ** t)) / (torch.sqrt(v / (1 - BETA2 ** t)) + EPS)
        out["P"][here] -= LR * DECAY * out["P"][here] + LR * step
        if s["Ms"] is None:
            out["M"][here], out["V"][here] = m, v
            continue
        for values, name, scales in ((m, "M", "Ms"), (v.sqrt(), "V", "Vs")):
            rows = torch.zeros((n + BLOCK - 1) // BLOCK * BLOCK, dtype=torch.float64, device=P.device)
            rows[:n] = values
            rows = rows.view(-1, BLOCK)
            unit = torch.exp2(torch.floor(torch.log2(rows.abs().amax(1))) - 7)
            out[scales][blocks] = unit.to(torch.float32)
            out[name][here] = (rows / unit[:, None]).view(-1)[:n]
    return out


# ---- what a pass cannot do without -------------------------------------------

def work(case):
    if case["op"] in ("loss", "grad"):
        T, V, k, r = case["T"], case["V"], case["k"], case["r"]
        read = 2 * T * k + 2 * V * k + 8 * T
        if case["op"] == "loss":
            return {"bytes": read + 8 * T + 2 * k * r + 2 * T * r, "flops": 2 * T * k * (V + r)}
        return {"bytes": read + 8 * T + 2 * T * r + 2 * T * k + 8 * V * r, "flops": 4 * T * V * k + 2 * T * V * r}
    if case["op"] == "norm":
        x, w = (2 if case["x"] == "bf16" else 4), (2 if case["w"] == "bf16" else 4)
        rows, width, params = case["rows"], case["width"], 2 if case["kind"] == "layer" else 1
        if not case["train"]:
            return {"bytes": 2 * rows * width * x + params * width * w, "flops": 8 * rows * width}
        return {"bytes": 4 * rows * width * x + 2 * params * width * w, "flops": 20 * rows * width}
    n = sum(_sizes(case))
    p, g = (2 if case["p"] == "bf16" else 4), (2 if case["g"] == "bf16" else 4)
    state = 16 if case["bits"] == 32 else 4 + 16 / BLOCK
    return {"bytes": n * (2 * p + g + state), "flops": 15 * n}
