"""The cases on which the operators of a policy's training step are measured.

What reinforcement learning needs around the sketched layers: the log
probabilities of the sampled tokens and the entropy of their distributions,
from the vocabulary head without its logits (`head`) or from logits at hand, with
the most likely alternatives (`logits`); the global norm of all gradients and
clipping (`clip`); and the norm of a residual stream together with the addition
that makes it (`residual`).

`own` false: each operator in elementary torch operations, in 32 bits (a long sum
in 64), rounded once at the end. `own` true: the calls of
rank_randomized_gradient_amd.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
NORM_EPS = 1e-5


def listed():
    return [
        # scoring one short answer against a small vocabulary: launch latency counts
        {"name": "head 24x8000x512", "op": "head", "T": 24, "V": 8000, "k": 512, "r": 16, "train": False},
        # a frozen head behind a trained body: an odd token count and an odd vocabulary
        {"name": "head 777x32001x1024 frozen train", "op": "head", "T": 777, "V": 32001, "k": 1024, "r": 0, "train": True},
        # a microbatch's policy loss and entropy bonus at the default layer's width, rank 128
        {"name": "head 4096x131072x4096 r128 train", "op": "head", "T": 4096, "V": 131072, "k": 4096, "r": 128, "train": True},
        # one step of a rollout: the sampled token's log probability beside the twenty most likely
        {"name": "logits 1x131072 top20", "op": "logits", "T": 1, "V": 131072, "z": "bf16", "top": 20, "pad": 0, "train": False},
        # a microbatch of responses scored by a reference model, eight alternatives kept for distillation
        {"name": "logits 4096x131072 top8", "op": "logits", "T": 4096, "V": 131072, "z": "bf16", "top": 8, "pad": 0,
         "train": False},
        # an odd vocabulary in fp32, whose rows start at odd addresses, with the gradient
        {"name": "logits 1003x50021 fp32 top5 train", "op": "logits", "T": 1003, "V": 50021, "z": "fp32", "top": 5, "pad": 0,
         "train": True},
        # the gains of every norm of a 36-layer model: many small tensors
        {"name": "clip 145x4096 norm", "op": "clip", "n": 145, "numel": 4096, "spread": 0, "g": "bf16", "write": False},
        # one embedding's gradient of 32768 x 4096
        {"name": "clip 134M norm", "op": "clip", "n": 1, "numel": 134217728, "spread": 0, "g": "bf16", "write": False},
        # ragged tensors of both types (gains, biases, small matrices), clipped in place
        {"name": "clip 60 ragged in place", "op": "clip", "n": 60, "numel": 1000003, "spread": 16411, "g": "mixed",
         "write": True},
        # the tokens of a small batch of rollouts, one each
        {"name": "residual 16x4096 rms forward", "op": "residual", "rows": 16, "width": 4096, "kind": "rms", "x": "bf16",
         "w": "bf16", "train": False},
        # two microbatches through a pre-norm block's norm, forward and backward
        {"name": "residual 8192x4096 rms", "op": "residual", "rows": 8192, "width": 4096, "kind": "rms", "x": "bf16",
         "w": "fp32", "train": True},
        # an odd width in fp32, a layer norm with a bias
        {"name": "residual 5000x1003 fp32 layer", "op": "residual", "rows": 5000, "width": 1003, "kind": "layer", "x": "fp32",
         "w": "fp32", "train": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["head", "logits", "clip", "residual"])
    if op == "head":
        r, V, train = rng.choice([0, 4, 16, 64, 128]), _log(rng, 1000, 131072), rng.random() < 0.6
        if r and train:
            V = 8 * (V // 8)  # a head whose gradient is sketched has a multiple of 8 rows
        return {"op": op, "T": _log(rng, 1, 4096), "V": V, "k": 8 * _log(rng, 32, 512), "r": r, "train": train}
    if op == "logits":
        return {"op": op, "T": _log(rng, 1, 4096), "V": _log(rng, 1000, 131072), "z": rng.choice(["bf16", "fp32"]),
                "top": rng.choice([0, 1, 5, 8, 20]), "pad": rng.choice([0, 0, 1, 64]), "train": rng.random() < 0.5}
    if op == "clip":
        n = _log(rng, 1, 200)
        numel = _log(rng, 64, 40000000 // n)
        return {"op": op, "n": n, "numel": numel, "spread": numel // (n + 1) if rng.random() < 0.5 else 0,
                "g": rng.choice(["bf16", "fp32", "mixed"]), "write": rng.random() < 0.5}
    return {"op": op, "rows": _log(rng, 1, 16384), "width": _log(rng, 64, 8192), "kind": rng.choice(["layer", "rms"]),
            "x": rng.choice(["bf16", "bf16", "fp32"]), "w": rng.choice(["bf16", "fp32"]), "train": rng.random() < 0.75}


def _sizes(case):
    return [case["numel"] - i * case["spread"] for i in range(case["n"])]


def _types(case):
    pair = {"bf16": ("bf16", "bf16"), "fp32": ("fp32", "fp32"), "mixed": ("bf16", "fp32")}[case["g"]]
    return [pair[i % 2] for i in range(case["n"])]


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=gen, device=dev) * std).to(dtype)

    op = case["op"]
    s = {"case": case}
    if op in ("head", "logits"):
        T, V = case["T"], case["V"]
        tokens = torch.randint(0, V, (T,), generator=gen, device=dev)
        if op == "head":
            k, r = case["k"], case["r"]
            s["X"], s["W"] = normal(T, k), normal(V, k, std=0.02)
            s["P"] = normal(k, r) if r else None
            s["XP"] = normal(T, r, std=math.sqrt(k)) if r and case["train"] else None
            s["C"] = torch.zeros(V, r, device=dev) if r and case["train"] else None
        else:
            # rows from flat to peaked; a fiftieth of the vocabulary is forbidden
            z = torch.empty(T, V + case["pad"], dtype=DTYPES[case["z"]], device=dev)
            sharp = 1.0 + 2.0 * torch.rand(T, 1, generator=gen, device=dev)
            z[:, :V] = torch.randn(T, V, generator=gen, device=dev) * sharp
            z[:, V:] = 1e4  # what lies between the rows is nobody's logit
            allowed = torch.rand(V, generator=gen, device=dev) >= 0.02
            z[:, :V] = z[:, :V].masked_fill(~allowed, -math.inf)
            s["Z"] = z[:, :V]
            # half of the tokens are likely ones
            free = allowed.nonzero()[:, 0]
            tokens = free[tokens % len(free)]
            likely = torch.rand(T, generator=gen, device=dev) < 0.5
            tokens = torch.where(likely, s["Z"].max(1).indices, tokens)
        # prompt and padding tokens take no part
        s["tokens"] = torch.where(torch.rand(T, generator=gen, device=dev) < 0.1, -100, tokens)
        # the loss's gradients: an advantage and an entropy bonus over the token count
        s["grad_logp"] = normal(T, dtype=torch.float32) / T
        s["grad_entropy"] = -0.01 * torch.rand(T, generator=gen, device=dev) / T
        return s
    if op == "clip":
        sizes, types = _sizes(case), _types(case)
        s["flat"] = {}
        for t in sorted(set(types)):  # the tensors of a type lie in one buffer, each at a multiple of 16 elements
            total = sum((n + 15) // 16 * 16 for n, of in zip(sizes, types) if of == t)
            s["flat"][t] = torch.zeros(total, dtype=DTYPES[t], device=dev)
        s["G"], at = [], {t: 0 for t in s["flat"]}
        for n, t in zip(sizes, types):
            g = s["flat"][t][at[t]:at[t] + n]
            at[t] += (n + 15) // 16 * 16
            # every tensor with gradients of its own size
            g.copy_(torch.randn(n, generator=gen, device=dev) *
                    torch.exp(torch.randn(1, generator=gen, device=dev) - 6.0))
            s["G"].append(g)
        # a tenth of what many tensors' gradients are expected to have, so that clipping nearly always has work to do
        s["max_norm"] = 0.1 * math.exp(-5.0) * math.sqrt(sum(sizes))
        return s
    rows, width, x, w = case["rows"], case["width"], DTYPES[case["x"]], DTYPES[case["w"]]
    # a residual stream, every row with its own size, and a block's output
    size = torch.exp(torch.randn(rows, 1, generator=gen, device=dev) * 0.5)
    s["R"] = (torch.randn(rows, width, generator=gen, device=dev) * size + 0.3).to(x)
    s["X"] = normal(rows, width, std=0.3, dtype=x)
    s["weight"] = (1 + normal(width, std=0.1, dtype=torch.float32)).to(w)
    s["bias"] = normal(width, std=0.1, dtype=w) if case["kind"] == "layer" else None
    if case["train"]:
        s["dY"], s["dS"] = normal(rows, width, std=1e-3, dtype=x), normal(rows, width, std=1e-3, dtype=x)
    return s


def run(state):
    op = state["case"]["op"]
    if op == "clip":
        state["max_norm"] *= 0.998  # the threshold decays, so that a pass over clipped gradients clips again
    if own:
        return {"head": _own_head, "logits": _own_logits, "clip": _own_clip, "residual": _own_residual}[op](state)
    return {"head": _head, "logits": _logits, "clip": _clip, "residual": _residual}[op](state)


# ---- the framework's calls ---------------------------------------------------

def _own_head(s):
    from rank_randomized_gradient_amd import rgc

    train = s["case"]["train"]
    logp, entropy, lse, XP = rgc.rgc_linear_log_prob_forward(s["X"], s["W"], s["tokens"], None if train else s["P"])
    out = {"logp": logp, "entropy": entropy, "lse": lse, "XP": XP}
    if train:
        out["dX"] = rgc.rgc_linear_log_prob_backward(s["X"], s["W"], s["tokens"], lse, entropy, s["grad_logp"],
                                                     s["grad_entropy"], s["XP"], s["C"])
        out["C"] = s["C"]
    return out


def _own_logits(s):
    from rank_randomized_gradient_amd import rgc

    logp, entropy, lse, top_logp, top_ids = rgc.rgc_log_prob_forward(s["Z"], s["tokens"], top=s["case"]["top"])
    out = {"logp": logp, "entropy": entropy, "lse": lse, "top_logp": top_logp, "top_ids": top_ids}
    if s["case"]["train"]:
        out["dZ"] = rgc.rgc_log_prob_backward(s["Z"], s["tokens"], lse, entropy, s["grad_logp"], s["grad_entropy"])
    return out


def _own_clip(s):
    from rank_randomized_gradient_amd import rgc

    norm, scale = rgc.rgc_grad_norm_batch(s["G"], s["max_norm"])
    out = {"norm": norm, "scale": scale}
    if s["case"]["write"]:
        rgc.rgc_scale_batch(s["G"], scale)
        out.update(s["flat"])
    return out


def _own_residual(s):
    from rank_randomized_gradient_amd import rgc

    kind = s["case"]["kind"]
    S, Y, mean, rstd = rgc.rgc_add_norm_forward(s["X"], s["R"], s["weight"], s["bias"], eps=NORM_EPS, kind=kind)
    if not s["case"]["train"]:
        return {"S": S, "Y": Y}
    dX, dweight, dbias = rgc.rgc_add_norm_backward(s["dY"], s["dS"], S, s["weight"], mean, rstd,
                                                   bias=s["bias"] is not None, kind=kind)
    return {"S": S, "Y": Y, "dX": dX, "dweight": dweight, "dbias": dbias}


# ---- the plain forms ---------------------------------------------------------

def _policy(z, tokens):
    """(kept, at, logp of every entry, p, entropy, lse) of rows of logits; entries of -inf are forbidden."""
    kept = (tokens >= 0) & (tokens < z.shape[1])
    at = torch.where(kept, tokens, 0)
    top = z.amax(1, keepdim=True)
    lse = top + torch.log(torch.exp(z - top).sum(1, keepdim=True))
    logp = z - lse
    p = torch.exp(logp)
    entropy = -torch.where(p > 0, p * logp, 0.0).sum(1)
    return kept, at, logp, p, entropy, lse[:, 0]


def _given(logp, kept, at, entropy):
    """The tokens' log probabilities and the entropies; 0 for a token that takes no part."""
    return torch.where(kept, logp.gather(1, at[:, None])[:, 0], 0.0), torch.where(kept, entropy, 0.0)


def _logit_gradient(s, kept, at, logp, p, entropy):
    gl, ge = s["grad_logp"][:, None], s["grad_entropy"][:, None]
    D = torch.where(p > 0, -p * (gl + ge * (logp + entropy[:, None])), 0.0)
    D[torch.arange(len(at), device=at.device), at] += s["grad_logp"]
    return torch.where(kept[:, None], D, 0.0)


def _head(s):
    z = s["X"].float() @ s["W"].float().T
    kept, at, logp, p, entropy, lse = _policy(z, s["tokens"])
    del z
    given, shown = _given(logp, kept, at, entropy)
    out = {"logp": given, "entropy": shown, "lse": lse, "XP": None}
    if not s["case"]["train"]:
        if s["P"] is not None:
            out["XP"] = (s["X"].float() @ s["P"].float()).to(torch.bfloat16)
        return out
    D = _logit_gradient(s, kept, at, logp, p, entropy)
    out["dX"] = (D @ s["W"].float()).to(torch.bfloat16)
    if s["C"] is not None:
        s["C"] += D.T @ s["XP"].float()
    out["C"] = s["C"]
    return out


def _logits(s):
    top = s["case"]["top"]
    z = s["Z"].float()
    kept, at, logp, p, entropy, lse = _policy(z, s["tokens"])
    given, shown = _given(logp, kept, at, entropy)
    out = {"logp": given, "entropy": shown, "lse": lse, "top_logp": None, "top_ids": None}
    if top:
        left, ids = z.clone(), []
        places = torch.arange(z.shape[1], device=z.device)
        for _ in range(top):  # the lowest index of the largest that is left
            best = torch.where(left == left.amax(1, keepdim=True), places, z.shape[1]).amin(1, keepdim=True)
            ids.append(best)
            left.scatter_(1, best, -math.inf)
        out["top_ids"] = torch.cat(ids, 1)
        out["top_logp"] = logp.gather(1, out["top_ids"])
    if s["case"]["train"]:
        out["dZ"] = _logit_gradient(s, kept, at, logp, p, entropy).to(s["Z"].dtype)
    return out


def _clip(s):
    total = torch.stack([G.double().square().sum() for G in s["G"]]).sum()
    norm = torch.sqrt(total)
    scale = torch.where(norm > s["max_norm"], s["max_norm"] / norm, 1.0).float()
    out = {"norm": norm.float().reshape(1), "scale": scale.reshape(1)}
    if s["case"]["write"]:
        for G in s["G"]:
            G.copy_(G.float() * scale)
        out.update(s["flat"])
    return out


def _residual(s):
    S = (s["X"].float() + s["R"].float()).to(s["X"].dtype)
    x = S.float()  # the norm is that of the stream as it is kept
    centre = s["case"]["kind"] == "layer"
    c = x - x.mean(1, keepdim=True) if centre else x
    rstd = 1.0 / torch.sqrt(c.square().mean(1, keepdim=True) + NORM_EPS)
    xhat = c * rstd
    w = s["weight"].float()
    y = xhat * w
    if s["bias"] is not None:
        y = y + s["bias"].float()
    y = y.to(S.dtype)
    if not s["case"]["train"]:
        return {"S": S, "Y": y}
    dy = s["dY"].float()
    h = dy * w
    dx = h - xhat * (h * xhat).mean(1, keepdim=True)
    if centre:
        dx = dx - h.mean(1, keepdim=True)
    dx = (dx * rstd + s["dS"].float()).to(S.dtype)
    dweight = (dy * xhat).sum(0).to(s["weight"].dtype)
    dbias = dy.sum(0).to(s["bias"].dtype) if s["bias"] is not None else None
    return {"S": S, "Y": y, "dX": dx, "dweight": dweight, "dbias": dbias}


# ---- the definitions in 64 bits ----------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"head": _exact_head, "logits": _exact_logits, "clip": _exact_clip, "residual": _exact_residual}[case["op"]](s)


def _exact_policy(z, s, want_gradient):
    """logp, entropy and lse by token, and the logits' gradient; z (in 64 bits) is used up."""
    y = s["tokens"]
    live = y.ge(0) & y.lt(z.shape[1])
    y = y.clamp(0, z.shape[1] - 1)[:, None]
    lse = torch.logsumexp(z, 1)
    logq = z.sub_(lse[:, None])
    given = logq.gather(1, y)[:, 0]
    q = logq.exp()
    surprise = torch.special.entr(q).sum(1)
    out = {"logp": given.masked_fill(~live, 0), "entropy": surprise.masked_fill(~live, 0), "lse": lse}
    if not want_gradient:
        return out, None
    # d logp / dz_v = [v = y] - q_v;  d entropy / dz_v = -q_v (log q_v + entropy)
    a = s["grad_logp"].double().masked_fill(~live, 0)[:, None]
    b = s["grad_entropy"].double().masked_fill(~live, 0)[:, None]
    slope = logq.masked_fill_(q == 0, 0).add_(surprise[:, None]).mul_(b).add_(a).mul_(q).neg_()
    slope.scatter_add_(1, y, a)
    return out, slope


def _exact_head(s):
    train = s["case"]["train"]
    W = s["W"].double()
    out, slope = _exact_policy(torch.mm(s["X"].double(), W.t()), s, train)
    out["XP"] = s["X"].double().mm(s["P"].double()) if s["P"] is not None and not train else None
    if train:
        out["dX"] = slope.mm(W)
        out["C"] = slope.t().mm(s["XP"].double()) if s["C"] is not None else None
    return out


def _exact_logits(s):
    top, train = s["case"]["top"], s["case"]["train"]
    z = s["Z"].double()
    best = torch.sort(z, dim=1, descending=True, stable=True) if top else None
    values, ids = (best.values[:, :top].clone(), best.indices[:, :top].clone()) if top else (None, None)
    del best
    out, slope = _exact_policy(z, s, train)
    out["top_logp"] = values - out["lse"][:, None] if top else None
    out["top_ids"] = ids
    if train:
        out["dZ"] = slope
    return out


def _exact_clip(s):
    limit = s["max_norm"] * 0.998
    length = math.sqrt(math.fsum(float(torch.dot(g, g)) for g in (G.double() for G in s["G"])))
    factor = limit / length if length > limit else 1.0
    out = {"norm": torch.tensor([length], dtype=torch.float64), "scale": torch.tensor([factor], dtype=torch.float64)}
    if s["case"]["write"]:
        out.update({t: x.double() * factor for t, x in s["flat"].items()})
    return out


def _exact_residual(s):
    S = (s["X"].double() + s["R"].double()).to(s["X"].dtype)  # kept in its own type: a rounding of the definition
    x, w = S.double(), s["weight"].double()
    centre = s["case"]["kind"] == "layer"
    mu = x.mean(1, keepdim=True) if centre else torch.zeros_like(x[:, :1])
    sigma = ((x - mu).pow(2).mean(1, keepdim=True) + NORM_EPS).sqrt()
    u = (x - mu) / sigma
    y = u * w + (s["bias"].double() if s["bias"] is not None else 0.0)
    if not s["case"]["train"]:
        return {"S": S.double(), "Y": y}
    dy = s["dY"].double()
    a = dy * w
    along = (a * u).sum(1, keepdim=True) / x.shape[1]
    flat = a.mean(1, keepdim=True) if centre else 0.0
    return {"S": S.double(), "Y": y, "dX": (a - flat - u * along) / sigma + s["dS"].double(),
            "dweight": torch.sum(dy * u, 0), "dbias": torch.sum(dy, 0) if s["bias"] is not None else None}


# ---- what a pass cannot do without -------------------------------------------

def work(case):
    if case["op"] == "head":
        T, V, k, r = case["T"], case["V"], case["k"], case["r"]
        read = 2 * T * k + 2 * V * k + 8 * T
        if not case["train"]:
            return {"bytes": read + 12 * T + 2 * k * r + 2 * T * r, "flops": 2 * T * k * (V + r)}
        return {"bytes": read + 8 * T + 12 * T + 2 * T * r + 2 * T * k + 8 * V * r, "flops": 4 * T * V * k + 2 * T * V * r}
    if case["op"] == "logits":
        T, V, z = case["T"], case["V"], 2 if case["z"] == "bf16" else 4
        if not case["train"]:
            return {"bytes": T * V * z + 8 * T + T * (12 + 12 * case["top"]), "flops": 6 * T * V}
        return {"bytes": 2 * T * V * z + 16 * T + T * (12 + 12 * case["top"]), "flops": 12 * T * V}
    if case["op"] == "clip":
        total = sum(n * (2 if t == "bf16" else 4) for n, t in zip(_sizes(case), _types(case)))
        n = sum(_sizes(case))
        return {"bytes": 2 * total + 8 if case["write"] else total + 8, "flops": 3 * n if case["write"] else 2 * n}
    x, w = (2 if case["x"] == "bf16" else 4), (2 if case["w"] == "bf16" else 4)
    rows, width, params = case["rows"], case["width"], 2 if case["kind"] == "layer" else 1
    if not case["train"]:
        return {"bytes": 4 * rows * width * x + params * width * w, "flops": 9 * rows * width}
    # X, R, dY and dS read, S, Y and dX written
    return {"bytes": 7 * rows * width * x + 2 * params * width * w, "flops": 22 * rows * width}
