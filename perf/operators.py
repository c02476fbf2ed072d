"""Cases that measure the operators beside the 4-bit linears: rotary positions, the vocabulary loss with its
gradient, and the product of a few tokens with a 4-bit weight that keeps one fp32 constant per block of 64.

Each operator has its plain form here (elementary torch operations in 32 bits, rounded once at the end); with
`own` set, `run` makes the calls that a user makes of the package instead. `exact` evaluates the operators'
definitions in 64 bits, apart from the plain forms.
"""
import math

import torch

own = False

DEVICE = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BLOCK = 64            # weights per constant
IGNORE = -100         # a target that takes no part in the loss


# ---- the cases ----------------------------------------------------------------------------------

def listed():
    return [
        # one generated token of a 64-head model: latency
        {"name": "rope_token", "op": "rope", "B": 1, "T": 1, "Hq": 64, "Hk": 64, "D": 128, "R": 128, "type": "bf16",
         "layout": "half", "scaling": "none", "far": 4096, "order": "tokens", "inverse": False},
        # a step of 16 sequences of 512 tokens, q and k read in place from one fused projection
        {"name": "rope_train", "op": "rope", "B": 16, "T": 512, "Hq": 32, "Hk": 32, "D": 128, "R": 128, "type": "bf16",
         "layout": "half", "scaling": "none", "far": 512, "order": "fused", "inverse": False},
        # gradients of a long packed batch with shared key heads, interleaved pairs, positions stretched 4 times
        {"name": "rope_grad_long", "op": "rope", "B": 2, "T": 8191, "Hq": 32, "Hk": 8, "D": 128, "R": 128,
         "type": "bf16", "layout": "interleaved", "scaling": "banded", "far": 131072, "order": "heads", "inverse": True},
        # odd sizes: a part of the head is turned, fp32, far positions
        {"name": "rope_part_f32", "op": "rope", "B": 3, "T": 1027, "Hq": 12, "Hk": 4, "D": 80, "R": 36, "type": "f32",
         "layout": "half", "scaling": "yarn", "far": 131072, "order": "tokens", "inverse": False},
        # scoring a short text: loss only
        {"name": "loss_score", "op": "loss", "T": 37, "V": 32000, "K": 4096, "grad": False, "reduction": "none",
         "ignored": 0.0},
        # one training sequence of the 65B-shaped decoder
        {"name": "loss_train_65b", "op": "loss", "T": 512, "V": 32000, "K": 8192, "grad": True, "reduction": "mean",
         "ignored": 0.0},
        # a step of 16 x 512 tokens of the 7B-shaped decoder, padding left out of the loss
        {"name": "loss_train_7b", "op": "loss", "T": 8192, "V": 32000, "K": 4096, "grad": True, "reduction": "mean",
         "ignored": 0.1},
        # a ragged batch over an odd vocabulary, weighted token by token
        {"name": "loss_ragged", "op": "loss", "T": 1201, "V": 50021, "K": 1032, "grad": True, "reduction": "none",
         "ignored": 0.3},
        # one token through the 65B-shaped layers, and 16 tokens (a batch of sequences) through int4 weights
        {"name": "matvec_8192", "op": "matvec", "T": 1, "N": 8192, "K": 8192, "book": "nf4"},
        {"name": "matvec_22016", "op": "matvec", "T": 1, "N": 22016, "K": 8192, "book": "nf4"},
        {"name": "matvec_16_tokens", "op": "matvec", "T": 16, "N": 8192, "K": 22016, "book": "int4"},
        # odd sizes, latency
        {"name": "matvec_odd", "op": "matvec", "T": 3, "N": 1003, "K": 1088, "book": "grid"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "loss", "matvec"])
    if op == "rope":
        D = rng.choice([64, 80, 96, 128, 192, 256])
        R = rng.choice([D, D, D // 2, 2 * rng.randint(1, D // 2)])
        Hk = rng.choice([1, 2, 4, 8, 16, 32])
        Hq = Hk * rng.choice([1, 1, 4, 7])
        B = rng.choice([1, 1, 2, 3, 16])
        most = 16 * 8192 * 64 * 128 // 16 // (B * (Hq + Hk) * D)
        T = _log(rng, 1, max(2, min(16384, most)))
        return {"op": op, "B": B, "T": T, "Hq": Hq, "Hk": Hk, "D": D, "R": R, "type": rng.choice(["bf16", "bf16", "f32"]),
                "layout": rng.choice(["half", "interleaved"]),
                "scaling": rng.choice(["none", "linear", "ntk", "banded", "yarn"]) if R > 2 else "none",
                "far": max(T, _log(rng, 512, 1 << 20)), "order": rng.choice(["tokens", "fused", "heads"]),
                "inverse": rng.random() < 0.5}
    if op == "loss":
        K = 8 * _log(rng, 8, 1024)
        V = _log(rng, 500, 131072)
        T = _log(rng, 1, max(2, min(8192, 8192 * 32000 * 4096 // (K * V), 8192 * 32000 // V)))
        return {"op": op, "T": T, "V": V, "K": K, "grad": rng.random() < 0.7,
                "reduction": rng.choice(["none", "sum", "mean"]), "ignored": rng.choice([0.0, 0.0, 0.2, 0.6])}
    K = 64 * _log(rng, 1, 344)
    return {"op": op, "T": rng.choice([1, 1, 1, 2, 4, 8, 16, rng.randint(1, 64)]),
            "N": _log(rng, 64, 22016), "K": K, "book": rng.choice(["nf4", "int4", "grid"])}


# ---- inputs --------------------------------------------------------------------------------------

def _generator(seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(int(seed))
    return g


def _config(case):
    """The rotary settings that a program keeps beside its model."""
    c = {"rotary_dim": case["R"], "layout": case["layout"], "base": 10000.0, "scaling": case["scaling"]}
    if case["scaling"] != "none":
        c["factor"] = 4.0
    if case["scaling"] in ("banded", "yarn"):
        c["original_length"] = 4096
    return c


def _rope_inputs(case, g):
    B, T, Hq, Hk, D, t = (case[k] for k in ("B", "T", "Hq", "Hk", "D", "type"))
    dtype = TYPES[t]
    if case["order"] == "fused":        # q, k and v beside one another, as one projection writes them
        qkv = torch.randn(B, T, Hq + 2 * Hk, D, device=DEVICE, generator=g).to(dtype)
        q, k = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hk]
    elif case["order"] == "heads":      # [batch, head, token, dim] in memory
        q = torch.randn(B, Hq, T, D, device=DEVICE, generator=g).to(dtype).transpose(1, 2)
        k = torch.randn(B, Hk, T, D, device=DEVICE, generator=g).to(dtype).transpose(1, 2)
    else:
        q = torch.randn(B, T, Hq, D, device=DEVICE, generator=g).to(dtype)
        k = torch.randn(B, T, Hk, D, device=DEVICE, generator=g).to(dtype)
    first = torch.randint(0, case["far"] - T + 1, (B, 1), device=DEVICE, generator=g)
    return {"q": q, "k": k, "positions": first + torch.arange(T, device=DEVICE), "config": _config(case),
            "inverse": case["inverse"]}


def _loss_inputs(case, g):
    T, V, K = case["T"], case["V"], case["K"]
    W = torch.empty(V, K, device=DEVICE, dtype=torch.bfloat16).normal_(0.0, 0.02, generator=g)
    targets = torch.randint(0, V, (T,), device=DEVICE, generator=g)
    # hidden states after the last norm; each leans towards its target by its own amount (target logits 0 .. 16)
    lean = torch.rand(T, 1, device=DEVICE, generator=g) * min(1.0, 16.0 / (0.02 * K))
    X = torch.randn(T, K, device=DEVICE, generator=g)
    X = (X + lean * W[targets].float() / 0.02).to(torch.bfloat16)
    out = torch.rand(T, device=DEVICE, generator=g) < case["ignored"]
    out[0] = False                      # a mean has at least one token
    targets[out] = IGNORE
    weights = torch.rand(T, device=DEVICE, generator=g) if case["reduction"] == "none" and case["grad"] else None
    return {"X": X, "W": W, "targets": targets, "reduction": case["reduction"], "grad": case["grad"], "dloss": weights}


def _levels(book):
    if book == "int4":
        return [k / 7 for k in range(-7, 8)]
    if book == "grid":
        return [k / 8 for k in range(-8, 8)]
    quantile = lambda p: torch.special.ndtri(p)  # noqa: E731
    up = quantile(torch.linspace(0.9677, 0.5, 9, dtype=torch.float64)[:-1])
    down = -quantile(torch.linspace(0.9677, 0.5, 8, dtype=torch.float64)[:-1])
    lv = torch.cat([down / up[0], torch.zeros(1, dtype=torch.float64), up.flip(0) / up[0]])
    lv[0] = -1.0
    return lv.to(torch.float32).tolist()


def _matvec_inputs(case, g):
    T, N, K = case["T"], case["N"], case["K"]
    lv = torch.tensor(_levels(case["book"]), device=DEVICE)
    between = (lv[1:] + lv[:-1]) / 2
    codes = torch.empty(N, K // 2, dtype=torch.uint8, device=DEVICE)
    absmax = torch.empty(N, K // BLOCK, device=DEVICE)
    for a in range(0, N, 4096):         # a slab of rows at a time keeps the inputs' own memory small
        w = torch.randn(min(4096, N - a), K // BLOCK, BLOCK, device=DEVICE, generator=g) * 0.02
        m = w.abs().amax(-1, keepdim=True)
        c = torch.bucketize(w / m, between).to(torch.uint8).view(-1, K // 2, 2)
        codes[a:a + 4096] = c[..., 0] << 4 | c[..., 1]
        absmax[a:a + 4096] = m[..., 0]
    X = torch.randn(T, K, device=DEVICE, generator=g).to(torch.bfloat16)
    return {"X": X, "codes": codes.view(-1), "absmax": absmax.view(-1), "N": N, "levels": _levels(case["book"])}


def prepare(case, seed):
    g = _generator(seed)
    make = {"rope": _rope_inputs, "loss": _loss_inputs, "matvec": _matvec_inputs}[case["op"]]
    return {"op": case["op"], **make(case, g)}


# ---- the plain forms -------------------------------------------------------------------------------

def _plain_frequencies(c, device):
    """Angle per position of each pair, and the factor on the result."""
    R, base, s = c["rotary_dim"], c["base"], c.get("factor", 1.0)
    i = torch.arange(R // 2, dtype=torch.float64, device=device)
    kind = c["scaling"]
    if kind == "ntk":
        base = base * s ** (R / (R - 2))
    theta = base ** (-2.0 * i / R)
    if kind == "linear":
        return theta / s, 1.0
    if kind == "banded":                # short waves stay, long ones are stretched, those between are mixed
        turns = c["original_length"] * theta / (2 * math.pi)
        mix = ((turns - 1.0) / (4.0 - 1.0)).clamp(0.0, 1.0)
        return (1 - mix) * theta / s + mix * theta, 1.0
    if kind == "yarn":
        at = lambda turns: R * math.log(c["original_length"] / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), R - 1)
        ramp = ((i - lo) / (hi - lo if hi > lo else 0.001)).clamp(0.0, 1.0)
        return theta / s * ramp + theta * (1 - ramp), 0.1 * math.log(s) + 1.0
    return theta, 1.0


def _plain_turn(x, cos, sin, R, layout):
    f = x.float()
    if layout == "half":
        a, b = f[..., :R // 2], f[..., R // 2:R]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = f[..., 0:R:2], f[..., 1:R:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([turned, f[..., R:]], -1).to(x.dtype)


def _plain_rope(s):
    c = s["config"]
    theta, m = _plain_frequencies(c, s["q"].device)
    angle = s["positions"].to(torch.float64)[..., None] * theta       # far positions need 64 bits
    cos, sin = (angle.cos() * m).float()[:, :, None], (angle.sin() * m).float()[:, :, None]
    if s["inverse"]:
        sin = -sin
    return (_plain_turn(s["q"], cos, sin, c["rotary_dim"], c["layout"]),
            _plain_turn(s["k"], cos, sin, c["rotary_dim"], c["layout"]))


def _plain_loss(s):
    X, W, targets = s["X"].float(), s["W"].float(), s["targets"]
    used = targets != IGNORE
    at = torch.where(used, targets, 0)[:, None]
    logits = X @ W.t()
    d = logits - logits.gather(1, at)                   # against the target's: small losses keep their digits
    top = d.amax(-1, keepdim=True)                      # >= 0
    e = (d - top).exp().scatter_(1, at, 0.0)
    rest, one = e.sum(-1, keepdim=True), (-top).exp()   # the other words, and the target
    loss = torch.where(used, torch.where(top > 0, top + (rest + one).log(), rest.log1p())[:, 0], 0.0)
    share = used / used.sum() if s["reduction"] == "mean" else used.float()
    if s["dloss"] is not None:
        share = share * s["dloss"]
    total = loss if s["reduction"] == "none" else (loss * share).sum()
    if not s["grad"]:
        return total, None
    p = e.scatter_(1, at, -rest) / (rest + one)         # softmax - 1 at the target
    return total, ((p * share[:, None]) @ W).to(s["X"].dtype)


def _plain_matvec(s):
    codes = s["codes"]
    lv = torch.tensor(s["levels"], dtype=torch.float32, device=codes.device)
    both = torch.stack([codes >> 4, codes & 15], -1).int()
    w = (lv[both].view(-1, BLOCK) * s["absmax"][:, None]).view(s["N"], -1)
    return (s["X"].float() @ w.t()).to(torch.bfloat16)


def run(state):
    op = state["op"]
    if own:
        import bit_nf4_quantized_14_b200 as q
        if op == "rope":
            return q.rotary(state["q"], state["k"], q.RotaryConfig(**state["config"]), positions=state["positions"],
                            inverse=state["inverse"])
        if op == "loss":
            return q.vocab_loss(state["X"], state["W"], state["targets"], ignore_index=IGNORE,
                                reduction=state["reduction"], dloss=state["dloss"], need_dx=state["grad"])
        return q.codebook_linear(state["X"], state["codes"], state["absmax"], state["N"], state["levels"])
    return {"rope": _plain_rope, "loss": _plain_loss, "matvec": _plain_matvec}[op](state)


def work(case):
    if case["op"] == "rope":
        tokens, heads = case["B"] * case["T"], case["Hq"] + case["Hk"]
        size = 2 if case["type"] == "bf16" else 4
        return {"bytes": 2 * tokens * heads * case["D"] * size + 8 * tokens, "flops": 3 * tokens * heads * case["R"]}
    if case["op"] == "loss":
        T, V, K = case["T"], case["V"], case["K"]
        return {"bytes": 2 * V * K + 8 * T + 2 * T * K * (2 if case["grad"] else 1) + 4 * T,
                "flops": 2 * T * V * K * (2 if case["grad"] else 1)}
    T, N, K = case["T"], case["N"], case["K"]
    return {"bytes": N * K // 2 + 4 * N * (K // BLOCK) + 2 * T * (N + K), "flops": 2 * T * N * K}


# ---- the definitions in 64 bits ----------------------------------------------------------------------

def _exact_rope(s):
    """Each pair as a complex number, multiplied by m exp(+-i p theta)."""
    c = s["config"]
    R, base, factor, kind = c["rotary_dim"], c["base"], c.get("factor", 1.0), c["scaling"]
    theta, m = [], 1.0
    for i in range(R // 2):
        t = math.pow(base * (factor ** (R / (R - 2)) if kind == "ntk" else 1.0), -2 * i / R)
        if kind == "linear":
            t /= factor
        elif kind == "banded":
            wave, L = 2 * math.pi / t, c["original_length"]
            if wave > L / 1.0:
                t /= factor
            elif wave >= L / 4.0:
                mix = (L / wave - 1.0) / 3.0
                t = (1 - mix) * t / factor + mix * t
        elif kind == "yarn":
            where = [R * math.log(c["original_length"] / (b * 2 * math.pi)) / (2 * math.log(base)) for b in (32, 1)]
            lo, hi = max(math.floor(where[0]), 0), min(math.ceil(where[1]), R - 1)
            ramp = min(max((i - lo) / (hi - lo if hi > lo else 0.001), 0.0), 1.0)
            t = (t / factor) * ramp + t * (1 - ramp)
            m = 0.1 * math.log(factor) + 1.0
        theta.append(t)
    theta = torch.tensor(theta, dtype=torch.float64, device=DEVICE)
    angle = s["positions"].double().unsqueeze(-1) * theta * (-1.0 if s["inverse"] else 1.0)
    turn = torch.polar(torch.full_like(angle, m), angle).unsqueeze(2)
    got = []
    for x in (s["q"], s["k"]):
        x = x.double()
        h = x[..., :R].unflatten(-1, (2, R // 2)).transpose(-1, -2) if c["layout"] == "half" else \
            x[..., :R].unflatten(-1, (R // 2, 2))
        y = torch.view_as_real(torch.view_as_complex(h.contiguous()) * turn)
        y = y.transpose(-1, -2).flatten(-2) if c["layout"] == "half" else y.flatten(-2)
        got.append(torch.cat([y, x[..., R:]], -1))
    return tuple(got)


def _exact_loss(s):
    X, W, targets = s["X"].double(), s["W"].double(), s["targets"]
    rows = (targets != IGNORE).nonzero()[:, 0]
    y = targets[rows]
    logits = X[rows] @ W.t()
    lse = torch.logsumexp(logits, 1)
    each = torch.zeros(X.shape[0], dtype=torch.float64, device=DEVICE)
    each[rows] = lse - logits[torch.arange(len(rows), device=DEVICE), y]
    total = {"none": each, "sum": each.sum(), "mean": each.sum() / max(1, len(rows))}[s["reduction"]]
    if not s["grad"]:
        return total, None
    g = torch.ones(len(rows), dtype=torch.float64, device=DEVICE) if s["dloss"] is None else s["dloss"][rows].double()
    if s["reduction"] == "mean":
        g = g / len(rows)
    p = logits.sub_(lse[:, None]).exp_()
    dX = torch.zeros_like(X)
    dX[rows] = (p @ W - W[y]) * g[:, None]
    return total, dX


def _exact_matvec(s):
    """Row slabs of the weight in 64 bits."""
    X, N = s["X"].double(), s["N"]
    K = X.shape[1]
    lv = torch.tensor(s["levels"], dtype=torch.float32, device=DEVICE).double()
    codes, absmax = s["codes"].view(N, K // 2), s["absmax"].view(N, K // BLOCK).double()
    got = []
    for a in range(0, N, 2048):
        c = codes[a:a + 2048]
        w = torch.empty(c.shape[0], K, dtype=torch.float64, device=DEVICE)
        w[:, 0::2] = lv[(c >> 4).long()]
        w[:, 1::2] = lv[(c & 15).long()]
        w *= absmax[a:a + 2048].repeat_interleave(BLOCK, dim=1)
        got.append(X @ w.t())
    return torch.cat(got, 1)


def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "loss": _exact_loss, "matvec": _exact_matvec}[s["op"]](s)
