"""The measured operators around the dispatch / combine path, with their plain forms.

  route     gate logits -> the k experts of each token and their weights
  balance   the balance loss of a routing, its per-expert counts and mean
            probabilities, per sequence
  gradient  the gradient of the gate logits from the routing weights, from the
            balance loss, or from both
  experts   the experts' products on the dispatched rows with 4-bit weights
            (E2M1 codes, one UE8M0 scale byte per 32 inputs), with or without
            the gated activation

With `own` false, run() computes them with elementary torch operations; with
`own` true it calls the package.  `exact` computes them in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
F32, F64, BF16, I32, U8 = torch.float32, torch.float64, torch.bfloat16, torch.int32, torch.uint8

# E2M1 magnitudes by code (bit 3 is the sign)
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------- the cases

def _routing(name, op, T, E, k, G=1, KG=1, score="softmax", norm=True, bf16=False, bias=False,
             pad=0.0, B=1, weights=True, loss=True):
    c = dict(op=op, T=T, E=E, k=k, G=G, KG=KG, score=score, norm=norm, bf16=bf16, bias=bias,
             pad=pad, B=B, weights=weights, loss=loss)
    return dict(c, name=name) if name else c


def _experts(name, T, E, k, K, N, cap=0, fmt=0, gated=False, skew=0.0):
    c = dict(op="experts", T=T, E=E, k=k, K=K, N=N, cap=cap, fmt=fmt, gated=gated, skew=skew)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one token of a decode step: the choice before its dispatch
        _routing("route 1 token", "route", 1, 256, 8, G=8, KG=4),
        # a large prefill of the group-limited model, with the sigmoid gate, a
        # choice bias and padding at the end of the batch
        _routing("route 16384 grouped", "route", 16384, 256, 8, G=8, KG=4, score="sigmoid",
                 bias=True, pad=0.02),
        # a prefill of the 64-expert model, bf16 logits, plain softmax weights
        _routing("route 8192 of 64 bf16", "route", 8192, 64, 6, norm=False, bf16=True),
        # training: the loss over four sequences with padding
        _routing("balance 16384", "balance", 16384, 256, 8, G=8, KG=4, B=4, pad=0.05),
        # a small training batch of odd sequences
        _routing("balance 1000 bf16", "balance", 1000, 64, 6, score="sigmoid", bf16=True, B=8),
        # the training step's gradient from both, at the largest batch
        _routing("gradient 16384", "gradient", 16384, 256, 8, G=8, KG=4, B=4, pad=0.05),
        # a small ragged batch whose experts fill no power of two, bf16
        _routing("gradient 1999 of 96 bf16", "gradient", 1999, 96, 6, score="sigmoid", bf16=True,
                 loss=False),
        # one decoded token: gate and up products of its eight experts
        _experts("experts 1 token", 1, 256, 8, 7168, 2048, gated=True),
        # the decode batch: every expert's weights are read, FP8 rows in the
        # fixed-capacity layout that dispatch leaves
        _experts("experts decode fp8", 128, 256, 8, 7168, 2048, cap=128, fmt=1, gated=True),
        # its second product, back to the hidden size, on bf16 rows
        _experts("experts decode down", 128, 256, 8, 2048, 7168, cap=128),
        # a mid-size batch with skewed routing: hot experts hold many rows
        _experts("experts skewed 512", 512, 64, 6, 4096, 1408, gated=True, skew=1.2),
        # a tiny model: odd output size, UE8M0 row scales
        _experts("experts tiny", 64, 8, 2, 256, 999, fmt=2),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "balance", "gradient", "experts", "experts"])
    if op != "experts":
        E = _log_int(rng, 4, 256)
        G = rng.choice([g for g in range(1, 17) if E % g == 0 and E // g >= 2])
        KG = rng.randint((G + 1) // 2, G)
        k = rng.randint(1, min(12, KG * (E // G)))
        B = 1 if op == "route" else rng.randint(1, 16)
        T = _log_int(rng, 1 if op == "route" else 2 * B, 16000)
        T = max(1, T // B) * B
        w, l = rng.choice([(True, True), (True, False), (False, True)])
        # a single normalised weight is 1 whatever the logits: no gradient
        norm = rng.random() < 0.5 and (k > 1 or op != "gradient")
        return _routing(None, op, T, E, k, G, KG, rng.choice(["softmax", "sigmoid"]),
                        norm, rng.random() < 0.5, rng.random() < 0.3,
                        rng.choice([0.0, 0.0, 0.1]), B, w, l)
    E = rng.choice([8, 16, 32, 64, 128, 256])
    k = rng.randint(1, 8)
    T = _log_int(rng, 1, 512)
    fmt = rng.choice([0, 0, 1, 2])
    unit = 128 if fmt else 32
    K = unit * max(1, _log_int(rng, 256, 7168) // unit)
    gated = rng.random() < 0.5
    most = 256 * 2048 * 7168 // (E * K * (2 if gated else 1))
    N = _log_int(rng, 48, max(48, min(7168, most)))
    cap = rng.choice([0, 0, max(1, math.ceil(T * k / E)), T])
    return _experts(None, T, E, k, K, N, cap, fmt, gated, rng.choice([0.0, 1.0]))


def work(case):
    c = case
    T, E, k = c["T"], c["E"], c["k"]
    if c["op"] == "experts":
        # experts that some token chose (expected number at uniform routing)
        hit = min(E, T * k) if T == 1 else E * (1 - (1 - k / E) ** T)
        n2 = c["N"] * (2 if c["gated"] else 1)
        row = c["K"] * 2 if c["fmt"] == 0 else c["K"] + c["K"] // 128 * (4 if c["fmt"] == 1 else 1)
        rows = T * k
        return {"bytes": hit * n2 * (c["K"] // 2 + c["K"] // 32) + rows * (row + c["N"] * 2),
                "flops": 2.0 * rows * n2 * c["K"]}
    el = 2 if c["bf16"] else 4
    logits = T * E * el
    if c["op"] == "route":
        return {"bytes": logits + T * k * 8 + (E * 4 if c["bias"] else 0), "flops": 4.0 * T * E}
    if c["op"] == "balance":
        return {"bytes": logits + T * k * 4 + c["B"] * (E * 8 + 4) + 4, "flops": 6.0 * T * E}
    return {"bytes": 2 * logits + T * k * 4 + (T * k * 4 if c["weights"] else 0)
            + (c["B"] * (E * 4 + 4) + 4 if c["loss"] else 0), "flops": 8.0 * T * E}


# ---------------------------------------------------------------- the inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _gate_logits(c, g):
    """Logits as a trained gate gives them: a common preference for some
    experts on top of what each token asks for."""
    x = torch.randn((c["T"], c["E"]), generator=g, device=DEV)
    x = 1.5 * x + 0.3 * torch.randn((1, c["E"]), generator=g, device=DEV)
    return x.to(BF16) if c["bf16"] else x


def prepare(case, seed):
    c, g = case, _gen(seed)
    if c["op"] == "experts":
        return _prepare_experts(c, g)
    T, E, k, B = c["T"], c["E"], c["k"], c["B"]
    s = dict(case=c, logits=_gate_logits(c, g), bias=None, valid=None)
    if c["bias"]:
        s["bias"] = 0.2 * torch.randn(E, generator=g, device=DEV)
    if c["pad"]:
        L = T // B
        at = torch.arange(L, device=DEV).repeat(B, 1)
        ends = L - (2 * c["pad"] * L * torch.rand((B, 1), generator=g, device=DEV)).long()
        s["valid"] = (at < ends).reshape(-1).to(U8)
    if c["op"] == "route":
        s["idx"] = torch.empty((T, k), dtype=I32, device=DEV)
        s["w"] = torch.empty((T, k), dtype=F32, device=DEV)
        return s
    s["coef"] = 0.01
    s["idx"] = _choose(c, s["logits"], s["bias"], s["valid"])
    if c["op"] == "balance":
        s["counts"] = torch.empty((B, E), dtype=I32, device=DEV)
        s["mean"] = torch.empty((B, E), dtype=F32, device=DEV)
        s["n"] = torch.empty(B, dtype=I32, device=DEV)
        s["loss"] = torch.empty(1, dtype=F32, device=DEV)
        s["space"] = torch.empty(64 << 20, dtype=U8, device=DEV)
        return s
    s["dw"] = torch.randn((T, k), generator=g, device=DEV) if c["weights"] else None
    s["dx"] = torch.empty_like(s["logits"])
    s["counts"] = s["n"] = s["dloss"] = None
    if c["loss"]:
        s["counts"], s["n"] = _counts(c, s["idx"], s["valid"])
        s["dloss"] = torch.rand(1, generator=g, device=DEV) + 0.5
    return s


def _codes_of_normals():
    """E2M1 codes of 256 equally likely values of a normal variable whose
    block maximum lands on 6."""
    z = torch.distributions.Normal(0.0, 1.0).icdf((torch.arange(256) + 0.5) / 256) * (6 / 2.6)
    near = (z.abs()[:, None] - torch.tensor(E2M1)[None]).abs().argmin(1)
    return (near + 8 * (z < 0)).to(U8)


def _prepare_experts(c, g):
    T, E, k, K, N, cap = c["T"], c["E"], c["k"], c["K"], c["N"], c["cap"]
    # distinct experts per token; skew: popularity falls with the rank
    pop = -c["skew"] * torch.log(torch.arange(1, E + 1, device=DEV, dtype=F32))
    noise = -torch.log(-torch.log(torch.rand((T, E), generator=g, device=DEV).clamp(1e-9, 1 - 1e-7)))
    idx = (pop + noise).topk(k, 1).indices.reshape(-1)
    count = torch.bincount(idx, minlength=E)
    offset = torch.zeros(E + 1, dtype=torch.int64, device=DEV)
    offset[1:] = count.cumsum(0)
    R = T * k if cap == 0 else E * cap
    n2 = N * (2 if c["gated"] else 1)
    bits = torch.randint(0, 256, (E, n2, K // 2, 2), generator=g, device=DEV, dtype=U8)
    code = _codes_of_normals().to(DEV)[bits.int()]
    codes = code[..., 0] | (code[..., 1] << 4)
    del bits, code
    mid = 127 - 1 - round(math.log2(2.0 * math.sqrt(K)))
    scales = torch.randint(mid, mid + 3, (E, n2, K // 32), generator=g, device=DEV, dtype=U8)
    x = torch.randn((R, K), generator=g, device=DEV)
    row_scales = None
    if c["fmt"]:
        a = x.view(R, K // 128, 128).abs().amax(2)
        if c["fmt"] == 1:
            sc = row_scales = a / 448
        else:
            e = torch.ceil(torch.log2(a / 448)).clamp(-127, 127)
            sc, row_scales = torch.exp2(e), (e + 127).to(U8)
        x = (x.view(R, K // 128, 128) / sc[..., None]).clamp(-448, 448)
        x = x.view(R, K).to(torch.float8_e4m3fn).view(U8)
    else:
        x = x.to(BF16)
    return dict(case=c, x=x, row_scales=row_scales, codes=codes, scales=scales,
                count=count.to(I32), offset=offset.to(I32),
                slot_of=torch.empty((T, k), dtype=I32, device=DEV),
                src=torch.empty(R, dtype=I32, device=DEV),
                status=torch.zeros(2, dtype=I32, device=DEV),
                out=torch.zeros((R, N), dtype=BF16, device=DEV))


# ------------------------------------------------------------- the plain forms

def _on(x):
    """Experts that a token may take: those with a finite logit."""
    return torch.isfinite(x)


def _choose(c, logits, bias, valid):
    x = logits.float()
    key = x if bias is None else x + bias
    inf = float("inf")
    key = torch.where(_on(x) & torch.isfinite(key), key, -inf)
    if valid is not None:
        key = torch.where(valid[:, None] != 0, key, -inf)
    if c["G"] > 1:
        by = key.view(c["T"], c["G"], -1)
        low = -float(torch.finfo(F32).max)
        top = by.topk(min(2, by.shape[2]), 2).values.double().clamp(min=low).sum(2)
        keep = top.sort(dim=1, descending=True, stable=True).indices[:, :c["KG"]]
        kept = torch.zeros_like(top, dtype=torch.bool).scatter_(1, keep, True)
        key = torch.where(kept[:, :, None], by, -inf).view(c["T"], -1)
    top = key.sort(dim=1, descending=True, stable=True)
    return torch.where(top.values[:, :c["k"]] > -inf, top.indices[:, :c["k"]], -1).to(I32)


def _log_score(c, x):
    """Scores whose softmax is the weight: the logits, or their log sigmoids."""
    if c["score"] == "softmax":
        return x
    return x.clamp(max=0) - torch.log1p(torch.exp(-x.abs()))


def _softmax(l, on):
    m = torch.where(on, l, -float("inf")).amax(1, keepdim=True)
    e = torch.where(on, torch.exp(torch.where(on, l - m, 0)), 0)
    return e / e.sum(1, keepdim=True).clamp(min=1e-30)


def _probs(c, x):
    return _softmax(_log_score(c, x), _on(x))


def _entries(c, logits, idx):
    """Logits at the chosen experts, and which entries are there."""
    x = logits.float().gather(1, idx.long().clamp(min=0))
    return x, (idx >= 0) & _on(x)


def _weights(c, logits, idx):
    x, there = _entries(c, logits, idx)
    if c["norm"]:
        return _softmax(_log_score(c, x), there)
    if c["score"] == "sigmoid":
        return torch.where(there, 1 / (1 + torch.exp(-x)), 0)
    return torch.where(there, _probs(c, logits.float()).gather(1, idx.long().clamp(min=0)), 0)


def _counts(c, idx, valid):
    E, B, k = c["E"], c["B"], c["k"]
    live = torch.ones(c["T"], dtype=I32, device=DEV) if valid is None else (valid != 0).to(I32)
    use = (idx >= 0) & (live[:, None] != 0)
    at = torch.where(use, idx, E).view(B, -1).long()
    counts = torch.zeros((B, E + 1), dtype=I32, device=DEV)
    counts.scatter_add_(1, at, torch.ones_like(at, dtype=I32))
    return counts[:, :E].contiguous(), live.view(B, -1).sum(1).to(I32)


def _plain_route(s):
    c = s["case"]
    idx = _choose(c, s["logits"], s["bias"], s["valid"])
    return idx, _weights(c, s["logits"], idx)


def _plain_balance(s):
    c = s["case"]
    E, B = c["E"], c["B"]
    p = _probs(c, s["logits"].float())
    if s["valid"] is not None:
        p = torch.where(s["valid"][:, None] != 0, p, 0)
    counts, n = _counts(c, s["idx"], s["valid"])
    m = n.clamp(min=1).double()[:, None]
    mean = p.view(B, -1, E).sum(1, dtype=F64) / m
    loss = (counts.double() * E / (c["k"] * m) * mean).sum() * (s["coef"] / B)
    return counts, mean.float(), n, loss.float().view(1)


def _plain_gradient(s):
    c = s["case"]
    T, E, B = c["T"], c["E"], c["B"]
    x = s["logits"].float()
    dx = torch.zeros_like(x)
    sig = c["score"] == "sigmoid"
    slope = 1 / (1 + torch.exp(x)) if sig else 1.0      # of the log score
    if c["loss"]:
        n = s["n"].clamp(min=1).float()
        a = s["counts"].float() * (s["coef"] * E / (B * c["k"]) * s["dloss"] / (n * n))[:, None]
        a = a[:, None, :].expand(B, T // B, E).reshape(T, E)
        p = _probs(c, x)
        dx = dx + p * (a - (a * p).sum(1, keepdim=True)) * slope
    if c["weights"]:
        xe, there = _entries(c, s["logits"], s["idx"])
        at = s["idx"].long().clamp(min=0)
        g = torch.where(there, s["dw"], 0)
        if c["norm"]:
            q = _softmax(_log_score(c, xe), there)
            d = q * (g - (g * q).sum(1, keepdim=True))
            if sig:
                d = d / (1 + torch.exp(xe))
        elif sig:
            y = 1 / (1 + torch.exp(-xe))
            d = g * y * (1 / (1 + torch.exp(xe)))
        else:
            p = _probs(c, x)
            q = torch.where(there, p.gather(1, at), 0)
            dx = dx - p * (g * q).sum(1, keepdim=True)
            d = g * q
        dx = dx.scatter_add(1, at, torch.where(there, d, 0))
    dx = torch.where(_on(x), dx, 0)
    if s["valid"] is not None:
        dx = torch.where(s["valid"][:, None] != 0, dx, 0)
    return dx.to(s["logits"].dtype)


def _plain_experts(s):
    c = s["case"]
    T, E, k, K, N, cap = c["T"], c["E"], c["k"], c["K"], c["N"], c["cap"]
    R = s["x"].shape[0]
    if c["fmt"]:
        x = s["x"].view(torch.float8_e4m3fn).float()
        sc = s["row_scales"] if c["fmt"] == 1 else torch.exp2(s["row_scales"].float() - 127)
        x = (x.view(R, K // 128, 128) * sc[..., None]).view(R, K)
    else:
        x = s["x"].float()
    r = torch.arange(R, device=DEV)
    if cap:
        e, at = r // cap, r % cap
    else:
        e = torch.searchsorted(s["offset"][1:].contiguous(), r.to(I32), right=True).clamp(max=E - 1)
        at = r - s["offset"][e]
    if not cap and R < E:                 # fewer rows than experts: each row with its expert's weights
        y = _products(x[:, None], s["codes"][e], s["scales"][e], c)[:, 0]
        return y.to(BF16)
    M = cap if cap else T                 # a token takes an expert at most once
    m = torch.arange(M, device=DEV)
    use = m[None] < s["count"][:, None]
    start = torch.arange(E, device=DEV) * cap if cap else s["offset"][:E].long()
    rows = (start[:, None] + m[None]).clamp(max=R - 1)
    y = _products(torch.where(use[..., None], x[rows], 0), s["codes"], s["scales"], c)
    at = at.clamp(0, M - 1)
    return torch.where(use[e, at][:, None], y[e, at].to(BF16), s["out"])


def _products(x, codes, scales, c):
    """x [B, M, K] with the weights of each B, decoded; the gated activation."""
    K, N = c["K"], c["N"]
    mag = torch.tensor(E2M1, device=DEV)
    value = torch.cat([mag, -mag])
    byte = torch.arange(256, device=DEV)
    pair = torch.stack([value[byte & 15], value[byte >> 4]], 1)
    w = pair[codes.int()].view(len(codes), -1, K // 32, 32)
    w = w.mul_(torch.exp2(scales.float() - 127)[..., None]).view(len(codes), -1, K)
    y = torch.bmm(w, x.transpose(1, 2).contiguous()).transpose(1, 2)
    if c["gated"]:
        gate, up = y[..., :N], y[..., N:]
        y = gate / (1 + torch.exp(-gate)) * up
    return y


# -------------------------------------------------------------- the package's

def _package_run(s):
    import combine_ep_layout_09_amd as ep
    c = s["case"]
    if c["op"] == "experts":
        prob = ep.Problem(c["T"], c["K"], c["k"], c["E"], c["cap"], c["fmt"])
        mm = ep.ExpertW4(c["K"], c["N"], in_format=c["fmt"], activation=int(c["gated"]))
        lay = ep.Layout(s["count"], s["offset"], s["slot_of"], s["src"], s["status"])
        ep.ep_expert_w4(prob, mm, s["x"], lay, s["codes"], s["scales"], s["out"],
                        row_scales=s["row_scales"])
        return s["out"]
    rt = ep.Routing(c["T"], c["E"], c["k"], num_groups=c["G"], topk_groups=c["KG"],
                    score=c["score"], normalize=c["norm"], num_seqs=c["B"])
    if c["op"] == "route":
        ep.ep_route(rt, s["logits"], s["idx"], s["w"], expert_bias=s["bias"], valid=s["valid"])
        return s["idx"], s["w"]
    if c["op"] == "balance":
        ep.ep_balance_loss(rt, s["logits"], s["idx"], s["coef"], s["counts"], s["mean"], s["n"],
                           s["loss"], s["space"], valid=s["valid"])
        return s["counts"], s["mean"], s["n"], s["loss"]
    ep.ep_route_backward(rt, s["logits"], s["idx"], s["dx"], d_weights=s["dw"], coef=s["coef"],
                         counts=s["counts"], num_valid=s["n"], d_loss=s["dloss"],
                         valid=s["valid"])
    return s["dx"]


def run(state):
    if own:
        return _package_run(state)
    return {"route": _plain_route, "balance": _plain_balance, "gradient": _plain_gradient,
            "experts": _plain_experts}[state["case"]["op"]](state)


# ---------------------------------------------------------- the 64-bit answers

def _exact_scores(c, x):
    """Probabilities over a token's experts, [T, E] in 64 bits."""
    ok = torch.isfinite(x)
    if c["score"] == "sigmoid":
        z = torch.sigmoid(x).masked_fill(~ok, 0)
        return z / z.sum(1, keepdim=True)
    return torch.softmax(x.masked_fill(~ok, -float("inf")), 1).nan_to_num(0)


def _exact_weights(c, x, idx):
    pos = idx.long().clamp(min=0)
    if c["score"] == "sigmoid" and not c["norm"]:
        z = torch.sigmoid(x).gather(1, pos)
    else:
        z = _exact_scores(c, x).gather(1, pos)
    z = z * (idx >= 0)
    if c["norm"]:
        t = z.sum(1, keepdim=True)
        z = z / torch.where(t > 0, t, torch.ones_like(t))
    return z


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    if c["op"] == "experts":
        return _exact_experts(s)
    x = s["logits"].double()
    if c["op"] == "route":
        idx = _choose(c, s["logits"], s["bias"], s["valid"])
        return None, _exact_weights(c, x, idx)
    B, E = c["B"], c["E"]
    live = torch.ones(c["T"], dtype=F64, device=DEV) if s["valid"] is None else s["valid"].double()
    hot = torch.zeros((c["T"], E), dtype=F64, device=DEV)
    hot.scatter_add_(1, s["idx"].long().clamp(min=0), (s["idx"] >= 0).double())
    f = (hot * live[:, None]).view(B, -1, E).sum(1)
    n = live.view(B, -1).sum(1)

    def total(z):
        mean = (_exact_scores(c, z) * live[:, None]).view(B, -1, E).sum(1) / n[:, None]
        return mean, s["coef"] / B * (E / c["k"] * f / n[:, None] * mean).sum()

    if c["op"] == "balance":
        mean, loss = total(x)
        return None, mean, None, loss.view(1)
    x.requires_grad_(True)
    goal = 0.0
    if c["loss"]:
        goal = goal + total(x)[1] * s["dloss"].double().sum()
    if c["weights"]:
        goal = goal + (_exact_weights(c, x, s["idx"]) * s["dw"].double() * live[:, None]).sum()
    return torch.autograd.grad(goal, x)[0]


def _exact_experts(s):
    c = s["case"]
    K, N, cap = c["K"], c["N"], c["cap"]
    out = s["out"].double()
    code = torch.arange(16, device=DEV)
    man, ex = (code & 1).double(), ((code >> 1) & 3).double()
    value = torch.where(ex == 0, man / 2, (1 + man / 2) * 2.0 ** (ex - 1)) * (1 - 2.0 * (code >> 3))
    count, offset = s["count"].tolist(), s["offset"].tolist()
    for e in range(c["E"]):
        a = e * cap if cap else offset[e]
        b = a + (min(count[e], cap) if cap else count[e])
        if a == b:
            continue
        x = s["x"][a:b]
        if c["fmt"]:
            x = x.view(torch.float8_e4m3fn).double()
            sc = s["row_scales"][a:b].double()
            x = x * (sc if c["fmt"] == 1 else 2.0 ** (sc - 127)).repeat_interleave(128, 1)
        else:
            x = x.double()
        q = s["codes"][e].long()
        w = torch.empty((q.shape[0], K), dtype=F64, device=DEV)
        w[:, 0::2] = value[q % 16]
        w[:, 1::2] = value[q // 16]
        w *= (2.0 ** (s["scales"][e].double() - 127)).repeat_interleave(32, 1)
        y = x @ w.t().contiguous()
        out[a:b] = torch.nn.functional.silu(y[:, :N]) * y[:, N:] if c["gated"] else y
    return out
