"""Cases for the operators on either side of the output head: the residual addition with its
root-mean-square norm (plain, 8-bit, gradient), the log probabilities of given tokens from logits
(with gradient), and the same straight from hidden rows and a head.

`run` computes a case in its plain form (elementary torch operations in 32 bits) or, with `own`
set, through the package's entry points; `exact` gives the values in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
EPS = 1e-6


def listed():
    return [
        # the hidden rows of one verify round (three drafts and the bonus position) before the head: latency
        {"name": "norm 4x2048", "op": "norm", "T": 4, "H": 2048, "dtype": "bf16", "out": "same"},
        # a prefill's rows on their way into 8-bit layers
        {"name": "norm int8 16384x2048", "op": "norm", "T": 16384, "H": 2048, "dtype": "bf16", "out": "int8"},
        # a training step's norm
        {"name": "norm grad 8192x2048", "op": "norm_grad", "T": 8192, "H": 2048, "dtype": "bf16"},
        # ragged token count, odd width, full precision
        {"name": "norm grad 301x2561", "op": "norm_grad", "T": 301, "H": 2561, "dtype": "f32"},
        # sampled tokens of one verify round over the full vocabulary, with the alternatives an API returns
        {"name": "logprobs 4x248320", "op": "logprobs", "R": 4, "V": 248320, "dtype": "f32", "top": 20, "masked": 0.0},
        # an odd vocabulary with most entries masked by a grammar
        {"name": "logprobs 129x40001", "op": "logprobs", "R": 129, "V": 40001, "dtype": "f16", "top": 5, "masked": 0.7},
        # a training step over a 64K vocabulary: no alternatives wanted
        {"name": "logprobs 2048x65536", "op": "logprobs", "R": 2048, "V": 65536, "dtype": "bf16", "top": 0, "masked": 0.0},
        # and its gradient
        {"name": "logprobs grad 2048x65536", "op": "logprobs_grad", "R": 2048, "V": 65536, "dtype": "bf16", "masked": 0.0},
        # gradient of a few rows of an odd masked vocabulary in full precision
        {"name": "logprobs grad 33x40001", "op": "logprobs_grad", "R": 33, "V": 40001, "dtype": "f32", "masked": 0.5},
        # one sequence's verify rows against the full head
        {"name": "head 4x248320x2048", "op": "head", "R": 4, "V": 248320, "H": 2048, "top": 20},
        # 64 sequences' verify rows against the full head
        {"name": "head 256x248320x2048", "op": "head", "R": 256, "V": 248320, "H": 2048, "top": 20},
        # scoring a sequence over the candidate table: many rows, no alternatives
        {"name": "head 2048x65536x2048", "op": "head", "R": 2048, "V": 65536, "H": 2048, "top": 0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "logprobs", "logprobs_grad", "head"])
    if op in ("norm", "norm_grad"):
        H = rng.choice([256, 512, 1024, 2048, 2560, 4096, 5120, 8192, 2 * rng.randrange(64, 4096) + 1])
        T = min(_log(rng, 1, 16384), 16384 * 2048 // H) | 1
        if op == "norm":
            return {"op": op, "T": T, "H": H, "dtype": rng.choice(["bf16", "bf16", "f16", "f32"]),
                    "out": rng.choice(["same", "int8", "e4m3"])}
        return {"op": op, "T": T // 2 | 1, "H": H, "dtype": rng.choice(["bf16", "f16", "f32"])}
    if op in ("logprobs", "logprobs_grad"):
        V = rng.choice([32768, 65536, 248320, _log(rng, 1000, 250000) | 1])
        R = max(1, min(_log(rng, 1, 2048), 2048 * 65536 // 2 // V))
        case = {"op": op, "R": R, "V": V, "dtype": rng.choice(["bf16", "f16", "f32"]),
                "masked": rng.choice([0.0, 0.0, rng.uniform(0.1, 0.95)])}
        if op == "logprobs":
            case["top"] = rng.choice([0, 1, 5, 20, 32])
        return case
    H = rng.choice([256, 512, 1024, 2048, 2560, 4096, 16 * (2 * rng.randrange(8, 64) + 1)])
    V = rng.choice([32768, 65536, 248320, _log(rng, 1000, 248320) | 1])
    V = min(V, 248320 * 2048 // H)
    R = max(1, min(_log(rng, 1, 2048), 256 * 248320 * 2048 // (V * H)))
    return {"op": "head", "R": R, "V": V, "H": H, "top": rng.choice([0, 1, 5, 20])}


# ---------------------------------------------------------------------------
# Inputs


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _tokens(g, R, V):
    """Given tokens: any id, and every eighth row a padding position with none."""
    t = torch.randint(0, V, (R,), generator=g, device="cuda", dtype=torch.int32)
    t[7::8] = -100
    return t


def _logits(g, R, V, dtype, masked):
    """Logits as a head gives them: a per-token bias (frequent tokens score higher), noise, and masked places at -inf."""
    bias = _randn(g, V) * 1.5
    x = _randn(g, R, V)
    x = x.mul_(1.5).add_(bias)
    if masked > 0:
        x.masked_fill_(torch.rand(R, V, generator=g, device="cuda") < masked, -math.inf)
        x[:, 0] = 0.5  # the end-of-sequence token stays allowed
    return x.to(dtype)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = {"case": dict(case)}
    if op in ("norm", "norm_grad"):
        T, H, dt = case["T"], case["H"], DTYPES[case["dtype"]]
        channel = 1 + 20 * (torch.rand(H, generator=g, device="cuda") < 0.003)  # a few outlier channels of the stream
        s["weight"] = (1 + 0.1 * _randn(g, H)).to(dt)
        s["residual"] = (_randn(g, T, H) * 2 * channel).to(dt)
        s["x"] = _randn(g, T, H).to(dt)
        s["h"] = torch.empty_like(s["x"])
        if op == "norm":
            out = {"same": dt, "int8": torch.int8, "e4m3": torch.float8_e4m3fn}[case["out"]]
            s["y"] = torch.empty(T, H, dtype=out, device="cuda")
            s["scales"] = torch.empty(T, dtype=torch.float32, device="cuda")
        else:
            s["h"].copy_(s["residual"])           # what the forward pass saved
            s["dy"] = (_randn(g, T, H) * 1e-2).to(dt)
            s["dh"] = s["x"].mul_(1e-2)           # the stream's own gradient
            s["dx"] = torch.empty_like(s["dy"])
            s["dweight"] = torch.empty(H, dtype=torch.float32, device="cuda")
    elif op in ("logprobs", "logprobs_grad"):
        R, V = case["R"], case["V"]
        s["logits"] = _logits(g, R, V, DTYPES[case["dtype"]], case["masked"])
        s["tokens"] = _tokens(g, R, V)
        if op == "logprobs_grad":
            _, s["entropy"], s["lse"] = _plain_stats(s["logits"].float(), s["tokens"])
            s["g_logprob"] = _randn(g, R)
            s["g_entropy"] = _randn(g, R) * 0.1
            s["dlogits"] = torch.empty_like(s["logits"])
    else:
        # Hidden rows and weights on grids of 1/16 and 1/1024: every score is then exact in 32 bits in
        # whatever order it is summed, so that the alternatives' ids can be compared.
        R, V, H = case["R"], case["V"], case["H"]
        s["hidden"] = (_randn(g, R, H).mul_(16).round_().clamp_(-100, 100).div_(16)).to(torch.bfloat16)
        s["W"] = (_randn(g, V, H).mul_(0.02 * 1024).round_().clamp_(-120, 120).div_(1024)).to(torch.bfloat16)
        s["tokens"] = _tokens(g, R, V)
    if op in ("logprobs", "head"):
        R, N = case["R"], case["top"]
        s["logprob"], s["entropy"], s["lse"] = (torch.empty(R, dtype=torch.float32, device="cuda") for _ in range(3))
        s["top_ids"] = torch.empty(R, N, dtype=torch.int32, device="cuda")
        s["top_logprobs"] = torch.empty(R, N, dtype=torch.float32, device="cuda")
    s["ws"] = {}  # the program's workspaces, made by the first call that needs one and kept
    return s


# ---------------------------------------------------------------------------
# Plain form


def _plain_norm(s, case):
    h = s["x"].float() + s["residual"].float()
    u = h * s["weight"].float()
    rstd = torch.rsqrt((h * h).mean(1, keepdim=True) + EPS)
    out = case["out"]
    if out == "same":
        return (u * rstd).to(s["x"].dtype), h.to(s["x"].dtype)
    top = 127.0 if out == "int8" else 448.0
    amax = u.abs().amax(1, keepdim=True)
    q = u * torch.where(amax > 0, top / amax, torch.zeros_like(amax))
    q = torch.round(q).to(torch.int8) if out == "int8" else q.to(torch.float8_e4m3fn)
    return q, (amax * rstd / top)[:, 0], h.to(s["x"].dtype)


def _plain_norm_grad(s):
    h, dy = s["h"].float(), s["dy"].float()
    rstd = torch.rsqrt((h * h).mean(1, keepdim=True) + EPS)
    n = h * rstd
    g = dy * s["weight"].float()
    dx = rstd * (g - n * (g * n).mean(1, keepdim=True)) + s["dh"].float()
    return dx.to(s["dy"].dtype), (dy * n).sum(0)


def _plain_stats(x, tokens):
    """(logprob, entropy, lse) of fp32 logits; a row's masked places (-inf) carry no probability."""
    lse = torch.logsumexp(x, 1)
    logp = x - lse[:, None]
    p = logp.exp()
    entropy = -(p * torch.where(p > 0, logp, torch.zeros_like(logp))).sum(1)
    given = tokens >= 0
    lp = logp.gather(1, tokens.clamp(min=0).long()[:, None])[:, 0]
    return torch.where(given, lp, torch.zeros_like(lp)), entropy, lse


def _plain_top(x, lse, n):
    """The n largest logits of each row, equal ones by lowest id: sorted as integers of the value's order and the id."""
    b = (x + 0.0).view(torch.int32).long()
    order = torch.where(b < 0, -2147483648 - b, b)
    ids = torch.arange(x.shape[1], device=x.device)
    key = torch.topk(order * 4294967296 + (4294967295 - ids), n, dim=1).values
    ids = 4294967295 - (key & 4294967295)
    return ids.int(), x.gather(1, ids) - lse[:, None]


def _plain_logprobs(x, tokens, n):
    lp, entropy, lse = _plain_stats(x, tokens)
    return (lp, entropy, lse) + (_plain_top(x, lse, n) if n else ())


def _plain_logprobs_grad(s):
    x = s["logits"].float()
    logp = x - s["lse"][:, None]
    p = logp.exp()
    t = s["tokens"]
    gl = torch.where(t >= 0, s["g_logprob"], torch.zeros_like(s["g_logprob"]))[:, None]
    d = -gl * p - s["g_entropy"][:, None] * p * (torch.where(p > 0, logp, torch.zeros_like(logp)) + s["entropy"][:, None])
    d.scatter_add_(1, t.clamp(min=0).long()[:, None], gl)
    return (d.to(s["logits"].dtype),)


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "norm":
        return _plain_norm(s, case)
    if op == "norm_grad":
        return _plain_norm_grad(s)
    if op == "logprobs":
        return _plain_logprobs(s["logits"].float(), s["tokens"], case["top"])
    if op == "logprobs_grad":
        return _plain_logprobs_grad(s)
    return _plain_logprobs(s["hidden"].float() @ s["W"].float().t(), s["tokens"], case["top"])


# ---------------------------------------------------------------------------
# The package's operators


def _workspace(s, make):
    if "ws" not in s["ws"]:
        s["ws"]["ws"] = make()
    return s["ws"]["ws"]


def _own(s):
    import verify_head_gb300 as vh
    case = s["case"]
    op = case["op"]
    if op == "norm":
        if case["out"] == "same":
            return vh.add_rmsnorm(s["x"], s["residual"], s["weight"], EPS, y=s["y"], h=s["h"])
        return vh.add_rmsnorm_q8(s["x"], s["residual"], s["weight"], EPS, q=s["y"], scales=s["scales"], h=s["h"])
    if op == "norm_grad":
        ws = _workspace(s, lambda: vh.add_rmsnorm_grad_workspace(case["T"], case["H"]))
        return vh.add_rmsnorm_grad(s["dy"], s["h"], s["weight"], EPS, dh=s["dh"], dx=s["dx"], dweight=s["dweight"], ws=ws)
    if op == "logprobs_grad":
        return (vh.logits_logprobs_grad(s["logits"], s["tokens"], s["lse"], s["entropy"], s["g_logprob"], s["g_entropy"],
                                        dlogits=s["dlogits"]),)
    outs = dict(logprob=s["logprob"], entropy=s["entropy"], lse=s["lse"], top_ids=s["top_ids"],
                top_logprobs=s["top_logprobs"])
    n = case["top"]
    if op == "logprobs":
        ws = _workspace(s, lambda: vh.logits_logprobs_workspace(case["R"], case["V"], n))
        got = vh.logits_logprobs(s["logits"], s["tokens"], n, ws=ws, **outs)
    else:
        ws = _workspace(s, lambda: vh.head_logprobs_workspace(case["R"], case["V"], n))
        got = vh.head_logprobs(s["hidden"], s["W"], s["tokens"], n, ws=ws, **outs)
    return got if n else got[:3]


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# What a pass cannot do without


def work(case):
    op = case["op"]
    if op == "norm":
        T, H, b = case["T"], case["H"], SIZE[case["dtype"]]
        out = b if case["out"] == "same" else 1
        return {"bytes": T * H * (3 * b + out) + H * b + (0 if case["out"] == "same" else 4 * T), "flops": 6 * T * H}
    if op == "norm_grad":
        T, H, b = case["T"], case["H"], SIZE[case["dtype"]]
        return {"bytes": 4 * T * H * b + H * (b + 4), "flops": 14 * T * H}
    R, V = case["R"], case["V"]
    if op == "logprobs_grad":
        return {"bytes": 2 * R * V * SIZE[case["dtype"]] + 20 * R, "flops": 8 * R * V}
    small = R * (16 + 8 * case["top"])
    if op == "logprobs":
        return {"bytes": R * V * SIZE[case["dtype"]] + small, "flops": 6 * R * V}
    return {"bytes": 2 * (V + R) * case["H"] + small, "flops": 2 * R * V * case["H"]}


# ---------------------------------------------------------------------------
# 64 bits


def _exact_rows(x, tokens, n, with_top=True):
    """Row statistics of float64 logits by the definitions: shifted sums, then logs."""
    top = x.max(1).values
    e = torch.exp(x - top[:, None])
    total = e.sum(1)
    p = e / total[:, None]
    plogp = torch.special.xlogy(p, p).sum(1)
    lse = top + total.log()
    at = x[torch.arange(x.shape[0], device=x.device), tokens.clamp(min=0).long()]
    lp = torch.where(tokens >= 0, at - lse, torch.zeros_like(lse))
    best = torch.sort(x, dim=1, descending=True).values[:, :n] - lse[:, None] if n else None
    return lp, -plogp, lse, best


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    d = {k: v.double() for k, v in s.items() if torch.is_tensor(v) and k in
         ("x", "residual", "weight", "h", "dy", "dh", "lse", "entropy", "g_logprob", "g_entropy")}
    if op == "norm":
        h = d["x"] + d["residual"]
        rms = torch.sqrt(h.pow(2).sum(1, keepdim=True) / case["H"] + EPS)
        y = h / rms * d["weight"]
        if case["out"] == "same":
            return y, h
        return None, y.abs().max(1).values / (127 if case["out"] == "int8" else 448), h
    if op == "norm_grad":
        H = case["H"]
        h, g = d["h"], d["dy"] * d["weight"]
        rms = torch.sqrt(h.pow(2).sum(1, keepdim=True) / H + EPS)
        dx = g / rms - h * (g * h).sum(1, keepdim=True) / (H * rms.pow(3)) + d["dh"]
        return dx, (d["dy"] * h / rms).sum(0)
    if op == "logprobs_grad":
        x = s["logits"].double()
        p = torch.exp(x - d["lse"][:, None])
        gl = d["g_logprob"] * (s["tokens"] >= 0)
        dx = -p * gl[:, None] - d["g_entropy"][:, None] * (torch.special.xlogy(p, p) + p * d["entropy"][:, None])
        rows = torch.arange(case["R"], device=x.device)
        dx[rows, s["tokens"].clamp(min=0).long()] += gl
        return (dx,)
    n = case["top"]
    parts = []
    if op == "logprobs":
        for r in range(0, case["R"], 256):
            parts.append(_exact_rows(s["logits"][r:r + 256].double(), s["tokens"][r:r + 256], n))
    else:
        W = s["W"].double().t()
        for r in range(0, case["R"], 256):
            parts.append(_exact_rows(s["hidden"][r:r + 256].double() @ W, s["tokens"][r:r + 256], n))
    lp, entropy, lse = (torch.cat([q[k] for q in parts]) for k in range(3))
    return (lp, entropy, lse, None, torch.cat([q[3] for q in parts])) if n else (lp, entropy, lse)
