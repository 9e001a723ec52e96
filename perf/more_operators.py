"""Cases for the operators around a 4-bit head and behind any head: rounding rows to block-scaled 4 bits
and back, the product of two 4-bit matrices (activations rounded on the way), and what a server does to
logits before it samples (biases, penalties for repeated tokens, temperature, grammar masks), with its
gradient.

`run` computes a case in its plain form (elementary torch operations in 32 bits, the choice of 4-bit and
8-bit codes in 64) or, with `own` set, through the package's entry points; `exact` gives the values in
64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
TOP = 6.0 * 448.0  # the largest 4-bit value times the largest block scale


def listed():
    return [
        # the hidden rows of one verify round (three drafts and the bonus position): latency
        {"name": "round 4x2048", "op": "round", "T": 4, "H": 2048, "dtype": "bf16", "scale": "rows"},
        # a training step's activations through a 4-bit layer's rounding
        {"name": "round 16384x2048", "op": "round", "T": 16384, "H": 2048, "dtype": "bf16", "scale": "rows"},
        # ragged rows of an odd number of blocks, full precision, a calibrated scale
        {"name": "round 301x2576", "op": "round", "T": 301, "H": 2576, "dtype": "f32", "scale": "tensor"},
        # one sequence's verify rows against a 4-bit candidate table
        {"name": "linear 4x65536x2048", "op": "linear", "T": 4, "V": 65536, "H": 2048, "dtype": "bf16", "out": "bf16",
         "scale": "rows"},
        # a ragged batch against an odd vocabulary, logits in full precision
        {"name": "linear 37x40001x2560", "op": "linear", "T": 37, "V": 40001, "H": 2560, "dtype": "f16", "out": "f32",
         "scale": "rows"},
        # 64 sequences' verify rows against the full head
        {"name": "linear 256x248320x2048", "op": "linear", "T": 256, "V": 248320, "H": 2048, "dtype": "bf16",
         "out": "bf16", "scale": "rows"},
        # a prefill through a wide layer with a calibrated scale
        {"name": "linear 4096x8192x8192", "op": "linear", "T": 4096, "V": 8192, "H": 8192, "dtype": "bf16", "out": "bf16",
         "scale": "tensor"},
        # one sequence's verify rows over the full vocabulary: penalties of a chat's history, no mask
        {"name": "process 4x248320", "op": "process", "S": 1, "m": 4, "V": 248320, "L": 1500, "nb": 8, "dtype": "f32",
         "out": "f32", "masked": 0.0},
        # a server's verify rows, long histories
        {"name": "process 256x248320", "op": "process", "S": 64, "m": 4, "V": 248320, "L": 4096, "nb": 32,
         "dtype": "bf16", "out": "bf16", "masked": 0.0},
        # single tokens of sequences that a grammar holds, odd vocabulary, 32-bit scores for the sampler
        {"name": "process 129x40001", "op": "process", "S": 129, "m": 1, "V": 40001, "L": 700, "nb": 3, "dtype": "f16",
         "out": "f32", "masked": 0.7},
        # a policy's update on the distribution it was sampled from: the gradient back to the head's logits
        {"name": "process grad 2048x65536", "op": "process_grad", "S": 2048, "m": 1, "V": 65536, "L": 512, "nb": 4,
         "dtype": "bf16", "out": "bf16", "masked": 0.0},
        # a few rows of an odd masked vocabulary in full precision
        {"name": "process grad 33x40001", "op": "process_grad", "S": 11, "m": 3, "V": 40001, "L": 300, "nb": 5,
         "dtype": "f32", "out": "f32", "masked": 0.5},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["round", "linear", "linear", "process", "process", "process_grad"])
    if op == "round":
        H = 16 * _log(rng, 4, 512)
        T = min(_log(rng, 1, 16384), 16384 * 2048 // H) | 1
        return {"op": op, "T": T, "H": H, "dtype": rng.choice(["bf16", "f16", "f32"]), "scale": rng.choice(["rows", "tensor"])}
    if op == "linear":
        H = rng.choice([512, 1024, 2048, 4096, 8192, 16 * _log(rng, 8, 400)])
        V = rng.choice([4096, 8192, 65536, 248320, _log(rng, 500, 100000) | 1])
        V = min(V, 248320 * 2048 // H)
        T = max(1, min(_log(rng, 1, 4096), 256 * 248320 // V, 256 * 248320 * 2048 // (V * H)))
        return {"op": op, "T": T, "V": V, "H": H, "dtype": rng.choice(["bf16", "f16", "f32"]),
                "out": rng.choice(["bf16", "f16", "f32"]), "scale": rng.choice(["rows", "tensor"])}
    V = rng.choice([32768, 65536, 248320, _log(rng, 1000, 250000) | 1])
    m = rng.choice([1, 1, 2, 3, 4, 8])
    dtype = rng.choice(["bf16", "f16", "f32"])
    S = max(1, min(_log(rng, 1, 2048), 1024 * 65536 // (V * m)))
    return {"op": op, "S": S, "m": m, "V": V, "L": min(_log(rng, 1, 32768), 1 + 2000000 // S), "nb": rng.choice([0, 1, 16, 300]),
            "dtype": dtype, "out": rng.choice([dtype, "f32"]) if op == "process" else dtype,
            "masked": rng.choice([0.0, 0.0, rng.uniform(0.1, 0.99)])}


# ---------------------------------------------------------------------------
# Inputs


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _rand(g, *shape):
    return torch.rand(*shape, generator=g, device="cuda")


def _randint(g, lo, hi, *shape):
    return torch.randint(lo, hi, shape, generator=g, device="cuda", dtype=torch.int32)


def _activations(g, T, H, dtype):
    """Hidden rows: a few outlier channels, rows of different size."""
    channel = 1 + 20 * (_rand(g, H) < 0.003)
    return (_randn(g, T, H) * channel * torch.exp(0.5 * _randn(g, T, 1))).to(dtype)


def _weights(g, V, H):
    """4-bit weights as a checkpoint holds them: codes [V, H/2] (element 2i in the low half of byte i),
    e4m3 scales [V, H/16], one tensor scale."""
    scale = 0.12 / TOP
    codes = torch.empty(V, H // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(V, H // 16, dtype=torch.uint8, device="cuda")
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    step = max(1, (1 << 26) // H)
    for v in range(0, V, step):
        w = _randn(g, min(step, V - v), H // 16, 16).mul_(0.02)
        s = (w.abs().amax(2) / (6 * scale)).to(torch.float8_e4m3fn)
        c = torch.bucketize(w.abs() / (s.float() * scale)[:, :, None], mids) + 8 * (w < 0)
        c = c.to(torch.uint8).view(-1, H)
        codes[v:v + step] = c[:, ::2] | (c[:, 1::2] << 4)
        scales[v:v + step] = s.view(torch.uint8)
    return codes, scales, scale


def tiles_bytes(rows, H):
    return -(-rows // 128) * -(-H // 256) * 18432


def _tiles(codes, scales):
    """The tiled copy of a 4-bit matrix that a program makes when it loads one: records of 128 rows x 256
    elements, each 128 lines of 128 code bytes whose 16-byte pieces lie at piece ^ (row % 8), then four
    times 512 bytes of scales, row r's four at (r % 32) * 16 + (r / 32) * 4."""
    V, H = codes.shape[0], codes.shape[1] * 2
    nv, nh = -(-V // 128), -(-H // 256)
    out = torch.empty(nv, nh, 18432, dtype=torch.uint8, device="cuda")
    c = torch.zeros(nv * 128, nh * 128, dtype=torch.uint8, device="cuda")
    c[:V, :H // 2] = codes
    c = c.view(nv, 128, nh, 8, 16).permute(0, 2, 1, 3, 4)
    piece = torch.arange(8, device="cuda")[None, :] ^ (torch.arange(128, device="cuda") % 8)[:, None]
    out[:, :, :16384] = torch.gather(c, 3, piece[None, None, :, :, None].expand(nv, nh, 128, 8, 16)).reshape(nv, nh, 16384)
    s = torch.zeros(nv * 128, nh * 16, dtype=torch.uint8, device="cuda")
    s[:V, :H // 16] = scales
    s = s.view(nv, 4, 32, nh, 4, 4).permute(0, 3, 4, 2, 1, 5)  # row / 32, row % 32, .., 64 elements, 16 elements
    out[:, :, 16384:] = s.reshape(nv, nh, 2048)
    return out.view(-1)


def _logits(g, R, V, dtype):
    """Logits as a head gives them: a per-token bias (frequent tokens score higher) and noise."""
    bias = _randn(g, V) * 1.5
    return _randn(g, R, V).mul_(1.5).add_(bias).to(dtype)


def _history(s, g, S, m, V, L):
    """Each sequence's tokens so far: common ones come back, every seventh sequence has just begun (none),
    the rest of its row is padding; and the draft of the round, row by row."""
    ids = (_rand(g, S, L).pow(3) * V).int().clamp_(max=V - 1)
    n = _randint(g, (L + 1) // 2, L + 1, S)
    n[6::7] = 0
    ids[torch.arange(L, device="cuda")[None, :] >= n[:, None]] = -1
    s["history"], s["history_len"] = ids, n
    s["prompt_len"] = (n.float() * _rand(g, S)).int()
    s["draft_ids"] = (_rand(g, S, m - 1).pow(3) * V).int().clamp_(max=V - 1) if m > 1 else None


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = {"case": dict(case)}
    if op in ("round", "linear"):
        T, H, dt = case["T"], case["H"], DTYPES[case["dtype"]]
        s["x"] = _activations(g, T, H, dt)
        s["x_scale"] = 60.0 / TOP if case["scale"] == "tensor" else None  # calibrated: the largest few saturate
        s["row_scales"] = torch.empty(T, dtype=torch.float32, device="cuda") if case["scale"] == "rows" else None
    if op == "round":
        s["codes"] = torch.empty(T, H // 2, dtype=torch.uint8, device="cuda")
        s["scales"] = torch.empty(T, H // 16, dtype=torch.uint8, device="cuda")
        s["y"] = torch.empty_like(s["x"])
    elif op == "linear":
        V = case["V"]
        s["w_codes"], s["w_scales"], s["w_scale"] = _weights(g, V, H)
        s["w_tiles"] = _tiles(s["w_codes"], s["w_scales"])
        s["x_tiles"] = torch.empty(tiles_bytes(T, H), dtype=torch.uint8, device="cuda")
        s["y"] = torch.empty(T, V, dtype=DTYPES[case["out"]], device="cuda")
    else:
        S, m, V, L, nb = (case[k] for k in ("S", "m", "V", "L", "nb"))
        R = S * m
        s["logits"] = _logits(g, R, V, DTYPES[case["dtype"]])
        _history(s, g, S, m, V, L)
        s["repetition"] = 1 + 0.3 * _rand(g, S)
        s["frequency"] = 0.5 * _rand(g, S)
        s["presence"] = 0.5 * _rand(g, S)
        s["repetition"][1::5] = 1.0
        s["temperature"] = 0.5 + 0.7 * _rand(g, S)
        s["temperature"][7::8] = 0.0  # greedy sequences
        if nb:
            s["bias_ids"] = _randint(g, 1, max(2, V // nb), S, nb).cumsum(1).int() - 1
            s["bias"] = 4 * _randn(g, S, nb)
        else:
            s["bias_ids"] = s["bias"] = None
        s["allowed"] = None
        if case["masked"] > 0:
            words = -(-V // 32)
            on = _rand(g, R, words * 32) >= case["masked"]
            on[:, 0] = True
            on[15::16] = False  # a grammar at a dead end
            bit = torch.ones(32, dtype=torch.int64, device="cuda") << torch.arange(32, device="cuda")
            w = (on.view(R, words, 32) * bit).sum(2)
            s["allowed"] = torch.where(w >= 1 << 31, w - (1 << 32), w).int()
        if op == "process":
            s["out"] = torch.empty(R, V, dtype=DTYPES[case["out"]], device="cuda")
        else:
            s["dout"] = (_randn(g, R, V) * 1e-2).to(DTYPES[case["dtype"]])
            s["dlogits"] = torch.empty_like(s["dout"])
    return s


# ---------------------------------------------------------------------------
# Plain form


def _grid(v, bits, lowest):
    """v >= 0 (64 bits) to the nearest number of `bits` mantissa bits and exponents from `lowest` on, ties to even."""
    e = (torch.frexp(v).exponent - 1).clamp(min=lowest)
    step = torch.ldexp(torch.ones_like(v), e - bits)
    return torch.round(v / step) * step


def _plain_round(x, tensor_scale):
    """(values' magnitudes and signs as code * block scale [T, H], row or tensor scale [T, 1] or float) in 32 bits."""
    T, H = x.shape
    x = x.float()
    scale = tensor_scale
    if scale is None:
        scale = x.abs().amax(1, keepdim=True)
        scale = scale / torch.full_like(scale, TOP)  # the quotient: a number's reciprocal would be multiplied with
    else:
        scale = torch.full((T, 1), scale, dtype=torch.float32, device=x.device)
    b = x.view(T, H // 16, 16).double()
    g = scale.double()[:, :, None]
    amax = b.abs().amax(2, keepdim=True)
    s = _grid(torch.where(g > 0, amax / (6 * g), torch.zeros_like(amax)), 3, -6).clamp(max=448)
    step = s * g
    u = torch.where(step > 0, b.abs() / step, torch.zeros_like(b)).clamp(max=6)
    v = _grid(u, 1, 0) * s * b.sign()
    return v.float().view(T, H), scale


_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def _values(codes, scales, dtype):
    """code * block scale of a 4-bit matrix."""
    grid = torch.tensor(_E2M1, dtype=dtype, device=codes.device)
    c = torch.stack((codes & 15, codes >> 4), 2).view(codes.shape[0], -1, 16)
    return (grid[c.int()] * scales.view(torch.float8_e4m3fn).to(dtype)[:, :, None]).view(codes.shape[0], -1)


def _plain_linear(s):
    x, xs = _plain_round(s["x"], s["x_scale"])
    y = x @ _values(s["w_codes"], s["w_scales"], torch.float32).t()
    return y.mul_(xs).mul_(s["w_scale"]).to(s["y"].dtype)


def _plain_counts(s, case):
    """([R, V] occurrences in prompt, output and draft so far, [R, V] those in output and draft)."""
    S, m, V, L = (case[k] for k in ("S", "m", "V", "L"))
    ids, at = s["history"], torch.arange(L, device="cuda")[None, :]
    ok = (at < s["history_len"][:, None]) & (ids >= 0) & (ids < V)
    where = ids.clamp(0, V - 1).long()
    every = torch.zeros(S, V, device="cuda").scatter_add_(1, where, ok.float())
    output = torch.zeros(S, V, device="cuda").scatter_add_(1, where, (ok & (at >= s["prompt_len"][:, None])).float())
    every, output = every.repeat_interleave(m, 0), output.repeat_interleave(m, 0)
    if m > 1:
        before = torch.arange(m, device="cuda")[:, None] > torch.arange(m - 1, device="cuda")[None, :]
        before = before[None].expand(S, m, m - 1).reshape(S * m, m - 1).float()
        d = s["draft_ids"].long().repeat_interleave(m, 0)
        every.scatter_add_(1, d, before)
        output.scatter_add_(1, d, before)
    return every, output


def _plain_allowed(s, V):
    bits = s["allowed"][:, :, None] >> torch.arange(32, dtype=torch.int32, device="cuda")
    return (bits & 1).view(s["allowed"].shape[0], -1)[:, :V] != 0


def _rows_of(s, name, m):
    return s[name].repeat_interleave(m)[:, None]


def _plain_biased(s, case):
    z = s["logits"].float()
    if case["nb"]:
        b = torch.zeros(case["S"], case["V"], device="cuda").scatter_(1, s["bias_ids"].long(), s["bias"])
        z = z + b.repeat_interleave(case["m"], 0)
    return z


def _plain_process(s, case):
    m, V = case["m"], case["V"]
    every, output = _plain_counts(s, case)
    z = _plain_biased(s, case)
    rep, t = _rows_of(s, "repetition", m), _rows_of(s, "temperature", m)
    z = torch.where(every > 0, torch.where(z > 0, z / rep, z * rep), z)
    z = z - _rows_of(s, "frequency", m) * output - _rows_of(s, "presence", m) * (output > 0)
    z = z / torch.where(t > 0, t, torch.ones_like(t))
    if s["allowed"] is not None:
        z = torch.where(_plain_allowed(s, V), z, torch.full_like(z, -math.inf))
    return z.to(s["out"].dtype)


def _plain_process_grad(s, case):
    m, V = case["m"], case["V"]
    every, _ = _plain_counts(s, case)
    z = _plain_biased(s, case)
    rep, t = _rows_of(s, "repetition", m), _rows_of(s, "temperature", m)
    d = s["dout"].float() / torch.where(t > 0, t, torch.ones_like(t))
    d = torch.where(every > 0, torch.where(z > 0, d / rep, d * rep), d)
    if s["allowed"] is not None:
        d = torch.where(_plain_allowed(s, V), d, torch.zeros_like(d))
    return d.to(s["dlogits"].dtype)


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "round":
        v, scale = _plain_round(s["x"], s["x_scale"])
        y = (v * scale).to(s["y"].dtype)
        return (y, scale[:, 0]) if s["x_scale"] is None else (y,)
    if op == "linear":
        return (_plain_linear(s),)
    return (_plain_process(s, case) if op == "process" else _plain_process_grad(s, case),)


# ---------------------------------------------------------------------------
# The package's operators


def _own(s):
    import verify_head_gb300 as vh
    case = s["case"]
    op = case["op"]
    if op == "round":
        vh.nvfp4_quantize(s["x"], s["x_scale"], codes=s["codes"], scales=s["scales"], row_scales=s["row_scales"])
        scale = s["row_scales"] if s["x_scale"] is None else s["x_scale"]
        y = vh.nvfp4_dequantize(s["codes"], s["scales"], scale, out=s["y"])
        return (y, s["row_scales"]) if s["x_scale"] is None else (y,)
    if op == "linear":
        vh.nvfp4_quantize_tiles(s["x"], s["x_scale"], tiles=s["x_tiles"], row_scales=s["row_scales"])
        scale = s["row_scales"] if s["x_scale"] is None else s["x_scale"]
        return (vh.nvfp4_matmul(s["x_tiles"], scale, s["w_tiles"], s["w_scale"], case["T"], case["V"], case["H"], out=s["y"]),)
    args = dict(history=s["history"], history_len=s["history_len"], prompt_len=s["prompt_len"], draft_ids=s["draft_ids"],
                repetition=s["repetition"], frequency=s["frequency"], presence=s["presence"], bias_ids=s["bias_ids"],
                bias=s["bias"], allowed=s["allowed"], temperature=s["temperature"])
    if op == "process":
        return (vh.logits_process(s["logits"], out=s["out"], **args),)
    return (vh.logits_process_grad(s["dout"], s["logits"], dlogits=s["dlogits"], **args),)


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# What a pass cannot do without


def work(case):
    op = case["op"]
    if op == "round":
        T, H, b = case["T"], case["H"], SIZE[case["dtype"]]
        return {"bytes": T * H * 2 * b + T * H * 9 // 16 + 4 * T, "flops": 6 * T * H}
    if op == "linear":
        T, V, H = case["T"], case["V"], case["H"]
        return {"bytes": V * H * 9 // 16 + T * H * SIZE[case["dtype"]] + T * V * SIZE[case["out"]], "flops": 2 * T * V * H}
    R, V = case["S"] * case["m"], case["V"]
    n = R * V * (SIZE[case["dtype"]] + SIZE[case["out"]]) + (R * V // 8 if case["masked"] else 0)
    return {"bytes": n + 4 * case["S"] * (case["L"] + 2 * case["nb"] + 8), "flops": 4 * R * V}


# ---------------------------------------------------------------------------
# 64 bits


def _nearest(v, grid):
    """Nearest of an ascending grid, a tie to the even place: by the distances to the two neighbours."""
    grid = torch.tensor(grid, dtype=torch.float64, device=v.device)
    hi = torch.searchsorted(grid, v.contiguous()).clamp(1, len(grid) - 1)
    lo = hi - 1
    dl, dh = v - grid[lo], grid[hi] - v
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    return grid[torch.where(up, hi, lo)]


def _exact_round(x, tensor_scale):
    """(code * block scale in 64 bits, scale [T] in 64 bits): the scale is the 32-bit number that is handed out."""
    e4m3 = [(c & 7) * 2.0 ** -9 if c < 8 else (8 + (c & 7)) * 2.0 ** ((c >> 3) - 10) for c in range(127)]
    x = x.double()
    T, H = x.shape
    if tensor_scale is None:
        g = (x.abs().max(1).values / TOP).float().double()
    else:
        g = torch.tensor(tensor_scale, dtype=torch.float32).double().to(x.device).expand(T)
    blocks = x.reshape(-1, 16)
    gb = g.repeat_interleave(H // 16)
    some = gb > 0
    safe = torch.where(some, gb, torch.ones_like(gb))
    s = _nearest(blocks.abs().max(1).values / 6 / safe, e4m3) * some
    step = torch.where(s > 0, s * safe, torch.ones_like(s))
    mag = _nearest(blocks.abs() / step[:, None], list(_E2M1[:8]))
    return (torch.copysign(mag, blocks) * s[:, None]).view(T, H), g


def _exact_process(s, case):
    """Sequence by sequence, its own tokens counted one kind at a time."""
    S, m, V = case["S"], case["m"], case["V"]
    grad = case["op"] == "process_grad"
    out = s["dout"].double() if grad else s["logits"].double()
    logits = s["logits"].double()
    n, p = s["history_len"].tolist(), s["prompt_len"].tolist()
    p32 = {k: s[k].double().tolist() for k in ("repetition", "frequency", "presence", "temperature")}
    for i in range(S):
        said = s["history"][i, :n[i]].long()
        rows = slice(i * m, (i + 1) * m)
        z = logits[rows]
        if case["nb"]:
            z[:, s["bias_ids"][i].long()] += s["bias"][i].double()
        t = p32["temperature"][i] if p32["temperature"][i] > 0 else 1.0
        base_all, base_out = torch.bincount(said, minlength=V), torch.bincount(said[p[i]:], minlength=V)
        for j in range(m):
            if j:
                one = torch.bincount(s["draft_ids"][i, :j].long(), minlength=V)
                c_all, c_out = base_all + one, base_out + one
            else:
                c_all, c_out = base_all, base_out
            seen = c_all > 0
            f = torch.ones(V, dtype=torch.float64, device="cuda")
            f[seen & (z[j] > 0)] = 1 / p32["repetition"][i]
            f[seen & ~(z[j] > 0)] = p32["repetition"][i]
            if grad:
                out[i * m + j] *= f / t
            else:
                out[i * m + j] = (z[j] * f - p32["frequency"][i] * c_out - p32["presence"][i] * (c_out > 0)) / t
    if s["allowed"] is not None:
        word = torch.arange(V, device="cuda")
        off = torch.div(s["allowed"].long()[:, word // 32] % (1 << 32), 2 ** (word % 32), rounding_mode="floor") % 2 == 0
        out[off] = 0.0 if grad else -math.inf
    return (out,)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("round", "linear"):
        v, g = _exact_round(s["x"], s["x_scale"])
        if op == "round":
            y = v * g[:, None]
            return (y, s["x"].double().abs().max(1).values / TOP) if s["x_scale"] is None else (y,)
        V, parts = case["V"], []
        step = max(1, (1 << 28) // case["H"])
        for r in range(0, V, step):
            parts.append(v @ _values(s["w_codes"][r:r + step], s["w_scales"][r:r + step], torch.float64).t())
        return (torch.cat(parts, 1) * g[:, None] * s["w_scale"],)
    if case["S"] > 4096:
        return None
    return _exact_process(s, case)
