"""64-bit definitions of the 4-bit rows and of the processing of logits, and the tiled layout in numpy."""
import math

import numpy as np
import torch

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0])
E4M3 = np.array([(c & 7) * 2.0 ** -9 if c < 8 else (8 + (c & 7)) * 2.0 ** ((c >> 3) - 10) for c in range(127)] + [math.nan])


def codes64(codes):
    """[V, H/2] bytes -> [V, H] values of the codes."""
    c = codes.cpu().numpy()
    return E2M1[np.stack((c & 15, c >> 4), 2).reshape(c.shape[0], -1)]


def values64(codes, scales):
    """code * block scale, exactly."""
    return codes64(codes) * np.repeat(E4M3[scales.cpu().numpy() & 127], 16, axis=1)


def tiles_bytes(rows, H):
    return -(-rows // 128) * -(-H // 256) * 18432


def tile(codes, scales, byte=0):
    """The tiled layout, place by place as its definition says; lines past V keep `byte`."""
    V, H = codes.shape[0], codes.shape[1] * 2
    nt = -(-H // 256)
    out = np.full((-(-V // 128), nt, 18432), byte, np.uint8)
    c, s = codes.cpu().numpy(), scales.cpu().numpy()
    for k in range(nt * 16):
        r = np.arange(V)
        q, t, kk = r // 128, k // 16, k % 16
        at = (r % 128) * 128 + ((kk // 2) ^ (r % 8)) * 16 + (kk % 2) * 8
        real = k < H // 16
        for b in range(8):
            out[q, t, at + b] = c[:, k * 8 + b] if real else 0
        out[q, t, 16384 + kk // 4 * 512 + r % 32 * 16 + r % 128 // 32 * 4 + kk % 4] = s[:, k] if real else 0
    return out.reshape(-1)


def process64(logits, S, rules, dout=None):
    """logits_process (or its gradient, with dout) row by row in 64 bits."""
    R, V = logits.shape
    m = R // S
    get = lambda n: rules.get(n)  # noqa: E731
    num = lambda n, s, d: d if get(n) is None else float(get(n)[s].double())  # noqa: E731
    x = logits.double().cpu()
    out = torch.empty(R, V, dtype=torch.float64)
    for r in range(R):
        s, j = r // m, r % m
        z = x[r].clone()
        if get("bias_ids") is not None:
            for i, b in zip(get("bias_ids")[s].tolist(), get("bias")[s].double().tolist()):
                if 0 <= i < V:
                    z[i] = x[r, i] + b  # the last entry counts
        hist = [] if get("history") is None else get("history")[s].tolist()
        n = len(hist) if get("history_len") is None else max(0, min(len(hist), int(get("history_len")[s])))
        p = 0 if get("prompt_len") is None else int(get("prompt_len")[s])
        hist = hist[:n]
        prompt, output = hist[:max(0, p)], hist[max(0, p):]
        if get("draft_ids") is not None:
            output = output + get("draft_ids")[s, :j].tolist()
        c_out = np.zeros(V)
        seen = np.zeros(V, bool)
        for t in output:
            if 0 <= t < V:
                c_out[t] += 1
                seen[t] = True
        for t in prompt:
            if 0 <= t < V:
                seen[t] = True
        c_out, seen = torch.from_numpy(c_out), torch.from_numpy(seen)
        rep, t = num("repetition", s, 1.0), num("temperature", s, 1.0)
        t = t if t > 0 else 1.0
        if dout is None:
            y = torch.where(seen, torch.where(z > 0, z / rep, z * rep), z)
            y = torch.where(c_out > 0, y - num("frequency", s, 0.0) * c_out - num("presence", s, 0.0), y) / t
        else:
            d = dout[r].double().cpu()
            y = torch.where(seen, torch.where(z > 0, d / rep, d * rep), d) / t
        if get("allowed") is not None:
            w = get("allowed")[r].cpu().numpy().astype(np.int64) & 0xFFFFFFFF
            v = np.arange(V)
            y = torch.where(torch.from_numpy((w[v // 32] >> (v % 32)) & 1 != 0), y,
                            torch.full_like(y, -math.inf if dout is None else 0.0))
        out[r] = y
    return out
