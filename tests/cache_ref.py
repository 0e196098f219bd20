"""The paged 8-bit token cache in plain 64-bit code (tests only): sequences one
after another, tokens one after another, no code shared with the library.

A cache here is a dict of CPU tensors: k, v (e4m3 codes as float64 values, NaN
where a code is NaN), k_scale, v_scale (float64), page_table. append() returns
for every written code its value before rounding.
"""
import math

import torch

E_MIN, E_MAX = -40, 60
F8 = torch.float8_e4m3fn


def host(cache):
    """CPU float64 view of a flare.FlareCache."""
    return {"k": cache.k.cpu().double(), "v": cache.v.cpu().double(), "k_scale": cache.k_scale.cpu().double(),
            "v_scale": cache.v_scale.cpu().double(), "page_table": cache.page_table.cpu()}


def exponent(amax):
    if amax == 0:
        return E_MIN
    m, e = math.frexp(amax)
    e = (e - 1 if m == 0.5 else e) - 8
    return max(E_MIN, min(E_MAX, e))


def rotate(x, pos, inv_freq, interleaved):
    """x [..., D] float64 at position pos."""
    y = x.clone()
    half = len(inv_freq)
    a = pos * inv_freq.double()
    c, s = torch.cos(a), torch.sin(a)
    lo = slice(0, 2 * half, 2) if interleaved else slice(0, half)
    hi = slice(1, 2 * half, 2) if interleaved else slice(half, 2 * half)
    p, q = x[..., lo], x[..., hi]
    y[..., lo], y[..., hi] = p * c - q * s, p * s + q * c
    return y


def append(cache, K, V, lens, counts, inv_freq=None, interleaved=False):
    """K, V: CPU [T, H, D] (any type). Returns (cache after, with k and v the
    codes' values before their rounding where this call wrote or rescaled them;
    written [P, page] of the new slots; rescaled [P, H, page, 2])."""
    out = {n: t.clone() for n, t in cache.items()}
    P, H, page, D = cache["k"].shape
    new = torch.zeros((P, page), dtype=torch.bool)
    again = {n: torch.zeros((P, H, page), dtype=torch.bool) for n in "kv"}
    t = 0
    for b, (at, n) in enumerate(zip(lens, counts)):
        i = 0
        while i < n:
            pos = at + i
            off = pos % page
            m = min(page - off, n - i)
            p = int(cache["page_table"][b, pos // page])
            raw = {"k": K[t + i:t + i + m].double(), "v": V[t + i:t + i + m].double()}
            ok = {x: y.isfinite().all(dim=2) for x, y in raw.items()}
            good = ok["k"] & ok["v"]                                  # [m, H]
            for x in "kv":
                for h in range(H):
                    y = raw[x][:, h]
                    fin = y[y.isfinite()]
                    e = exponent(float(fin.abs().max()) if fin.numel() else 0.0)
                    scale = 2.0 ** e
                    if off:
                        old = float(out[x + "_scale"][p, h])
                        if scale > old:
                            out[x][p, h, :off] *= old / scale
                            again[x][p, h, :off] = True
                        scale = max(scale, old)
                    out[x + "_scale"][p, h] = scale
                    for j in range(m):
                        r = y[j]
                        if x == "k" and inv_freq is not None:
                            r = rotate(r, pos + j, inv_freq, interleaved)
                        if not good[j, h]:
                            r = torch.full_like(r, math.nan if x == "k" else 0.0)
                        out[x][p, h, off + j] = r / scale
            new[p, off:off + m] = True
            i += m
        t += n
    return out, new, again


def half_step(y):
    """Half the spacing of e4m3 at |y| (up to the largest code, 448)."""
    e = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6)))
    return 2.0 ** (e - 4)


def tokens(cache, b, length):
    """Keys and values [length, H, D] that sequence b holds, float64."""
    H, page, D = cache["k"].shape[1:]
    pages = cache["page_table"][b, : -(-length // page)].long()
    return [(cache[x][pages] * cache[x + "_scale"][pages][:, :, None, None]).transpose(1, 2).reshape(-1, H, D)[:length]
            for x in "kv"]


def attn(cache, Q, lens, counts, causal, scale=None):
    """Q CPU [T, Hq, D]. Returns (O, L, A, E) in float64: A the outputs' weighted
    absolute values sum_n p_n |v_n|, E [T, Hq] the largest s sum_d |q_d k_nd|
    over the tokens seen, both for error bounds."""
    T, Hq, D = Q.shape
    H = cache["k"].shape[1]
    G = Hq // H
    s = D ** -0.5 if scale is None else scale
    Q = Q.double()
    O, A = torch.zeros((T, Hq, D), dtype=torch.float64), torch.zeros((T, Hq, D), dtype=torch.float64)
    L, E = torch.full((T, Hq), -math.inf, dtype=torch.float64), torch.zeros((T, Hq), dtype=torch.float64)
    t = 0
    for b, (length, n) in enumerate(zip(lens, counts)):
        K, V = tokens(cache, b, length)
        first = max(0, n - length) if causal else (0 if length else n)     # rows before see nothing
        for h in range(H):
            rows, heads = slice(t + first, t + n), slice(h * G, (h + 1) * G)
            q = Q[rows, heads]                                             # [n, G, D]
            if not q.shape[0]:
                continue
            S = s * (q @ K[:, h].T)
            size = s * (q.abs() @ K[:, h].abs().T)
            if causal:
                last = length - n + torch.arange(first, n)
                hidden = (torch.arange(length) > last[:, None])[:, None]
                S = S.masked_fill(hidden, -math.inf)
                size = size.masked_fill(hidden, 0.0)
            L[rows, heads] = torch.logsumexp(S, dim=2)
            w = torch.exp(S - L[rows, heads][..., None])
            O[rows, heads], A[rows, heads] = w @ V[:, h], w @ V[:, h].abs()
            E[rows, heads] = size.amax(dim=2)
        t += n
    return O, L, A, E
