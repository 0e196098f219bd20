"""Cases of the paged 8-bit token cache: appending tokens to it (with the rotation
of positions on the way) and attention over it.

The cache holds keys and values as e4m3 codes in pages [P, H, page, D] with one
power-of-two fp32 scale for each page and head, [P, H]; page_table [B, W] gives
the pages of each sequence. Where `own` is false the operators are computed in
their plain form with elementary torch operations; where it is true by the
framework's entry points. Length and position vectors follow from a case alone;
values and the order of the pages from the seed.
"""
import random

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
F8 = torch.float8_e4m3fn
E_MIN, E_MAX = -40, 60            # exponents that a page's scale may take
NAN_CODE = 0x7F                   # what slots that no token was written to hold here


def listed():
    return [
        # one sequence generating: its next token enters the cache (latency)
        _append("append_one", B=1, n_lo=1, n_hi=1, at_lo=4999, at_hi=4999),
        # a serving batch generating one token each, some of them far into a long context
        _append("append_batch", B=96, n_lo=1, n_hi=1, at_lo=0, at_hi=1_000_000, page=32),
        # prompts of mixed lengths entering together, some on top of what is cached
        _append("append_prompts", B=8, n_lo=1, n_hi=6000, at_lo=0, at_hi=2000),
        # fp32 tokens of a mixer with 64 channels a head, pairs rotated side by side
        _append("append_fp32", B=4, n_lo=2051, n_hi=2051, at_lo=0, at_hi=333, dtype="fp32", H=16, Hq=0, D=64,
                rot=48, inter=True, page=16),
        # one short conversation, one token (latency)
        _attn("decode_short", B=1, n_lo=1, n_hi=1, len_lo=1500, len_hi=1500),
        # a serving batch of mixed lengths, one token each
        _attn("decode_batch", B=32, n_lo=1, n_hi=1, len_lo=0, len_hi=16000),
        # one token against a million cached ones
        _attn("decode_long", B=1, n_lo=1, n_hi=1, len_lo=1_000_003, len_hi=1_000_003, page=128),
        # a few proposed tokens a sequence, five queries a shared head
        _attn("decode_few", B=6, n_lo=3, n_hi=3, len_lo=2, len_hi=9000, H=4, G=5, D=64, page=16),
        # fp32 queries
        _attn("decode_fp32", B=4, n_lo=1, n_hi=1, len_lo=500, len_hi=7000, H=4, G=4, D=64, dtype="fp32", page=32),
        # pieces of prompts on top of what is cached
        _attn("prompts", B=2, n_lo=1500, n_hi=2100, len_lo=6000, len_hi=11000),
        # the latent queries of a mixer over a long token set held in 8 bits
        _attn("latents_long", B=1, n_lo=64, n_hi=64, len_lo=1_048_576, len_hi=1_048_576, G=1, causal=False),
        # twice as many heads, 256 latents of 64 channels
        _attn("latents_wide", B=2, n_lo=256, n_hi=256, len_lo=131_072, len_hi=131_072, H=16, G=1, D=64, causal=False),
    ]


def _append(name, *, B, n_lo, n_hi, at_lo, at_hi, dtype="bf16", H=8, Hq=32, D=128, page=64, rot=None, inter=False):
    """Appends n_lo..n_hi tokens to each of B sequences that hold at_lo..at_hi."""
    c = dict(op="append", B=B, n_lo=n_lo, n_hi=n_hi, at_lo=at_lo, at_hi=at_hi, dtype=dtype, H=H, Hq=Hq, D=D, page=page,
             rot=D if rot is None else rot, inter=inter)
    return dict(c, name=name) if name else c


def _attn(name, *, B, n_lo, n_hi, len_lo, len_hi, H=8, G=4, D=128, page=64, causal=True, dtype="bf16"):
    """n_lo..n_hi queries a sequence, H * G heads, over len_lo..len_hi cached tokens."""
    c = dict(op="attn", B=B, n_lo=n_lo, n_hi=n_hi, len_lo=len_lo, len_hi=len_hi, H=H, G=G, D=D, page=page, causal=causal, dtype=dtype)
    return dict(c, name=name) if name else c


def draw(rng):
    log = lambda lo, hi: int(round(lo * (hi / lo) ** rng.random()))  # noqa: E731
    page = rng.choice([16, 32, 64, 128])
    D = rng.choice([64, 64, 128, 128, 128, 32, 96])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    kind = rng.choice(["append_token", "append_prompt", "decode", "decode", "decode_long", "few", "prompts", "latents"])
    H = rng.choice([1, 2, 3, 4, 8, 8, 16])
    if kind.startswith("append"):
        rot = rng.choice([0, D, D, D // 2])
        more = dict(dtype=dtype, H=H, Hq=rng.choice([0, H, 4 * H]), D=D, page=page, rot=rot, inter=rng.random() < 0.5)
        if kind == "append_token":
            return _append("", B=log(1, 128), n_lo=1, n_hi=rng.choice([1, 1, 4]), at_lo=0, at_hi=log(100, 1_000_000), **more)
        B = rng.randint(1, 8)
        return _append("", B=B, n_lo=1, n_hi=log(64, 16000 // B), at_lo=0, at_hi=log(10, 4000), **more)
    G = rng.choice([1, 2, 3, 4, 5, 7, 8])
    if kind == "decode":
        B = log(1, 64)
        return _attn("", B=B, n_lo=1, n_hi=1, len_lo=rng.choice([0, 1, 100]), len_hi=log(200, 500_000 // B), H=H, G=G, D=D, page=page, dtype=dtype)
    if kind == "decode_long":
        n = log(60_000, 1_000_000)
        return _attn("", B=1, n_lo=1, n_hi=1, len_lo=n, len_hi=n, H=min(H, 8), G=G, D=D, page=page)
    if kind == "few":
        B = log(1, 16)
        return _attn("", B=B, n_lo=1, n_hi=rng.randint(2, 9), len_lo=1, len_hi=log(64, 16000), H=H, G=G, D=D, page=page,
                     causal=rng.random() < 0.8, dtype=dtype)
    if kind == "prompts":
        B = rng.randint(1, 3)
        n = log(40, 4000 // B)
        return _attn("", B=B, n_lo=max(1, n // 2), n_hi=n, len_lo=n // 2, len_hi=n + log(8, 8000), H=min(H, 8), G=min(G, 4), D=D, page=page)
    n, M = log(4_000, 300_000), rng.choice([16, 33, 64, 128, 200, 256])
    return _attn("", B=rng.randint(1, 2), n_lo=M, n_hi=M, len_lo=n, len_hi=n, H=min(H, 8), G=1, D=D, page=page, causal=False)


# ---- lengths, work ---------------------------------------------------------------
def _spread(case, lo, hi, what):
    """B whole numbers of lo..hi, the two ends among them where there are two or more."""
    r = random.Random("%s %s" % (what, sorted((k, v) for k, v in case.items() if k != "name")))
    v = [r.randint(lo, hi) for _ in range(case["B"])]
    if len(v) > 1:
        v[0], v[-1] = hi, lo
    return v


def _sizes(case):
    """(new tokens or queries a sequence, tokens that it holds before an append or at an attention call)"""
    n = _spread(case, case["n_lo"], case["n_hi"], "n")
    lo, hi = (case["at_lo"], case["at_hi"]) if case["op"] == "append" else (case["len_lo"], case["len_hi"])
    return n, _spread(case, lo, hi, "at")


def _seen(case, n, at):
    """Pairs of a query and a token that it sees, over the sequences."""
    if not case["causal"]:
        return sum(x * y for x, y in zip(n, at))
    return sum(sum(max(0, y - x + i + 1) for i in range(x)) for x, y in zip(n, at))


def work(case):
    n, at = _sizes(case)
    H, D, es = case["H"], case["D"], 2 if case["dtype"] == "bf16" else 4
    T = sum(n)
    if case["op"] == "append":
        pages = sum((a + x - 1) // case["page"] - a // case["page"] + 1 for x, a in zip(n, at) if x)
        kv = 2 * T * H * D * (es + 1) + 2 * 4 * H * pages                  # tokens in, codes and scales out
        return {"bytes": kv + 2 * es * T * case["Hq"] * D, "flops": T * (4 * H * D + 3 * (H + case["Hq"]) * case["rot"])}
    pages = sum(-(-a // case["page"]) for a in at)
    rows = T * H * case["G"]
    cache = 2 * H * D * sum(at) + 2 * 4 * H * pages + 4 * pages
    return {"bytes": cache + 2 * es * rows * D + 4 * rows, "flops": 4 * D * H * case["G"] * _seen(case, n, at)}


# ---- inputs ------------------------------------------------------------------------
def _exponent(amax):
    """Whole e with 2^(e+7) < amax <= 2^(e+8): amax * 2^-e is at most 256, so that a
    rotated pair (at most sqrt(2) longer in one channel) stays under e4m3's 448."""
    m, e = torch.frexp(amax)
    e = torch.where(m == 0.5, e - 1, e) - 8
    return torch.where(amax > 0, e, E_MIN).clamp(E_MIN, E_MAX)


def _two_to(e):
    return torch.ldexp(torch.ones_like(e, dtype=torch.float32), e)


def _tokens(g, shape, dtype):
    """Keys or values: N(0, 1), one token in a hundred eight times as large."""
    x = torch.randn(shape, generator=g, device=DEV)
    x *= 1 + 7 * (torch.rand(shape[:-1], generator=g, device=DEV) < 0.01).float()[..., None]
    return x.to(dtype)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed) * 2 + 1)
    n, at = _sizes(case)
    H, D, page, dtype = case["H"], case["D"], case["page"], TYPES[case["dtype"]]
    T, ragged = sum(n), case["n_lo"] != case["n_hi"]
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    s = {"case": case, "n_max": max(n), "lens": ints(at)}
    s["cu"] = ints([0] + [sum(n[: i + 1]) for i in range(len(n))]) if ragged else None
    lead = (T,) if ragged else (case["B"], n[0])
    append = case["op"] == "append"
    # the pages that a call touches, in a random order in the pool; what an append does not
    # touch of a long context (its earlier pages) has no page of its own here
    first = [a // page if append else 0 for a in at]
    ends = [-(-(a + x) // page) if append else -(-a // page) for x, a in zip(n, at)]
    W = max(1, max(ends))
    P = sum(e - f for e, f in zip(ends, first)) + 3
    order = torch.randperm(P, generator=g, device=DEV, dtype=torch.int32)
    table, used = torch.zeros((case["B"], W), dtype=torch.int32, device=DEV), 0
    for b, (f, e) in enumerate(zip(first, ends)):
        table[b, f:e] = order[used:used + e - f]
        used += e - f
    k, v = (torch.empty((P, H, page, D), dtype=torch.uint8, device=DEV) for _ in range(2))
    ks, vs = (torch.empty((P, H), device=DEV) for _ in range(2))
    step = max(1, (1 << 27) // (H * page * D))
    for codes, scale in ((k, ks), (v, vs)):
        for p in range(0, P, step):
            x = _tokens(g, (min(step, P - p), H, page, D), torch.float32)
            scale[p:p + step] = _two_to(_exponent(x.abs().amax(dim=(2, 3))))
            codes[p:p + step] = (x / scale[p:p + step, :, None, None]).to(F8).view(torch.uint8)
    # slots behind a sequence's last token hold what memory held
    for b, a in enumerate(at):
        if a % page:
            p = int(table[b, a // page])
            k[p, :, a % page:] = NAN_CODE
            v[p, :, a % page:] = NAN_CODE
    s["cache"] = (k.view(F8), v.view(F8), ks, vs, table)
    if append:
        s["K"], s["V"] = _tokens(g, (*lead, H, D), dtype), _tokens(g, (*lead, H, D), dtype)
        s["Q"] = torch.randn((*lead, case["Hq"], D), generator=g, device=DEV).to(dtype) if case["Hq"] else None
        r = case["rot"]
        s["inv_freq"] = (10000.0 ** (-torch.arange(0, r, 2, device=DEV, dtype=torch.float64) / r)).float() if r else None
    else:
        s["Q"] = torch.randn((*lead, H * case["G"], D), generator=g, device=DEV).to(dtype)
    return s


# ---- one pass ------------------------------------------------------------------------
def run(s):
    c = s["case"]
    if own:
        from latent_query_split_gb300 import flare
        cache = flare.FlareCache(*s["cache"])
        if c["op"] == "append":
            lens, q = flare.flare_cache_append(cache, s["K"], s["V"], s["lens"], cu_seqlens=s["cu"], Q=s["Q"],
                                               inv_freq=s["inv_freq"], interleaved=c["inter"])
        else:
            o, l = flare.flare_cache_attn(s["Q"], cache, s["lens"], cu_seqlens=s["cu"], causal=c["causal"])
    elif c["op"] == "append":
        lens, q = _plain_append(s)
    else:
        o, l = _plain_attn(s)
    if c["op"] == "append":
        k, v, ks, vs, _ = s["cache"]
        return {"k": k, "v": v, "k_scale": ks, "v_scale": vs, "lens": lens, "q": q}
    return {"o": o, "l": l}


def _places(s):
    """Of every new token: its sequence, and its place among that sequence's new ones."""
    c = s["case"]
    if s["cu"] is None:
        t = torch.arange(c["B"] * s["n_max"], device=DEV)
        return t // s["n_max"], t % s["n_max"]
    t = torch.arange(s["Q" if s["Q"] is not None else "K"].shape[0], device=DEV)
    b = torch.searchsorted(s["cu"][1:].long(), t, right=True)
    return b, t - s["cu"][b]


def _rotate(x, cos, sin, inter):
    """x [T, heads, D] with its first 2 * cos.shape[1] channels rotated by pairs."""
    r = cos.shape[1]
    cos, sin = cos[:, None], sin[:, None]
    if inter:
        a, b = x[..., 0:2 * r:2], x[..., 1:2 * r:2]
        turned = torch.stack((a * cos - b * sin, a * sin + b * cos), dim=-1).flatten(-2)
    else:
        a, b = x[..., :r], x[..., r:2 * r]
        turned = torch.cat((a * cos - b * sin, a * sin + b * cos), dim=-1)
    return torch.cat((turned, x[..., 2 * r:]), dim=-1)


def _plain_append(s):
    c = s["case"]
    k, v, ks, vs, table = s["cache"]
    page, H, D = c["page"], c["H"], c["D"]
    b, i = _places(s)
    pos = s["lens"][b] + i
    at, slot = table[b, pos // page].long(), pos % page
    K, V = (s[x].reshape(-1, H, D).float() for x in ("K", "V"))
    Q = None if s["Q"] is None else s["Q"].reshape(-1, c["Hq"], D).float()
    amax = [x.abs().amax(dim=2) for x in (K, V)]
    if s["inv_freq"] is not None:
        angle = pos.double()[:, None] * s["inv_freq"].double()
        cos, sin = angle.cos().float(), angle.sin().float()
        K = _rotate(K, cos, sin, c["inter"])
        Q = None if Q is None else _rotate(Q, cos, sin, c["inter"])
    n = s["n_max"] if s["cu"] is None else s["cu"][1:] - s["cu"][:-1]
    # the page that a sequence's first new token falls into, where it holds earlier ones
    cut = s["lens"] % page
    old = table.gather(1, (s["lens"] // page).clamp(max=table.shape[1] - 1).long()[:, None])[:, 0].long()
    kept = (torch.arange(page, device=DEV) < cut[:, None])[:, None, :, None]
    keeps = ((cut > 0) & (torch.zeros_like(cut) + n > 0))
    for x, a, codes, scale in ((K, amax[0], k, ks), (V, amax[1], v, vs)):
        top = torch.zeros_like(scale).scatter_reduce_(0, at[:, None].expand_as(a), a, "amax")
        was = scale[old]
        scale[at] = _two_to(_exponent(top))[at]
        now = torch.where(keeps[:, None], torch.maximum(scale[old], was), scale[old])
        scale[old] = now
        bytes_, before = codes.view(torch.uint8), codes.view(torch.uint8)[old]
        again = (before.view(F8).float() * (was / now)[:, :, None, None]).to(F8).view(torch.uint8)
        bytes_[old] = torch.where(kept & keeps[:, None, None, None], again, before)
        bytes_[at, :, slot] = (x / scale[at][:, :, None]).to(F8).view(torch.uint8)
    dtype = TYPES[c["dtype"]]
    return (s["lens"] + n).int(), None if Q is None else Q.to(dtype).view_as(s["Q"])


def _plain_attn(s):
    c = s["case"]
    k, v, ks, vs, table = s["cache"]
    B, H, G, D, n = c["B"], c["H"], c["G"], c["D"], s["n_max"]
    rows = table.long()
    tokens = torch.arange(rows.shape[1] * c["page"], device=DEV)
    held = tokens < s["lens"][:, None]                                       # [B, L]
    if s["cu"] is None:
        Q, count = s["Q"].float(), torch.full((B,), n, device=DEV)
    else:
        count = (s["cu"][1:] - s["cu"][:-1]).long()
        Q = s["Q"][(s["cu"][:-1, None] + torch.arange(n, device=DEV)).clamp(max=s["Q"].shape[0] - 1)].float()
    K, V = (x[rows].float().mul_(y[rows][..., None, None]).transpose(1, 2).reshape(B, H, -1, D) for x, y in ((k, ks), (v, vs)))
    V.masked_fill_(~held[:, None, :, None], 0)
    Q = Q.view(B, n, H, G, D).permute(0, 2, 1, 3, 4).reshape(B, H, n * G, D)
    S = torch.matmul(Q * D ** -0.5, K.transpose(2, 3)).view(B, H, n, G, -1)
    seen = held[:, None]
    if c["causal"]:
        last = s["lens"][:, None] - count[:, None] + torch.arange(n, device=DEV)      # [B, n]
        seen = seen & (tokens <= last[..., None])
    S.masked_fill_(~seen[:, None, :, None], float("-inf"))
    top = S.amax(dim=-1, keepdim=True)
    top = torch.where(top == float("-inf"), 0.0, top)
    S = S.sub_(top).exp_()
    total = S.sum(dim=-1, keepdim=True)
    O = torch.matmul(S.view(B, H, n * G, -1), V).view(B, H, n, G, D) / torch.where(total == 0, 1.0, total)
    L = (top + total.log())[..., 0]
    O, L = O.permute(0, 2, 1, 3, 4).reshape(B, n, H * G, D), L.permute(0, 2, 1, 3).reshape(B, n, H * G)
    if s["cu"] is not None:
        b, i = _places(s)
        O, L = O[b, i], L[b, i]
    return O.to(s["Q"].dtype), L.contiguous()


# ---- the definition in 64 bits, sequence by sequence -------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return _exact_append(s) if case["op"] == "append" else _exact_attn(s)


def _exact_append(s):
    """What each written code stands for before its rounding, in units of its page's scale."""
    c = s["case"]
    n, at = _sizes(c)
    k, v, ks, vs, table = s["cache"]
    page, table = c["page"], table.tolist()
    out = {"k": k.double(), "v": v.double(), "k_scale": ks.double(), "v_scale": vs.double(), "lens": None}
    K, V = (s[x].reshape(-1, c["H"], c["D"]).double() for x in ("K", "V"))
    Q = None if s["Q"] is None else s["Q"].reshape(-1, c["Hq"], c["D"]).double().clone()
    start = 0
    for b in range(c["B"]):
        own_k, own_v = K[start:start + n[b]].clone(), V[start:start + n[b]]
        plain_k = K[start:start + n[b]]
        if c["rot"]:
            half = c["rot"] // 2
            where = torch.arange(at[b], at[b] + n[b], device=DEV, dtype=torch.float64)
            turn = torch.polar(torch.ones((), device=DEV, dtype=torch.float64), where[:, None, None] * s["inv_freq"].double())
            lo = slice(0, 2 * half, 2) if c["inter"] else slice(0, half)
            hi = slice(1, 2 * half, 2) if c["inter"] else slice(half, 2 * half)
            for x in (own_k, None if Q is None else Q[start:start + n[b]]):
                if x is not None:
                    z = torch.complex(x[..., lo], x[..., hi]) * turn
                    x[..., lo], x[..., hi] = z.real.clone(), z.imag.clone()
        done = 0
        while done < n[b]:
            pos = at[b] + done
            p, off = table[b][pos // page], pos % page
            m = min(page - off, n[b] - done)
            for name, new, raw in (("k", own_k, plain_k), ("v", own_v, V[start:start + n[b]])):
                need = raw[done:done + m].abs().amax(dim=(0, 2))
                e = torch.where(need > 0, torch.ceil(torch.log2(need)) - 8, float(E_MIN)).clamp(E_MIN, E_MAX)
                scale = torch.exp2(e)
                if off:
                    before = out[name + "_scale"][p].clone()
                    scale = torch.maximum(scale, before)
                    out[name][p, :, :off] *= (before / scale)[:, None, None]
                out[name + "_scale"][p] = scale
                out[name][p, :, off:off + m] = (new[done:done + m] / scale[:, None]).transpose(0, 1)
            done += m
        start += n[b]
    out["q"] = None if Q is None else Q.view(s["Q"].shape)
    return out


def _exact_attn(s):
    c = s["case"]
    n, at = _sizes(c)
    k, v, ks, vs, table = s["cache"]
    H, G, D, page = c["H"], c["G"], c["D"], c["page"]
    Q = s["Q"].reshape(-1, H, G, D)
    O = torch.zeros(Q.shape, device=DEV, dtype=torch.float64)
    L = torch.full(Q.shape[:-1], float("-inf"), device=DEV, dtype=torch.float64)
    start = 0
    for b in range(c["B"]):
        pages = table[b, : -(-at[b] // page)].long()
        for h in range(H if at[b] else 0):
            K, V = ((x[pages, h].double() * y[pages, h].double()[:, None, None]).reshape(-1, D)[: at[b]] for x, y in ((k, ks), (v, vs)))
            step = max(1, (1 << 27) // (at[b] * G))
            for i in range(0, n[b], step):
                m = min(step, n[b] - i)
                q = Q[start + i:start + i + m, h].reshape(m * G, D).double()
                S = q @ K.T / D ** 0.5
                if c["causal"]:
                    last = at[b] - n[b] + torch.arange(i, i + m, device=DEV).repeat_interleave(G)
                    S[torch.arange(at[b], device=DEV) > last[:, None]] = float("-inf")
                l = torch.logsumexp(S, dim=1)
                w = torch.where(l[:, None] == float("-inf"), 0.0, torch.exp(S - l[:, None]))
                O[start + i:start + i + m, h] = (w @ V).view(m, G, D)
                L[start + i:start + i + m, h] = l.view(m, G)
        start += n[b]
    return {"o": O.view(s["Q"].shape), "l": L.view(s["Q"].shape[:-1])}
