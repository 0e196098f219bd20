"""The paged 8-bit token cache on the GPU against the plain 64-bit reference.

Bounds. Append: a code is the nearest e4m3 to the value over its scale, within
half a step; a rotated value is off by fp32 roundings before that (cos, sin,
two products, a sum: within 2^-21 of the pair's length). Attention, with S the
scores, p the weights and |q||k| short for E = max_n s sum_d |q_d k_nd|:
  a score is off by at most e = (D + 8) 2^-23 E + 2^-20 (a sum of D products in
  fp32 in any order, whether it rounds or cuts; the scale; exp2 of the
  difference from the maximum, right to 2^-22), a weight by the factor e;
  L by e + 2^-22 |L|;
  O by 2 e A + N 2^-23 A with A = sum_n p_n |v_n| (numerator and sum, N terms
  added in fp32); the kernels for bf16 round weights to fp16, 2^-11 A more, or
  for many rows a head to bf16, 2^-8 A more; the output's own rounding, 2^-8 |O|
  for bf16.
"""
import math

import pytest
import torch

import cache_ref
from guards import guarded
from latent_query_split_gb300 import flare

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
I32 = dict(dtype=torch.int32, device="cuda")


def make_cache(B, W, H, D, page, spare=3, seed=0, fill=0x7F):
    """A cache whose pages are handed out in a random order; every slot holds a
    NaN code and every scale is NaN until something is written."""
    g = torch.Generator().manual_seed(seed)
    P = B * W + spare
    table = torch.randperm(P, generator=g)[: B * W].view(B, W).to(**I32)
    cache = flare.flare_cache_alloc(P, H, D, page, page_table=table.contiguous())
    for x in (cache.k, cache.v):
        x.view(torch.uint8).fill_(fill)
    for x in (cache.k_scale, cache.v_scale):
        x.fill_(math.nan)
    return cache


def fill(cache, lens, seed=0, big=8.0):
    """Random tokens in the slots that the sequences hold, written here with torch:
    exponents of the scales differ from page to page."""
    g = torch.Generator().manual_seed(seed)
    P, H, page, D = cache.k.shape
    for codes, scale in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        c, s = codes.view(torch.uint8).cpu(), scale.cpu()
        for b, n in enumerate(lens):
            for w in range(-(-n // page)):
                p, m = int(cache.page_table[b, w]), min(page, n - w * page)
                x = torch.randn((H, m, D), generator=g) * (100 if torch.rand((), generator=g) < 0.5 else 60)
                e = torch.randint(-9, -4, (H,), generator=g)
                if torch.rand((), generator=g) < 0.1:
                    e += int(math.log2(big))
                s[p] = torch.exp2(e.float())
                c[p, :, :m] = x.clamp(-448, 448).to(cache_ref.F8).view(torch.uint8)
        codes.view(torch.uint8).copy_(c)
        scale.copy_(s)


def ints(x):
    return torch.tensor(list(x), **I32)


def starts(counts):
    return ints([sum(counts[:i]) for i in range(len(counts) + 1)])


def check_attn(O, L, Q, cache, lens, counts, causal, scale=None, kernel="auto", o_f32=False):
    T, Hq, D = Q.shape
    room = cache.page_table.shape[1] * cache.k.shape[2]
    many = D in (64, 128) and T * Hq // (cache.k.shape[1] * len(lens)) > (16 if room > 16384 else 32)
    step = 0.0 if kernel == "simt" or Q.dtype == torch.float32 else 2.0 ** -8 if many else 2.0 ** -11
    ref = cache_ref.host(cache)
    o, l, A, E = cache_ref.attn(ref, Q.cpu(), lens, counts, causal, scale)
    O, L = O.reshape(T, Hq, D).cpu().double(), L.reshape(T, Hq).cpu().double()
    N = max(max(lens), 1)
    e = (D + 8) * 2.0 ** -23 * E + 2.0 ** -20
    bf16 = Q.dtype == torch.bfloat16
    tol_o = (2 * e[..., None] + N * 2.0 ** -23 + step) * A
    tol_o = tol_o + (2.0 ** -8 * 1.01 if bf16 and not o_f32 else 2.0 ** -23) * o.abs() + 1e-37
    empty = l == -math.inf
    assert torch.equal(L == -math.inf, empty), "rows that see nothing"
    assert (O[empty] == 0).all()
    assert not O.isnan().any() and not L.isnan().any()
    worst = ((O - o).abs() / tol_o).max().item()
    assert worst <= 1, f"O is {worst:.3g} of its bound off"
    d = ((L - l).abs() / (e + 2.0 ** -22 * l.abs()))[~empty]
    assert d.numel() == 0 or d.max().item() <= 1, f"L is {d.max().item():.3g} of its bound off"


# ---- append ------------------------------------------------------------------------
def run_append(cache, K, V, Q, lens, counts, inv_freq=None, interleaved=False, ragged=True):
    B = cache.page_table.shape[0]
    cu = starts(counts) if ragged else None
    if not ragged:
        K, V = (x.unflatten(0, (B, -1)) for x in (K, V))
        Q = None if Q is None else Q.unflatten(0, (B, -1))
    return flare.flare_cache_append(cache, K, V, ints(lens), cu_seqlens=cu, Q=Q, inv_freq=inv_freq, interleaved=interleaved)


def check_append(cache, before, K, V, Q, lens, counts, inv_freq, interleaved, lens_out, q_out):
    want, new, again = cache_ref.append(before, K.cpu(), V.cpu(), lens, counts, None if inv_freq is None else inv_freq.cpu(),
                                        interleaved)
    got = cache_ref.host(cache)
    assert lens_out.tolist() == [x + y for x, y in zip(lens, counts)]
    for x in "kv":
        s, t = got[x + "_scale"], want[x + "_scale"]
        assert torch.equal(s[~t.isnan()], t[~t.isnan()]) and torch.equal(s.isnan(), t.isnan()), x + "_scale"
        y, z = want[x], got[x]
        assert torch.equal(y.isnan(), z.isnan()), x
        touched = (new[:, None] | again[x])[..., None].expand_as(y) & ~y.isnan()
        same = ~touched & ~y.isnan()
        assert torch.equal(y[same], z[same]), x + ": a slot that was not written changed"
        tol = cache_ref.half_step(y[touched])
        if x == "k" and inv_freq is not None:
            tol = tol + 362 * 2.0 ** -21
        assert ((y - z).abs()[touched] <= tol * (1 + 1e-9)).all(), x
    if q_out is not None:
        t, q = 0, Q.double().cpu()
        for at, n in zip(lens, counts):
            for i in range(n):
                if inv_freq is not None:
                    r = cache_ref.rotate(q[t], at + i, inv_freq.cpu(), interleaved)
                    tol = 2.0 ** -21 * q[t].abs().max() * 2 ** 0.5
                else:
                    r, tol = q[t], 0.0
                half = 2.0 ** -8 if Q.dtype == torch.bfloat16 else 2.0 ** -24
                d = (q_out.reshape(Q.shape)[t].cpu().double() - r).abs()
                assert (d <= tol + half * r.abs() * (1 + 2.0 ** -7)).all()
                t += 1


def freqs(rot, base=10000.0):
    return (base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float().cuda() if rot else None


# Calls of few tokens a sequence, of many (a page and some heads a block: one, two
# and four tasks a thread, several heads at once), and of rotations whose pairs do
# not lie in runs of eight.
APPENDS = [  # dtype, H, Hq, D, page, rot, interleaved, lens, counts
    ("bf16", 2, 4, 64, 16, 64, False, [0, 5, 16, 31], [1, 1, 1, 1]),
    ("bf16", 1, 3, 128, 64, 128, False, [0, 63, 64, 100], [70, 1, 0, 129]),
    ("bf16", 3, 3, 96, 32, 48, True, [7, 0, 95], [33, 200, 1]),
    ("bf16", 2, 0, 16, 128, 2, False, [127, 128, 129], [1, 128, 127]),
    ("bf16", 2, 2, 128, 16, 20, False, [3, 1], [40, 41]),
    ("fp32", 2, 4, 64, 32, 64, True, [1, 0, 31], [0, 64, 66]),
    ("fp32", 2, 2, 32, 64, 0, False, [10], [300]),
    ("fp32", 1, 5, 112, 128, 112, False, [200, 0], [1, 2]),
    ("fp32", 4, 0, 128, 64, 100, False, [64] * 5, [0, 0, 3, 0, 61]),
    ("bf16", 8, 32, 128, 64, 128, True, [63, 0], [130, 5]),
    ("bf16", 3, 9, 128, 128, 64, False, [100, 0], [400, 129]),
    ("fp32", 2, 4, 128, 128, 128, True, [5], [260]),
    ("bf16", 5, 5, 32, 16, 32, False, [9, 0, 16], [40, 33, 100]),
    ("bf16", 9, 0, 64, 16, 16, True, [15, 0], [90, 17]),
    ("fp32", 3, 6, 80, 32, 80, False, [31, 1], [70, 64]),
    ("bf16", 2, 18, 128, 32, 128, False, [31, 0, 5], [2, 1, 4]),
    ("fp32", 9, 9, 96, 16, 32, True, [15, 3], [1, 8]),
]


@pytest.mark.parametrize("dtype,H,Hq,D,page,rot,inter,lens,counts", APPENDS)
def test_append(dtype, H, Hq, D, page, rot, inter, lens, counts):
    W = max(x + y for x, y in zip(lens, counts)) // page + 2
    cache = make_cache(len(lens), W, H, D, page)
    fill(cache, lens, seed=1)
    before = cache_ref.host(cache)
    g = torch.Generator().manual_seed(2)
    T = sum(counts)
    K, V = ((torch.randn((T, H, D), generator=g) * torch.exp2(torch.randint(-6, 7, (T, 1, 1), generator=g).float())).to(DT[dtype]).cuda()
            for _ in range(2))
    Q = torch.randn((T, Hq, D), generator=g).to(DT[dtype]).cuda() if Hq else None
    f = freqs(rot)
    lens_out, q_out = run_append(cache, K, V, Q, lens, counts, f, inter)
    flare.flare_device_status()
    check_append(cache, before, K, V, Q, lens, counts, f, inter, lens_out, q_out)


def test_append_equal_rows_from_a_fused_projection():
    """[B, n, ...] slices of one wide projection: token strides that are not dense."""
    B, n, H, Hq, D, page, lens = 3, 5, 2, 4, 64, 16, [14, 0, 33]
    cache = make_cache(B, 4, H, D, page)
    fill(cache, lens, seed=3)
    before = cache_ref.host(cache)
    x = torch.randn((B, n, Hq + 2 * H, D), generator=torch.Generator().manual_seed(4)).bfloat16().cuda()
    Q, K, V = x[:, :, :Hq], x[:, :, Hq:Hq + H], x[:, :, Hq + H:]
    f = freqs(D)
    lens_out, q_out = flare.flare_cache_append(cache, K, V, ints(lens), Q=Q, inv_freq=f)
    flat = lambda y: y.reshape(B * n, *y.shape[2:])  # noqa: E731
    check_append(cache, before, flat(K), flat(V), flat(Q), lens, [n] * B, f, False, lens_out, q_out)


@pytest.mark.parametrize("n", [2, 40])
def test_append_of_any_alignment(n):
    """Tensors that begin at odd elements."""
    H, Hq, D, page, lens = 2, 4, 64, 16, [14]
    cache = make_cache(1, 5, H, D, page)
    fill(cache, lens, seed=13)
    before = cache_ref.host(cache)
    g = torch.Generator().manual_seed(14)
    off = lambda heads: torch.randn(n * heads * D + 1, generator=g).bfloat16().cuda()[1:].view(1, n, heads, D)  # noqa: E731
    K, V, Q, f = off(H), off(H), off(Hq), freqs(D)
    out, q = flare.flare_cache_append(cache, K, V, ints(lens), Q=Q, inv_freq=f)
    check_append(cache, before, K[0], V[0], Q[0], lens, [n], f, False, out, q[0])
    O = off(Hq)
    flare.flare_cache_attn(Q, cache, out, O=O)
    L = flare.flare_cache_attn(Q, cache, out)[1]
    check_attn(O[0], L[0], Q[0], cache, out.tolist(), [n], True)


@pytest.mark.parametrize("at", [0, 1000, 999_999, (1 << 30) - 200])
def test_append_far_positions(at):
    """Angles are right at any position: the cache's table reaches 2^30 tokens (its
    earlier entries name one page, which is not touched)."""
    page, D = 128, 128
    W = (at + 40) // page + 1
    cache = make_cache(1, 3, 1, D, page, spare=0)
    if at % page:
        fill(cache, [3 * page], seed=5)
    wide = torch.zeros((1, W), **I32) + int(cache.page_table[0, 2])
    w = at // page
    wide[0, w], last = cache.page_table[0, 0], (at + 39) // page
    if last > w:
        wide[0, last] = cache.page_table[0, 1]
    cache = cache._replace(page_table=wide)
    before = cache_ref.host(cache)
    g = torch.Generator().manual_seed(6)
    K, V, Q = (torch.randn((40, 1, D), generator=g).cuda() for _ in range(3))
    f = freqs(D)
    f[-1] = 0.0
    f[-2] = 7.0                                           # more than a turn a position
    out, q = run_append(cache, K, V, Q, [at], [40], f)
    flare.flare_device_status()
    check_append(cache, before, K, V, Q, [at], [40], f, False, out, q)


def test_append_grows_a_pages_scale():
    """Token after token, each larger than the last: the page's codes are rescaled;
    a smaller one leaves them."""
    cache = make_cache(1, 1, 1, 32, 16)
    g = torch.Generator().manual_seed(7)
    for i, size in enumerate([2.0 ** -30, 1.0, 1.0, 16.0, 0.25, 2.0 ** 40, 0.0]):
        before = cache_ref.host(cache)
        K, V = (torch.randn((1, 1, 32), generator=g).mul(size).cuda() for _ in range(2))
        out, _ = run_append(cache, K, V, None, [i], [1])
        check_append(cache, before, K, V, None, [i], [1], None, False, out, None)


@pytest.mark.parametrize("pieces", [[20], [4, 3, 10, 3]])
def test_append_holds_what_is_not_finite_as_nan_keys(pieces):
    cache = make_cache(1, 2, 2, 64, 16)
    K, V = (torch.randn((20, 2, 64), generator=torch.Generator().manual_seed(s)).bfloat16() for s in (8, 9))
    K[3, 0, 5], K[4, 1, 0], V[6, 0, 63], V[17, 1, 1] = math.nan, math.inf, -math.inf, math.nan
    at = 0
    for n in pieces:
        before = cache_ref.host(cache)
        k, v = K[at:at + n], V[at:at + n]
        out, _ = run_append(cache, k.cuda(), v.cuda(), None, [at], [n], freqs(64))
        check_append(cache, before, k, v, None, [at], [n], freqs(64), False, out, None)
        at += n
    assert not cache.v.float()[cache.page_table[0].long()].transpose(1, 2).reshape(32, 2, 64)[:20].isnan().any()
    Q = torch.randn((20, 2, 64), generator=torch.Generator().manual_seed(10)).bfloat16().cuda()
    for kernel in ("simt", "auto"):
        O, L = flare.flare_cache_attn(Q, cache, out, cu_seqlens=ints([0, 20]), kernel=kernel)
        bad = O.isnan().any(dim=2).cpu()                                  # [20, 2]
        want = torch.zeros((20, 2), dtype=torch.bool)
        want[6:, 0] = want[4:, 1] = want[3:, 0] = True
        assert torch.equal(bad, want) and torch.equal(L.isnan().cpu(), want)


def test_append_extreme_magnitudes():
    cache = make_cache(1, 1, 1, 16, 16)
    K = torch.zeros((4, 1, 16))
    K[0, 0, 0], K[1, 0, 0], K[2, 0, 0], K[3, 0, 0] = 3.3e38, 1e-45, 2.0 ** 68, -2.0 ** 60
    before = cache_ref.host(cache)
    out, _ = run_append(cache, K.cuda(), K.cuda() * 0, None, [0], [4])
    p = int(cache.page_table[0, 0])
    assert cache.k_scale[p, 0].item() == 2.0 ** 60 and cache.v_scale[p, 0].item() == 2.0 ** -40
    k = cache.k[p, 0, :4, 0].double()
    assert k.tolist() == [448.0, 0.0, 256.0, -1.0] and (cache.v[p, 0, :4].float() == 0).all()
    assert before["k"].isnan().all()


def test_append_drops_what_does_not_fit_and_says_so():
    """Lengths beyond the table, pages outside the pool, offsets out of order: what
    they name is skipped, the rest is written, the status says so."""
    B, H, D, page, W = 4, 1, 32, 16, 2
    cache = make_cache(B, W, H, D, page)
    table = cache.page_table.clone()
    table[1, 0], table[2, 0] = -1, cache.k.shape[0]
    cache = cache._replace(page_table=table)
    snap = {x: getattr(cache, x).clone() for x in ("k", "v", "k_scale", "v_scale")}
    K = torch.randn((B * 8, H, D)).cuda()
    lens = [28, 0, 3, 2 ** 31 - 1]
    out, _ = run_append(cache, K, K, None, lens, [8] * B)
    with pytest.raises(flare.FlareError) as e:
        flare.flare_device_status()
    assert e.value.status == flare.FLARE_ERR_CACHE
    flare.flare_device_status()                                          # and is cleared
    assert out.tolist() == [32, 8, 11, 32]
    p = int(table[0, 1])
    changed = (cache.k.view(torch.uint8) != snap["k"].view(torch.uint8)).any(dim=3).nonzero().tolist()
    assert changed == [[p, 0, s] for s in range(12, 16)]
    cu = ints([0, 8, 4, 2 ** 31 - 1, -5])
    flare.flare_cache_append(cache, K, K, ints([0] * B), cu_seqlens=cu)
    with pytest.raises(flare.FlareError):
        flare.flare_device_status()


def test_append_nothing():
    cache = make_cache(3, 2, 1, 32, 16)
    K = torch.zeros((0, 1, 32), device="cuda")
    out, _ = flare.flare_cache_append(cache, K, K, ints([4, 0, 32]), cu_seqlens=ints([0, 0, 0, 0]))
    assert out.tolist() == [4, 0, 32] and cache.k.float().isnan().all()


def test_append_many_sequences():
    """More sequences than a block has threads, most of them without a new token."""
    B, H, D, page = 700, 1, 16, 16
    g = torch.Generator().manual_seed(11)
    lens = torch.randint(0, 40, (B,), generator=g).tolist()
    counts = [n if i % 3 == 0 else 0 for i, n in enumerate(torch.randint(0, 5, (B,), generator=g).tolist())]
    cache = make_cache(B, 4, H, D, page)
    fill(cache, lens, seed=12)
    before = cache_ref.host(cache)
    K, V = (torch.randn((sum(counts), H, D), generator=g).cuda() for _ in range(2))
    out, _ = run_append(cache, K, V, None, lens, counts, freqs(16))
    flare.flare_device_status()
    check_append(cache, before, K, V, None, lens, counts, freqs(16), False, out, None)


@pytest.mark.parametrize("dtype,H,Hq,D,page,rot,inter", [
    ("bf16", 2, 18, 128, 32, 128, False), ("fp32", 9, 9, 96, 16, 32, True), ("bf16", 1, 0, 16, 16, 0, False),
    ("fp32", 3, 6, 64, 128, 64, False), ("bf16", 4, 4, 112, 64, 16, True),
])
def test_append_few_tokens_of_more_than_eight_sequences(dtype, H, Hq, D, page, rot, inter):
    """Step after step, magnitudes growing and shrinking from one to the next, some
    channels not finite: a warp a page and head."""
    g = torch.Generator().manual_seed(71)
    B = 11
    lens = torch.randint(0, 3 * page, (B,), generator=g).tolist()
    cache = make_cache(B, 5, H, D, page)
    fill(cache, lens, seed=72)
    f = freqs(rot)
    for size in (1.0, 2.0 ** 9, 2.0 ** -6):
        counts = torch.randint(0, 9, (B,), generator=g).tolist()
        before = cache_ref.host(cache)
        T = sum(counts)
        K, V = ((size * torch.randn((T, H, D), generator=g)).to(DT[dtype]) for _ in range(2))
        K[T // 2, 0, D - 1], V[T // 3, H - 1, 0] = math.inf, math.nan
        Q = torch.randn((T, Hq, D), generator=g).to(DT[dtype]).cuda() if Hq else None
        out, q = run_append(cache, K.cuda(), V.cuda(), Q, lens, counts, f, inter)
        flare.flare_device_status()
        check_append(cache, before, K, V, Q, lens, counts, f, inter, out, q)
        lens = out.tolist()


# ---- attention -----------------------------------------------------------------------
ATTNS = [  # dtype, H, G, D, page, lens, counts, causal
    ("bf16", 2, 4, 128, 64, [1500], [1], True),
    ("bf16", 2, 4, 128, 16, [0, 1, 15, 16, 17, 127, 128, 129, 600], [1] * 9, True),
    ("bf16", 1, 1, 64, 32, [1, 300, 0, 77], [1] * 4, False),
    ("bf16", 3, 5, 64, 16, [2, 90, 1000], [3, 3, 3], True),
    ("bf16", 2, 7, 96, 32, [40, 555], [9, 2], True),
    ("bf16", 1, 3, 32, 128, [700, 130, 0], [1, 0, 4], True),
    ("bf16", 2, 1, 16, 64, [513], [33], False),
    ("bf16", 1, 8, 112, 64, [260, 129], [8, 1], True),
    ("bf16", 2, 2, 128, 128, [300, 40, 700], [150, 60, 1], True),
    ("bf16", 1, 4, 64, 64, [1000], [260], True),
    ("bf16", 1, 1, 128, 64, [2049, 1111], [64, 64], False),
    ("bf16", 2, 1, 64, 32, [900, 5], [256, 256], False),
    ("bf16", 1, 1, 128, 16, [500], [200], False),
    ("bf16", 1, 3, 128, 32, [170], [171], True),
    ("bf16", 1, 2, 80, 32, [400], [100], True),
    ("fp32", 2, 4, 64, 32, [1, 1200, 0], [1] * 3, True),
    ("fp32", 1, 1, 128, 64, [700], [70], True),
    ("fp32", 2, 3, 48, 16, [50, 260], [5, 30], False),
    ("fp32", 1, 9, 112, 128, [300], [2], True),
]


@pytest.mark.parametrize("kernel", ["simt", "auto"])
@pytest.mark.parametrize("dtype,H,G,D,page,lens,counts,causal", ATTNS)
def test_attn(kernel, dtype, H, G, D, page, lens, counts, causal):
    cache = make_cache(len(lens), max(lens) // page + 2, H, D, page)
    fill(cache, lens, seed=20)
    g = torch.Generator().manual_seed(21)
    Q = torch.randn((sum(counts), H * G, D), generator=g).to(DT[dtype]).cuda()
    T, Hq = Q.shape[:2]
    O, go = guarded((T + 2, Hq, D), DT[dtype], fill=7.0)
    L, gl = guarded((T + 2, Hq), fill=7.0)
    need = flare.flare_cache_workspace_bytes(flare.flare_cache_dims(cache, Hq, Q.dtype, kernel=kernel), T + 2)
    ws, gw = guarded((need,), torch.uint8)
    tail = torch.full((2, Hq, D), math.nan, dtype=Q.dtype, device="cuda")       # rows behind the last sequence
    flare.flare_cache_attn(torch.cat((Q, tail)), cache, ints(lens), cu_seqlens=starts(counts), causal=causal, O=O, L=L,
                           workspace=ws, kernel=kernel)
    flare.flare_device_status()
    check_attn(O[:T], L[:T], Q, cache, lens, counts, causal, kernel=kernel)
    assert (O[T:] == 7).all() and (L[T:] == 7).all(), "rows behind the last sequence were written"
    for x, name in ((go, "O"), (gl, "L"), (gw, "workspace")):
        x.check(name)


EQUAL = [  # dtype, H, G, D, page, lens, n, causal: equal sequences (small ones are a cluster's)
    ("bf16", 2, 4, 128, 64, [1500], 1, True),
    ("bf16", 2, 5, 64, 16, [2, 900, 33, 128, 0, 17], 3, True),
    ("bf16", 1, 3, 96, 32, [100, 1], 9, False),
    ("bf16", 4, 8, 128, 128, [129] * 5, 4, True),
    ("fp32", 2, 4, 64, 32, [1, 1200, 0, 300], 1, True),
    ("fp32", 1, 9, 112, 16, [260, 500], 4, True),
    ("bf16", 8, 2, 32, 16, [5000, 31, 700], 2, False),
]


@pytest.mark.parametrize("dtype,H,G,D,page,lens,n,causal", EQUAL)
def test_attn_equal_sequences(dtype, H, G, D, page, lens, n, causal):
    B = len(lens)
    cache = make_cache(B, max(lens) // page + 2, H, D, page)
    fill(cache, lens, seed=70)
    Q = torch.randn((B, n, H * G, D), generator=torch.Generator().manual_seed(71)).to(DT[dtype]).cuda()
    O, go = guarded(Q.shape, DT[dtype], fill=7.0)
    L, gl = guarded(Q.shape[:-1], fill=7.0)
    flare.flare_cache_attn(Q, cache, ints(lens), causal=causal, O=O, L=L)
    flare.flare_device_status()
    check_attn(O, L, Q.reshape(B * n, H * G, D), cache, lens, [n] * B, causal)
    go.check("O")
    gl.check("L")


@pytest.mark.parametrize("kernel", ["simt", "auto"])
@pytest.mark.parametrize("n", [1, 40, 140])
def test_attn_equal_rows_strided_queries_and_scale(kernel, n):
    B, H, G, D, page, lens = 2, 2, 2, 64, 32, [333, 150]
    cache = make_cache(B, 12, H, D, page)
    fill(cache, lens, seed=22)
    wide = torch.randn((B, n, H * G + 3, D), generator=torch.Generator().manual_seed(23)).bfloat16().cuda()
    Q = wide[:, :, 1:1 + H * G]
    for causal in (True, False):
        O, L = flare.flare_cache_attn(Q, cache, ints(lens), causal=causal, scale=0.3, kernel=kernel)
        check_attn(O, L, Q.reshape(B * n, H * G, D), cache, lens, [n] * B, causal, scale=0.3)


@pytest.mark.parametrize("kernel", ["simt", "auto"])
@pytest.mark.parametrize("dtype,n", [("bf16", 1), ("bf16", 130), ("fp32", 2)])
def test_attn_sharp_scores(kernel, dtype, n):
    """Scores in the hundreds, the largest anywhere in the sequence."""
    H, D, page, lens = 2, 64, 16, [700]
    cache = make_cache(1, 44, H, D, page)
    fill(cache, lens, seed=24, big=64.0)
    for s in (25, 26):
        Q = (20 * torch.randn((n, H, D), generator=torch.Generator().manual_seed(s))).to(DT[dtype]).cuda()
        O, L = flare.flare_cache_attn(Q, cache, ints(lens), cu_seqlens=ints([0, n]), kernel=kernel)
        check_attn(O, L, Q, cache, lens, [n], True)


@pytest.mark.parametrize("kernel", ["simt", "auto"])
@pytest.mark.parametrize("n", [1, 30, 140])
def test_attn_value_scales_far_apart(kernel, n):
    """Pages whose value scales differ by 2^60: the sum of the weights and the
    small pages' rows stay right."""
    H, D, page, lens = 1, 64, 16, [256]
    cache = make_cache(1, 17, H, D, page)
    fill(cache, lens, seed=27)
    w = cache.page_table[0].long()
    cache.v_scale[w[:6]] = 2.0 ** 30
    cache.v_scale[w[6:]] = 2.0 ** -30
    Q = torch.randn((n, H, D), generator=torch.Generator().manual_seed(28)).bfloat16().cuda()
    for lens in ([256], [96]):
        O, L = flare.flare_cache_attn(Q, cache, ints(lens), cu_seqlens=ints([0, n]), causal=False, kernel=kernel)
        check_attn(O, L, Q, cache, lens, [n], False)
    cache.v_scale[w[:6]] = 2.0 ** -30
    cache.v_scale[w[6:]] = 2.0 ** 30
    O, L = flare.flare_cache_attn(Q, cache, ints([256]), cu_seqlens=ints([0, n]), causal=False, kernel=kernel)
    check_attn(O, L, Q, cache, [256], [n], False)


@pytest.mark.parametrize("kernel", ["simt", "auto"])
@pytest.mark.parametrize("n", [1, 20, 200])
def test_attn_query_rows_that_are_not_finite(kernel, n):
    H, D, page, lens = 2, 128, 64, [300]
    cache = make_cache(1, 6, H, D, page)
    fill(cache, lens, seed=29)
    Q = torch.randn((n, H, D), generator=torch.Generator().manual_seed(30)).bfloat16()
    clean = Q.clone()
    Q[0, 0, 3], Q[n // 2, 1, 100] = math.nan, math.inf
    args = dict(cu_seqlens=ints([0, n]), kernel=kernel)
    O, L = flare.flare_cache_attn(Q.cuda(), cache, ints(lens), **args)
    want, wl = flare.flare_cache_attn(clean.cuda(), cache, ints(lens), **args)
    bad = torch.zeros((n, H), dtype=torch.bool)
    bad[0, 0] = bad[n // 2, 1] = True
    assert O.cpu()[bad].isnan().all() and L.cpu()[bad].isnan().all()
    assert torch.equal(O.cpu()[~bad], want.cpu()[~bad]) and torch.equal(L.cpu()[~bad], wl.cpu()[~bad])


@pytest.mark.parametrize("kernel", ["simt", "auto"])
@pytest.mark.parametrize("n", [1, 30, 130])
def test_attn_zero_and_wide_ranged_queries(kernel, n):
    """Query rows of zeros, and rows whose channels span 2^-40 .. 2^10."""
    H, D, page, lens = 1, 64, 32, [200]
    cache = make_cache(1, 8, H, D, page)
    fill(cache, lens, seed=31)
    g = torch.Generator().manual_seed(32)
    Q = (torch.randn((n, H, D), generator=g) * torch.exp2(torch.randint(-40, 3, (n, H, D), generator=g).float())).bfloat16()
    Q[::2] *= 2.0 ** -60
    Q[-1] = 0
    Q = Q.cuda()
    O, L = flare.flare_cache_attn(Q, cache, ints(lens), cu_seqlens=ints([0, n]), kernel=kernel)
    check_attn(O, L, Q, cache, lens, [n], True)


@pytest.mark.parametrize("kernel", ["simt", "auto"])
@pytest.mark.parametrize("n", [1, 150])
def test_attn_skips_bad_pages_and_says_so(kernel, n):
    B, H, D, page, lens = 3, 1, 64, 16, [100, 60, 2 ** 31 - 1]
    cache = make_cache(B, 8, H, D, page)
    fill(cache, [100, 60, 128], seed=33)
    table = cache.page_table.clone()
    table[0, 1], table[1, 3] = -7, 2 ** 31 - 1
    Q = torch.randn((B * n, H, D), generator=torch.Generator().manual_seed(34)).bfloat16().cuda()
    O, L = flare.flare_cache_attn(Q, cache._replace(page_table=table), ints(lens), cu_seqlens=starts([n] * B), causal=False,
                                  kernel=kernel)
    with pytest.raises(flare.FlareError) as e:
        flare.flare_device_status()
    assert e.value.status == flare.FLARE_ERR_CACHE
    # the same sequences without those tokens; the third's length is the table's
    short = cache.page_table.clone()
    short[0, :-1] = cache.page_table[0, [0, 2, 3, 4, 5, 6, 7]]
    check_attn(O, L, Q, cache._replace(page_table=short), [84, 48, 128], [n] * B, False)


@pytest.mark.parametrize("kernel", ["simt", "auto"])
@pytest.mark.parametrize("D,n", [(64, 1), (128, 20), (64, 130), (128, 140)])
def test_attn_every_code(kernel, D, n):
    """Every finite code, subnormal ones too, as keys and as values: tokens of the
    smallest codes alone, and of all of them."""
    page, H = 32, 1
    cache = make_cache(1, 9, H, D, page)
    fill(cache, [256], seed=60)
    codes = torch.tensor([c for c in range(256) if c & 0x7F != 0x7F], dtype=torch.uint8)
    tiny = torch.tensor([1, 2, 3, 4, 5, 6, 7, 0x81, 0x82, 0x83, 0x85, 0x87, 0, 0x80], dtype=torch.uint8)
    g = torch.Generator().manual_seed(61)
    Q = torch.randn((n, H, D), generator=g).bfloat16().cuda()
    for pick in (tiny, codes):
        for x in (cache.k, cache.v):
            b = x.view(torch.uint8)
            b.copy_(pick[torch.randint(0, len(pick), b.shape, generator=g)])
        O, L = flare.flare_cache_attn(Q, cache, ints([256]), cu_seqlens=ints([0, n]), causal=False, kernel=kernel)
        check_attn(O, L, Q, cache, [256], [n], False, kernel=kernel)


@pytest.mark.parametrize("kernel", ["simt", "auto"])
@pytest.mark.parametrize("D,n", [(64, 1), (128, 40), (64, 130), (128, 300)])
def test_attn_scores_that_grow(kernel, D, n):
    """Keys that double from tile to tile: the largest score moves by more than any
    reference leaves room for, inside a tile and from one to the next."""
    page, H, lens = 32, 1, [1024]
    cache = make_cache(1, 33, H, D, page)
    fill(cache, lens, seed=62)
    for w in range(32):
        cache.k_scale[int(cache.page_table[0, w])] = 2.0 ** (w - 24)
    for seed in (63, 64):
        Q = torch.randn((n, H, D), generator=torch.Generator().manual_seed(seed)).bfloat16().cuda()
        O, L = flare.flare_cache_attn(Q, cache, ints(lens), cu_seqlens=ints([0, n]), causal=False, kernel=kernel, scale=0.02)
        check_attn(O, L, Q, cache, lens, [n], False, scale=0.02, kernel=kernel)


@pytest.mark.parametrize("D", [64, 128])
def test_attn_wide_row_tiles(D):
    """Row tiles of 256 (ragged calls of more than 896 rows a sequence on average): the
    causal edge inside tiles, a sequence that ends inside one, keys that double."""
    page, lens, counts = 64, [1300, 950, 3], [1250, 949, 600]
    cache = make_cache(3, 21, 1, D, page)
    fill(cache, lens, seed=65)
    Q = torch.randn((sum(counts), 1, D), generator=torch.Generator().manual_seed(66)).bfloat16().cuda()
    O, L = flare.flare_cache_attn(Q, cache, ints(lens), cu_seqlens=starts(counts))
    flare.flare_device_status()
    check_attn(O, L, Q, cache, lens, counts, True)
    for w in range(20):
        cache.k_scale[int(cache.page_table[0, w])] = 2.0 ** (w - 18)
    O, L = flare.flare_cache_attn(Q, cache, ints(lens), cu_seqlens=starts(counts), causal=False, scale=0.02)
    check_attn(O, L, Q, cache, lens, counts, False, scale=0.02)


@pytest.mark.parametrize("D,n", [(64, 20), (128, 17), (128, 32)])
def test_attn_some_rows_over_a_long_table(D, n):
    """17 to 32 rows a sequence where the table has room for more than 16,384 tokens."""
    page, lens = 128, [700, 0, 1, 129]
    cache = make_cache(4, 130, 1, D, page)
    fill(cache, lens, seed=67)
    Q = torch.randn((4, n, 1, D), generator=torch.Generator().manual_seed(68)).bfloat16().cuda()
    for causal in (True, False):
        O, L = flare.flare_cache_attn(Q, cache, ints(lens), causal=causal)
        check_attn(O, L, Q.reshape(4 * n, 1, D), cache, lens, [n] * 4, causal)


@pytest.mark.parametrize("M,D", [(3, 64), (40, 64), (150, 64), (64, 128), (200, 128), (700, 128)])
def test_rows_that_one_token_fills(M, D):
    """A late token whose score is far above all others': Z (fp32) is its value. The
    weights' rounding (2^-8 or 2^-11) must not show in it: of the others' share r of the
    row at most 2^-7 r max|v| of it can, on top of the bounds above."""
    H, page, lens = 1, 64, [900]
    cache = make_cache(1, 16, H, D, page)
    fill(cache, lens, seed=69)
    g = torch.Generator().manual_seed(70)
    Q = (0.1 * torch.randn((H, M, D), generator=g)).abs().bfloat16().cuda()
    p, s = int(cache.page_table[0, 13]), 17                               # token 849
    cache.k_scale[p] = 2.0 ** -4
    cache.k.view(torch.uint8)[p, 0, s] = torch.full((D,), 400.0).to(cache_ref.F8).view(torch.uint8).cuda()
    Z, L = flare.flare_cache_encoder_fwd(Q, cache, ints(lens))
    q = Q[0][:, None]
    o, l, A, E = cache_ref.attn(cache_ref.host(cache), q.cpu(), lens, [M], False, None)
    v = cache.v[p, 0, s].double().cpu() * cache.v_scale[p, 0].double().cpu()
    big = max((cache.v[int(x), 0, :].double().cpu().nan_to_num().abs().max() * cache.v_scale[int(x), 0].double().cpu()).item()
              for x in cache.page_table[0, :15])
    k = cache.k[p, 0, s].double().cpu() * cache.k_scale[p, 0].double().cpu()
    rest = 1 - torch.exp((q.double().cpu()[:, 0] @ k) * D ** -0.5 - l[:, 0])                      # share of the other tokens
    assert rest.max() < 2.0 ** -6                 # (the bound below is of `rest`, and holds for any: this is for its sharpness)
    e = (D + 8) * 2.0 ** -23 * E[:, 0] + 2.0 ** -20
    tol = (2 * rest[:, None] * e[:, None] + 900 * 2.0 ** -23) * A[:, 0] + 2.0 ** -7 * rest.clamp(min=0)[:, None] * big + 1e-9 * big
    worst = ((Z[0, 0].double().cpu() - o[:, 0]).abs() / tol).max().item()
    assert worst <= 1, f"Z is {worst:.3g} of its bound off"
    assert ((o[:, 0] - v).abs() <= 2 * rest[:, None].clamp(min=0) * big + 1e-12 * big).all()


@pytest.mark.parametrize("dtype,G", [("bf16", 4), ("bf16", 11), ("fp32", 2)])
def test_attn_short_and_empty_sequences_among_long_ones(dtype, G):
    """Items of no tile at all, of one and of many: spans begin and end inside them."""
    H, D, page, B = 2, 64, 32, 60
    g = torch.Generator().manual_seed(73)
    lens = [0 if i % 4 == 0 else int(x) for i, x in enumerate(torch.randint(0, 40, (B,), generator=g) ** 2 % 1500)]
    lens[7], lens[-1], lens[-2], lens[-3] = 5000, 0, 0, 0
    cache = make_cache(B, 160, H, D, page, spare=1)
    fill(cache, lens, seed=74)
    Q = torch.randn((B, H * G, D), generator=g).to(DT[dtype]).cuda()
    O, L = flare.flare_cache_attn(Q, cache, ints(lens), cu_seqlens=starts([1] * B))
    flare.flare_device_status()
    check_attn(O, L, Q, cache, lens, [1] * B, True)


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("fp32", 32)])
def test_attn_one_item_over_every_span(dtype, D):
    """One head of one long sequence: as many pieces as there are spans."""
    page, lens = 128, [70_001]
    cache = make_cache(1, 548, 1, D, page)
    fill(cache, lens, seed=75)
    Q = torch.randn((1, 2, 3, D), generator=torch.Generator().manual_seed(76)).to(DT[dtype]).cuda()
    O, L = flare.flare_cache_attn(Q, cache, ints(lens))
    check_attn(O, L, Q[0], cache, lens, [2], True)


@pytest.mark.parametrize("dtype,n", [("bf16", 1), ("bf16", 130), ("fp32", 1)])
def test_attn_pool_beyond_32_bits(dtype, n):
    """A pool of more than 2^32 bytes each for keys and values: pages at both ends."""
    H, D, page = 2, 128, 128
    P = (1 << 32) // (H * D * page) + 40
    table = torch.tensor([[P - 1, 0, P - 2, 1, P - 3]], **I32)
    cache = flare.flare_cache_alloc(P, H, D, page, page_table=table)
    lens = [400]
    small = make_cache(1, 5, H, D, page, spare=0)
    fill(small, lens, seed=35)
    at, src = table[0].long(), small.page_table[0].long()
    for x in ("k", "v"):
        getattr(cache, x).view(torch.uint8)[at] = getattr(small, x).view(torch.uint8)[src]
    cache.k_scale[at], cache.v_scale[at] = small.k_scale[src], small.v_scale[src]
    g = torch.Generator().manual_seed(36)
    K, V, Q = (torch.randn((n, H, D), generator=g).to(DT[dtype]).cuda() for _ in range(3))
    before = cache_ref.host(small)
    out, _ = run_append(cache, K, V, None, lens, [n], None)
    O, L = flare.flare_cache_attn(Q, cache, out, cu_seqlens=ints([0, n]))
    out2, _ = run_append(small, K, V, None, lens, [n], None)
    check_append(small, before, K, V, None, lens, [n], None, False, out2, None)
    for x in ("k", "v"):
        assert torch.equal(getattr(cache, x).view(torch.uint8)[at], getattr(small, x).view(torch.uint8)[src])
    check_attn(O, L, Q, small, out2.tolist(), [n], True)


@pytest.mark.parametrize("n", [1, 140])
def test_attn_many_sequences(n):
    B, H, G, D, page = 400, 1, 2, 64, 16
    g = torch.Generator().manual_seed(37)
    lens = torch.randint(0, 150, (B,), generator=g).tolist()
    counts = [n if i % 50 == 0 else int(x) for i, x in enumerate(torch.randint(0, 3, (B,), generator=g))]
    cache = make_cache(B, 10, H, D, page)
    fill(cache, lens, seed=38)
    Q = torch.randn((sum(counts), H * G, D), generator=g).bfloat16().cuda()
    O, L = flare.flare_cache_attn(Q, cache, ints(lens), cu_seqlens=starts(counts))
    flare.flare_device_status()
    check_attn(O, L, Q, cache, lens, counts, True)


@pytest.mark.parametrize("kernel", ["simt", "auto"])
def test_attn_shared_pages(kernel):
    """Two sequences whose first pages are the same ones; the same rows twice give
    the same bits."""
    H, D, page = 2, 64, 16
    cache = make_cache(2, 8, H, D, page)
    fill(cache, [100, 120], seed=39)
    table = cache.page_table.clone()
    table[1, :4] = table[0, :4]
    cache = cache._replace(page_table=table)
    Q = torch.randn((2, 1, 4, D), generator=torch.Generator().manual_seed(40)).bfloat16().cuda()
    O, L = flare.flare_cache_attn(Q, cache, ints([100, 120]), kernel=kernel)
    check_attn(O, L, Q.reshape(2, 4, D), cache, [100, 120], [1, 1], True)
    for _ in range(3):
        O2, L2 = flare.flare_cache_attn(Q, cache, ints([100, 120]), kernel=kernel)
        assert torch.equal(O, O2) and torch.equal(L, L2)


# ---- the run of them together ---------------------------------------------------------
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_prompt_then_tokens(dtype):
    """A prompt in two pieces, then token after token: rotation, append, attention;
    every attention agrees with the plain one over what the cache holds."""
    B, H, G, D, page = 2, 2, 3, 64, 16
    cache = make_cache(B, 20, H, D, page)
    f, g = freqs(D), torch.Generator().manual_seed(41)
    lens = ints([0, 0])
    for counts in ([150, 33], [70, 1], [1, 1], [1, 1], [0, 1], [4, 2]):
        T = sum(counts)
        K, V = (torch.randn((T, H, D), generator=g).to(DT[dtype]).cuda() for _ in range(2))
        Q = torch.randn((T, H * G, D), generator=g).to(DT[dtype]).cuda()
        cu, was, before = starts(counts), lens.tolist(), cache_ref.host(cache)
        lens, q = flare.flare_cache_append(cache, K, V, lens, cu_seqlens=cu, Q=Q, inv_freq=f)
        check_append(cache, before, K, V, Q, was, counts, f, False, lens, q)
        O, L = flare.flare_cache_attn(q, cache, lens, cu_seqlens=cu)
        check_attn(O, L, q, cache, lens.tolist(), counts, True)
    flare.flare_device_status()


@pytest.mark.parametrize("n", [1, 36])
def test_captured_step_follows_the_lengths(n):
    """One step captured in a graph, replayed while the sequences grow; two graphs
    in turn share one workspace."""
    B, H, G, D, page = 2, 2, 4, 128, 16
    cache = make_cache(B, 40, H, D, page)
    lens = ints([0, 45])
    fill(cache, lens.tolist(), seed=42)
    K, V = (torch.zeros((B, n, H, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    Q = torch.zeros((B, n, H * G, D), dtype=torch.bfloat16, device="cuda")
    O, L, after = torch.empty_like(Q), torch.empty(Q.shape[:-1], device="cuda"), torch.empty_like(lens)
    ws = torch.empty(flare.flare_cache_workspace_bytes(flare.flare_cache_dims(cache, H * G, Q.dtype), B * n), dtype=torch.uint8,
                     device="cuda")
    f = freqs(D)

    def step():
        _, q = flare.flare_cache_append(cache, K, V, lens, Q=Q, inv_freq=f, seq_lens_out=after)
        flare.flare_cache_attn(q, cache, after, O=O, L=L, workspace=ws)
        lens.copy_(after)
        return q
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            q = step()
        graphs.append((graph, q))
    g = torch.Generator().manual_seed(43)
    for i in range(6):
        for x in (K, V, Q):
            x.copy_(torch.randn(x.shape, generator=g))
        graph, q = graphs[i % 2]
        graph.replay()
        torch.cuda.synchronize()
        assert lens.tolist() == [n * (i + 2), 45 + n * (i + 2)]
        check_attn(O, L, q.reshape(B * n, H * G, D), cache, lens.tolist(), [n] * B, True)


def test_two_streams_at_once():
    """Two calls that may overlap, each with its own workspace and stream."""
    H, G, D, page = 2, 4, 64, 32
    caches, want = [], []
    Q = torch.randn((1, 1, H * G, D), generator=torch.Generator().manual_seed(44)).bfloat16().cuda()
    for s in range(2):
        c = make_cache(1, 200, H, D, page, seed=s)
        fill(c, [6000], seed=45 + s)
        caches.append(c)
        want.append(flare.flare_cache_attn(Q, c, ints([6000])))
    lens = ints([6000])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(20):
        for s in range(2):
            with torch.cuda.stream(streams[s]):
                got[s].append(flare.flare_cache_attn(Q, caches[s], lens))
    torch.cuda.synchronize()
    for s in range(2):
        for O, L in got[s]:
            assert torch.equal(O, want[s][0]) and torch.equal(L, want[s][1])


def test_given_stream():
    """Calls with `stream` run there, and what they allocate belongs to it."""
    H, G, D, page = 2, 4, 64, 32
    cache = make_cache(1, 40, H, D, page)
    fill(cache, [600], seed=47)
    g = torch.Generator().manual_seed(48)
    K, V, Q = (torch.randn((1, 40, h, D), generator=g).bfloat16().cuda() for h in (H, H, H * G))
    side, lens = torch.cuda.Stream(), ints([600])
    side.wait_stream(torch.cuda.current_stream())
    before = cache_ref.host(cache)
    for stream in (side, side.cuda_stream):
        out, q = flare.flare_cache_append(cache, K, V, lens, Q=Q, inv_freq=freqs(D), stream=stream)
        O, L = flare.flare_cache_attn(q, cache, out, stream=stream)
        Z, _ = flare.flare_cache_encoder_fwd(Q[0].transpose(0, 1)[:H].contiguous(), cache, out, stream=stream)
    side.synchronize()
    check_append(cache, before, K[0], V[0], Q[0], [600], [40], freqs(D), False, out, q[0])
    check_attn(O[0], L[0], q[0], cache, [640], [40], True)


# ---- the FLARE encoder and mixer over the cache ------------------------------------------
@pytest.mark.parametrize("dtype,M,D,per_batch", [("bf16", 64, 64, False), ("bf16", 128, 128, True), ("bf16", 256, 64, False),
                                                 ("bf16", 20, 32, True), ("fp32", 16, 32, False), ("fp32", 33, 64, True)])
def test_encoder_over_the_cache(dtype, M, D, per_batch):
    B, H, page, lens = 3, 2, 32, [700, 0, 133]
    cache = make_cache(B, 24, H, D, page)
    fill(cache, lens, seed=50)
    g = torch.Generator().manual_seed(51)
    Q = torch.randn(((B,) if per_batch else ()) + (H, M, D), generator=g).to(DT[dtype]).cuda()
    for kernel in ("simt", "auto"):
        Z, gz = guarded((B, H, M, D))
        L, gl = guarded((B, H, M))
        flare.flare_cache_encoder_fwd(Q, cache, ints(lens), Z=Z, L=L, kernel=kernel)
        flare.flare_device_status()
        rows = Q.expand(B, H, M, D).transpose(1, 2).reshape(B * M, H, D).contiguous()
        check_attn(Z.transpose(1, 2), L.transpose(1, 2), rows, cache, lens, [M] * B, False, o_f32=True)
        gz.check("Z")
        gl.check("L")


@pytest.mark.parametrize("dtype,M", [("bf16", 64), ("fp32", 16)])
def test_mixer_over_a_growing_cache(dtype, M):
    """Three pieces of a token set enter one after another; each piece's outputs are
    the decode of its tokens against the latents of everything held so far, and the
    last latents agree with the encoder over the dense tokens of the same values."""
    B, H, D, page = 2, 2, 64, 64
    cache = make_cache(B, 10, H, D, page)
    lens, g = ints([0, 70]), torch.Generator().manual_seed(52)
    fill(cache, lens.tolist(), seed=53)
    Q = (0.5 * torch.randn((H, M, D), generator=g)).to(DT[dtype]).cuda()
    for N in (100, 1, 250):
        K, V = (torch.randn((B, N, H, D), generator=g).to(DT[dtype]).cuda() for _ in range(2))
        before, was = cache_ref.host(cache), lens.tolist()
        Y, Z, L, lens = flare.flare_cache_fwd(Q, cache, K, V, lens)
        flare.flare_device_status()
        check_append(cache, before, K.flatten(0, 1), V.flatten(0, 1), None, was, [N] * B, None, False, lens, None)
        rows = Q.expand(B, H, M, D).transpose(1, 2).reshape(B * M, H, D).contiguous()
        check_attn(Z.transpose(1, 2), L.transpose(1, 2), rows, cache, lens.tolist(), [M] * B, False, o_f32=True)
        assert torch.equal(Y, flare.flare_decode_fwd(Q, Z, K))
    n = lens.tolist()
    host = cache_ref.host(cache)
    for b in range(B):
        k, v = (x[None].to(DT[dtype]).cuda() for x in cache_ref.tokens(host, b, n[b]))       # exact: 4 bits and a power of two
        _, _, Zd, Ld = flare.flare_encoder_fwd(Q, k, v)
        tol = 2e-2 if dtype == "bf16" else 1e-4                          # the dense encoder's own bound
        assert (Zd[0] - Z[b]).abs().max() <= tol and (Ld[0] - L[b]).abs().max() <= 1e-3


def test_binding_refuses_mixed_up_tensors():
    cache = make_cache(2, 2, 2, 64, 16)
    Q = torch.zeros((2, 1, 4, 64), dtype=torch.bfloat16, device="cuda")
    lens = ints([1, 1])
    with pytest.raises(ValueError):
        flare.flare_cache_attn(Q[:1], cache, lens)
    with pytest.raises(ValueError):
        flare.flare_cache_attn(Q, cache, lens.long())
    with pytest.raises(ValueError):
        flare.flare_cache_attn(Q, cache, ints([1, 1, 1]))
    with pytest.raises(TypeError):
        flare.flare_cache_attn(Q.half(), cache, lens)
    with pytest.raises(ValueError):
        flare.flare_cache_attn(Q.cpu(), cache, lens)
    with pytest.raises(ValueError):
        flare.flare_cache_attn(Q, cache, lens, O=torch.zeros_like(Q, dtype=torch.float32))
    with pytest.raises(ValueError):
        flare.flare_cache_append(cache, Q[:, :, :2], Q[:, :, :2].cpu(), lens)
    with pytest.raises(flare.FlareError):
        flare.flare_cache_append(cache, Q[:, :, :2], Q[:, :, :2], lens, seq_lens_out=lens)
    with pytest.raises(flare.FlareError):
        flare.flare_cache_attn(Q[:, :, :3], cache, lens)
