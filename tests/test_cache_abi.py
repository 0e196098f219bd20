"""Argument checks of the paged token cache's entry points, at the C ABI with
made-up addresses (nothing is launched before they pass) and in the binding, and
the plain 64-bit reference that the GPU tests compare with (CPU only)."""
import ctypes
import math

import pytest
import torch

import cache_ref
from latent_query_split_gb300 import build, flare

INVALID, UNSUPPORTED, WORKSPACE = flare.FLARE_ERR_INVALID_ARG, flare.FLARE_ERR_UNSUPPORTED, flare.FLARE_ERR_WORKSPACE
A = [1 << (12 + i) for i in range(24)]


@pytest.fixture(scope="module")
def lib():
    build.build()
    return flare.load_library()


def _dims(**kw):
    d = dict(B=2, H=2, Hq=4, D=64, page=64, W=8, P=16, scale=0.0, dtype=flare.FLARE_BF16, kernel=0)
    d.update(kw)
    return flare.FlareCacheDims(**d)


def _cache(**kw):
    d = dict(k=A[0], v=A[1], k_scale=A[2], v_scale=A[3], page_table=A[4])
    d.update(kw)
    return flare.FlareCachePtrs(**d)


def test_dims_struct_layout_matches_header():
    assert ctypes.sizeof(flare.FlareCacheDims) == 48 and flare.FlareCacheDims.P.offset == 24
    assert ctypes.sizeof(flare.FlareCachePtrs) == 40
    d = _dims(B=1, H=2, Hq=4, D=64, page=16, W=7, P=2 ** 33, scale=0.5, dtype=1, kernel=2)
    assert flare._PACK_DIMS(1, 2, 4, 64, 16, 7, 2 ** 33, 0.5, 1, 2) == bytes(d)
    assert flare._PACK_PTRS(*A[:5]) == bytes(_cache())


BAD_DIMS = [(dict(B=-1), INVALID), (dict(H=0), INVALID), (dict(Hq=3), INVALID), (dict(Hq=-2), INVALID),
            (dict(D=8), UNSUPPORTED), (dict(D=72), UNSUPPORTED), (dict(D=144), UNSUPPORTED),
            (dict(page=8), UNSUPPORTED), (dict(page=48), UNSUPPORTED), (dict(page=256), UNSUPPORTED),
            (dict(W=0), INVALID), (dict(W=1 << 25), INVALID), (dict(P=0), INVALID), (dict(P=1 << 31), INVALID),
            (dict(P=1 << 25), INVALID), (dict(dtype=2), INVALID), (dict(kernel=3), INVALID),
            (dict(scale=math.inf), INVALID), (dict(scale=math.nan), INVALID), (dict(B=1 << 21), UNSUPPORTED)]


def _append(lib, dims, cache=None, K=A[5], V=A[6], ks=0, vs=0, T=4, lens=A[7], cu=None, Q=A[8], qs=0, Qo=A[9],
            f=A[10], rot=64, out=A[11]):
    return lib.flare_cache_append(bytes(dims), bytes(cache or _cache()), K, V, ks, vs, T, lens, cu, Q, qs,
                                  Qo, f, rot, 0, out, None)


def _attn(lib, dims, cache=None, Q=A[8], qs=0, T=4, lens=A[7], cu=None, O=A[9], L=A[10], ws=1 << 40, wsb=1 << 40):
    return lib.flare_cache_attn(bytes(dims), bytes(cache or _cache()), Q, qs, T, lens, cu, 1, O, L, ws, wsb,
                                None)


@pytest.mark.parametrize("change,status", BAD_DIMS)
def test_bad_sizes_are_refused(lib, change, status):
    d = _dims(**change)
    assert _append(lib, d) == status and _attn(lib, d) == status
    assert lib.flare_last_error_string()
    assert lib.flare_cache_workspace_bytes(bytes(d), 4) == ctypes.c_size_t(-1).value
    assert lib.flare_cache_encoder_fwd(bytes(d), bytes(_cache()), 16, A[5], 0, A[6], A[7], A[8], A[9], 1 << 40,
                                       None) == status
    assert lib.flare_cache_fwd(bytes(d), bytes(_cache()), 16, 3, A[5], 0, A[6], A[7], A[8], A[9], A[10], A[11],
                               A[12], 1 << 40, 1 << 40, None) == status


@pytest.mark.parametrize("name", ["k", "v", "k_scale", "v_scale", "page_table"])
def test_cache_pointers_are_checked(lib, name):
    for bad in (None, A[0] + 2):
        c = _cache(**{name: bad})
        assert _append(lib, _dims(), c) == INVALID and _attn(lib, _dims(), c) == INVALID


@pytest.mark.parametrize("kw", [dict(K=None), dict(V=None), dict(T=-1), dict(T=5), dict(lens=None), dict(lens=A[7] + 2),
                                dict(Q=None), dict(Qo=None), dict(ks=127), dict(vs=-128), dict(qs=255), dict(rot=63),
                                dict(rot=0), dict(rot=66), dict(out=A[7]), dict(Qo=A[8]), dict(K=A[5] + 1), dict(f=A[10] + 1),
                                dict(T=1 << 31)])
def test_append_refuses(lib, kw):
    assert _append(lib, _dims(), **kw) == INVALID


@pytest.mark.parametrize("kw", [dict(Q=None), dict(O=None), dict(T=-2), dict(T=3), dict(lens=None), dict(qs=255), dict(L=A[10] + 2),
                                dict(Q=A[8] + 1), dict(ws=(1 << 40) + 64), dict(cu=A[12] + 1)])
def test_attn_refuses(lib, kw):
    assert _attn(lib, _dims(), **kw) == INVALID


@pytest.mark.parametrize("D,dtype", [(64, flare.FLARE_BF16), (128, flare.FLARE_BF16), (96, flare.FLARE_BF16), (128, flare.FLARE_F32)])
def test_the_workspace_is_enough_for_equal_and_ragged_rows(lib, D, dtype):
    """What the query names passes the size check of either form of the call (the
    address, which is checked next, is refused: nothing is launched)."""
    for W in (8, 1024):
        for n in (1, 5, 8, 9, 16, 17, 32, 33, 64, 65, 75, 128, 192, 193, 256, 257, 320, 448, 449, 512, 1000, 4096):
            d = _dims(D=D, dtype=dtype, W=W)
            need = lib.flare_cache_workspace_bytes(bytes(d), 2 * n)
            for cu in (None, A[12]):
                assert _attn(lib, d, T=2 * n, cu=cu, ws=(1 << 40) + 64, wsb=need) == INVALID, (W, n, cu)
                assert "256-byte" in lib.flare_last_error_string().decode()


def test_attn_needs_its_workspace_and_query_heads(lib):
    need = lib.flare_cache_workspace_bytes(bytes(_dims()), 4)
    assert need > 0
    assert _attn(lib, _dims(), cu=A[12], wsb=need - 1) == WORKSPACE and _attn(lib, _dims(), cu=A[12], ws=None) == WORKSPACE
    assert _attn(lib, _dims(), T=400, ws=None) == WORKSPACE and _attn(lib, _dims(W=8192), ws=None) == WORKSPACE
    assert _attn(lib, _dims(Hq=0)) == INVALID
    assert _append(lib, _dims(Hq=0)) == INVALID
    assert _append(lib, _dims(H=4, Hq=0), Q=A[8], Qo=A[9]) == INVALID


def test_nothing_to_do_is_fine(lib):
    assert _attn(lib, _dims(B=0), T=0) == 0 and _attn(lib, _dims(), T=0) == 0
    assert lib.flare_cache_workspace_bytes(bytes(_dims()), 0) == 0


def test_mixer_checks_every_stage_before_launching(lib):
    def call(d=None, M=16, N=3, Q=A[5], qbs=0, K=A[6], V=A[7], lens=A[8], out=A[9], Y=A[10], Z=A[11], L=A[12],
             ws=1 << 40, wsb=1 << 40):
        return lib.flare_cache_fwd(bytes(d or _dims()), bytes(_cache()), M, N, Q, qbs, K, V, lens, out, Y, Z, L,
                                   ws, wsb, None)
    for kw in (dict(M=0), dict(N=-1), dict(Q=None), dict(qbs=5), dict(K=None), dict(V=None), dict(lens=None), dict(out=None),
               dict(out=A[8]), dict(Y=None), dict(Z=None), dict(L=None), dict(ws=1 + (1 << 40))):
        assert call(**kw) == INVALID, kw
    assert call(wsb=0, M=128) == WORKSPACE
    assert call(M=300) == UNSUPPORTED              # the decode's latents


def test_binding_refuses_what_it_cannot_pass_on():
    table = torch.zeros((2, 4), dtype=torch.int32)
    cache = flare.flare_cache_alloc(8, 2, 64, 16, page_table=table, device="cpu")
    assert cache.k.shape == (8, 2, 16, 64) and cache.v_scale.shape == (8, 2)
    with pytest.raises(ValueError):
        flare._cache_args(cache)                                                   # not on a device
    with pytest.raises(TypeError):
        flare._cache_args(cache._replace(k=cache.k.float()))
    with pytest.raises(TypeError):
        flare._cache_args(cache._replace(page_table=table.long()))
    with pytest.raises(ValueError):
        flare._cache_args(cache._replace(v=cache.v[:4]))
    x = torch.zeros((2, 3, 2, 64), dtype=torch.bfloat16)
    rows = lambda x, cu=None, heads=2: flare._rows(x, "K", heads, 64, 2, cu, torch.bfloat16, x.device)  # noqa: E731
    assert rows(x)[1:] == (0, 6)
    wide = torch.zeros((2, 3, 6, 64), dtype=torch.bfloat16)
    assert rows(wide[:, :, 2:4])[1:] == (384, 6)                                   # a slice of a fused projection
    assert rows(wide[:, :1, 2:4])[1:] == (3 * 384, 2)
    for bad in (x.float(), x.transpose(0, 1), x[..., ::2], x[:, :, :1].expand(2, 3, 2, 64), x[:, :1].expand(2, 3, 2, 64),
                wide[:, :2, 2:4], x.transpose(2, 3).contiguous().transpose(2, 3), x[0]):
        with pytest.raises((ValueError, TypeError)):
            rows(bad)
    with pytest.raises(ValueError):
        rows(x, cu=torch.zeros(3, dtype=torch.int32))


def test_reference_quantisation_rule():
    """The scale leaves room for the rotation: a magnitude in (128, 256] of the scale."""
    for a in (1e-3, 0.5, 1.0, 1.0000001, 3.9, 256.0, 447.0, 1e6):
        u = a * 2.0 ** -cache_ref.exponent(a)
        assert 128 < u <= 256 and u * math.sqrt(2) < 448
    assert cache_ref.exponent(0.0) == -40 and cache_ref.exponent(1e30) == 60 and cache_ref.exponent(1e-30) == -40


def test_reference_attention_against_a_written_out_softmax():
    torch.manual_seed(0)
    table = torch.tensor([[2, 0], [1, 3]], dtype=torch.int32)
    cache = {"k": torch.randn(4, 2, 16, 16).double(), "v": torch.randn(4, 2, 16, 16).double(),
             "k_scale": torch.full((4, 2), 0.5).double(), "v_scale": torch.full((4, 2), 2.0).double(), "page_table": table}
    Q = torch.randn(5, 4, 16)
    O, L, _, _ = cache_ref.attn(cache, Q, [20, 1], [3, 2], True)
    assert (O[3] == 0).all() and (L[3] == -math.inf).all()                         # sequence 1: its first row sees nothing
    for i in range(3):
        for hq in range(4):
            w, acc = 0.0, torch.zeros(16).double()
            for n in range(20 - 3 + i + 1):
                p, slot = int(table[0, n // 16]), n % 16
                e = math.exp(float(Q[i, hq].double() @ cache["k"][p, hq // 2, slot]) * 0.5 / 4)
                w, acc = w + e, acc + e * 2.0 * cache["v"][p, hq // 2, slot]
            assert abs(float(L[i, hq]) - math.log(w)) < 1e-12
            assert (O[i, hq] - acc / w).abs().max() < 1e-12
