"""Host side of the decoding entry points (CPU): refusals before anything is launched,
workspace sizes, and the rotation's frequencies and fixed-point words."""

import ctypes
import math
from fractions import Fraction

import pytest

import long_context_causal_flash_b200 as gqa
from long_context_causal_flash_b200 import _lib, rotary
from long_context_causal_flash_b200.build import build
from oracle import decode

INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE = -1, -2, -3, -4
P = 1 << 20  # a pointer value that is never read


@pytest.fixture(scope="module")
def lib():
    build()
    return _lib.load()


def _rows(data=P, sb=1 << 16, sh=1 << 12, sl=256, H=4):
    return _lib.Rows(data, sb, sh, sl, H)


def _cache(dtype=1, **over):
    e4m3 = dtype == _lib.GQA_E4M3
    a = dict(k=P, v=P, k_scale=P if e4m3 else None, v_scale=P if e4m3 else None, status=P, sp=4 * 64 * 256, sh=64 * 256,
             st=256, n=10, Hkv=4, page=64, dtype=dtype)
    a.update(over)
    return _lib.Cache(a["k"], a["v"], a["k_scale"], a["v_scale"], a["status"], a["sp"], a["sh"], a["st"], a["n"],
                      a["Hkv"], a["page"], a["dtype"])


def _rope(turns=P, rot=64, layout=0):
    return _lib.Rope(turns, None, 0, 0, 1.0, rot, layout)


def _ref(x):
    return None if x is None else ctypes.byref(x)


def test_rope_refusals(lib):
    def call(x=_rows(), y=_rows(), x2=None, y2=None, B=2, L=5, d=256, dtype=1, rope=_rope()):
        return lib.gqa_attn_rope(_ref(x), _ref(y), _ref(x2), _ref(y2), B, L, d, dtype, _ref(rope), 0, None)

    assert call(x=None) == INVALID
    assert call(x=_rows(data=None)) == INVALID
    assert call(rope=None) == INVALID
    assert call(rope=_rope(turns=None)) == INVALID
    assert call(rope=_rope(rot=24)) == INVALID
    assert call(rope=_rope(rot=272)) == INVALID
    assert call(rope=_rope(rot=0)) == INVALID
    assert call(rope=_rope(layout=2)) == INVALID
    assert call(x2=_rows()) == INVALID                 # half a pair
    assert call(x2=_rows(), y2=_rows(H=5)) == INVALID
    assert call(y=_rows(H=5)) == INVALID
    assert call(B=-1) == INVALID
    assert call(L=-1) == INVALID
    assert call(dtype=2) == INVALID
    assert call(dtype=3) == INVALID
    assert call(d=128) == UNSUPPORTED
    assert call(x=_rows(data=P + 8)) == MISALIGNED
    assert call(y=_rows(sl=260)) == MISALIGNED
    assert call(x=_rows(sb=12)) == MISALIGNED
    assert call(x=_rows(sh=4), dtype=1) == MISALIGNED
    assert call(B=0) == 0 and call(L=0) == 0           # nothing to do, nothing launched


def test_cache_write_and_read_refusals(lib):
    def write(cache=_cache(), k=_rows(), v=_rows(), table=P, max_pages=3, start=P, B=2, L=5, d=256, dtype=1, rope=None):
        return lib.gqa_attn_cache_write(_ref(cache), _ref(k), _ref(v), table, max_pages, start, None, B, L, d, dtype,
                                        _ref(rope), None)

    def read(cache=_cache(), table=P, max_pages=3, lens=P, k=P, v=P, B=2, L=5, d=256, dtype=1):
        return lib.gqa_attn_cache_read(_ref(cache), table, max_pages, lens, k, v, B, L, d, dtype, None)

    for call in (write, read):
        assert call(cache=None) == INVALID
        assert call(table=None) == INVALID
        assert call(cache=_cache(k=None)) == INVALID
        assert call(cache=_cache(n=0)) == INVALID
        assert call(cache=_cache(Hkv=0)) == INVALID
        assert call(cache=_cache(dtype=2)) == INVALID
        assert call(cache=_cache(page=48)) == INVALID
        assert call(cache=_cache(page=4)) == INVALID
        assert call(cache=_cache(page=2048)) == INVALID
        assert call(cache=_cache(dtype=3, k_scale=None)) == INVALID   # codes without scales
        assert call(cache=_cache(v_scale=P)) == INVALID               # scales without codes
        assert call(cache=_cache(k=P + 4)) == MISALIGNED
        assert call(cache=_cache(st=260)) == MISALIGNED
        assert call(cache=_cache(dtype=3, st=264)) == MISALIGNED      # codes: sixteen to a unit
        assert call(max_pages=0) == INVALID
        assert call(B=-1) == INVALID
        assert call(L=-1) == INVALID
        assert call(dtype=3) == INVALID
        assert call(d=64) == UNSUPPORTED
        assert call(B=0) == 0 and call(L=0) == 0
    assert write(start=None) == INVALID
    assert write(k=_rows(H=3)) == INVALID
    assert write(v=_rows(data=P + 2)) == MISALIGNED
    assert write(rope=_rope(rot=40)) == INVALID
    assert read(lens=None) == INVALID
    assert read(k=None) == INVALID
    assert read(v=P + 8) == MISALIGNED


def test_tree_refusals_and_workspace(lib):
    def call(q=_rows(H=16), cache=_cache(), table=P, max_pages=3, ctx=P, mask=None, mask_sb=0, out=P, lse=P, B=2, T=5,
             d=256, dtype=1, ws=P, n=1 << 40):
        return lib.gqa_attn_fwd_tree(_ref(q), _ref(cache), table, max_pages, ctx, None, mask, mask_sb, out, lse, B, T, d,
                                     dtype, ws, n, None)

    assert call(q=None) == INVALID
    assert call(cache=None) == INVALID
    assert call(table=None) == INVALID
    assert call(ctx=None) == INVALID
    assert call(out=None) == INVALID
    assert call(lse=None) == INVALID
    assert call(B=0) == INVALID
    assert call(T=0) == INVALID
    assert call(mask=P, mask_sb=-1) == INVALID
    assert call(q=_rows(H=15)) == INVALID
    assert call(dtype=2) == INVALID
    assert call(cache=_cache(page=100)) == INVALID
    assert call(cache=_cache(dtype=3, v_scale=None)) == INVALID
    assert call(d=128) == UNSUPPORTED
    assert call(q=_rows(H=12)) == UNSUPPORTED
    assert call(T=1025) == UNSUPPORTED
    assert call(q=_rows(H=16, sl=100)) == MISALIGNED
    assert call(out=P + 8) == MISALIGNED
    assert call(ws=None) == WORKSPACE
    assert call(ws=P + 8) == MISALIGNED
    size = lambda T, Hq=16, B=2, pages=1000, page=64, dtype=1, kind=1: lib.gqa_attn_tree_workspace_bytes(  # noqa: E731
        B, Hq, 4, T, pages, page, 256, dtype, kind)
    assert size(1) > 0 and size(1024) > 0 and size(1025) == 0 and size(0) == 0 and size(1, Hq=12) == 0
    assert call(n=size(5, pages=3) - 1) == WORKSPACE
    # the longest cache needs no more than a bounded workspace: partial results per worker, not per key
    assert size(64, pages=1 << 20) < 200 << 20
    assert size(64, pages=1 << 20) == size(64, pages=1 << 24)


@pytest.mark.parametrize("scaling", [None, "linear", "ntk", "yarn"])
def test_frequencies(scaling):
    rot, base, s, n = 64, 10000.0, 8.0, 4096
    t = rotary.Table(rot=rot, base=base, scaling=scaling, factor=s, original_length=n)
    plain = [base ** (-2 * i / rot) for i in range(rot // 2)]
    if scaling is None:
        assert t.inv_freq == pytest.approx(plain, rel=1e-14) and t.magnitude == 1
    elif scaling == "linear":
        assert t.inv_freq == pytest.approx([f / s for f in plain], rel=1e-14) and t.magnitude == 1
    elif scaling == "ntk":
        assert t.inv_freq[0] == 1 and t.inv_freq[-1] == pytest.approx(plain[-1] / s, rel=1e-12)
        assert all(b < a for a, b in zip(plain[1:], t.inv_freq[1:])) and t.magnitude == 1
    else:
        assert t.magnitude == pytest.approx(0.1 * math.log(s) + 1)
        for f, g in zip(plain, t.inv_freq):
            turns = n * f / (2 * math.pi)
            if turns >= 32:
                assert g == pytest.approx(f, rel=1e-14)
            elif turns <= 1:
                assert g == pytest.approx(f / s, rel=1e-14)
            else:
                assert f / s < g < f


def test_words_are_exact_fractions_of_a_turn():
    own = [1.0, 0.123, 1e-6, 0.0, -0.5, 7.0, 1e-4, 2.5]
    t = rotary.Table(rot=16, inv_freq=own, magnitude=1.25)
    assert t.magnitude == 1.25
    for f, w in zip(own, t._words.tolist()):
        want = Fraction(f) / (2 * decode._PI)
        want -= math.floor(want)
        off = abs(Fraction(w % (1 << 64), 1 << 64) - want)
        assert min(off, 1 - off) <= Fraction(1, 1 << 62)
    # a far position's angle from the words: p * w modulo 2^64
    for p in (1_048_575, (1 << 31) - 1, -(1 << 31)):
        turns = (p * t._words.tolist()[1]) % (1 << 64) / 2.0 ** 64
        want = decode.angle(p, own[1]) / (2 * math.pi) % 1.0
        assert abs(turns - want) < 2.0 ** -30


def test_table_refusals():
    for kw in (dict(rot=24), dict(rot=0), dict(rot=288), dict(layout="pairs"), dict(scaling="dynamic"),
               dict(inv_freq=[1.0]), dict(magnitude=2.0)):
        with pytest.raises(ValueError):
            rotary.Table(**kw)
    for kw in (dict(base=1.0), dict(factor=0.5, scaling="linear"), dict(scaling="yarn", factor=2.0),
               dict(scaling="yarn", factor=2.0, original_length=100, beta_fast=1.0), dict(base=float("nan")),
               dict(rot=16, inv_freq=[float("inf")] * 8)):
        with pytest.raises(gqa.GqaAttnError):
            rotary.Table(**kw)


def test_host_tensors_are_refused():
    import torch

    from long_context_causal_flash_b200 import cache

    x = torch.zeros(1, 4, 3, 256)
    with pytest.raises(ValueError):
        rotary.rotate(x, None, rotary.Table())
    with pytest.raises(ValueError):
        cache.PagedCache(torch.zeros(2, 4, 16, 256), torch.zeros(2, 4, 16, 256))
    with pytest.raises(ValueError):
        cache.PagedCache(torch.zeros(2, 4, 16, 256, dtype=torch.float16), torch.zeros(2, 4, 16, 256,
                                                                                      dtype=torch.float16))


def test_workspace_of_the_largest_shapes(lib):
    """Sizes that pass 32 bits on the way: counted, or refused."""
    size = lib.gqa_attn_tree_workspace_bytes
    for code in (_lib.GQA_F32, _lib.GQA_BF16):
        assert 0 < size(1, 16, 4, 1, 0x7fffffff, 1024, 256, code, code) < 1 << 26
        assert 0 < size(1 << 20, 1 << 10, 1 << 6, 1024, 0x7fffffff, 1024, 256, code, code) < 1 << 28
        assert size(1 << 24, 1 << 8, 1 << 4, 1, 10, 64, 256, code, code) == 0
        # a page table of one page: no more workers than tiles
        assert size(1, 4, 4, 1, 1, 8, 256, code, code) <= 4 * 2 * 16 * (1024 + 4) + 256
