"""The paged cache on the GPU: rows written (rotated, quantised) and read back, against the
float64 definitions.  Unrotated rows are compared exactly: bf16 and fp32 pages hold the
input rounded once, e4m3 pages a division by a power of two (exact) and one rounding to
nearest even.  A rotated key is off by 8 e (|x1| + |x2|) m before its rounding (see
test_rotary), e = 2^-24, and by half a step of the page's type after it: 2^-8 of the value
(bf16), 2^-4 or, below the least normal number, 2^-10 scales (e4m3)."""

import numpy as np
import pytest
import torch

import long_context_causal_flash_b200 as gqa
from long_context_causal_flash_b200 import cache, rotary
from oracle import decode

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn
E = 2.0 ** -24


def _x(shape, dtype, seed, spread=True):
    x = torch.randn(shape, generator=torch.Generator().manual_seed(seed))
    if spread:  # rows of very different sizes
        x = x * torch.logspace(-4, 4, shape[2])[None, None, :, None]
    return x.to(dtype)


def _pool(n, Hkv, page, dtype, dev):
    pool = cache.PagedCache.empty(n, Hkv, page, dtype, dev)
    pool.k.view(torch.uint8).fill_(0xff)  # NaN in every type that pages have
    pool.v.view(torch.uint8).fill_(0xff)
    return pool


def _table(B, per, n, seed, dev):
    ids = torch.randperm(n, generator=torch.Generator().manual_seed(seed))[: B * per]
    return ids.view(B, per).to(torch.int32).to(dev)




def _stored(pool, table, b, places):
    j = torch.as_tensor(places)
    page, slot = table[b].cpu().long()[j // pool.page_size], j % pool.page_size
    out = []
    for t, s in ((pool.k, pool.k_scale), (pool.v, pool.v_scale)):
        raw = t.view(torch.uint8).cpu().view(*t.shape[:3], -1)[page, :, slot].contiguous().view(t.dtype)
        scale = None if s is None else s.cpu()[page, :, slot]
        out.append((raw.double().transpose(0, 1).numpy(), None if scale is None else scale.double().T.numpy()))
    return out


@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16, E4M3], ids=["f32", "bf16", "e4m3"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["from_f32", "from_bf16"])
@pytest.mark.parametrize("B,L,Hkv,page", [(1, 1, 1, 8), (3, 29, 5, 16), (2, 70, 4, 64)])
def test_write_and_read(cuda_device, kind, dtype, B, L, Hkv, page):
    per = 4 + -(-L // page)
    n = B * per + 2
    pool, table = _pool(n, Hkv, page, kind, cuda_device), _table(B, per, n, 1, cuda_device)
    k, v = _x((B, Hkv, L, 256), dtype, 2), _x((B, Hkv, L, 256), dtype, 3)
    if L > 1:
        k[0, 0, 1] = 0.0
    start = torch.tensor([(7 * b + 5) % (3 * page) for b in range(B)], dtype=torch.int32)
    before = pool.k.view(torch.uint8).clone()
    cache.write(pool, k.to(cuda_device), v.to(cuda_device), table, start.to(cuda_device))
    touched = torch.zeros((n, page), dtype=torch.bool)
    for b in range(B):
        places = int(start[b]) + np.arange(L)
        for (got, scale), x in zip(_stored(pool, table, b, places), (k[b], v[b])):
            if kind == E4M3:
                want, s = decode.quantise(x)
                assert np.array_equal(scale, s) and np.array_equal(got, want)
            else:
                assert np.array_equal(got, x.to(kind).double().numpy())
        j = torch.as_tensor(places)
        touched[table[b].cpu().long()[j // page], j % page] = True
    same = (pool.k.view(torch.uint8).view(n, Hkv, page, -1) == before.view(n, Hkv, page, -1)).all(-1).cpu()
    assert same[~touched[:, None].expand(n, Hkv, page)].all()  # slots of no token are as they were
    assert cache.status(pool) == 0
    # reading back: the first lens[b] places; those before start hold NaN
    lens = start + L
    lens[0] = 0 if B > 1 else lens[0]
    top = int(lens.max()) + 3
    for out_dtype in (torch.float32, torch.bfloat16):
        kd, vd = cache.read(pool, table, lens.to(cuda_device), top, dtype=out_dtype)
        for b in range(B):
            m = int(lens[b])
            (kw, ks), (vw, vs) = _stored(pool, table, b, np.arange(m)) if m else ((None, None), (None, None))
            for got, w, s in ((kd, kw, ks), (vd, vw, vs)):
                assert not got[b, :, m:].any()
                if m:
                    value = torch.as_tensor(w if s is None else w * s[..., None]).to(out_dtype)
                    assert torch.equal(got[b, :, :m].cpu().nan_to_num(-7.0), value.nan_to_num(-7.0))


@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16, E4M3], ids=["f32", "bf16", "e4m3"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("given", [False, True])
def test_write_rotates_the_keys(cuda_device, kind, layout, given):
    B, L, Hkv, page, rot = 2, 19, 3, 16, 96
    t = rotary.Table(rot, layout=layout, scaling="yarn", factor=4.0, original_length=512)
    pool, table = _pool(20, Hkv, page, kind, cuda_device), _table(B, 6, 20, 4, cuda_device)
    k, v = _x((B, Hkv, L, 256), torch.bfloat16, 5, False), _x((B, Hkv, L, 256), torch.bfloat16, 6, False)
    start = torch.tensor([3, 40], dtype=torch.int32)
    pos = torch.tensor([[900_000 + i // 2 for i in range(L)], [5 * i for i in range(L)]], dtype=torch.int32)
    kw = dict(positions=pos.to(cuda_device)) if given else dict(pos_offset=1000)
    cache.write(pool, k.to(cuda_device), v.to(cuda_device), table, start.to(cuda_device), rope=t, **kw)
    p = pos.numpy() if given else start.numpy()[:, None] + np.arange(L) + 1000
    want = decode.rotate(k, p, t.inv_freq, t.magnitude, layout)
    size = k.double().abs().numpy()
    lo, hi = (slice(0, rot // 2), slice(rot // 2, rot)) if layout == "half" else (slice(0, rot, 2), slice(1, rot, 2))
    before = np.zeros_like(size)
    before[..., lo] = before[..., hi] = 8 * E * t.magnitude * (size[..., lo] + size[..., hi])
    for b in range(B):
        (kg, ks), (vg, vs) = _stored(pool, table, b, int(start[b]) + np.arange(L))
        if kind == E4M3:
            tol = before[b] + np.maximum((np.abs(want[b]) + before[b]) * 2.0 ** -4, 2.0 ** -10 * ks[..., None])
            kg = kg * ks[..., None]
            vw, vsw = decode.quantise(v[b])
            assert np.array_equal(vg, vw) and np.array_equal(vs, vsw)
        else:
            step = 2.0 ** -8 if kind == torch.bfloat16 else E
            tol = before[b] + np.abs(want[b]) * step
            assert np.array_equal(vg, v[b].to(kind).double().numpy())
        assert np.all(np.abs(kg - want[b]) <= tol)


def test_special_values(cuda_device):
    """Infinities saturate, NaN stays, neither sets the scale; tiny and huge rows keep theirs in range."""
    pool, table = _pool(2, 1, 8, E4M3, cuda_device), torch.tensor([[1]], dtype=torch.int32, device=cuda_device)
    x = torch.zeros(1, 1, 6, 256)
    x[0, 0, 0, :4] = torch.tensor([float("inf"), -float("inf"), float("nan"), 3.0])
    x[0, 0, 1, :2] = torch.tensor([1e-38, 3e-39])
    x[0, 0, 2, :2] = torch.tensor([3.4e38, -1e38])
    x[0, 0, 3, :3] = torch.tensor([448.0, 1.0, 2.0 ** -9])
    x[0, 0, 4, :3] = torch.tensor([-448.5, 1.0, 2.0 ** -9])
    zero = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    cache.write(pool, x.to(cuda_device), x.to(cuda_device), table, zero)
    for got, scale in _stored(pool, table, 0, np.arange(6)):
        want, s = decode.quantise(x[0])
        assert np.array_equal(scale, s)
        assert np.array_equal(np.isnan(got), np.isnan(want))
        assert np.array_equal(np.nan_to_num(got), np.nan_to_num(want))


def test_ragged_lengths_and_strides(cuda_device):
    B, L, Hkv, page = 4, 10, 2, 8
    pool, table = _pool(40, Hkv, page, torch.bfloat16, cuda_device), _table(B, 5, 40, 7, cuda_device)
    x = _x((B, Hkv, L, 256), torch.bfloat16, 8, False)
    lens = torch.tensor([10, 0, -3, 99], dtype=torch.int32, device=cuda_device)
    start = torch.tensor([0, 4, 4, 9], dtype=torch.int32, device=cuda_device)
    tokens = torch.stack((x, -x), 3).transpose(1, 2).contiguous().to(cuda_device)  # [B, L, Hkv, 2, 256]
    cache.write(pool, tokens[:, :, :, 0].transpose(1, 2), tokens[:, :, :, 1].transpose(1, 2), table, start, lens=lens)
    written = (pool.v.float().isfinite()).all(-1).sum().item()
    assert written == Hkv * (10 + 0 + 0 + 10)
    for b in (0, 3):
        (k, _), (v, _) = _stored(pool, table, b, int(start[b]) + np.arange(L))
        assert np.array_equal(k, x[b].double().numpy()) and np.array_equal(v, -x[b].double().numpy())
    # pages whose tokens lie outside their heads
    base = torch.zeros((40, page, Hkv, 2, 256), dtype=torch.bfloat16, device=cuda_device)
    other = cache.PagedCache(base[:, :, :, 0].transpose(1, 2), base[:, :, :, 1].transpose(1, 2))
    cache.write(other, tokens[:, :, :, 0].transpose(1, 2), tokens[:, :, :, 1].transpose(1, 2), table, start, lens=lens)
    for b in (0, 3):
        (k, _), (v, _) = _stored(other, table, b, int(start[b]) + np.arange(L))
        assert np.array_equal(k, x[b].double().numpy()) and np.array_equal(v, -x[b].double().numpy())


def test_bad_pages_and_lengths_are_skipped_and_recorded(cuda_device):
    Hkv, page = 2, 8
    x = _x((3, Hkv, 6, 256), torch.bfloat16, 9, False).to(cuda_device)

    def write(table, start):
        pool = _pool(4, Hkv, page, torch.bfloat16, cuda_device)
        cache.write(pool, x, x, torch.tensor(table, dtype=torch.int32, device=cuda_device),
                    torch.tensor(start, dtype=torch.int32, device=cuda_device))
        return pool, int(pool.k.float().isfinite().all(-1).sum()) // Hkv, cache.status(pool)

    assert write([[0, 1], [2, 9], [3, -1]], [0, 0, 2])[1:] == (18, 0)      # entries not reached are not read
    assert write([[0, 1], [2, 9], [3, -1]], [0, 4, 4])[1:] == (14, -7)     # two tokens each into bad pages
    assert write([[0, 1], [2, 3], [1, 0]], [0, 14, -2])[1:] == (12, -7)    # past the table, before the start
    pool, _, _ = write([[0, 1], [2, 3], [1, 0]], [0, 0, 0])
    table = torch.tensor([[0, 1], [-5, 3], [2, 4]], dtype=torch.int32, device=cuda_device)
    lens = torch.tensor([6, 12, 40], dtype=torch.int32, device=cuda_device)
    k, _ = cache.read(pool, table, lens, 17)
    assert cache.status(pool) == gqa._lib.GQA_ERR_DEVICE_BOUNDS
    assert torch.equal(k[0, :, :6], x[0]) and not k[0, :, 6:].any()
    assert not k[1, :, :8].any() and not k[2, :, 8:].any()
    # without a status word nothing is recorded, and nothing else changes
    bare = cache.PagedCache(pool.k, pool.v)
    again, _ = cache.read(bare, table, lens, 17)
    assert torch.equal(again.nan_to_num(-7.0), k.nan_to_num(-7.0))
    with pytest.raises(ValueError):
        cache.status(bare)


def test_offsets_past_32_bits(cuda_device):
    Hkv, page = 4, 64
    n = (1 << 31) // (Hkv * page * 256) + 5
    pool = cache.PagedCache.empty(n, Hkv, page, E4M3, cuda_device)
    table = torch.tensor([[0, n - 1], [n - 2, n - 3]], dtype=torch.int32, device=cuda_device)
    x = _x((2, Hkv, 100, 256), torch.bfloat16, 10, False)
    zero = torch.zeros(2, dtype=torch.int32, device=cuda_device)
    cache.write(pool, x.to(cuda_device), (-x).to(cuda_device), table, zero)
    k, v = cache.read(pool, table, zero + 100, 100, dtype=torch.float32)
    want, s = decode.quantise(x)
    assert np.array_equal(k.double().cpu().numpy(), want * s[..., None]) and torch.equal(v, -k)
    q = _x((2, 16, 1, 256), torch.bfloat16, 11, False)
    out, lse = cache.attend(q.to(cuda_device), pool, table, zero + 99)
    for b in range(2):
        value = want[b] * s[b][..., None]
        o, l, _ = decode.tree_attention(q[b], value, -value, 99, 1)
        assert np.abs(lse[b].double().cpu().numpy() - l).max() <= 2e-4
        assert np.abs(out[b].double().cpu().numpy() - o).max() <= 2e-2


def test_streams_and_graphs(cuda_device):
    """A captured step follows its lengths, table and inputs as they change in place."""
    B, Hkv, page = 3, 2, 16
    t = rotary.Table(64, device=cuda_device)
    pool, table = _pool(30, Hkv, page, E4M3, cuda_device), _table(B, 8, 30, 12, cuda_device)
    k = _x((B, Hkv, 1, 256), torch.bfloat16, 13, False).to(cuda_device)
    start = torch.zeros(B, dtype=torch.int32, device=cuda_device)
    g = torch.cuda.CUDAGraph()
    cache.write(pool, k, k, table, start, rope=t)
    with torch.cuda.graph(g):
        cache.write(pool, k, k, table, start, rope=t)
    ref = _pool(30, Hkv, page, E4M3, cuda_device)
    side = torch.cuda.Stream()
    for step in range(20):
        k.copy_(_x(k.shape, torch.bfloat16, 20 + step, False))
        start.fill_(step)
        g.replay()
        side.wait_stream(torch.cuda.current_stream())
        cache.write(ref, k, k, table, start, rope=t, stream=side)
        torch.cuda.current_stream().wait_stream(side)
    lens = start + 1
    for a, b in zip(cache.read(pool, table, lens, 20), cache.read(ref, table, lens, 20)):
        assert torch.equal(a, b) and a.isfinite().all()


def test_nothing_to_write_or_read(cuda_device):
    pool = cache.PagedCache.empty(2, 2, 8, torch.bfloat16, cuda_device)
    empty = torch.zeros((0, 1), dtype=torch.int32, device=cuda_device)
    one = torch.zeros((1, 1), dtype=torch.int32, device=cuda_device)
    x = torch.zeros((1, 2, 0, 256), device=cuda_device)
    cache.write(pool, x, x, one, one[0])
    x = torch.zeros((0, 2, 3, 256), device=cuda_device)
    cache.write(pool, x, x, empty, empty[:, 0])
    assert cache.read(pool, one, one[0], 0)[0].shape == (1, 2, 0, 256)
    assert cache.read(pool, empty, empty[:, 0].contiguous(), 4)[0].shape == (0, 2, 4, 256)


def test_refusals(cuda_device):
    dev = cuda_device
    k = torch.zeros(4, 2, 16, 256, dtype=E4M3, device=dev)
    s = torch.ones(4, 2, 16, device=dev)
    for a in ((k, k), (k, k, s), (k, k, s, s[:, :, :8]), (k, k, s, s.double()), (k.float(), k.float(), s, s),
              (k.half(), k.half()), (k.float(), k.bfloat16()), (k[:, :, :12].float(), k[:, :, :12].float()),
              (k[..., :128].float(), k[..., :128].float()), (k.float()[:1].expand(4, 2, 16, 256),) * 2,
              (k.float().cpu(), k.float().cpu()), (k.float(), k.float().transpose(0, 1).contiguous().transpose(0, 1)),
              (k, k, s, s, torch.zeros(1, device=dev))):
        with pytest.raises(ValueError):
            cache.PagedCache(*a)
    pool = cache.PagedCache(k, k.clone(), s, s.clone())
    x = torch.zeros(2, 2, 3, 256, device=dev)
    table = torch.zeros(2, 3, dtype=torch.int32, device=dev)
    start = torch.zeros(2, dtype=torch.int32, device=dev)
    good = dict(k=x, v=x, page_table=table, start=start)
    for kw in (dict(k=x[:, :1], v=x[:, :1]), dict(v=x[:, :, :2]), dict(v=x.bfloat16()), dict(page_table=table[:1]),
               dict(page_table=table.long()), dict(page_table=table.cpu()), dict(page_table=table[:, :2]),
               dict(start=start[:1]), dict(start=start.long()), dict(lens=start.cpu()), dict(lens=table),
               dict(positions=table), dict(pos_offset=4), dict(k=x.half(), v=x.half()),
               dict(rope=rotary.Table(64), positions=table, pos_offset=1), dict(rope=rotary.Table(64), positions=start)):
        with pytest.raises(ValueError):
            cache.write(pool, **{**good, **kw})
    for kw in (dict(lens=start[:1]), dict(max_len=-1), dict(dtype=E4M3), dict(out=(x, x)), dict(page_table=start)):
        with pytest.raises(ValueError):
            cache.read(pool, **{**dict(page_table=table, lens=start, max_len=4), **kw})


@pytest.mark.parametrize("kind", [torch.bfloat16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("given", [False, True])
def test_write_of_ragged_lengths_rotates_what_it_writes(cuda_device, kind, given):
    """lens and rope together, from a projection's view: the first lens[b] tokens turned to their
    places (or to the positions given), every other slot as it was."""
    B, L, Hkv, page = 3, 11, 2, 16
    t = rotary.Table(64, layout="interleaved", device=cuda_device)
    pool, table = _pool(20, Hkv, page, kind, cuda_device), _table(B, 4, 20, 40, cuda_device)
    tokens = _x((B, L, 2 * Hkv, 256), torch.bfloat16, 41, False).to(cuda_device)
    k, v = tokens[:, :, :Hkv].transpose(1, 2), tokens[:, :, Hkv:].transpose(1, 2)
    lens, start = torch.tensor([11, 0, 4], dtype=torch.int32), torch.tensor([5, 9, 40], dtype=torch.int32)
    pos = torch.arange(3 * L, dtype=torch.int32).view(B, L) * 7
    kw = dict(positions=pos.to(cuda_device)) if given else dict(pos_offset=100)
    cache.write(pool, k, v, table, start.to(cuda_device), lens=lens.to(cuda_device), rope=t, **kw)
    whole = _pool(20, Hkv, page, kind, cuda_device)
    places = start.to(cuda_device)[:, None] + 100 + torch.arange(L, dtype=torch.int32, device=cuda_device)
    # the same rows as one call for each sequence writes, which the tests above hold against the definition
    for b in range(B):
        n = int(lens[b])
        at = pos[b:b + 1, :n].to(cuda_device) if given else places[b:b + 1, :n]
        cache.write(whole, k[b:b + 1, :, :n], v[b:b + 1, :, :n], table[b:b + 1], start[b:b + 1].to(cuda_device), rope=t,
                    positions=at.contiguous())
    for a, w in ((pool.k, whole.k), (pool.v, whole.v)):
        assert torch.equal(a.view(torch.uint8), w.view(torch.uint8))
    if kind == E4M3:
        assert torch.equal(pool.k_scale, whole.k_scale) and torch.equal(pool.v_scale, whole.v_scale)
    assert cache.status(pool) == 0
