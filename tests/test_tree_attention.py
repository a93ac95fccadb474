"""Attention of drafted tokens over the paged cache on the GPU against the float64 definition.

Tolerances.  fp32 queries: the repository's bars for unit-variance inputs (out 2e-5, LSE
1e-5), scaled by the size of the values where those are larger.  bf16 queries: products
of bf16 (and e4m3) numbers are exact in fp32, so scores are off by the fp32 sums only, or, where a query is taken
apart into two e4m3 pieces, by 2^-10 steps of a row scaled to 448: 2^-18.8 of its
largest element times sum |k| / 16, below 2e-4 for these inputs, which bounds the LSE.
Each probability is rounded to at least 8 bits, off by at most 2^-8 of itself, and so is the output: out is
off by at most 2^-8 (|out| + sum p |v| / sum p) plus the scores' share, 2 x 2e-4 of
that sum.
Over e4m3 values, that holds for probabilities down to 2^-6 of the largest p s (s: the
value's scale).  16 p s / m is stored, m at most that largest, in two e4m3 pieces whose
smallest step is 2^-9: a smaller p is off by at most 2^-10 / 16 = 2^-14 of max(p s) / s, and
out by 2^-14 max(p) / sum p x (sum of the |v| a row sees) x (largest s / smallest s), which is
2 for rows of 256 normal numbers, whose largest lies in (1.75, 7].  Where a row sees few keys
of very different weights (``small``) this is added.  (Such were two e4m3 pieces.  Three e5m2 ones
are off by 2^-8.8 of a probability down to 2^-20 of the largest, and by 2^-28 of that below: the later
tests here take no such allowance.)
"""

import functools

import numpy as np
import pytest
import torch

import long_context_causal_flash_b200 as gqa
from long_context_causal_flash_b200 import cache, rotary
from oracle import decode

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn
F32, BF16 = torch.float32, torch.bfloat16
PAIRS = [(F32, F32), (BF16, BF16), (BF16, E4M3), (F32, BF16), (F32, E4M3), (BF16, F32)]
IDS = ["f32", "bf16", "bf16_e4m3", "f32_bf16", "f32_e4m3", "bf16_f32"]


def _tree(T, seed):
    rng = np.random.default_rng(seed)
    mask = np.eye(T, dtype=bool)
    for t in range(1, T):
        mask[t] |= mask[rng.integers(0, t)]
    return mask


class Problem:
    """Filled pages (garbage, NaN by default, in every slot that no sequence holds) and what they stand for."""

    def __init__(self, dev, B, Hq, Hkv, T, ctx, page, dtype, kind, seed=0, drafted=None, garbage=0xff, gain=1.0):
        g = torch.Generator().manual_seed(seed)
        self.ctx = list(ctx)
        self.drafted = list(drafted) if drafted is not None else [T] * B
        per = max(1, -(-(max(self.ctx) + T) // page))
        n = B * per + 2
        self.pool = cache.PagedCache.empty(n, Hkv, page, kind, dev)
        for t in (self.pool.k, self.pool.v):
            t.view(torch.uint8).fill_(garbage)
        if kind == E4M3:
            for t in (self.pool.k_scale, self.pool.v_scale):
                t.fill_(float("nan"))
        self.table = torch.randperm(n, generator=g)[: B * per].view(B, per).to(torch.int32)
        L = max(c + d for c, d in zip(self.ctx, self.drafted))
        self.k, self.v = (torch.randn((B, Hkv, max(L, 1), 256), generator=g).to(BF16) * gain for _ in range(2))
        lens = torch.tensor([c + d for c, d in zip(self.ctx, self.drafted)], dtype=torch.int32)
        self.table = self.table.to(dev)
        cache.write(self.pool, self.k.to(dev), self.v.to(dev), self.table,
                    torch.zeros(B, dtype=torch.int32, device=dev), lens=lens.to(dev))
        if kind == E4M3:
            self.k, self.v = (torch.as_tensor(y * s[..., None]) for y, s in map(decode.quantise, (self.k, self.v)))
        self.q = torch.randn((B, Hq, T, 256), generator=g).to(dtype)
        self.dev, self.ctx_dev = dev, torch.tensor(self.ctx, dtype=torch.int32, device=dev)
        self.drafted_dev = torch.tensor(self.drafted, dtype=torch.int32, device=dev) if drafted is not None else None

    def attend(self, mask=None, **kw):
        if mask is not None:
            mask = torch.as_tensor(mask).to(self.dev)
        return cache.attend(self.q.to(self.dev), self.pool, self.table, self.ctx_dev, tree_mask=mask,
                            tree_lens=self.drafted_dev, **kw)

    def small(self, b, mask):
        """What e4m3 probabilities below 2^-6 of the largest lose: see the tolerances above."""
        n, T, G = self.ctx[b] + self.drafted[b], self.q.shape[2], self.q.shape[1] // self.k.shape[1]
        sees = np.zeros((T, n), dtype=bool)
        d = self.drafted[b]
        sees[:d, : self.ctx[b]] = True
        sees[:d, self.ctx[b]:] = np.tril(np.ones((d, d), dtype=bool)) if mask is None else np.asarray(mask)[:d, :d]
        k, v = (x[b, :, :n].double().numpy().repeat(G, 0) for x in (self.k, self.v))
        x = np.where(sees, self.q[b].double().numpy() @ k.transpose(0, 2, 1) / 16.0, -np.inf)
        w = np.exp(x - np.max(x, -1, keepdims=True, initial=-1e300))
        return 2.0 ** -13 / np.maximum(w.sum(-1, keepdims=True), 1.0) * (sees @ np.abs(v))

    def check(self, out, lse, mask=None, rows=None, small=False):
        exact = self.q.dtype == F32
        out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
        for b in range(len(self.ctx)) if rows is None else rows:
            m = None if mask is None else np.asarray(mask)[b] if np.ndim(mask) == 3 else np.asarray(mask)
            o, l, spread = decode.tree_attention(self.q[b], self.k[b], self.v[b], self.ctx[b], self.drafted[b], m)
            empty = np.isneginf(l)
            assert np.array_equal(np.isneginf(lse[b]), empty), "rows without a visible key"
            assert not out[b][empty].any()
            fin = ~empty
            if not fin.any():
                continue
            if exact:
                tol_o, tol_l = 2e-5 * max(1.0, float(np.abs(o).max())), 1e-5
            else:
                tol_o, tol_l = 2.0 ** -8 * (np.abs(o) + spread) + 4e-4 * spread, 2e-4
            if small:
                tol_o = tol_o + self.small(b, m)
            d_l = np.abs(lse[b][fin] - l[fin]).max()
            d_o = np.abs(out[b] - o)
            assert d_l <= tol_l, f"sequence {b}: LSE off by {d_l:.2e}"
            assert np.all(d_o <= tol_o), f"sequence {b}: out off by {(d_o - tol_o).max():.2e} more than allowed"


@pytest.mark.parametrize("dtype,kind", PAIRS, ids=IDS)
@pytest.mark.parametrize("ctx", [0, 1, 127, 128, 700])
def test_one_token(cuda_device, dtype, kind, ctx):
    p = Problem(cuda_device, 1, 16, 4, 1, [ctx], 16, dtype, kind, seed=ctx)
    p.check(*p.attend())
    assert cache.status(p.pool) == 0


@pytest.mark.parametrize("dtype,kind", PAIRS, ids=IDS)
@pytest.mark.parametrize("T,page", [(3, 8), (13, 64), (70, 128)])
def test_trees(cuda_device, dtype, kind, T, page):
    ctx = [130, 0, 259]
    p = Problem(cuda_device, 3, 8, 2, T, ctx, page, dtype, kind, seed=T)
    p.check(*p.attend())
    masks = np.stack([_tree(T, b) for b in range(3)])
    p.check(*p.attend(masks), mask=masks)
    p.check(*p.attend(masks[0]), mask=masks[0])
    p.check(*p.attend(masks.astype(np.uint8) * 3), mask=masks)


@pytest.mark.parametrize("dtype,kind", PAIRS[:3], ids=IDS[:3])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (5, 5), (6, 3), (8, 1), (16, 1), (32, 4)])
def test_head_layouts(cuda_device, dtype, kind, Hq, Hkv):
    p = Problem(cuda_device, 2, Hq, Hkv, 5, [37, 301], 32, dtype, kind, seed=Hq)
    masks = _tree(5, 3)
    p.check(*p.attend(masks), mask=masks)


@pytest.mark.parametrize("dtype,kind", PAIRS[:3], ids=IDS[:3])
def test_empty_and_padded_rows(cuda_device, dtype, kind):
    T = 6
    p = Problem(cuda_device, 5, 16, 4, T, [0, 50, 0, 300, 0], 16, dtype, kind, seed=5, drafted=[6, 2, 0, 0, 3])
    p.check(*p.attend())
    mask = _tree(T, 1)
    mask[2] = mask[5] = False  # rows that name nobody: empty where there is no context
    p.check(*p.attend(mask), mask=mask)
    mask[:] = False
    p.check(*p.attend(mask), mask=mask)
    # outputs are written whole: what was in them does not stay
    out = torch.full(p.q.shape, float("nan"), dtype=dtype, device=cuda_device)
    lse = torch.full(p.q.shape[:3], float("nan"), device=cuda_device)
    got = p.attend(mask, out=out, lse=lse)
    assert got[0] is out and got[1] is lse
    p.check(out, lse, mask=mask)
    # nothing at all
    p = Problem(cuda_device, 3, 4, 4, 2, [0, 0, 0], 16, dtype, kind, drafted=[0, 0, 0])
    p.check(*p.attend())


@pytest.mark.parametrize("dtype,kind", [(F32, F32), (BF16, BF16), (F32, BF16)], ids=["f32", "bf16", "f32_bf16"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), 3.3e38], ids=["nan", "inf", "-inf", "max"])
@pytest.mark.parametrize("T,ctx", [(5, 20), (33, 200)])
def test_hidden_values_do_not_reach_a_row(cuda_device, dtype, kind, bad, T, ctx):
    """One drafted token's value (then its key) is bad: rows that do not see it are as if it
    were good, the others show it in that column (or in all)."""
    p = Problem(cuda_device, 2, 4, 2, T, [ctx, ctx + 3], 16, dtype, kind, seed=8)
    mask = _tree(T, 2)
    u = 3
    sees = mask[:, u]
    assert sees.any() and not sees.all()
    good, good_lse = p.attend(mask)
    where = [(int(p.table[b, (c + u) // 16]), (c + u) % 16) for b, c in enumerate(p.ctx)]
    for pages, column in ((p.pool.v, 77), (p.pool.k, 5)):
        kept = pages.clone()
        for page, slot in where:
            pages[page, :, slot, column] = bad
        out, lse = p.attend(mask)
        pages.copy_(kept)
        hidden = torch.as_tensor(~sees)
        assert torch.equal(out[:, :, hidden], good[:, :, hidden])
        assert torch.equal(lse[:, :, hidden], good_lse[:, :, hidden])
        if abs(bad) > 3e38 and bad == bad and not np.isinf(bad):
            continue
        if pages is p.pool.v:
            seen = out[:, :, ~hidden].float()
            assert not seen[..., column].isfinite().any()
            assert torch.equal(out[:, :, ~hidden][..., :column], good[:, :, ~hidden][..., :column])
            assert torch.equal(lse, good_lse)


@pytest.mark.parametrize("dtype,kind", PAIRS[:3], ids=IDS[:3])
def test_long_context_of_one_sequence_among_short_ones(cuda_device, dtype, kind):
    """The work list is cut across sequences and heads: boundaries fall anywhere."""
    ctx = [5, 9000, 1, 0, 640, 129, 4000]
    p = Problem(cuda_device, 7, 8, 2, 2, ctx, 64, dtype, kind, seed=21)
    p.check(*p.attend(), rows=range(7))


@pytest.mark.parametrize("dtype,kind", PAIRS[:3], ids=IDS[:3])
@pytest.mark.parametrize("T,page", [(1, 128), (12, 32), (20, 64)])
def test_long_runs_of_tiles(cuda_device, dtype, kind, T, page):
    """Eight tiles or more to a worker: every ring of slots goes round several times.  Calls in
    a row, with nothing between them, give the same bits."""
    p = Problem(cuda_device, 1, 16, 4, T, [38_000], page, dtype, kind, seed=40 + T)
    got = [p.attend() for _ in range(12)]
    p.check(*got[0])
    for out, lse in got[1:]:
        assert torch.equal(out, got[0][0]) and torch.equal(lse, got[0][1])


@pytest.mark.parametrize("dtype,kind", PAIRS[:3], ids=IDS[:3])
def test_many_sequences(cuda_device, dtype, kind):
    rng = np.random.default_rng(4)
    ctx = [int(c) for c in rng.integers(0, 200, 150)]
    p = Problem(cuda_device, 150, 4, 4, 1, ctx, 16, dtype, kind, seed=22)
    p.check(*p.attend())


@pytest.mark.parametrize("dtype,kind", PAIRS[:3], ids=IDS[:3])
def test_most_tokens(cuda_device, dtype, kind):
    """T = 1024 of 16 heads to a key/value head, the most rows a call takes: checked by a chain's last rows."""
    T = 1024
    p = Problem(cuda_device, 1, 16, 1, T, [200], 128, dtype, kind, seed=23)
    out, lse = p.attend()
    k, v = p.k[0], p.v[0]
    for t in (0, 1, 500, 1023):
        o, l, spread = decode.tree_attention(p.q[0][:, t:t + 1], k, v, 200 + t, 1)
        assert np.abs(lse[0, :, t].double().cpu().numpy() - l[:, 0]).max() <= 2e-4
        d = np.abs(out[0, :, t].double().cpu().numpy() - o[:, 0])
        assert np.all(d <= 2.0 ** -8 * (np.abs(o[:, 0]) + spread[:, 0]) + 4e-4 * spread[:, 0])


@pytest.mark.parametrize("T", [2, 20])
def test_rows_of_zeros_among_quantised_values(cuda_device, T):
    """A value of zeros, which is written with scale 1, takes its weight and nothing else: the
    other values, of scales about 2^-7, keep their precision.  (A zero scale is as good.)"""
    p = Problem(cuda_device, 2, 16, 4, T, [1000, 333], 32, BF16, E4M3, seed=50)
    zero = torch.zeros((2, 4, 1, 256), dtype=BF16, device=cuda_device)
    for place in (0, 5, 128, 300):
        at = torch.full((2,), place, dtype=torch.int32, device=cuda_device)
        k = torch.randn((2, 4, 1, 256), generator=torch.Generator().manual_seed(place)).to(BF16)
        cache.write(p.pool, k.to(cuda_device), zero, p.table, at)
        y, s = decode.quantise(k)
        p.k[:, :, place:place + 1] = torch.as_tensor(y * s[..., None])
        p.v[:, :, place] = 0.0
    out, lse = p.attend()
    p.check(out, lse)
    for b in range(2):  # the scale of one of them by the user's own rule
        p.pool.v_scale[p.table[b, 5 // 32], :, 5 % 32] = 0.0
    again, lse2 = p.attend()
    p.check(again, lse2)


@pytest.mark.parametrize("dtype,kind", PAIRS[:3], ids=IDS[:3])
@pytest.mark.parametrize("gain", [30.0, 1e-3])
def test_peaked_and_flat_scores(cuda_device, dtype, kind, gain):
    """Large scores (standard deviation 30: the maximum moves from tile to tile) and nearly equal ones."""
    p = Problem(cuda_device, 2, 4, 2, 3, [900, 333], 32, dtype, kind, seed=24, gain=gain)
    out, lse = p.attend()
    for b in range(2):
        o, l, spread = decode.tree_attention(p.q[b], p.k[b], p.v[b], p.ctx[b], 3)
        # The bars of the module's head, for rows of unit variance, scale with the keys: scores are gain times larger.
        share = (1e-5 if dtype == F32 else 2e-4) * max(1.0, gain)
        assert np.abs(lse[b].double().cpu().numpy() - l).max() <= share
        step = 0.0 if dtype == F32 else 2.0 ** -8
        tol = step * (np.abs(o) + spread) + (2 * share + 2e-5) * spread
        assert np.all(np.abs(out[b].double().cpu().numpy() - o) <= tol)


def test_strided_queries_and_pages(cuda_device):
    p = Problem(cuda_device, 2, 8, 2, 3, [70, 11], 16, BF16, BF16, seed=25)
    want, want_lse = p.attend()
    q = p.q.transpose(1, 2).contiguous().to(cuda_device).transpose(1, 2)
    got, lse = cache.attend(q, p.pool, p.table, p.ctx_dev)
    assert torch.equal(got, want) and torch.equal(lse, want_lse) and got.is_contiguous()
    both = torch.stack((p.pool.k, p.pool.v), 3).transpose(1, 2).contiguous()  # [n, page, Hkv, 2, 256]
    pool = cache.PagedCache(both[:, :, :, 0].transpose(1, 2), both[:, :, :, 1].transpose(1, 2))
    got, lse = cache.attend(q, pool, p.table, p.ctx_dev)
    assert torch.equal(got, want) and torch.equal(lse, want_lse)


def test_bad_pages_and_lengths(cuda_device):
    """A bad page's keys are absent, a length past the table ends with the table; both are recorded."""
    for dtype, kind in PAIRS[:3]:
        p = Problem(cuda_device, 2, 4, 2, 1, [60, 60], 16, dtype, kind, seed=26)
        p.table[0, 1] = p.pool.k.shape[0]
        out, lse = p.attend()
        assert cache.status(p.pool) == gqa._lib.GQA_ERR_DEVICE_BOUNDS
        p.check(out, lse, rows=[1])
        keep = [j for j in range(61) if not 16 <= j < 32]
        p.k[0, :, :len(keep)], p.v[0, :, :len(keep)] = p.k[0][:, keep], p.v[0][:, keep]
        p.ctx[0] = len(keep) - 1
        p.check(out, lse, rows=[0])
        p = Problem(cuda_device, 1, 4, 2, 1, [63], 16, dtype, kind, seed=27)
        p.ctx_dev.fill_(1 << 30)
        out, lse = p.attend()
        assert cache.status(p.pool) == gqa._lib.GQA_ERR_DEVICE_BOUNDS
        p.check(out, lse)  # the table's 64 tokens
        p = Problem(cuda_device, 1, 4, 2, 1, [0], 16, dtype, kind, seed=28)
        p.ctx_dev.fill_(-5)
        out, lse = p.attend()
        assert cache.status(p.pool) == gqa._lib.GQA_ERR_DEVICE_BOUNDS
        p.check(out, lse)


@pytest.mark.parametrize("dtype,kind", PAIRS[:3], ids=IDS[:3])
def test_equal_calls_streams_and_graphs(cuda_device, dtype, kind):
    """Equal calls give equal bits, alone, together on two streams and replayed."""
    p = Problem(cuda_device, 3, 16, 4, 4, [2000, 10, 777], 32, dtype, kind, seed=29)
    o = Problem(cuda_device, 2, 16, 4, 4, [500, 3000], 32, dtype, kind, seed=30)
    mask = torch.as_tensor(_tree(4, 1)).to(cuda_device)
    want, other = p.attend(mask), o.attend(mask)
    torch.cuda.synchronize()
    q, q2 = p.q.to(cuda_device), o.q.to(cuda_device)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (s1, s2):
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(5):
        got.append((cache.attend(q, p.pool, p.table, p.ctx_dev, tree_mask=mask, stream=s1),
                    cache.attend(q2, o.pool, o.table, o.ctx_dev, tree_mask=mask, stream=s2)))
    torch.cuda.synchronize()
    for a, b in got:
        assert torch.equal(a[0], want[0]) and torch.equal(a[1], want[1])
        assert torch.equal(b[0], other[0]) and torch.equal(b[1], other[1])
    ws = torch.empty(cache.workspace_bytes(3, 16, 4, p.pool, p.table.shape[1], dtype), dtype=torch.uint8,
                     device=cuda_device)
    out, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
    g, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    for graph in (g, g2):  # two captured steps that share a workspace, replayed in order
        with torch.cuda.graph(graph):
            cache.attend(q, p.pool, p.table, p.ctx_dev, tree_mask=mask, out=out, lse=lse, workspace=ws)
    for ctx in ([2000, 10, 777], [1500, 0, 700], [3, 8, 1]):
        p.ctx_dev.copy_(torch.tensor(ctx, dtype=torch.int32))
        for graph in (g, g2):
            out.fill_(float("nan"))
            graph.replay()
            eager = cache.attend(q, p.pool, p.table, p.ctx_dev, tree_mask=mask)
            assert torch.equal(out, eager[0]) and torch.equal(lse, eager[1])


def test_refusals(cuda_device):
    p = Problem(cuda_device, 2, 16, 4, 3, [20, 30], 16, BF16, BF16)
    q, dev = p.q.to(cuda_device), cuda_device
    mask = torch.ones(3, 3, dtype=torch.bool, device=dev)
    good = dict(q=q, pool=p.pool, page_table=p.table, context_lens=p.ctx_dev)
    for kw in (dict(q=q.cpu()), dict(q=q.half()), dict(q=q[0]), dict(q=q[..., :128]), dict(page_table=p.table[:1]),
               dict(page_table=p.table.long()), dict(context_lens=p.ctx_dev.long()), dict(context_lens=p.ctx_dev[:1]),
               dict(tree_lens=p.ctx_dev.cpu()), dict(tree_mask=mask.float()), dict(tree_mask=mask[:2]),
               dict(tree_mask=mask.cpu()), dict(tree_mask=mask.expand(2, 3, 3)),
               dict(out=torch.empty_like(q, dtype=F32)), dict(lse=torch.empty(2, 16, 4, device=dev)),
               dict(lse=torch.empty(2, 16, 3, device=dev, dtype=torch.float64)),
               dict(workspace=torch.empty(1 << 20, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            cache.attend(**{**good, **kw})
    for kw in (dict(q=q[:, :15]), dict(q=q[:, :12]), dict(workspace=torch.empty(64, dtype=torch.uint8, device=dev)),
               dict(q=torch.zeros(2, 16, 0, 256, dtype=BF16, device=dev)),
               dict(q=torch.zeros(2, 16, 1025, 256, dtype=BF16, device=dev))):
        with pytest.raises(gqa.GqaAttnError):
            cache.attend(**{**good, **kw})


@pytest.mark.parametrize("dtype,kind", [(F32, F32), (BF16, BF16), (BF16, E4M3)], ids=IDS[:3])
def test_a_decoder_with_the_operators_together(cuda_device, dtype, kind):
    """A prompt written with rotated keys, decoded token by token, then a drafted tree whose
    accepted branch is kept: against the float64 attention of the rotated rows, and for
    unquantised pages against the dense ``fwd`` over what ``read`` gives back."""
    dev, Hq, Hkv, L, page = cuda_device, 16, 4, 150, 16
    t = rotary.Table(128, layout="interleaved", scaling="linear", factor=2.0, device=dev)
    g = torch.Generator().manual_seed(31)
    pool = cache.PagedCache.empty(40, Hkv, page, kind, dev)
    table = torch.randperm(40, generator=g)[:20].view(1, 20).to(torch.int32).to(dev)
    n = torch.zeros(1, dtype=torch.int32, device=dev)

    def token(T):
        return [torch.randn((1, h, T, 256), generator=g).to(dtype).to(dev) for h in (Hq, Hkv, Hkv)]

    def bar(out, lse, q, ctx, T, mask=None):
        kd, vd = cache.read(pool, table, n * 0 + ctx + T, ctx + T, dtype=F32)
        o, l, spread = decode.tree_attention(q[0], kd[0], vd[0], ctx, T, mask)
        tol_o = 2e-5 if dtype == F32 else 2.0 ** -8 * (np.abs(o) + spread) + 4e-4 * spread
        assert np.all(np.abs(out[0].double().cpu().numpy() - o) <= tol_o)
        assert np.abs(lse[0].double().cpu().numpy() - l).max() <= (1e-5 if dtype == F32 else 2e-4)

    q, k, v = token(L)
    cache.write(pool, k, v, table, n, rope=t)
    q, _ = rotary.rotate(q, None, t)
    if kind != E4M3:  # the prompt's own attention, dense, over the cache read back
        kd, vd = cache.read(pool, table, n + L, L, dtype=dtype)
        assert torch.equal(vd, v)
        full, full_lse = gqa.fwd(q, kd, vd)
        out, lse = cache.attend(q[:, :, -1:], pool, table, n + L - 1)
        tol = 4e-5 if dtype == F32 else 2e-2
        assert (out - full[:, :, -1:]).abs().max() <= tol and (lse - full_lse[:, :, -1:]).abs().max() <= tol
    n += L
    for _ in range(5):
        q, k, v = token(1)
        cache.write(pool, k, v, table, n, rope=t)
        q, _ = rotary.rotate(q, None, t, positions=n[:, None])
        out, lse = cache.attend(q, pool, table, n)
        bar(out, lse, q, int(n), 1)
        n += 1
    parent, depth = [-1, 0, 0, 1, 1, 2], [0, 1, 1, 2, 2, 2]
    mask = np.eye(6, dtype=bool)
    for i, p in enumerate(parent):
        if p >= 0:
            mask[i] |= mask[p]
    q, k, v = token(6)
    pos = n[:, None] + torch.tensor([depth], dtype=torch.int32, device=dev)
    cache.write(pool, k, v, table, n, rope=t, positions=pos)
    q, _ = rotary.rotate(q, None, t, positions=pos)
    out, lse = cache.attend(q, pool, table, n, tree_mask=torch.as_tensor(mask).to(dev))
    bar(out, lse, q, int(n), 6, mask)
    # accept 0 -> 1 -> 4: its keys written behind the context; its last row sees what the tree's row 4 saw
    path = [0, 1, 4]
    cache.write(pool, k[:, :, path], v[:, :, path], table, n, rope=t)
    out2, lse2 = cache.attend(q[:, :, path], pool, table, n)
    bar(out2, lse2, q[:, :, path], int(n), 3)
    tol = 4e-5 if dtype == F32 else 2e-2
    assert (out2[:, :, 2] - out[:, :, 4]).abs().max() <= tol and (lse2[:, :, 2] - lse[:, :, 4]).abs().max() <= 4e-4
    assert cache.status(pool) == 0


@pytest.mark.parametrize("dtype,kind", PAIRS, ids=IDS)
@pytest.mark.parametrize("bits", [0x7fc00000, -1, 0x7f800001])
def test_a_visible_nan_reaches_its_rows(cuda_device, dtype, kind, bits):
    """A NaN of any payload in a key makes the rows that see it NaN and no other; in a value, their column."""
    p = Problem(cuda_device, 1, 4, 2, 3, [40], 16, dtype, kind, seed=31)
    clean, _ = p.attend()
    nan = torch.tensor([bits], dtype=torch.int32).view(F32)
    for pool, column in ((p.pool.k, None), (p.pool.v, 77)):
        at = pool[p.table[0, 2], 0, 9]  # token 41, drafted token 1, of key/value head 0
        kept = at.clone()
        if kind == F32:
            at[77] = nan.to(cuda_device)[0]
        elif kind == BF16:
            at.view(torch.int16)[77] = {0x7fc00000: 0x7fc0, -1: -1, 0x7f800001: 0x7f81}[bits]
        else:
            at.view(torch.int8)[77] = {0x7fc00000: 0x7f, -1: -1, 0x7f800001: 0x7f}[bits]
        out, _ = p.attend()
        nans = torch.zeros_like(out, dtype=torch.bool)
        nans[0, :2, 1:, slice(None) if column is None else column] = True
        assert torch.equal(out.isnan(), nans)
        same = ~nans if column is not None else ~nans.any(-1, keepdim=True).expand_as(nans)
        assert torch.equal(out[same], clean[same])
        at.copy_(kept)


@pytest.mark.parametrize("dtype,kind", [(BF16, BF16), (BF16, E4M3)], ids=["bf16", "bf16_e4m3"])
@pytest.mark.parametrize("T,Hq,page", [(40, 16, 8), (64, 16, 16), (33, 32, 64), (128, 16, 128), (96, 16, 32)])
def test_many_rows(cuda_device, dtype, kind, T, Hq, page):
    """Two to four tiles of 128 rows to a head, ragged contexts and trees, padding rows."""
    ctx = [0, 130, 700, 63]
    p = Problem(cuda_device, 4, Hq, 4, T, ctx, page, dtype, kind, seed=T, drafted=[T, T - 3, 1, 0])
    p.check(*p.attend(), small=kind == E4M3)
    mask = np.stack([_tree(T, 60 + b) for b in range(4)])
    mask[0, 5] = False  # a row that sees nothing where there is no context
    p.check(*p.attend(mask), mask=mask, small=kind == E4M3)
    assert cache.status(p.pool) == 0


@pytest.mark.parametrize("column", [3, 127, 128, 250])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")], ids=["nan", "inf", "-inf"])
def test_hidden_values_of_many_rows(cuda_device, bad, column):
    """Two tiles of rows: a bad value in any column reaches the rows that see it, in that column."""
    T = 48
    p = Problem(cuda_device, 1, 16, 4, T, [100], 32, BF16, BF16, seed=9)
    mask = _tree(T, 4)
    clean, clean_lse = p.attend(mask)
    at = p.pool.v[p.table[0, (100 + 7) // 32].item(), 2, (100 + 7) % 32]
    at[column] = bad
    out, lse = p.attend(mask)
    sees = torch.zeros((1, 16, T, 256), dtype=torch.bool)
    sees[0, 8:12, torch.as_tensor(mask[:, 7]), column] = True
    assert torch.equal(lse, clean_lse)
    assert torch.equal(out[~sees.to(out.device)], clean[~sees.to(out.device)])
    got = out[sees.to(out.device)].float()
    assert got.numel() and bool((got.isnan() if bad != bad else got == bad).all())


@pytest.mark.parametrize("kind", [BF16, E4M3], ids=["bf16", "e4m3"])
def test_many_rows_over_long_contexts(cuda_device, kind):
    """Rings go round many times, workers cross heads; equal calls give equal bits, also replayed."""
    p = Problem(cuda_device, 2, 16, 4, 40, [9000, 4100], 16, BF16, kind, seed=41)
    first, lse = p.attend()
    p.check(first, lse)
    for _ in range(20):
        out, l2 = p.attend()
        assert torch.equal(out, first) and torch.equal(l2, lse)
    q, graph = p.q.to(cuda_device), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, l2 = cache.attend(q, p.pool, p.table, p.ctx_dev)
    for _ in range(3):
        graph.replay()
    assert torch.equal(out, first) and torch.equal(l2, lse)


def test_calls_of_all_kinds_in_a_row(cuda_device):
    """Calls of every kernel behind one another on one stream, sharing a workspace (each may start
    while the one before ends), the same on two streams at once, and captured as one graph of
    two branches: the same bits as alone."""
    kinds = [(F32, F32, 5), (BF16, BF16, 1), (BF16, BF16, 40), (BF16, E4M3, 40), (BF16, E4M3, 3), (F32, BF16, 1),
             (BF16, BF16, 12), (BF16, F32, 2), (BF16, BF16, 20)]
    problems = [Problem(cuda_device, 2, 16, 4, T, [1500, 37], 32, dtype, kind, seed=70 + i)
                for i, (dtype, kind, T) in enumerate(kinds)]
    qs = [p.q.to(cuda_device) for p in problems]
    size = max(cache.workspace_bytes(2, 16, p.q.shape[2], p.pool, p.table.shape[1], p.q.dtype) for p in problems)

    def call(i, ws=None, **kw):
        p = problems[i]
        return cache.attend(qs[i], p.pool, p.table, p.ctx_dev, workspace=ws, **kw)

    want = []
    for i in range(len(kinds)):
        want.append(call(i))
        torch.cuda.synchronize()

    def same(got):
        torch.cuda.synchronize()
        for i, (out, lse) in got:
            assert torch.equal(out, want[i][0]) and torch.equal(lse, want[i][1]), f"call {i}"

    order = [i for r in range(4) for i in np.random.default_rng(r).permutation(len(kinds))]
    ws = [torch.empty(size, dtype=torch.uint8, device=cuda_device) for _ in range(2)]
    same([(i, call(i, ws[0])) for i in order])

    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    same([(i, call(i, ws[k], stream=streams[k])) for i in order for k in range(2)])

    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph):
        fork = torch.cuda.current_stream()
        side.wait_stream(fork)
        got = [(i, call(i, ws[0])) for i in order[:9]]
        with torch.cuda.stream(side):
            got += [(i, call(i, ws[1])) for i in order[9:18]]
        fork.wait_stream(side)
    for _ in range(3):
        for _, (out, _) in got:
            out.zero_()
        graph.replay()
        same(got)


@pytest.mark.parametrize("dtype,kind,T", [(BF16, BF16, 1), (BF16, BF16, 40), (BF16, E4M3, 40), (F32, F32, 5)])
def test_captured_behind_copies_and_joined_streams(cuda_device, dtype, kind, T):
    """In a graph: behind a copy of the lengths, behind a cleared output, and behind two streams
    that join; the lengths change between replays."""
    p = Problem(cuda_device, 2, 16, 4, T, [1500, 37], 32, dtype, kind, seed=90 + T)
    q, ctx, source = p.q.to(cuda_device), p.ctx_dev.clone(), p.ctx_dev.clone()
    out = [torch.empty_like(q) for _ in range(3)]
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        ctx.copy_(source)
        cache.attend(q, p.pool, p.table, ctx, out=out[0])
        side.wait_stream(main)
        with torch.cuda.stream(side):
            out[1].zero_()
            cache.attend(q, p.pool, p.table, ctx, out=out[1])
        out[2].zero_()
        main.wait_stream(side)
        cache.attend(q, p.pool, p.table, ctx, out=out[2])
    for lens in ([1500, 37], [200, 30], [0, 1]):
        source.copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        want, _ = cache.attend(q, p.pool, p.table, source)
        torch.cuda.synchronize()
        for o in out:
            assert torch.equal(o, want)


@pytest.mark.parametrize("T", [1, 12, 24, 64])
def test_scales_of_one_throughout(cuda_device, T):
    """A pool quantised with the scale 1 for every value: any row may then be one of zeros, so the
    kernels look at each of them, tile after tile, over many rounds of the rings.  Equal calls
    give equal bits and no wait runs out."""
    p = Problem(cuda_device, 2, 16, 4, T, [9000, 4100], 32, BF16, E4M3, seed=110 + T)
    codes = p.pool.v.float().cpu()[p.table.cpu().long()].transpose(1, 2).flatten(2, 3)  # up to 448 each
    p.v = codes[:, :, : p.v.shape[2]].nan_to_num(0.0)  # (behind a sequence's end the pages hold NaN)
    p.pool.v_scale.fill_(1.0)
    first, lse = p.attend()
    p.check(first, lse)
    for _ in range(20):
        out, again = p.attend()
        assert torch.equal(out, first) and torch.equal(again, lse)
    assert cache.status(p.pool) == 0


@functools.lru_cache(maxsize=2)
def _long_pages(dev, flat, n):
    """Pages of n + 65 tokens of four heads: unit-normal keys (all zeros with ``flat``) but for the first
    column and the first key, values with a common mean."""
    g = torch.Generator().manual_seed(1000 + n)
    k, v = (torch.randn((1, 4, n + 65, 256), generator=g) for _ in range(2))
    if flat:
        k.zero_()
    k[..., 0] = 0.0
    v += 0.5
    per = -(-(n + 65) // 128)
    pool = cache.PagedCache.empty(per, 4, 128, E4M3, dev)
    table = torch.arange(per, dtype=torch.int32, device=dev)[None]
    cache.write(pool, k.to(dev), v.to(dev), table, torch.zeros(1, dtype=torch.int32, device=dev))
    return pool, table, [torch.as_tensor(y * s[..., None]) for y, s in map(decode.quantise, (k, v))]


class Sink:
    """One key that holds `share` of every row's weight before `n` others, whose scores are unit
    normals (or, `flat`, all equal); 40 sequences of four key/value heads share the pages, so that a
    worker has a whole head's keys.  The first column of every query is 8 and that of the other
    keys 0, so the first key's score is half of its first column."""

    def __init__(self, dev, T, n, share, flat, B=40):
        self.pool, table, (k, v) = _long_pages(dev, flat, n)
        first = torch.zeros(1, 4, 1, 256)
        mass = float(np.log(n)) + (0.0 if flat else 0.5)  # log of the other keys' sum
        first[..., 0] = 2.0 * (mass + np.log(share / (1.0 - share)))
        zero = torch.zeros(1, dtype=torch.int32, device=dev)
        cache.write(self.pool, first.to(dev), v[:, :, :1].float().to(dev), table, zero)
        y, s = decode.quantise(first)
        self.k, self.v = k[0].clone(), v[0]
        self.k[:, :1] = torch.as_tensor(y * s[..., None])[0]
        self.table = table.expand(B, -1).contiguous()
        q = torch.randn((B, 16, T, 256), generator=torch.Generator().manual_seed(2000 + T))
        q[..., 0] = 8.0
        self.q, self.ctx = q.to(BF16), n + 1
        self.lens = torch.full((B,), n + 1, dtype=torch.int32, device=dev)

    def check(self, out, lse, rows):
        T = self.q.shape[2]
        for b in rows:
            for t in sorted({0, T // 2, T - 1}):  # of a chain
                o, l, spread = decode.tree_attention(self.q[b][:, t:t + 1], self.k, self.v, self.ctx + t, 1)
                assert np.abs(lse[b, :, t:t + 1].double().cpu().numpy() - l).max() <= 2e-4
                tol = 2.0 ** -8 * (np.abs(o) + spread) + 4e-4 * spread
                off = np.abs(out[b, :, t:t + 1].double().cpu().numpy() - o) / tol
                assert off.max() <= 1.0, f"sequence {b}, token {t}: {off.max():.1f} times the tolerance"


@pytest.mark.parametrize("share", [0.05, 0.2, 0.5, 0.95])
@pytest.mark.parametrize("flat", [False, True], ids=["normal", "flat"])
@pytest.mark.parametrize("T", [1, 5, 12, 24, 64])
def test_one_key_outweighs_a_long_context(cuda_device, T, flat, share):
    """Quantised pages keep the weight of many small probabilities beside a large one, at the
    plain tolerance of the module's head: a probability is off by 2^-9 + 2^-11 of itself, or by 2^-28 of the
    largest, 2^-13 of it for all 32,768 keys together.  Alone and in a batch alike."""
    p = Sink(cuda_device, T, 32_768, share, flat)
    q = p.q.to(cuda_device)
    p.check(*cache.attend(q, p.pool, p.table, p.lens), rows=(0, 39))
    p.check(*cache.attend(q[:1], p.pool, p.table[:1], p.lens[:1]), rows=(0,))
    assert cache.status(p.pool) == 0


@pytest.mark.parametrize("T,Hq,page", [(3, 8, 16), (40, 16, 8), (64, 16, 16), (33, 32, 64)])
def test_few_quantised_keys_at_the_plain_tolerance(cuda_device, T, Hq, page):
    """Rows that see few keys of very different weights: the pieces of a probability need no
    allowance for its size."""
    p = Problem(cuda_device, 4, Hq, 4, T, [0, 130, 700, 63], page, BF16, E4M3, seed=140 + T, drafted=[T, T - 2, 1, 0])
    p.check(*p.attend())
    mask = np.stack([_tree(T, 60 + b) for b in range(4)])
    p.check(*p.attend(mask), mask=mask)


@pytest.mark.parametrize("dtype,kind", PAIRS, ids=IDS)
@pytest.mark.parametrize("Hq", [4, 32])
def test_a_single_token_that_its_mask_hides(cuda_device, dtype, kind, Hq):
    """T = 1 and a mask of 0: the row sees its context alone, whatever the token's key and value are."""
    p = Problem(cuda_device, 2, Hq, 2, 1, [37, 128], 16, dtype, kind, seed=120)
    mask = np.zeros((1, 1), dtype=bool)
    good, good_lse = p.attend(mask)
    p.check(good, good_lse, mask=mask)
    for pages in (p.pool.v, p.pool.k):
        for b, c in enumerate(p.ctx):
            pages.view(torch.uint8).view(*pages.shape[:3], -1)[p.table[b, c // 16], :, c % 16] = 0xff  # NaN
        out, lse = p.attend(mask)
        assert torch.equal(out, good) and torch.equal(lse, good_lse)
    if kind != E4M3:
        for b, c in enumerate(p.ctx):
            p.pool.v[p.table[b, c // 16], :, c % 16] = float("inf")
        assert torch.equal(p.attend(mask)[0], good)
    both = np.stack([mask, ~mask])  # one sequence's token hides, the other's does not
    out, lse = p.attend(both)
    assert torch.equal(out[0], good[0]) and out[1].isnan().all()


@pytest.mark.parametrize("dtype,kind", PAIRS, ids=IDS)
@pytest.mark.parametrize("T", [1, 12, 24])
def test_scores_far_below_zero(cuda_device, dtype, kind, T):
    """Each row sees its own token only, at a score of -6.25e32: that token's value, not nothing."""
    p = Problem(cuda_device, 1, 16, 4, T, [0], 16, dtype, kind, seed=121)
    mask = np.eye(T, dtype=bool)
    p.q.zero_()
    p.q[..., 0] = 1e17
    k = torch.zeros(1, 4, T, 256)
    k[..., 0] = -1e17
    k, v = k.to(BF16), torch.randn((1, 4, T, 256), generator=torch.Generator().manual_seed(122)).to(BF16)
    cache.write(p.pool, k.to(cuda_device), v.to(cuda_device), p.table, torch.zeros_like(p.ctx_dev))
    if kind == E4M3:
        k, v = (torch.as_tensor(y * s[..., None]) for y, s in map(decode.quantise, (k, v)))
    out, lse = p.attend(mask)
    o, l, _ = decode.tree_attention(p.q[0], k[0], v[0], 0, T, mask)
    # one product, its scale and the factors 1 / ln 2 and ln 2: each rounds by 2^-24 of the score, and the e4m3
    # pieces of a query leave 2^-18 of it
    assert np.all(np.abs(lse[0].double().cpu().numpy() - l) <= np.abs(l) * (8 * 2.0 ** -24 + 2.0 ** -18))
    # weight 1: a probability's rounding (2^-8), the output's (2^-8)
    assert np.all(np.abs(out[0].double().cpu().numpy() - o) <= 2.0 ** -7 * np.abs(o))


@pytest.mark.parametrize("T", [1, 5, 12, 24])
def test_value_scales_of_any_sign_and_size(cuda_device, T):
    """The value of a row is code x scale for any fp32 scale: of either sign, zero or subnormal,
    tiny or huge throughout; a scale that is not a number stays behind the mask that hides it."""
    dev, ctx = cuda_device, [700, 40]
    p = Problem(dev, 2, 16, 4, T, ctx, 32, BF16, E4M3, seed=130 + T)
    n, per = p.v.shape[2], p.table.shape[1]
    at = p.table.cpu().long()
    place = torch.arange(n)
    where = [(at[b][place // 32], place % 32) for b in range(2)]

    def scales(fill):  # fill(b, j, head) -> a factor of the scale, for every place
        kept = p.pool.v_scale.clone()
        f = torch.ones(2, n, 4)
        fill(f)
        s = p.pool.v_scale.cpu()
        value = p.v.clone()
        for b in range(2):
            page, slot = where[b]
            s[page, :, slot] = s[page, :, slot] * f[b]
            value[b] = p.v[b] * f[b].double().T[..., None]
        p.pool.v_scale.copy_(s)
        got = p.attend()
        p.pool.v_scale.copy_(kept)
        return got, value

    def check(fill):
        (out, lse), value = scales(fill)
        for b in range(2):
            o, l, spread = decode.tree_attention(p.q[b], p.k[b], value[b], ctx[b], T)
            assert np.abs(lse[b].double().cpu().numpy() - l).max() <= 2e-4
            tol = 2.0 ** -8 * (np.abs(o) + spread) + 4e-4 * spread
            assert np.all(np.abs(out[b].double().cpu().numpy() - o) <= tol)

    g = torch.Generator().manual_seed(131)
    sign = torch.where(torch.rand((2, n, 4), generator=g) < 0.5, -1.0, 1.0)
    check(lambda f: f.copy_(sign))
    check(lambda f: f[:, ::3].fill_(0.0))
    check(lambda f: f[:, ::3].fill_(2.0 ** -126))  # subnormal: too little to reach the output
    for size in (2.0 ** -111, 2.0 ** -40, 2.0 ** 50, 2.0 ** 100):
        check(lambda f: f.fill_(size))

    def with_zeros(f):  # zero rows as the writer leaves them, beside large ones
        f.fill_(2.0 ** 50)
        f[:, 1::2] = 0.0

    check(with_zeros)
    if T > 1:  # a drafted token whose scale is not a number, hidden from the rows before it
        good, good_lse = p.attend()
        for bad in (float("nan"), float("inf"), 1e-42):
            kept = p.pool.v_scale.clone()
            for b in range(2):
                j = ctx[b] + T - 1
                p.pool.v_scale[at[b][j // 32], :, j % 32] = bad
            out, lse = p.attend()
            p.pool.v_scale.copy_(kept)
            assert torch.equal(out[:, :, :-1], good[:, :, :-1]) and torch.equal(lse[:, :, :-1], good_lse[:, :, :-1])


@pytest.mark.parametrize("T,Hq", [(1, 16), (2, 16), (5, 8), (8, 16)])
def test_probabilities_of_few_rows_are_not_rounded_to_bf16(cuda_device, T, Hq):
    """Up to 32 rows of a head over bf16 pages: a probability is off by 2^-15 of itself, so an output
    by its own rounding, 2^-8 of it, and the scores' share.  A score's 255 additions are each off
    by 2^-24 of at most sum |q k|, below 220 for these inputs: 255 x 220 x 2^-24 / 16 = 2.1e-4, twice
    that in a probability."""
    p = Problem(cuda_device, 12, Hq, 4, T, [0, 1, 2, 3, 4, 5, 1, 2, 3, 1, 2, 40], 16, BF16, BF16, seed=150 + T)
    size = np.abs(p.q.double().numpy()).reshape(12, 4, -1, 256) @ p.k.double().abs().numpy().swapaxes(2, 3)
    assert size.max() < 220
    out, lse = p.attend()
    for b in range(12):
        o, l, spread = decode.tree_attention(p.q[b], p.k[b], p.v[b], p.ctx[b], T)
        assert np.abs(lse[b].double().cpu().numpy() - l).max() <= 2.1e-4 + 1e-5
        tol = 2.0 ** -8 * np.abs(o) + (2.0 ** -15 + 4.2e-4) * spread
        assert np.all(np.abs(out[b].double().cpu().numpy() - o) <= tol)


@pytest.mark.parametrize("dtype,kind", PAIRS, ids=IDS)
@pytest.mark.parametrize("T,page", [(1, 256), (12, 1024), (40, 512)])
def test_large_pages_and_one_page_pools(cuda_device, dtype, kind, T, page):
    """Pages of more keys than a tile, and a pool of a single page of one head, whose strides
    of the dimensions of one mean nothing."""
    p = Problem(cuda_device, 2, 8, 2, T, [1500, 255], page, dtype, kind, seed=160 + T)
    p.check(*p.attend())
    p = Problem(cuda_device, 1, 4, 1, T, [100], page, dtype, kind, seed=161)
    only = int(p.table[0, 0])
    first = lambda t: None if t is None else t[only:only + 1].contiguous()  # noqa: E731
    pool = cache.PagedCache(*(first(t) for t in (p.pool.k, p.pool.v, p.pool.k_scale, p.pool.v_scale)))
    out, lse = cache.attend(p.q.to(cuda_device), pool, torch.zeros_like(p.table), p.ctx_dev)
    p.check(out, lse)


def test_a_thousand_sequences(cuda_device):
    """More sequences than a warp's lanes many times over, most of them short, some empty."""
    B = 1000
    rng = np.random.default_rng(5)
    ctx = [int(c) for c in rng.integers(0, 40, B)]
    drafted = [int(d) for d in rng.integers(0, 3, B)]
    p = Problem(cuda_device, B, 4, 2, 2, ctx, 8, BF16, BF16, seed=170, drafted=drafted)
    p.check(*p.attend(), rows=list(range(0, B, 7)) + [B - 1])
    assert cache.status(p.pool) == 0
