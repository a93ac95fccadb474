"""Pins of the decoding oracle against library routines, closed forms and invariants (CPU)."""

import math

import numpy as np
import pytest
import torch

import oracle
from oracle import decode


def test_angle_of_near_and_far_positions():
    for p, f in ((0, 0.3), (7, 1.0), (-5, 0.25), (100, 0.01)):
        want = math.remainder(p * f, 2 * math.pi)
        assert decode.angle(p, f) == pytest.approx(want, abs=1e-13)
    # cos and sin take any float64 argument exactly: 3 * 2^28 * 0.75 is a whole float
    p, f = 3 << 28, 0.75
    a = decode.angle(p, f)
    assert math.cos(a) == pytest.approx(math.cos(p * f), abs=1e-12)
    assert math.sin(a) == pytest.approx(math.sin(p * f), abs=1e-12)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rotation_preserves_norms_and_relative_positions(layout):
    rng = np.random.default_rng(0)
    f = [10000.0 ** (-2 * i / 32) for i in range(16)]
    q, k = rng.standard_normal((2, 1, 1, 1, 256))
    at = lambda x, p: decode.rotate(x, [[p]], f, layout=layout)  # noqa: E731
    assert np.linalg.norm(at(q, 12345)) == pytest.approx(np.linalg.norm(q), rel=1e-13)
    near, far = np.sum(at(q, 9) * at(k, 4)), np.sum(at(q, 1_000_009) * at(k, 1_000_004))
    assert near == pytest.approx(far, abs=1e-9)
    back = decode.rotate(at(q, 77), [[77]], f, layout=layout, sign=-1.0)
    assert np.allclose(back, q, atol=1e-13)
    assert np.array_equal(at(q, 5)[..., 32:], q[..., 32:])


def test_quantise_matches_the_float8_cast():
    g = torch.Generator().manual_seed(3)
    x = torch.randn((50, 256), generator=g) * torch.logspace(-3, 3, 50)[:, None]
    y, s = decode.quantise(x)
    want = (x / torch.tensor(s, dtype=torch.float32)[:, None]).to(torch.float8_e4m3fn)
    assert np.array_equal(y, want.double().numpy())
    assert np.all(np.abs(y).max(-1) <= 448) and np.all(np.abs(y).max(-1) > 223)
    y, s = decode.quantise(np.array([[0.0] * 4, [448.0, 0, 0, 1.0], [449.0, 0, np.inf, np.nan]]))
    assert list(s) == [1.0, 1.0, 2.0] and y[2, 2] == 448 and np.isnan(y[2, 3])


def test_chain_is_causal_attention():
    rng = np.random.default_rng(1)
    ctx, T = 13, 4
    q, k, v = (rng.standard_normal((1, h, n, 256)) for h, n in ((4, T), (2, ctx + T), (2, ctx + T)))
    want, want_lse = oracle.attention(q, k, v, q_pos_offset=ctx)
    out, lse, spread = decode.tree_attention(q[0], k[0], v[0], ctx, T)
    assert np.allclose(out, want[0], atol=1e-12) and np.allclose(lse, want_lse[0], atol=1e-12)
    assert np.all(spread >= np.abs(out) - 1e-12)


def test_tree_rows_are_the_chains_along_their_branches():
    rng = np.random.default_rng(2)
    ctx, parent = 5, [-1, 0, 0, 1, 2]
    T = len(parent)
    mask = np.eye(T, dtype=bool)
    for t, p in enumerate(parent):
        if p >= 0:
            mask[t] |= mask[p]
    q, k, v = (rng.standard_normal((h, n, 256)) for h, n in ((2, T), (1, ctx + T), (1, ctx + T)))
    out, lse, _ = decode.tree_attention(q, k, v, ctx, T, mask)
    path = [0, 2, 4]  # the branch of the last token
    rows = list(range(ctx)) + [ctx + u for u in path]
    chain, chain_lse, _ = decode.tree_attention(q[:, path], k[:, rows], v[:, rows], ctx, 3)
    assert np.allclose(out[:, 4], chain[:, 2]) and np.allclose(lse[:, 4], chain_lse[:, 2])
    # nothing visible
    out, lse, _ = decode.tree_attention(q, k, v, 0, T, np.zeros((T, T), bool))
    assert not out.any() and np.all(np.isneginf(lse))
    out, lse, _ = decode.tree_attention(q, k, v, ctx, 2)
    assert not out[:, 2:].any() and np.all(np.isneginf(lse[:, 2:])) and np.all(np.isfinite(lse[:, :2]))
