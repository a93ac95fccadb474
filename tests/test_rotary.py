"""Rotary positions on the GPU against the float64 definition.

Tolerances, in units of e = 2^-24 (half a step of fp32) times m (|x1| + |x2|), the size of
the terms: the angle within a quarter turn, at most pi / 4, is rounded to fp32 and multiplied by
a rounded constant, off by at most 3 pi e / 4 < 2.4 e, plus 2^-31 pi < 0.03 e for the bits cut
off; the series leave out less than 0.03 e and round by half a step of their result, 0.5 e, and
less than 0.5 e before; the product with m, the product with x and the sum round once each, 1 e
apiece.  6.5 e in all, 8 e taken.  bf16 outputs add half a step, 2^-8 of the value.
"""

import numpy as np
import pytest
import torch

from long_context_causal_flash_b200 import rotary
from oracle import decode

pytestmark = pytest.mark.gpu

E = 2.0 ** -24


def _x(shape, dtype, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


def _check(got, x, positions, table, sign=1.0):
    pos = np.broadcast_to(np.asarray(positions), (x.shape[0], x.shape[2]))
    want = decode.rotate(x, pos, table.inv_freq, table.magnitude, table.layout, sign)
    size = x.double().abs().numpy()
    R = table.rot
    lo, hi = (slice(0, R // 2), slice(R // 2, R)) if table.layout == "half" else (slice(0, R, 2), slice(1, R, 2))
    tol = np.zeros_like(size)
    tol[..., lo] = tol[..., hi] = 8 * E * table.magnitude * (size[..., lo] + size[..., hi])
    if got.dtype == torch.bfloat16:
        tol[..., :R] += 2.0 ** -8 * np.abs(want[..., :R])
    off = np.abs(got.double().cpu().numpy() - want) - tol
    assert off.max() <= 0, f"off by {off.max():.2e} more than allowed"


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("rot,scaling", [(256, None), (64, "linear"), (16, None), (96, "ntk"), (128, "yarn")])
@pytest.mark.parametrize("B,L", [(1, 1), (3, 17)])
def test_matches_the_definition(cuda_device, dtype, layout, rot, scaling, B, L):
    t = rotary.Table(rot, layout=layout, scaling=scaling, factor=4.0, original_length=2048, device=cuda_device)
    q, k = _x((B, 5, L, 256), dtype, 1), _x((B, 2, L, 256), dtype, 2)
    qo, ko = rotary.rotate(q.to(cuda_device), k.to(cuda_device), t, pos_offset=1000)
    pos = [1000 + np.arange(L)]
    _check(qo, q, pos, t)
    _check(ko, k, pos, t)
    back, none = rotary.rotate(q.to(cuda_device), None, t, pos_offset=1000, inverse=True)
    assert none is None
    _check(back, q, pos, t, sign=-1.0)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_far_negative_and_given_positions(cuda_device, dtype):
    t = rotary.Table(64, layout="interleaved")
    B, L = 2, 9
    pos = torch.randint(-(1 << 31), (1 << 31) - 1, (B, L), generator=torch.Generator().manual_seed(5)).to(torch.int32)
    q = _x((B, 3, L, 256), dtype, 3)
    qo, _ = rotary.rotate(q.to(cuda_device), None, t, positions=pos.to(cuda_device))
    _check(qo, q, pos.numpy(), t)
    qo, _ = rotary.rotate(q.to(cuda_device), None, t, positions=pos[1].to(cuda_device))
    _check(qo, q, pos[1:2].numpy(), t)
    wide = torch.zeros((B, 2 * L), dtype=torch.int32, device=cuda_device)  # rows of a wider table
    wide[:, :L] = pos.to(cuda_device)
    qo, _ = rotary.rotate(q.to(cuda_device), None, t, positions=wide[:, :L])
    _check(qo, q, pos.numpy(), t)
    qo, _ = rotary.rotate(q.to(cuda_device), None, t, pos_offset=(1 << 33) + 11)
    _check(qo, q, [(1 << 33) + 11 + np.arange(L)], t)


def test_strided_inputs_and_in_place(cuda_device):
    B, L, t = 2, 33, rotary.Table(128)
    qkv = _x((B, L, 8, 256), torch.bfloat16, 4)
    q, k = qkv[:, :, :4].transpose(1, 2), qkv[:, :, 4:6].transpose(1, 2)
    dev = qkv.to(cuda_device)
    qd, kd = dev[:, :, :4].transpose(1, 2), dev[:, :, 4:6].transpose(1, 2)
    qo, ko = rotary.rotate(qd, kd, t)
    _check(qo, q, [np.arange(L)], t)
    _check(ko, k, [np.arange(L)], t)
    assert qo.is_contiguous()
    a, b = rotary.rotate(qd, kd, t, out=qd, out_k=kd)
    assert a is qd and b is kd
    assert torch.equal(qd, qo) and torch.equal(kd, ko)
    assert torch.equal(dev[:, :, 6:], qkv[:, :, 6:].to(cuda_device))  # the values between them untouched
    same = _x((1, 3, L, 256), torch.bfloat16, 9)  # one sequence for all of a batch
    qo, _ = rotary.rotate(same.to(cuda_device).expand(4, 3, L, 256), None, t)
    for row in qo:
        _check(row[None], same, [np.arange(L)], t)


def test_nothing_to_rotate(cuda_device):
    t = rotary.Table()
    for shape in ((0, 2, 5, 256), (2, 2, 0, 256)):
        q, _ = rotary.rotate(torch.empty(shape, device=cuda_device), None, t)
        assert q.shape == shape


def test_nan_and_infinity_stay_in_their_pair(cuda_device):
    t = rotary.Table(64)
    x = _x((1, 1, 4, 256), torch.float32, 6)
    x[0, 0, 1, 3], x[0, 0, 2, 200] = float("nan"), float("inf")
    y = rotary.rotate(x.to(cuda_device), None, t)[0].cpu()
    bad = (~torch.isfinite(y)).nonzero().tolist()
    assert bad == [[0, 0, 1, 3], [0, 0, 1, 35], [0, 0, 2, 200]]


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_gradients(cuda_device, layout):
    """Against the formula, and against differences of the forward: the map is linear, so a
    central difference has no truncation error and fp32 inputs of unit size and step 1 leave
    the rounding of the two outputs, 8 e (|x1| + |x2|) each with terms below 12."""
    t = rotary.Table(96, layout=layout, scaling="yarn", factor=4.0, original_length=64)
    B, L = 2, 21
    q, k = _x((B, 4, L, 256), torch.float32, 7), _x((B, 2, L, 256), torch.float32, 8)
    dq, dk = _x(q.shape, torch.float32, 9), _x(k.shape, torch.float32, 10)
    qd, kd = q.to(cuda_device).requires_grad_(), k.to(cuda_device).requires_grad_()
    qo, ko = rotary.rotate_autograd(qd, kd, t, pos_offset=50)
    gq, gk = torch.autograd.grad((qo, ko), (qd, kd), (dq.to(cuda_device), dk.to(cuda_device)))
    pos = [50 + np.arange(L)]
    _check(gq, dq, pos, t, sign=-1.0)
    _check(gk, dk, pos, t, sign=-1.0)
    at = lambda x: rotary.rotate(x, None, t, pos_offset=50)[0].double()  # noqa: E731
    for i, c in ((0, 0), (3, 47), (2, 50), (1, 95), (0, 96), (3, 255)):
        step = torch.zeros_like(qd)
        step[1, i, 5, c] = 1.0
        diff = (at(qd.detach() + step) - at(qd.detach() - step)) / 2
        want = float((diff[1, i, 5] * dq[1, i, 5].double().to(cuda_device)).sum())
        assert abs(float(gq[1, i, 5, c]) - want) <= 2 * 8 * E * 12 * 2 * 4


def test_gradients_one_sided_and_expanded(cuda_device):
    t = rotary.Table(64)
    q, k = _x((2, 2, 7, 256), torch.bfloat16, 11), _x((2, 1, 7, 256), torch.bfloat16, 12)
    qd, kd = q.to(cuda_device).requires_grad_(), k.to(cuda_device).requires_grad_()
    qo, ko = rotary.rotate_autograd(qd, kd, t)
    qo.float().sum().backward()  # an expanded gradient; none for k's output
    ones = torch.ones(q.shape, dtype=torch.bfloat16)
    _check(qd.grad, ones, [np.arange(7)], t, sign=-1.0)
    assert kd.grad is None or not kd.grad.any()
    base = _x((1, 2, 7, 256), torch.float32, 13).to(cuda_device).requires_grad_()
    out, _ = rotary.rotate_autograd(base.expand(3, 2, 7, 256), None, t)  # a broadcast input sums its gradients
    out.backward(torch.ones_like(out))
    one = decode.rotate(np.ones((1, 2, 7, 256)), [np.arange(7)], t.inv_freq, sign=-1.0)
    assert np.abs(base.grad.double().cpu().numpy() - 3 * one).max() <= 3 * (8 + 2) * E * 2


def test_streams_and_graphs(cuda_device):
    t = rotary.Table(256, device=cuda_device)
    q = _x((2, 4, 300, 256), torch.bfloat16, 14).to(cuda_device)
    pos = torch.arange(300, dtype=torch.int32, device=cuda_device)
    want, _ = rotary.rotate(q, None, t, positions=pos)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got, _ = rotary.rotate(q, None, t, positions=pos, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    out = torch.empty_like(q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        rotary.rotate(q, None, t, positions=pos, out=out)
    pos.add_(7)
    g.replay()
    want, _ = rotary.rotate(q, None, t, pos_offset=7)
    assert torch.equal(out, want)


def test_refusals(cuda_device):
    t = rotary.Table(64)
    q = torch.zeros(2, 3, 8, 256, device=cuda_device)
    ids = torch.zeros(8, dtype=torch.int32, device=cuda_device)
    bad = [dict(positions=ids.long()), dict(positions=ids[:7]), dict(positions=ids.cpu()),
           dict(positions=ids, pos_offset=3), dict(out=torch.empty_like(q, dtype=torch.bfloat16)),
           dict(out=torch.empty(2, 3, 9, 256, device=cuda_device)), dict(out=q[:1].expand(2, 3, 8, 256)),
           dict(out_k=q)]
    for kw in bad:
        with pytest.raises(ValueError):
            rotary.rotate(q, None, t, **kw)
    for x in (q.half(), q[..., :128], q.transpose(2, 3), q[0]):
        with pytest.raises(ValueError):
            rotary.rotate(x, None, t)
    with pytest.raises(ValueError):
        rotary.rotate(q, q[:, :, :4], t)
    from long_context_causal_flash_b200 import GqaAttnError

    raw = torch.zeros(2 * 3 * 8 * 256 + 1, device=cuda_device)
    with pytest.raises(GqaAttnError):
        rotary.rotate(raw[1:].view(2, 3, 8, 256), None, t)


def test_second_derivatives(cuda_device):
    """The rotation is linear: the gradient's own gradient is the rotation, to any order."""
    t = rotary.Table(96, layout="interleaved", scaling="yarn", factor=4.0, original_length=64)
    q, k = _x((2, 3, 9, 256), torch.float32, 20), _x((2, 1, 9, 256), torch.float32, 21)
    dq, dk, uq, uk = (_x(x.shape, torch.float32, 22 + i) for i, x in enumerate((q, k, q, k)))
    qd, kd, dqd, dkd = (x.to(cuda_device).requires_grad_() for x in (q, k, dq, dk))
    pos = torch.tensor([[3, 900_000, 7, 0, 1, 2, 5, 9, 8]] * 2, dtype=torch.int32, device=cuda_device)
    out = rotary.rotate_autograd(qd, kd, t, positions=pos)
    gq, gk = torch.autograd.grad(out, (qd, kd), (dqd, dkd), create_graph=True)
    hq, hk = torch.autograd.grad((gq, gk), (dqd, dkd), (uq.to(cuda_device), uk.to(cuda_device)), create_graph=True)
    _check(gq.detach(), dq, pos.cpu().numpy(), t, sign=-1.0)
    _check(hq.detach(), uq, pos.cpu().numpy(), t)
    _check(hk.detach(), uk, pos.cpu().numpy(), t)
    # a penalty on the gradient's size, as a user writes it: d / dq of |dL / dq|^2 / 2 with L = |rotated q|^2 / 2
    m = t.magnitude
    out, _ = rotary.rotate_autograd(qd, None, t, positions=pos)
    (g,) = torch.autograd.grad(0.5 * out.square().sum(), qd, create_graph=True)
    (p,) = torch.autograd.grad(0.5 * g.square().sum(), qd)
    want = q.double().numpy().copy()
    want[..., :96] *= m ** 4  # turned and turned back twice, by m each time
    # four rotations, each off by 8 e m (|x1| + |x2|) (see the module's head), of pairs whose terms are below 12 m^3
    assert np.abs(p.double().cpu().numpy() - want).max() <= 4 * 8 * E * m * 24 * m ** 3


def test_gradients_that_nobody_asked_for_are_not_computed(cuda_device, monkeypatch):
    t = rotary.Table(64, device=cuda_device)
    q, k = (_x((2, h, 7, 256), torch.bfloat16, 30 + h).to(cuda_device) for h in (2, 1))
    turned = []
    real = rotary.rotate
    monkeypatch.setattr(rotary, "rotate", lambda a, b, *args, **kw: (turned.append((a is not None, b is not None)),
                                                                     real(a, b, *args, **kw))[1])

    def back(need_q, need_k, loss):
        qd, kd = q.clone().requires_grad_(need_q), k.clone().requires_grad_(need_k)
        qo, ko = rotary.rotate_autograd(qd, kd, t)
        turned.clear()
        loss(qo, ko).backward()
        return qd.grad, kd.grad

    both = lambda qo, ko: qo.float().square().sum() + ko.float().square().sum()  # noqa: E731
    gq, gk = back(True, False, both)
    assert turned == [(True, False)] and gk is None
    alone, _ = back(True, True, lambda qo, ko: qo.float().square().sum())
    assert turned == [(True, False)] and torch.equal(alone, gq)
    _, gk = back(True, True, lambda qo, ko: ko.float().square().sum())
    assert turned == [(True, False)] and gk is not None  # k's gradient alone, as the launch's first tensor
    gq2, gk2 = back(True, True, both)
    assert turned == [(True, True)] and torch.equal(gq2, gq) and torch.equal(gk2, gk)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gradients_off_their_alignment(cuda_device, dtype):
    """A gradient that starts anywhere in memory, as that of a tensor that was concatenated does."""
    t = rotary.Table(64, device=cuda_device)
    q = _x((2, 2, 7, 256), dtype, 33)
    w = _x((q.numel() + 1,), dtype, 34).to(cuda_device)
    qd = q.to(cuda_device).requires_grad_()
    out, _ = rotary.rotate_autograd(qd, None, t)
    head = torch.zeros(1, dtype=dtype, device=cuda_device, requires_grad=True)
    torch.cat((head, out.reshape(-1))).backward(w)
    _check(qd.grad, w[1:].view(q.shape).cpu(), [np.arange(7)], t, sign=-1.0)
