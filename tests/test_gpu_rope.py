"""Rotary positions on the GPU: rope / rope_backward against the fp64 oracle."""
import numpy as np
import pytest
import torch

import exact_tiled_attention_31_b200 as fa
from paged_helpers import check_rotated, f64, freqs_of, randn
from oracle import paged as op

pytestmark = pytest.mark.gpu


def _call(dev, q, k, freqs, **kw):
    fn = fa.rope_backward if kw.pop("backward", False) else fa.rope
    out = fn(q, k, torch.from_numpy(freqs).to(dev), **kw)
    fa.check_device_error()
    return out


@pytest.mark.parametrize("D,R", [(64, 64), (64, 16), (64, 48), (128, 128), (128, 32), (128, 112)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype,backward", [("bf16", False), ("fp16", True)])
def test_dense(cuda_device, D, R, interleaved, dtype, backward):
    gen = torch.Generator().manual_seed(D + R)
    B, Hq, Hkv, S = 2, 5, 2, 37
    q, k = randn(gen, dtype, B, Hq, S, D), randn(gen, dtype, B, Hkv, S, D)
    freqs, amp = freqs_of(R), 1.25
    yq, yk = _call(cuda_device, q.to(cuda_device), k.to(cuda_device), freqs, interleaved=interleaved, amp=amp,
                   backward=backward)
    for y, x in ((yq, q), (yk, k)):
        assert y.is_contiguous()
        check_rotated(y, x, np.arange(S), freqs, interleaved, amp, backward, f"D{D} R{R}")


@pytest.mark.parametrize("B,Hq,Hkv,S", [(1, 1, 1, 1), (3, 1, 1, 1), (1, 32, 8, 1), (2, 16, 1, 33), (1, 3, 3, 1000),
                                        (70, 4, 2, 5)])
def test_sizes_and_no_k(cuda_device, B, Hq, Hkv, S):
    gen = torch.Generator().manual_seed(S)
    q, k = randn(gen, "bf16", B, Hq, S, 128), randn(gen, "bf16", B, Hkv, S, 128)
    freqs = freqs_of(128)
    yq, yk = _call(cuda_device, q.to(cuda_device), k.to(cuda_device), freqs)
    check_rotated(yq, q, np.arange(S), freqs, False, 1.0, False, "q")
    check_rotated(yk, k, np.arange(S), freqs, False, 1.0, False, "k")
    only, none = _call(cuda_device, q.to(cuda_device), None, freqs)
    assert none is None and torch.equal(only, yq)


@pytest.mark.parametrize("interleaved", [False, True])
def test_views_in_place_and_positions(cuda_device, interleaved):
    """q, k, v as one projection leaves them, [B, S, H, D] interleaved; positions
    per batch row, shared, and far out in both directions; in place."""
    gen = torch.Generator().manual_seed(3)
    B, S, Hq, Hkv, D = 3, 29, 6, 2, 64
    both = randn(gen, "fp16", B, S, Hq + 2 * Hkv, D)
    dev = both.to(cuda_device)
    q, k = both[:, :, :Hq].transpose(1, 2), both[:, :, Hq:Hq + Hkv].transpose(1, 2)
    gq, gk = dev[:, :, :Hq].transpose(1, 2), dev[:, :, Hq:Hq + Hkv].transpose(1, 2)
    freqs = freqs_of(32)
    pos = torch.randint(-(1 << 31), (1 << 31) - 1, (B, S), generator=gen).to(torch.int32)
    yq, yk = _call(cuda_device, gq, gk, freqs, positions=pos.to(cuda_device), interleaved=interleaved)
    p = pos.numpy()[:, None].astype(np.int64)
    check_rotated(yq, q, p, freqs, interleaved, 1.0, False, "far q")
    check_rotated(yk, k, p, freqs, interleaved, 1.0, False, "far k")
    shared = (torch.arange(S, dtype=torch.int32) + 100000).to(cuda_device)
    for form in (shared, shared[None]):
        zq, _ = _call(cuda_device, gq, gk, freqs, positions=form, interleaved=interleaved)
        check_rotated(zq, q, shared.cpu().numpy(), freqs, interleaved, 1.0, False, "shared positions")
    rest = dev[:, :, Hq + Hkv:].clone()
    oq, ok = _call(cuda_device, gq, gk, freqs, positions=shared, interleaved=interleaved, out=(gq, gk))
    assert oq is gq and ok is gk and torch.equal(oq, zq) and torch.equal(dev[:, :, Hq + Hkv:], rest)
    wide = q[:1].to(cuda_device).expand(B, Hq, S, D)  # one row of the batch, broadcast
    ye, _ = _call(cuda_device, wide, None, freqs, positions=shared)
    assert torch.equal(ye[0], ye[B - 1]) and ye.is_contiguous()


@pytest.mark.parametrize("lens,tail", [([1], 0), ([5, 0, 300, 1, 64], 0), ([0, 17, 0], 9), ([2] * 200, 3)])
def test_packed(cuda_device, lens, tail):
    gen = torch.Generator().manual_seed(len(lens))
    T = sum(lens) + tail
    q, k = randn(gen, "bf16", 3, T, 64), randn(gen, "bf16", 1, T, 64)
    cu = np.concatenate([[0], np.cumsum(lens)])
    freqs = freqs_of(64)
    out = tuple(torch.full_like(x, 7.0).to(cuda_device) for x in (q, k))
    cu_dev = torch.tensor(cu, dtype=torch.int32, device=cuda_device)
    _call(cuda_device, q.to(cuda_device), k.to(cuda_device), freqs, cu_seqlens=cu_dev, out=out)
    pos, n = op.packed_positions(cu, T), sum(lens)
    for y, x in zip(out, (q, k)):
        check_rotated(y[:, :n], x[:, :n], pos[:n], freqs, False, 1.0, False, "packed")
        assert (y[:, n:] == 7.0).all()  # rows behind the last sequence
    given = torch.arange(T, dtype=torch.int32, device=cuda_device) + 11
    y, _ = _call(cuda_device, q.to(cuda_device), None, freqs, positions=given)
    check_rotated(y, q, np.arange(T) + 11, freqs, False, 1.0, False, "packed, given positions")


def test_backward_is_the_transpose(cuda_device):
    """<dy, rope(x)> = <rope_backward(dy), x>, and turning back undoes the turn."""
    gen = torch.Generator().manual_seed(9)
    x, dy = (randn(gen, "fp16", 1, 4, 50, 128).to(cuda_device) for _ in range(2))
    freqs, amp = fa.rope_freqs(96, scaling="yarn", factor=4.0, original_len=4096, device=cuda_device)
    kw = dict(amp=amp, interleaved=True)
    y, _ = fa.rope(x, None, freqs, **kw)
    dx, _ = fa.rope_backward(dy, None, freqs, **kw)
    a, b = (y.double() * dy.double()).sum(), (dx.double() * x.double()).sum()
    # both roundings: 2^-11 of each product
    size = 2.0 ** -11 * ((y.double() * dy.double()).abs().sum() + (dx.double() * x.double()).abs().sum())
    assert abs(float(a - b)) <= float(size)
    back, _ = fa.rope_backward(y, None, freqs, **kw)
    n = 96
    want = f64(x).copy()
    want[..., :n] *= amp * amp
    # y is rounded once (2^-11 of each of the pair's values), the way back once more
    err = np.abs(f64(back) - want)
    assert err.max() <= 2.0 ** -11 * (3 * 2 * amp * amp * np.abs(f64(x)).max())


def test_rope_then_attention_gradient(cuda_device):
    """dq of sum(dO * attention(rope(q), rope(k), v)) through rope_backward,
    against the fp64 formula and its central differences."""
    from oracle import attention as oa
    gen = torch.Generator().manual_seed(1)
    S, D = 40, 64
    q, k, v, do = (randn(gen, "fp16", 1, 2, S, D) for _ in range(4))
    freqs = freqs_of(32)
    F = torch.from_numpy(freqs).to(cuda_device)
    g = [x.to(cuda_device) for x in (q, k, v, do)]
    rq, rk = fa.rope(g[0], g[1], F)
    o, lse = fa.forward(rq, rk, g[2], True)
    dq, dk, _ = fa.backward(rq, rk, g[2], o, g[3], lse, True)
    dq, dk = fa.rope_backward(dq, dk, F)
    fa.check_device_error()
    pos, scale = np.arange(S), D ** -0.5

    def loss(qq, kk):
        a, b = op.rotate(qq, pos, freqs), op.rotate(kk, pos, freqs)
        return (oa.attention_forward(a, b, f64(v), scale, True)[0] * f64(do)).sum()

    gq, gk, _ = oa.attention_backward(op.rotate(q, pos, freqs), op.rotate(k, pos, freqs), f64(v), f64(do), scale, True)
    ref = [op.rotate(x, pos, freqs, backward=True) for x in (gq, gk)]
    for got, want in zip((dq, dk), ref):  # the attention gradients' own bound
        assert np.abs(f64(got) - want).max() <= 2e-2 * np.abs(want).max()
    h = 1e-5
    for i, want in enumerate(ref):
        for at in [(0, 0, 3, 5), (0, 1, 17, 20), (0, 0, 39, 60)]:
            ends = []
            for sign in (1, -1):
                xs = [f64(q).copy(), f64(k).copy()]
                xs[i][at] += sign * h
                ends.append(loss(*xs))
            assert abs((ends[0] - ends[1]) / (2 * h) - want[at]) <= 1e-6 * (1 + abs(want[at]))
