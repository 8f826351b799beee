"""Inputs and tolerances of the rotary and paged-cache tests.

Tolerances, elementwise, u = half a step of the output type (bf16 2^-8,
fp16 2^-11), t the smallest fp16 half step 2^-25:

* rotated values: the sine and cosine are within 2^-22 (sincospif, two units)
  plus the angle's own error (fp64 turns: |pos| f 2^-51; their fp32 rounding:
  2^-23 rad), the products and the sum round to fp32: with amp (|a| + |b|) the
  size of the pair, |y - ref| <= u |ref| + t + (2^-20 + |pos| f 2^-51) amp (|a| + |b|).
* decode: a score is off by at most e_s = (D + 8) 2^-24 size (fp32 sums of exact
  products; size = scale * sum |q_i k_i|) + 2^-22 |s|, an exponential by 2^-22
  relative, a weight by u more when rounded for the product, its normaliser
  likewise: |O - ref| <= u |ref| + t + (2 u + 2 (2 e_s + 2^-21)) mean|V|, and
  |LSE - ref| <= 2 e_s + 2^-20 + 2^-22 |ref|, e_s with |s| <= size.
"""
import numpy as np
import torch

from exact_tiled_attention_31_b200.inputs import torch_dtype
from oracle import paged as op

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = 2.0 ** -25


def f64(t):
    return t.detach().double().cpu().numpy()


def check_rotated(y, x, positions, freqs, interleaved, amp, backward, what):
    """y (GPU result) against x turned by positions [..., T], x [..., T, D]."""
    ref = op.rotate(x, positions, freqs, interleaved, amp, backward)
    R = 2 * len(freqs)
    size = np.zeros_like(ref)
    first, second = (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, R // 2), slice(R // 2, R))
    x = f64(x)
    pair = abs(amp) * (np.abs(x[..., first]) + np.abs(x[..., second]))
    ang = 2.0 ** -20 + np.abs(np.asarray(positions, dtype=np.float64))[..., None] * np.abs(freqs) * 2.0 ** -51
    size[..., first] = size[..., second] = pair * ang
    u = U[y.dtype]
    err, tol = np.abs(f64(y) - ref), u * np.abs(ref) + TINY + size
    assert np.isfinite(f64(y)).all(), what
    bad = np.unravel_index((err - tol).argmax(), err.shape)
    assert (err <= tol).all(), f"{what}: {f64(y)[bad]} vs {ref[bad]} (tolerance {tol[bad]:.3g}) at {bad}"
    # the columns that are not rotated are copied
    assert np.array_equal(f64(y)[..., R:], x[..., R:]), what


def check_decode(o, lse, q, ref, what):
    ro, rl, mean_v, size = ref
    D, u = q.shape[-1], U[o.dtype]
    e_s = ((D + 8) * 2.0 ** -24 + 2.0 ** -22) * size
    go, gl = f64(o), f64(lse)
    empty = np.isneginf(rl)
    assert (go[empty] == 0).all() and np.isneginf(gl[empty]).all(), f"{what}: empty rows"
    assert np.isfinite(go).all() and np.isfinite(gl[~empty]).all(), f"{what}: non-finite"
    err, tol = np.abs(go - ro), u * np.abs(ro) + TINY + (2 * u + 2 * (2 * e_s[..., None] + 2.0 ** -21)) * mean_v
    bad = np.unravel_index((err - tol).argmax(), err.shape)
    assert (err <= tol).all(), f"{what}: O {go[bad]} vs {ro[bad]} (tolerance {tol[bad]:.3g}) at {bad}"
    err = np.abs(np.where(empty, 0, gl) - np.where(empty, 0, rl))
    tol = 2 * e_s + 2.0 ** -20 + 2.0 ** -22 * np.abs(np.where(empty, 0, rl))
    bad = np.unravel_index((err - tol).argmax(), err.shape)
    assert (err <= tol).all(), f"{what}: LSE {gl[bad]} vs {rl[bad]} (tolerance {tol[bad]:.3g}) at {bad}"


def freqs_of(R, base=10000.0):
    return base ** (-np.arange(R // 2) * 2.0 / R)


def randn(gen, dtype, *shape):
    return torch.randn(*shape, generator=gen).to(torch_dtype(dtype))


def make_cache(gen, lens, Hkv, D, page, dtype, shared=0, spare=2, poison=True, interleaved=False):
    """Pools and a table for sequences of these lengths: pages in no order, the
    first `shared` pages the same for all; entries past a length -1 and rows
    past a length NaN (pages of no sequence too) when `poison`."""
    need = [max(-(-int(n) // page), shared) for n in lens]
    n_pages = shared + sum(n - shared for n in need) + spare
    ids = torch.randperm(n_pages, generator=gen).to(torch.int32)
    table = torch.full((len(lens), max(max(need), 1)), -1, dtype=torch.int32)
    at = shared
    for b, n in enumerate(need):
        table[b, :shared] = ids[:shared]
        table[b, shared:n] = ids[at:at + n - shared]
        at += n - shared
    pools = [randn(gen, dtype, n_pages, Hkv, page, D) for _ in range(2)]
    if poison:
        live = torch.zeros(n_pages, page, dtype=torch.bool)
        for b, n in enumerate(lens):
            for i in range(int(n)):
                live[table[b, i // page], i % page] = True
        live[ids[:shared].long()] = True
        for x in pools:
            x.masked_fill_(~live[:, None, :, None], float("nan"))
    if interleaved:  # one allocation [n_pages, 2, Hkv, page, D]
        both = torch.stack(pools, 1)
        pools = [both[:, 0], both[:, 1]]
    return pools[0], pools[1], table
