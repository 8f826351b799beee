"""CPU-side checks of the rotary and paged entry points: sizes, frequencies,
and refusals before anything touches a device; the oracle's own pins."""
import ctypes
import math

import numpy as np
import pytest
import torch

import exact_tiled_attention_31_b200 as fa
from exact_tiled_attention_31_b200 import api, build
from oracle import paged as op

E, U, OK = api.FA_ERR_INVALID_ARG, api.FA_ERR_UNSUPPORTED, api.FA_OK
A = 1 << 20  # a 16-byte aligned address that is never dereferenced


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build_library()
    return fa.load_library()


def rows(data=A, batch=0, head=1280, row=128, heads=2):
    return api._ROWS.pack(data, batch, head, row, heads)


def pages(k=A, v=A, stride=2 * 64 * 128, table=A, row=10, n=100, page=64, heads=2, most=10):
    return api._PAGES.pack(k, v, stride, table, row, n, page, heads, most)


# ---------------------------------------------------------------- frequencies

def _freqs(rot, **kw):
    f, amp = fa.rope_freqs(rot, device="cpu", **kw)
    assert f.dtype == torch.float64 and f.shape == (rot // 2,)
    return f.numpy(), amp


def test_frequencies_against_their_formulas():
    i = np.arange(32)
    plain, amp = _freqs(64)
    assert amp == 1.0 and np.allclose(plain, 10000.0 ** (-i / 32), rtol=1e-15, atol=0)
    lin, amp = _freqs(64, scaling="linear", factor=8.0)
    assert amp == 1.0 and np.allclose(lin, plain / 8, rtol=1e-15, atol=0)
    ntk, _ = _freqs(64, scaling="ntk", factor=4.0, base=500.0)
    assert np.allclose(ntk, (500.0 * 4.0 ** (64 / 62)) ** (-i / 32), rtol=1e-14, atol=0)
    # the last pair's wavelength grows by the factor exactly: that is what the larger base is for
    assert math.isclose(ntk[-1], 500.0 ** (-31 / 32) / 4.0, rel_tol=1e-13)


def test_yarn_keeps_fast_pairs_and_interpolates_slow_ones():
    f, amp = _freqs(128, scaling="yarn", factor=4.0, original_len=4096)
    plain, _ = _freqs(128)
    assert math.isclose(amp, 0.1 * math.log(4.0) + 1.0, rel_tol=1e-6)
    turns = 4096 * plain / (2 * math.pi)
    ratio = f / plain
    assert np.all(np.diff(ratio) <= 1e-15) and ratio[0] == 1.0 and math.isclose(ratio[-1], 0.25, rel_tol=1e-12)
    # one pair of slack: the ramp's ends are rounded outwards
    assert np.all(ratio[:-1][turns[1:] > 32] == 1.0) and np.allclose(ratio[1:][turns[:-1] < 1], 0.25)


def test_frequency_refusals():
    out, amp = (ctypes.c_double * 64)(), ctypes.c_float()
    call = lambda rot=64, base=10000.0, s=0, factor=1.0, n=0, bf=32.0, bs=1.0, o=out: fa.fa_rope_freqs(
        rot, base, s, factor, n, bf, bs, o, ctypes.byref(amp))
    assert call() == OK
    for bad in (dict(rot=0), dict(rot=7), dict(rot=-2), dict(base=1.0), dict(base=float("nan")), dict(s=9),
                dict(s=1, factor=0.5), dict(s=1, factor=float("inf")), dict(s=2, rot=2, factor=2.0),
                dict(s=3, factor=2.0), dict(s=3, factor=2.0, n=4096, bf=1.0, bs=2.0),
                dict(s=3, factor=2.0, n=4096, bs=0.0), dict(o=None)):
        assert call(**bad) == E, bad
    with pytest.raises(fa.FAError):
        fa.rope_freqs(64, scaling="linear", factor=0.1, device="cpu")
    with pytest.raises(ValueError):
        fa.rope_freqs(64, scaling="other", device="cpu")


# ---------------------------------------------------------------- refusals of the C entries

def test_rope_refusals():
    ok = dict(x=rows(), y=rows(A + (1 << 20)), n=1, f=A, rot=64, amp=1.0, pos=None, ps=0, cu=None, nseq=0, B=0, S=10,
              D=128, dt=0)

    def call(**kw):
        a = {**ok, **kw}
        return fa.fa_rope(a["x"], a["y"], a["n"], a["f"], a["rot"], 0, a["amp"], 0, a["pos"], a["ps"], a["cu"],
                          a["nseq"], a["B"], a["S"], a["D"], a["dt"], None)
    assert call() == OK and call(B=1, S=0) == OK                 # nothing to do
    assert call(cu=A, nseq=0, B=1) == OK
    for bad in (dict(n=0), dict(n=3), dict(amp=float("inf")), dict(amp=float("nan")), dict(B=-1), dict(S=-1),
                dict(dt=5), dict(ps=-1), dict(nseq=-1), dict(x=None), dict(y=None), dict(cu=A, nseq=1, B=2)):
        assert call(**{"B": 1, **bad}) == E, bad
    for bad in (dict(rot=8), dict(rot=24), dict(rot=144), dict(D=96), dict(D=64, rot=80), dict(rot=0)):
        assert call(**bad) == U, bad
    for bad in (dict(f=None), dict(f=A + 4), dict(pos=A + 2), dict(cu=A + 1, nseq=1), dict(x=rows(A + 8)),
                dict(x=rows(0)), dict(x=rows(row=100)), dict(x=rows(head=-8)), dict(x=rows(heads=0)),
                dict(y=rows(heads=3)), dict(y=rows(A + 2))):
        assert call(**{"B": 1, **bad}) == E, bad
    assert call(B=1 << 16, S=1 << 16) == U                       # rows are counted in 32 bits


def test_append_refusals():
    ok = dict(k=rows(), v=rows(), q=None, qo=None, pg=pages(), lens=A, cu=None, nseq=4, total=4, f=A, rot=64, amp=1.0,
              pos=None, D=128, dt=1)

    def call(**kw):
        a = {**ok, **kw}
        return fa.fa_append_paged(a["k"], a["v"], a["q"], a["qo"], a["pg"], a["lens"], a["cu"], a["nseq"], a["total"],
                                  a["f"], a["rot"], 0, a["amp"], a["pos"], a["D"], a["dt"], None)
    assert call(nseq=0, total=0) == OK and call(cu=A, total=0) == OK
    for bad in (dict(nseq=-1, total=-1), dict(dt=2), dict(total=5), dict(amp=float("nan")), dict(lens=None),
                dict(lens=A + 1), dict(cu=A + 2), dict(pos=A + 2), dict(f=A + 4), dict(k=None), dict(v=None),
                dict(k=rows(heads=3)), dict(v=rows(heads=1)), dict(k=rows(row=4)), dict(v=rows(A + 4)),
                dict(q=rows(heads=8)), dict(q=rows(heads=8), qo=rows(heads=4)),
                dict(q=rows(heads=8), qo=rows(heads=8), f=None), dict(pg=None), dict(pg=pages(k=A + 8)),
                dict(pg=pages(v=0)), dict(pg=pages(table=0)), dict(pg=pages(table=A + 2)), dict(pg=pages(n=0)),
                dict(pg=pages(most=0)), dict(pg=pages(heads=0)), dict(pg=pages(page=0)), dict(pg=pages(page=-16)),
                dict(pg=pages(stride=2 * 64 * 128 - 8)), dict(pg=pages(stride=2 * 64 * 128 + 4)),
                dict(pg=pages(row=-1)), dict(pg=pages(n=-1))):
        assert call(**bad) == E, bad
    for bad in (dict(D=96), dict(rot=40), dict(rot=256), dict(pg=pages(page=8, stride=1 << 20)),
                dict(pg=pages(page=48, stride=1 << 20)), dict(pg=pages(page=8192, stride=1 << 30)),
                dict(pg=pages(most=1 << 25)), dict(pg=pages(stride=1 << 39)),
                dict(pg=pages(heads=1 << 19, page=4096, stride=1 << 38), k=rows(heads=1 << 19), v=rows(heads=1 << 19))):
        assert call(**bad) == U, bad


def test_decode_refusals_and_workspace():
    size = fa.fa_decode_paged_workspace_size(4, 8, 2, 128)
    pre = fa.fa_decode_prefix_workspace_size(4, 8, 2, 640, 128)
    assert 0 < size == pre == fa.fa_decode_prefix_workspace_size(4, 8, 2, 0, 128)  # read for each sequence
    # a pass of its own takes fp32 parts of every row besides
    more = fa.fa_decode_prefix_workspace_size(64, 8, 2, 640, 128) - fa.fa_decode_paged_workspace_size(64, 8, 2, 128)
    assert more >= 2 * 64 * 8 * (128 + 1) * 4
    for bad in ((0, 8, 2, 128), (4, 0, 2, 128), (4, 8, 0, 128), (4, 9, 2, 128), (4, 34, 2, 128), (4, 8, 2, 96)):
        assert fa.fa_decode_paged_workspace_size(*bad) == 0, bad
    assert fa.fa_decode_prefix_workspace_size(4, 8, 2, -64, 128) == 0
    ok = dict(q=A, pg=pages(), lens=A, o=A, lse=A, B=4, Hq=8, D=128, scale=0.1, dt=0, ws=A, wsb=pre, P=640, pt=None)

    def both(only=None, **kw):
        a = {**ok, **kw}
        got = []
        if only != "prefix":
            got.append(fa.fa_decode_paged(a["q"], a["pg"], a["lens"], a["o"], a["lse"], a["B"], a["Hq"], a["D"],
                                          a["scale"], a["dt"], a["ws"], a["wsb"], None))
        got.append(fa.fa_decode_prefix(a["q"], a["pg"], a["lens"], a["P"], a["pt"], a["o"], a["lse"], a["B"], a["Hq"],
                                       a["D"], a["scale"], a["dt"], a["ws"], a["wsb"], None))
        return set(got)
    assert both(B=0) == {OK} and both(Hq=0) == {OK}
    for bad in (dict(B=-1), dict(Hq=-8), dict(dt=3), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
                dict(q=0), dict(q=A + 8), dict(o=A + 4), dict(lse=0), dict(lens=None), dict(lens=A + 3), dict(Hq=9),
                dict(ws=None), dict(ws=A + 128), dict(wsb=size - 1), dict(pg=None), dict(pg=pages(n=0)),
                dict(pg=pages(v=A + 2))):
        assert both(**bad) == {E}, bad
    for bad in (dict(D=80), dict(Hq=34), dict(pg=pages(page=24, stride=1 << 20)), dict(B=1 << 29)):
        assert both(**bad) == {U}, bad
    for bad in (dict(P=100), dict(P=-64), dict(P=704), dict(pt=A + 2), dict(wsb=pre - 1)):
        assert both("prefix", **bad) == {E}, bad


def test_decode_refuses_tables_of_too_many_tiles():
    """KV heads x sequences x (tiles of a full table + 2) is counted in 31 bits
    by the kernels.  128 sequences of 2^30 rows sum to 2^31 + 256 for one head,
    which is negative in 32 bits: refused before anything is launched."""
    def status(B, Hkv, prefix):
        pg = pages(stride=Hkv * 4096 * 128, row=1 << 18, page=4096, heads=Hkv, most=1 << 18)
        q, end = (A, pg, A), (A, A, B, Hkv, 128, 0.1, 0, A, 0, None)  # no room: what is not refused ends there
        return fa.fa_decode_paged(*q, *end) if prefix is None else fa.fa_decode_prefix(*q, prefix, None, *end)
    for prefix in (None, 0, 4096):
        for B, Hkv in ((128, 1), (64, 4), (300, 2)):
            assert status(B, Hkv, prefix) == U, (B, Hkv, prefix)
        for B in (127, 1):  # 127 * (2^24 + 2) < 2^31
            assert status(B, 1, prefix) == E, (B, prefix)


# ---------------------------------------------------------------- refusals of the tensor calls

def test_tensor_calls_want_cuda_tensors():
    x = torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16)
    f = torch.ones(32, dtype=torch.float64)
    with pytest.raises(ValueError, match="CUDA"):
        fa.rope(x, None, f)
    t = torch.zeros(1, 4, dtype=torch.int32)
    p = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    n = torch.ones(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        fa.append_paged(x[:, :, 0], x[:, :, 0], p, p, t, n)
    with pytest.raises(ValueError, match="CUDA"):
        fa.decode_paged(x[:, :, 0], p, p, t, n)


# ---------------------------------------------------------------- the oracle

def test_oracle_rotation_pins():
    rng = np.random.default_rng(0)
    x = rng.normal(size=(3, 7, 64))
    f = 10000.0 ** (-np.arange(16) / 16)
    pos = np.array([0, 1, 5, 1 << 20, (1 << 31) - 1, -3, 77])
    for inter in (False, True):
        y = op.rotate(x, pos, f, inter, amp=1.5)
        assert np.array_equal(y[..., 32:], x[..., 32:])
        assert np.allclose(y[:, 0, :32], 1.5 * x[:, 0, :32], atol=1e-14)              # position 0: the amplitude alone
        assert np.allclose((y[..., :32] ** 2).sum(-1), 2.25 * (x[..., :32] ** 2).sum(-1))
        back = op.rotate(y, pos, f, inter, amp=1 / 1.5, backward=True)
        assert np.allclose(back, x, atol=1e-12)
        # one pair by hand
        a, b = (0, 1) if inter else (0, 16)
        c, s = math.cos(5.0), math.sin(5.0)
        assert np.allclose(y[0, 2, a], 1.5 * (x[0, 2, a] * c - x[0, 2, b] * s))
        assert np.allclose(y[0, 2, b], 1.5 * (x[0, 2, b] * c + x[0, 2, a] * s))
    # scores depend on the distance alone
    q, k = rng.normal(size=(1, 1, 32)), rng.normal(size=(1, 1, 32))
    dot = lambda i, j: float((op.rotate(q, [i], f) * op.rotate(k, [j], f)).sum())
    assert math.isclose(dot(10, 3), dot(1 << 30, (1 << 30) - 7), rel_tol=1e-9)
    # the gradient is the transposed map: central differences of sum(w * rotate(x))
    w = rng.normal(size=x.shape)
    g = op.rotate(w, pos, f, False, 1.5, backward=True)
    for at in [(0, 2, 3), (1, 4, 20), (2, 6, 40)]:
        d = np.zeros_like(x)
        d[at] = 1e-6
        diff = ((op.rotate(x + d, pos, f, False, 1.5) - op.rotate(x - d, pos, f, False, 1.5)) * w).sum() / 2e-6
        assert abs(diff - g[at]) < 1e-7


def test_oracle_paged_decode_is_decode():
    from oracle import attention as oa
    rng = np.random.default_rng(1)
    B, Hq, Hkv, L, D, page = 2, 4, 2, 40, 16, 8
    q = rng.normal(size=(B, Hq, D))
    k, v = rng.normal(size=(B, Hkv, L, D)), rng.normal(size=(B, Hkv, L, D))
    table = rng.permutation(B * L // page).reshape(B, -1)
    pools = []
    for x in (k, v):
        pool = np.zeros((B * L // page, Hkv, page, D))
        for b in range(B):
            for i in range(L):
                pool[table[b, i // page], :, i % page] = x[b, :, i]
        pools.append(pool)
    o, lse, _, _ = op.decode_paged(q, *pools, table, [40, 13], 0.25)
    ro, rl = oa.decode_forward(q, k, v, np.array([40, 13]), 0.25)
    assert np.allclose(o, ro) and np.allclose(lse, rl)
    o, lse, _, _ = op.decode_paged(q, *pools, table, [0, 1], 0.25)
    assert (o[0] == 0).all() and np.isneginf(lse[0]).all() and np.allclose(o[1], np.repeat(v[1, :, 0], 2, axis=0))


# ---------------------------------------------------------------- how the work is cut

def _cut(B, Hkv, lens, start, grid, claim):
    """The runs that the kernel makes of a call (PagedRuns and the walk over
    them), in Python: every tile in one run, every part in one slot, and every
    cut unit's first and last run those that hold its parts."""
    KT, unit_cost, min_run, claim_tiles = 64, 2, 4, 48
    tiles = [max(1, -(-(n - start) // KT)) if n > start else 1 for n in lens]
    cost = np.concatenate([[0], np.cumsum([t + unit_cost for t in tiles])])
    total, units = int(cost[-1]) * Hkv, B * Hkv
    runs, waves = min(grid, max(units, total // min_run)), 1
    if claim and total // grid >= claim_tiles:
        waves, runs = 3, 3 * grid
    share = [0, 208, 240]

    def begin(c):
        if waves == 1:
            return c * total // runs
        step = total // grid * 256 + total % grid * 256 // grid  # of a 256th of a stretch, in 65536ths
        return total if c >= runs else (c // waves * 256 + share[c % waves]) * step >> 16

    def of(x):
        return max(c for c in range(runs) if begin(c) <= x)
    assert begin(runs) == total
    if waves > 1:
        assert sorted(i % grid * waves + i // grid for i in range(runs)) == list(range(runs))
    seen, slots, cuts = set(), {}, []
    for c in range(runs):
        t0, t1 = begin(c), begin(c + 1)
        b = int(np.searchsorted(cost * Hkv, t0, side="right")) - 1
        one = tiles[b] + unit_cost
        kvh, off = divmod(t0 - int(cost[b]) * Hkv, one)
        tile, left = max(0, off - unit_cost), t1 - t0 - max(0, unit_cost - off)
        while left > 0:
            n = min(tiles[b] - tile, left)
            for i in range(n):
                assert (b, kvh, tile + i) not in seen
                seen.add((b, kvh, tile + i))
            begins, ends = tile == 0, tile + n == tiles[b]
            if not (begins and ends):
                slot = 2 * c + begins
                assert slot not in slots
                slots[slot] = (b, kvh, n)
            if begins and not ends:
                cuts.append((b, kvh, c, of(t1 + tiles[b] - tile - n - 1)))
            left -= n + unit_cost
            tile = 0
            kvh += 1
            if kvh == Hkv:
                b, kvh = b + 1, 0
    assert len(seen) == Hkv * sum(tiles)
    used = set()
    for b, kvh, first, last in cuts:
        assert first < last < runs
        parts = [2 * first + 1] + [2 * c for c in range(first + 1, last + 1)]
        assert all(slots[s][:2] == (b, kvh) for s in parts) and sum(slots[s][2] for s in parts) == tiles[b]
        used.update(parts)
    assert used == set(slots)


@pytest.mark.parametrize("claim", [False, True])
def test_every_tile_is_in_one_run(claim):
    import random
    r = random.Random(5)
    for _ in range(60):
        B, Hkv = r.choice([1, 2, 3, 7, 64, 129]), r.choice([1, 2, 3, 8])
        most = r.choice([1, 64, 65, 300, 5000, 40000])
        lens = [r.choice([0, 1, most, r.randint(0, most)]) for _ in range(B)]
        _cut(B, Hkv, lens, r.choice([0, 64, 512]), r.choice([296, 5]), claim)
