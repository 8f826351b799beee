"""CPU-side refusals of the rotary and paged entry points, beside those of
test_paged_abi.py: nothing here touches a device."""
import pytest

import exact_tiled_attention_31_b200 as fa
from exact_tiled_attention_31_b200 import api, build

E, U, OK = api.FA_ERR_INVALID_ARG, api.FA_ERR_UNSUPPORTED, api.FA_OK
A = 1 << 20  # a 16-byte aligned address that is never dereferenced


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build_library()
    return fa.load_library()


def rows(data=A, batch=0, head=1280, row=128, heads=2):
    return api._ROWS.pack(data, batch, head, row, heads)


def pages(k=A, v=A + (1 << 30), stride=2 * 64 * 128, table=A, row=10, n=100, page=64, heads=2, most=10):
    return api._PAGES.pack(k, v, stride, table, row, n, page, heads, most)


def test_fill_entries_refuse_what_the_plain_ones_refuse():
    for call in (fa.fa_rope, fa.fa_rope_fill):
        def status(x=rows(), y=rows(A + (1 << 20)), n=1, f=A, rot=64, amp=1.0, cu=None, nseq=0, B=1, S=10, D=128, dt=0):
            return call(x, y, n, f, rot, 0, amp, 0, None, 0, cu, nseq, B, S, D, dt, None)
        assert status(B=0) == OK and status(S=0, cu=A, nseq=0) == OK
        for bad in (dict(n=3), dict(amp=float("nan")), dict(S=-1), dict(dt=2), dict(cu=A, nseq=-1), dict(cu=A, nseq=1, B=2),
                    dict(f=None), dict(x=rows(0)), dict(y=rows(heads=3)), dict(cu=A + 2, nseq=1)):
            assert status(**bad) == E, (call, bad)
        assert status(rot=8) == U and status(D=96) == U and status(B=1 << 16, S=1 << 16) == U
    for call in (fa.fa_append_paged, fa.fa_append_paged_fill):
        def status(k=rows(), v=rows(), q=None, qo=None, pg=pages(), lens=A, cu=None, nseq=4, total=4, f=A, rot=64, D=128):
            return call(k, v, q, qo, pg, lens, cu, nseq, total, f, rot, 0, 1.0, None, D, 0, None)
        assert status(nseq=0, total=0) == OK and status(cu=A, total=0) == OK
        for bad in (dict(total=5), dict(lens=None), dict(k=rows(heads=3)), dict(q=rows(heads=8)),
                    dict(q=rows(heads=8), qo=rows(heads=8), f=None), dict(pg=pages(n=0))):
            assert status(**bad) == E, (call, bad)
        assert status(D=96) == U and status(rot=40) == U
    # with no sequences the queries' rows are still written: their rows have to be valid
    bad = dict(pages=pages(), seq_lens=None, cu_seqlens=A, nseq=0, total=4, freqs=A, rot_dim=64, interleaved=0, amp=1.0,
               positions=None, D=128, dt=0, stream=None)
    assert fa.fa_append_paged(rows(), rows(), rows(), None, **bad) == OK
    assert fa.fa_append_paged_fill(rows(), rows(), rows(), None, **bad) == E


# ---------------------------------------------------------------- overlaps

def _hit(call):
    """Whether the call is refused.  What is not refused goes on to its launch, which fails here without a device."""
    st = call()
    assert st in (E, api.FA_ERR_CUDA), st
    return st == E


def _rope(x, y, B, S, D=64):
    return lambda: fa.fa_rope(b"".join(x), b"".join(y), len(x), A, 64, 0, 1.0, 0, None, 0, None, 0, B, S, D, 0, None)


def _places(r, B, S, D):
    import numpy as np
    data, batch, head, row, heads = api._ROWS.unpack(r)
    at = data // 2 + np.add.outer(np.add.outer(np.add.outer(np.arange(B) * batch, np.arange(heads) * head),
                                               np.arange(S) * row), np.arange(D))
    return at.ravel()


def _expected(x, y, B, S, D=64):
    """By listing the elements: an output over itself, another output, or an input that it is not in place of."""
    outs, ins = [_places(r, B, S, D) for r in y], [_places(r, B, S, D) for r in x]
    if any(len(set(o)) < len(o) for o in outs):
        return True
    sets = [set(o) for o in outs]
    for i, o in enumerate(sets):
        for j in range(len(x)):
            if not (i == j and (outs[i] == ins[j]).all()) and o & set(ins[j]):
                return True
    return len(y) == 2 and bool(sets[0] & sets[1])


@pytest.mark.skipif(__import__("torch").cuda.is_available(), reason="addresses that no launch may see")
def test_rope_overlaps_against_a_list_of_elements():
    import random
    rng = random.Random(11)
    D, seen = 64, {True: 0, False: 0}
    for _ in range(1500):
        B, S, hq, hk = rng.choice([1, 2, 3]), rng.choice([1, 2, 5]), rng.choice([1, 2, 4]), rng.choice([1, 2])
        x, y = [], []
        n = rng.choice([1, 2])
        kind = rng.choice(["fused", "fused", "arena", "any"])
        for i, h in enumerate((hq, hk)[:n]):
            both = []
            for _ in range(2):
                if kind == "fused":    # [B, S, 8 heads, D], some heads of it
                    at, st = 64 * rng.randrange(0, 9 - h), (S * 8 * 64, 64, 8 * 64)
                elif kind == "arena":  # a region of heads by rows or of rows by heads in each batch's 2048
                    at, st = 64 * rng.choice([0, 2, 5, 10, 16, 20]), (2048, *rng.choice([(S * 64, 64), (64, h * 64)]))
                else:
                    at, st = 8 * rng.randrange(0, 60), tuple(8 * rng.choice([0, 1, 4, 8, 9, 16, 24, 40, 72]) for _ in range(3))
                both.append(rows(A + 2 * at + (0 if rng.random() < 0.6 else 1 << 16), *st, h))
            x.append(both[0])
            y.append(both[0] if rng.random() < 0.4 else both[1])
        want = _expected(x, y, B, S)
        assert _hit(_rope(x, y, B, S)) == want, (kind, B, S, [api._ROWS.unpack(r) for r in x + y])
        seen[want] += 1
    assert min(seen.values()) > 300, seen


@pytest.mark.skipif(__import__("torch").cuda.is_available(), reason="addresses that no launch may see")
def test_rope_overlaps_of_large_buffers():
    """A fused projection of 4 x 8192 tokens, in place: no overlap, found without a walk over its rows."""
    import time
    B, S, H = 4, 8192, 48
    part = lambda first, heads, base=A: rows(base + 128 * first, S * H * 64, 64, H * 64, heads)
    q, k, v = part(0, 32), part(32, 8), part(40, 8)
    other = (part(0, 32, 1 << 40), part(32, 8, 1 << 40))
    t = time.perf_counter()
    for _ in range(100):
        assert not _hit(_rope((q, k), (q, k), B, S)) and not _hit(_rope((q, k), other, B, S))
    assert not _hit(_rope((q, k), (q, v), B, S))
    assert time.perf_counter() - t < 5
    for y in ((k, part(40, 8)), (q, part(31, 8)), (part(1, 32), k), (q, part(0, 8)), (part(8, 32), part(0, 8))):
        assert _hit(_rope((q, k), y, B, S)), y
    assert _hit(_rope((k, v), (v, k), B, S))                               # exchanged


@pytest.mark.skipif(__import__("torch").cuda.is_available(), reason="addresses that no launch may see")
def test_append_overlaps():
    def call(k=rows(A, 0, 640, 64), v=rows(A + (1 << 20), 0, 640, 64), q=None, qo=None, pg=pages(k=1 << 40, v=1 << 41), f=A):
        return lambda: fa.fa_append_paged(k, v, q, qo, pg, A, None, 10, 10, f, 64, 0, 1.0, None, 64, 0, None)
    at = lambda first: rows(A + 2 * first, 0, 64, 1024, 4)                  # [10 tokens, 16 heads, 64], heads from first / 64 on
    two = lambda first: rows(A + 2 * first, 0, 64, 1024, 2)
    assert not _hit(call()) and not _hit(call(q=at(0), qo=at(0), k=two(256), v=two(384)))
    assert not _hit(call(q=at(0), qo=at(512), k=two(256), v=two(384)))
    for first in (64, 192, 256, 320, 384, 448):                            # on q in part, k, v
        assert _hit(call(q=at(0), qo=at(first), k=two(256), v=two(384))), first
    assert _hit(call(q=at(0), qo=rows(A + (1 << 30), 0, 32, 1024, 4)))      # on itself
    assert _hit(call(q=at(0), qo=rows((1 << 40) + 4096, 0, 64, 1024, 4)))   # on the pools
    assert _hit(call(q=at(0), qo=rows((1 << 41) + 4096, 0, 64, 1024, 4)))
    page = 2 * 64 * 64
    inter = pages(k=1 << 40, v=(1 << 40) + 2 * page, stride=2 * page)       # one allocation, page by page
    assert not _hit(call(pg=inter))
    assert _hit(call(pg=pages(k=1 << 40, v=(1 << 40) + page, stride=2 * page)))
    one = pages(k=1 << 40, v=1 << 40)
    same = dict(k=rows(A, 0, 640, 64), v=rows(A, 0, 640, 64), pg=one)
    assert _hit(call(pg=one)) and _hit(call(**same)) and not _hit(call(**same, f=None))


# ---------------------------------------------------------------- numbers that do not fit

def test_numbers_beyond_32_bits_are_refused():
    """2^32 + 4096 is not 4096."""
    import torch
    x, p = torch.zeros(1, 2, 64, dtype=torch.bfloat16), torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    t, n = torch.zeros(1, 4, dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    for big in ((1 << 32) + 64, 1 << 31, -(1 << 32)):
        with pytest.raises(ValueError, match="32 bits"):
            fa.decode_prefix(x, p, p, t, n, big)
        with pytest.raises(ValueError, match="32 bits"):
            fa.rope_freqs(64, scaling="yarn", factor=4.0, original_len=big, device="cpu")
    for big in ((1 << 32) + 64, 1 << 31):
        with pytest.raises(ValueError, match="32 bits"):
            fa.rope_freqs(big, device="cpu")


@pytest.mark.skipif(__import__("torch").cuda.is_available(), reason="addresses that no launch may see")
def test_strides_beyond_every_address_are_refused():
    """Rows whose last index lies 2^47 bytes and more away, up to strides whose sums pass 64 bits."""
    far = (1 << 47, 1 << 60, (1 << 63) - 8)
    for s in far:
        for r in (rows(A, s, 640, 64), rows(A, 4096, s, 64), rows(A, 4096, 640, s)):
            other = rows(A + (1 << 30), 4096, 640, 64)
            assert _hit(_rope((r,), (other,), 2, 10)) and _hit(_rope((other,), (r,), 2, 10))
        for bad in (dict(k=rows(A, 0, s, 64)), dict(v=rows(A, 0, 640, s)), dict(q=rows(A, 0, s, 64), qo=rows(A, 0, s, 64))):
            a = {**dict(k=rows(), v=rows(A + (1 << 20)), q=None, qo=None), **bad}
            assert _hit(lambda: fa.fa_append_paged(a["k"], a["v"], a["q"], a["qo"], pages(k=1 << 40, v=1 << 41), A, None, 10,
                                                   10, A, 64, 0, 1.0, None, 64, 0, None)), (s, bad)
    assert _hit(lambda: fa.fa_append_paged(rows(), rows(A + (1 << 20)), None, None, pages(stride=1 << 38, n=(1 << 31) - 1), A,
                                           None, 10, 10, A, 64, 0, 1.0, None, 64, 0, None))
    assert not _hit(_rope((rows(A, 1 << 40, 640, 64),), (rows(A + (1 << 30), 1 << 40, 640, 64),), 2, 10))
