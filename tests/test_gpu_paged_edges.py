"""Edges of the rotary and paged calls: whose row of the table names the shared
pages, rows that nobody or only some may see, extreme scores, rows that a call
skips, outputs that overlap."""
import numpy as np
import pytest
import torch

import exact_tiled_attention_31_b200 as fa
from helpers import O_MAX
from paged_helpers import U, check_decode, f64, freqs_of, make_cache, randn
from oracle import paged as op

pytestmark = pytest.mark.gpu


def _i32(x, dev):
    return torch.tensor(x, dtype=torch.int32, device=dev)


# Sequences that share 320 rows of 2 KV heads of 128: shorter than them, as long
# and longer.  Once, the shared rows are read for each sequence; nine times over
# they take a pass of their own; 16 times over there are more sequences than
# threads that sum their lengths.
P, PAGE, HQ, HKV, D = 320, 32, 8, 2, 128
LENS = [0, 1, 31, 64, 129, 319, 320, 321, 400]


def _batch(many, lens=LENS, seed=5):
    gen = torch.Generator().manual_seed(seed)
    lens = list(lens) * many
    kp, vp, table = make_cache(gen, lens, HKV, D, PAGE, "bf16", shared=P // PAGE)
    return lens, kp, vp, table, randn(gen, "bf16", len(lens), HQ, D)


def _prefix(dev, lens, kp, vp, table, q, prefix_table=None):
    o, lse = fa.decode_prefix(q.to(dev), kp.to(dev), vp.to(dev), table.to(dev), _i32(lens, dev), P,
                              prefix_table=None if prefix_table is None else prefix_table.to(dev))
    fa.check_device_error()
    return o, lse


# ---------------------------------------------------------------- whose pages are the shared ones

@pytest.mark.parametrize("many", [1, 9, 16])
@pytest.mark.parametrize("first", ["none", "other pages", "its own rows alone"])
def test_shared_pages_without_the_first_sequence(cuda_device, many, first):
    """No prefix_table, and the first sequence is a padding row (its table row
    -1, or left over from other sequences) or shorter than the shared rows (-1
    behind its length): the pages are those of a sequence that has them all."""
    lens, kp, vp, table, q = _batch(many, LENS if first != "its own rows alone" else LENS[3:] + LENS[:3])
    given = table.clone()
    if first == "none":
        given[0] = -1
    elif first == "other pages":
        given[0] = given[8].flip(0)
    for b, n in enumerate(lens):  # entries past a length are never read, the shared ones neither
        if n < P and not (b == 0 and first == "other pages"):
            given[b, -(-n // PAGE):] = -1
    o, lse = _prefix(cuda_device, lens, kp, vp, given, q)
    check_decode(o, lse, q, op.decode_paged(q, kp, vp, table.numpy(), lens, D ** -0.5), first)


@pytest.mark.parametrize("many", [1, 30])
def test_shared_pages_that_no_sequence_has_all_of(cuda_device, many):
    """Every sequence ends inside the shared rows: the longest one's pages are theirs, its entries behind -1."""
    lens, kp, vp, table, q = _batch(many, [0, 17, 300, 288, 40])
    given = table.clone()
    for b, n in enumerate(lens):
        given[b, -(-n // PAGE):] = -1
    o, lse = _prefix(cuda_device, lens, kp, vp, given, q)
    check_decode(o, lse, q, op.decode_paged(q, kp, vp, table.numpy(), lens, D ** -0.5), "all of them shorter")
    o, lse = _prefix(cuda_device, [0] * len(lens), kp, vp, torch.full_like(table, -1), q)
    assert (o == 0).all() and torch.isneginf(lse).all()


def test_row_of_the_table_among_many_sequences(cuda_device):
    """600 sequences read their shared rows one by one; the only one that has them all comes late."""
    dev, gen = cuda_device, torch.Generator().manual_seed(2)
    shared, page = 64, 16
    lens = [i % 60 for i in range(600)]
    lens[417] = 90
    kp, vp, table = make_cache(gen, lens, 1, 64, page, "fp16", shared=shared // page)
    q = randn(gen, "fp16", len(lens), 3, 64)
    given = table.clone()
    given[:417, :4] = -1
    given[418:, :4] = -1
    o, lse = fa.decode_prefix(q.to(dev), kp.to(dev), vp.to(dev), given.to(dev), _i32(lens, dev), shared)
    fa.check_device_error()
    check_decode(o, lse, q, op.decode_paged(q, kp, vp, table.numpy(), lens, 0.125), "one full sequence")


# ---------------------------------------------------------------- what is in rows that a sequence does not see

@pytest.mark.parametrize("many", [1, 9])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_values_in_shared_rows_that_some_do_not_see(cuda_device, many, bad):
    """A value that is not finite reaches the sequences that see its row and no
    others, whether or not the shared rows take a pass of their own."""
    lens, kp, vp, table, q = _batch(many)
    ref = op.decode_paged(q, kp, vp, table.numpy(), lens, D ** -0.5)
    at, col = 200, 77
    vp[table[8, at // PAGE], 1, at % PAGE, col] = bad
    o, lse = _prefix(cuda_device, lens, kp, vp, table, q)
    hit = torch.zeros(o.shape, dtype=torch.bool, device=o.device)
    for b, n in enumerate(lens):
        hit[b, HQ // HKV:, col] = n > at
    assert hit.any() and not torch.isfinite(o[hit]).any()
    want = torch.from_numpy(ref[0]).to(o.device)
    check_decode(torch.where(hit, want.to(o.dtype), o), lse, q, ref, f"{bad} in one row")


@pytest.mark.parametrize("many", [1, 30])
def test_shared_rows_behind_every_length(cuda_device, many):
    """Shared rows at and past the longest length hold NaN."""
    lens, kp, vp, table, q = _batch(many, [0, 17, 300, 288, 40])
    for x in (kp, vp):
        x[table[0, 9], :, 300 % PAGE:] = float("nan")  # rows 300 to 319
    o, lse = _prefix(cuda_device, lens, kp, vp, table, q, prefix_table=table[0, :P // PAGE].clone())
    check_decode(o, lse, q, op.decode_paged(q, kp, vp, table.numpy(), lens, D ** -0.5), "NaN behind every length")


@pytest.mark.parametrize("many", [1, 9])
def test_shared_pages_named_by_one_row_alone(cuda_device, many):
    """The first sequence that has all shared rows names them; every other row of the table holds -1 there."""
    lens, kp, vp, table, q = _batch(many)
    given = table.clone()
    given[[b for b in range(len(lens)) if b != 6], :P // PAGE] = -1
    o, lse = _prefix(cuda_device, lens, kp, vp, given, q)
    check_decode(o, lse, q, op.decode_paged(q, kp, vp, table.numpy(), lens, D ** -0.5), "one row of the table")


@pytest.mark.parametrize("many", [4, 81])
def test_bad_shared_page_is_reported_where_it_is_seen(cuda_device, many):
    """A shared page outside the pool: an error if a sequence sees its rows, none if all end in front of it."""
    dev = cuda_device
    for n, seen in ((128, False), (P, True)):
        lens, kp, vp, table, q = _batch(1, [n, 128] * (many // 2) + [n] * (many % 2))
        prefix = table[0, :P // PAGE].clone()
        prefix[7] = kp.shape[0]  # rows 224 to 255
        o, lse = fa.decode_prefix(q.to(dev), kp.to(dev), vp.to(dev), table.to(dev), _i32(lens, dev), P,
                                  prefix_table=prefix.to(dev))
        if seen:
            with pytest.raises(fa.FAError) as e:
                fa.check_device_error()
            assert e.value.status == fa.api.FA_ERR_INVALID_ARG
        fa.check_device_error()
        short = [b for b in range(len(lens)) if lens[b] == 128]
        ref = op.decode_paged(q[short], kp, vp, table[short].numpy(), [128] * len(short), D ** -0.5)
        check_decode(o[short], lse[short], q[short], ref, "the sequences in front of it")


# ---------------------------------------------------------------- extreme scores

def _score_rows(scores):
    """Keys whose product with a query of ones in its first three columns is the score, to 2^-24 of it."""
    k = torch.zeros(len(scores), 64)
    rest = torch.tensor(scores, dtype=torch.float64)
    for i in range(3):
        k[:, i] = rest.to(torch.bfloat16).float()
        rest = rest - k[:, i].double()
    return k.to(torch.bfloat16)


@pytest.mark.parametrize("up", [7.0, 0.0])
def test_two_keys_of_nearly_one_weight(cuda_device, up):
    """Two keys share the weight; in log2 units one is 2^-8 + 2^-14, the other
    2^-8 - 2^-14 above 2^`up` times the largest weight in front of them, which
    is just above and just below a midpoint of bf16.  Relative to the exact
    maximum the larger weight is exactly 1 and the other within 2^-8, so O is
    off by at most w1 w2 2^-8 |v1 - v2| (w1 + w2 <= 1, w1 w2 <= 1 / 4) beside
    its own half step: 2^-7 for values of +-4, within the 1e-2 that forward and
    decode are held to.  Relative to an older maximum both would round, apart:
    2^-6."""
    dev = cuda_device
    B, Hkv, page, rows = 130, 8, 64, 8192
    scores = np.full(rows, -60.0)
    ln2 = np.log(2.0)
    scores[np.arange(40, 63) * 128] = 0.0
    one, two = 63 * 128 + 5, 63 * 128 + 70
    for at, d in ((one, -1), (two, 1)):
        scores[at] = (up + np.log2(1 + 2.0 ** -8 + d * 2.0 ** -14)) * ln2
    k, v = _score_rows(scores), torch.zeros(rows, 64)
    v[one], v[two] = 4.0, -4.0
    kp, vp = (x.to(torch.bfloat16).view(rows // page, 1, page, 64).expand(-1, Hkv, -1, -1).contiguous().to(dev)
              for x in (k, v))
    q = torch.zeros(B, Hkv, 64, dtype=torch.bfloat16)
    q[..., :3] = 1.0
    table = torch.arange(rows // page, dtype=torch.int32, device=dev).expand(B, -1).contiguous()
    args = (q.to(dev), kp, vp, table, _i32([rows] * B, dev))
    w = np.exp(k[:, :3].double().sum(-1).numpy())
    ref = 4.0 * (w[one] - w[two]) / w.sum()
    tol = 0.25 * 2.0 ** -8 * 8.0 + 2.0 ** -8 * abs(ref) + 2.0 ** -18
    assert tol < O_MAX
    for o, lse in (fa.decode_prefix(*args, rows, scale=1.0), fa.decode_paged(*args, scale=1.0)):
        fa.check_device_error()
        assert np.abs(f64(o) - ref).max() <= tol, (f64(o).flat[0], ref, tol)
        assert np.abs(f64(lse) - np.log(w.sum())).max() <= 1e-5


# ---------------------------------------------------------------- rows that a call skips

def _leave_nan(shape, dev):
    """What the next allocation of this size finds in its memory."""
    torch.cuda.synchronize()
    x = [torch.full(shape, float("nan"), dtype=torch.bfloat16, device=dev) for _ in range(4)]
    torch.cuda.synchronize()
    del x


@pytest.mark.parametrize("call", ["rope", "rope_backward"])
@pytest.mark.parametrize("lens,tail", [([5, 0, 40], 19), ([0], 7), ([], 5), ([64], 0)])
def test_rows_of_no_sequence_in_new_outputs_are_zero(cuda_device, call, lens, tail):
    """Rows behind the last sequence of outputs that the call allocates hold
    zeros, so that a product over all rows (a weight's gradient) stays finite."""
    dev, gen = cuda_device, torch.Generator().manual_seed(1)
    n, T = sum(lens), sum(lens) + tail
    q, k = randn(gen, "bf16", 6, T, 128).to(dev), randn(gen, "bf16", 2, T, 128).to(dev)
    freqs = torch.from_numpy(freqs_of(64)).to(dev)
    cu = _i32(np.concatenate([[0], np.cumsum(lens)]), dev)
    for x in (q, k):
        _leave_nan(x.shape, dev)
    got = getattr(fa, call)(q, k, freqs, cu_seqlens=cu)
    given = tuple(torch.full_like(x, 3.0) for x in (q, k))
    getattr(fa, call)(q, k, freqs, cu_seqlens=cu, out=given)
    fa.check_device_error()
    for x, y in zip(got, given):
        assert (x[:, n:] == 0).all() and torch.equal(x[:, :n], y[:, :n]) and (y[:, n:] == 3.0).all()


@pytest.mark.parametrize("one", [True, False])
def test_queries_of_padding_tokens_in_new_outputs_are_zero(cuda_device, one):
    """append_paged without q_out: the queries of tokens that are not written are zero, and with q_out left as they were."""
    dev, gen = cuda_device, torch.Generator().manual_seed(4)
    lens = [3, 0, 17, 0] if one else [3, 0, 17]
    new = [1] * 4 if one else [5, 2, 4]  # two tokens in front of the first sequence's rows, two of an empty one
    cu = np.concatenate([[0], np.cumsum(new)])
    T = int(cu[-1]) + (0 if one else 3)  # three behind the last sequence
    skipped = [1, 3] if one else [0, 1, 5, 6, 11, 12, 13]
    kp, vp, table = (x.to(dev) for x in make_cache(gen, [max(n, 1) for n in lens], 2, 64, 16, "bf16", poison=False))
    shape = (lambda h: (T, h, 64)) if one else (lambda h: (h, T, 64))
    q, k, v = (randn(gen, "bf16", *shape(h)).to(dev) for h in (5, 2, 2))
    kw = dict(q=q, freqs=torch.from_numpy(freqs_of(32)).to(dev), cu_seqlens=None if one else _i32(cu, dev))
    _leave_nan(q.shape, dev)
    got = fa.append_paged(k, v, kp, vp, table, _i32(lens, dev), **kw)
    given = torch.full_like(q, 3.0)
    fa.append_paged(k, v, kp, vp, table, _i32(lens, dev), q_out=given, **kw)
    fa.check_device_error()
    got, given = (x if one else x.transpose(0, 1) for x in (got, given))
    rest = [t for t in range(T) if t not in skipped]
    assert (got[skipped] == 0).all() and (given[skipped] == 3.0).all() and torch.equal(got[rest], given[rest])
    assert torch.isfinite(given).all() and not (given[rest] == 3.0).all()


def test_queries_of_no_sequences_are_zero(cuda_device):
    """Tokens without any sequence: append_paged writes nothing, and zeros to a new q."""
    dev, gen = cuda_device, torch.Generator().manual_seed(4)
    q, k = randn(gen, "bf16", 4, 9, 64).to(dev), randn(gen, "bf16", 2, 9, 64).to(dev)
    kp, vp = (torch.full((3, 2, 16, 64), 2.0, dtype=torch.bfloat16, device=dev) for _ in range(2))
    args = (k, k, kp, vp, torch.zeros(0, 3, dtype=torch.int32, device=dev), torch.zeros(0, dtype=torch.int32, device=dev))
    kw = dict(cu_seqlens=_i32([0], dev), freqs=torch.from_numpy(freqs_of(32)).to(dev))
    _leave_nan(q.shape, dev)
    assert (fa.append_paged(*args, q=q, **kw) == 0).all() and fa.append_paged(*args, **kw) is None
    given = torch.full_like(q, 3.0)
    fa.append_paged(*args, q=q, q_out=given, **kw)
    fa.check_device_error()
    assert (given == 3.0).all() and (kp == 2.0).all() and (vp == 2.0).all()


# ---------------------------------------------------------------- outputs that overlap

def test_overlapping_outputs_are_refused(cuda_device):
    """Each output is its own input, in place, or apart from everything else of the call."""
    bf = dict(dtype=torch.bfloat16, device=cuda_device)
    f = torch.ones(32, dtype=torch.float64, device=cuda_device)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device=cuda_device)
    q, k = (torch.randn(2, 4, 6, 64, **bf) for _ in range(2))
    buf = torch.zeros(2, 8, 6, 64, **bf)
    kp, vp = (torch.zeros(4, 2, 16, 64, **bf) for _ in range(2))
    t, n = i32(2, 2), i32(2) + 1
    t[1] = 1
    k1, q1 = torch.zeros(2, 2, 64, **bf), torch.zeros(2, 4, 64, **bf)
    one = torch.zeros(2, 8, 64, **bf)
    wrong = [
        lambda: fa.rope(q, k, f, out=(k, q)),                                  # exchanged
        lambda: fa.rope(q, k, f, out=(torch.empty_like(q), q)),                # k_out on q
        lambda: fa.rope(q, k, f, out=(buf[:, :4], buf[:, 2:6])),               # two outputs in part
        lambda: fa.rope(q, None, f, out=buf.view(-1).as_strided((2, 4, 6, 64), (1536, 384, 32, 1))),  # of itself
        lambda: fa.append_paged(k1, k1, kp, vp, t, n, q=one[:, :4], freqs=f, q_out=one[:, 2:6]),
        lambda: fa.append_paged(one[:, 4:6], k1, kp, vp, t, n, q=q1, freqs=f, q_out=one[:, 4:]),      # on k
        lambda: fa.append_paged(k1, one[:, 4:6], kp, vp, t, n, q=q1, freqs=f, q_out=one[:, 2:6]),     # on v
        lambda: fa.append_paged(k1, k1, kp, kp, t, n, freqs=f),                # keys and values into one pool
    ]
    for i, call in enumerate(wrong):
        with pytest.raises((ValueError, fa.FAError)):
            call()
            raise AssertionError(f"call {i} was not refused")
    fa.check_device_error()
    # one buffer of a fused projection, q and k in place or into another such buffer's places
    fused, other = (torch.randn(2, 6, 12, 64, **bf) for _ in range(2))
    parts = lambda x: (x[:, :, :8].transpose(1, 2), x[:, :, 8:10].transpose(1, 2))
    want = fa.rope(*parts(fused), f)
    rest = other[:, :, 10:].clone()
    fa.rope(*parts(fused), f, out=parts(other))
    fa.rope(*parts(fused), f, out=parts(fused))
    fa.check_device_error()
    for x in (fused, other):
        assert all(torch.equal(a, b) for a, b in zip(parts(x), want))
    assert torch.equal(other[:, :, 10:], rest)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("where", ["first tile", "inside", "all shared rows"])
def test_shared_rows_of_the_lowest_value_drop_out(cuda_device, dtype, where):
    """Keys of the type's lowest value against queries that are all positive:
    scores of -inf (bf16) or far below the others (fp16), in a pass of their own.
    Their weight is zero, the rest exact; with nothing else O is 0 and LSE -inf (bf16)."""
    dev, gen = cuda_device, torch.Generator().manual_seed(6)
    lens = [P] * 20 + [P + 1 + 3 * i for i in range(60)]
    kp, vp, table = make_cache(gen, lens, HKV, D, PAGE, dtype, shared=P // PAGE)
    q = randn(gen, dtype, len(lens), HQ, D).abs() + 0.125
    low = {"first tile": range(0, 128), "inside": range(130, 250), "all shared rows": range(P)}[where]
    keep = [i for i in range(P) if i not in low]
    for i in low:
        kp[table[0, i // PAGE], :, i % PAGE] = torch.finfo(kp.dtype).min
    o, lse = _prefix(dev, lens, kp, vp, table, q)
    if not keep:  # the sequences of shared rows alone
        if dtype == "bf16":
            assert (o[:20] == 0).all() and torch.isneginf(lse[:20]).all()
        else:
            assert torch.isfinite(o[:20]).all() and torch.isfinite(lse[:20]).all()
    first = 0 if keep else 20
    G, k, v = HQ // HKV, f64(kp), f64(vp)
    for b in range(first, len(lens)):
        rows = keep + list(range(P, lens[b]))
        kk, vv = (np.stack([x[table[b, i // PAGE], :, i % PAGE] for i in rows], 1).repeat(G, 0) for x in (k, v))
        s = np.einsum("hnd,hd->hn", kk, f64(q)[b]) * D ** -0.5
        e = np.exp(s - s.max(-1, keepdims=True))
        w = e / e.sum(-1, keepdims=True)
        e_s = ((D + 8) * 2.0 ** -24 + 2.0 ** -22) * np.einsum("hnd,hd->hn", np.abs(kk), f64(q)[b]).max(-1) * D ** -0.5
        ref, mean_v = np.einsum("hn,hnd->hd", w, vv), np.einsum("hn,hnd->hd", w, np.abs(vv))
        u = U[o.dtype]  # as in paged_helpers
        tol = u * np.abs(ref) + 2.0 ** -25 + (2 * u + 2 * (2 * e_s[:, None] + 2.0 ** -21)) * mean_v
        assert (np.abs(f64(o[b]) - ref) <= tol).all(), b
        assert (np.abs(f64(lse[b]) - s.max(-1) - np.log(e.sum(-1))) <= 2 * e_s + 2.0 ** -20 + 1e-5).all(), b


def test_outputs_between_the_rows_of_their_inputs(cuda_device):
    """An output in another place of its input's buffer, its rows between the input's."""
    bf = dict(dtype=torch.bfloat16, device=cuda_device)
    f = torch.from_numpy(freqs_of(64)).to(cuda_device)
    buf = torch.randn(2, 6, 16, 64, **bf).transpose(1, 2)
    q, k, rest = buf[:, :4], buf[:, 4:6], buf[:, 12:].clone()
    want = fa.rope(q, k, f)
    got = fa.rope(q, k, f, out=(buf[:, 6:10], buf[:, 10:12]))
    one = torch.randn(3, 12, 64, **bf)
    kp, vp = (torch.zeros(3, 2, 16, 64, **bf) for _ in range(2))
    args = (kp, vp, _i32([[0], [1], [2]], cuda_device), _i32([5, 6, 7], cuda_device))
    want1 = fa.append_paged(one[:, 4:6], one[:, 6:8], *args, q=one[:, :4], freqs=f)
    got1 = fa.append_paged(one[:, 4:6], one[:, 6:8], *args, q=one[:, :4], freqs=f, q_out=one[:, 8:])
    fa.check_device_error()
    assert all(torch.equal(a, b) for a, b in zip((*got, got1), (*want, want1))) and torch.equal(buf[:, 12:], rest)
    for call in (lambda: fa.rope(q, k, f, out=(k.repeat(1, 2, 1, 1), buf[:, 5:7])),
                 lambda: fa.append_paged(one[:, 4:6], one[:, 6:8], *args, q=one[:, :4], freqs=f, q_out=one[:, 3:7])):
        with pytest.raises(ValueError, match="overlaps"):
            call()
