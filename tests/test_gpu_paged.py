"""The paged KV cache on the GPU: append_paged, decode_paged and
decode_prefix against the fp64 oracle, apart and together."""
import numpy as np
import pytest
import torch

import exact_tiled_attention_31_b200 as fa
from paged_helpers import check_decode, check_rotated, f64, freqs_of, make_cache, randn
from oracle import paged as op

pytestmark = pytest.mark.gpu


def _i32(x, dev):
    return torch.tensor(x, dtype=torch.int32, device=dev)


# ---------------------------------------------------------------- append

def _append_case(dev, lens, new, Hq, Hkv, D, R, page, dtype, interleaved, one, seed, with_q=True, tail=0, pool2=False):
    """Sequences of `lens` rows, the last `new` of each just arriving."""
    gen = torch.Generator().manual_seed(seed)
    kp, vp, table = make_cache(gen, lens, Hkv, D, page, dtype, poison=False, interleaved=pool2)
    cu = np.concatenate([[0], np.cumsum(new)])
    T = int(cu[-1]) + tail
    shape = (lambda h: (T, h, D)) if one else (lambda h: (h, T, D))
    k, v, q = (randn(gen, dtype, *shape(h)) for h in (Hkv, Hkv, Hq))
    freqs = freqs_of(R)
    both = torch.stack([kp, vp], 1).to(dev) if pool2 else None
    gk, gv = (both[:, 0], both[:, 1]) if pool2 else (kp.to(dev), vp.to(dev))
    q_out = torch.full_like(q, 5.0).to(dev)
    got = fa.append_paged(k.to(dev), v.to(dev), gk, gv, table.to(dev), _i32(lens, dev),
                          cu_seqlens=None if one else _i32(cu, dev), q=q.to(dev) if with_q else None,
                          freqs=torch.from_numpy(freqs).to(dev), interleaved=interleaved, amp=1.1,
                          q_out=q_out if with_q else None)
    fa.check_device_error()
    assert got is (q_out if with_q else None)
    # the same rows as [H, T, D]
    k, v, q, yq = ((x.transpose(0, 1) if one else x) for x in (k, v, q, q_out.cpu()))
    written = torch.zeros(kp.shape[0], page, dtype=torch.bool)
    for b, (n, m) in enumerate(zip(lens, new)):
        first = max(0, m - n)  # tokens before row 0 are padding
        i = np.arange(n - m + first, n)
        t = slice(int(cu[b]) + first, int(cu[b + 1]))
        at, row = table[b, torch.from_numpy(i) // page].long(), torch.from_numpy(i) % page
        written[at, row] = True
        if len(i) == 0:
            continue
        check_rotated(gk.cpu()[at, :, row].transpose(0, 1), k[:, t], i, freqs, interleaved, 1.1, False, f"k of {b}")
        assert torch.equal(gv.cpu()[at, :, row].transpose(0, 1), v[:, t])
        if with_q:
            check_rotated(yq[:, t], q[:, t], i, freqs, interleaved, 1.1, False, f"q of {b}")
        if with_q and first:
            assert (yq[:, int(cu[b]):int(cu[b]) + first] == 5.0).all()
    if with_q:
        assert (yq[:, int(cu[-1]):] == 5.0).all()
    for x, y in ((kp, gk), (vp, gv)):  # every other row as it was
        keep = ~written[:, None, :, None].expand(x.shape)
        assert torch.equal(x[keep], y.cpu()[keep])


@pytest.mark.parametrize("page", [16, 64, 512])
@pytest.mark.parametrize("Hq,Hkv,D,R,dtype,interleaved", [(8, 2, 128, 128, "bf16", False), (3, 3, 64, 32, "fp16", True),
                                                          (16, 1, 64, 64, "bf16", True)])
def test_append_step(cuda_device, page, Hq, Hkv, D, R, dtype, interleaved):
    """One token each: first rows, page ends and starts, a padding row (length 0)."""
    lens = [1, 0, 16, 17, 64, 65, 300, 128]
    _append_case(cuda_device, lens, [1] * len(lens), Hq, Hkv, D, R, page, dtype, interleaved, True, seed=page)


@pytest.mark.parametrize("new,old,tail", [([7], [0], 0), ([130, 0, 1, 33], [0, 10, 63, 500], 0), ([1, 64, 65], [15, 0, 63], 6),
                                          ([3] * 300, [2] * 300, 1)])
@pytest.mark.parametrize("with_q", [True, False])
def test_append_packed(cuda_device, new, old, tail, with_q):
    lens = [a + b for a, b in zip(new, old)]
    _append_case(cuda_device, lens, new, 4, 2, 128, 96, 32, "bf16", False, False, seed=len(new), with_q=with_q, tail=tail,
                 pool2=True)


def test_append_padding_tokens_of_a_sequence(cuda_device):
    """More new tokens than the sequence has rows: the surplus in front is padding."""
    _append_case(cuda_device, [3, 40], [8, 40], 4, 4, 64, 64, 16, "fp16", False, False, seed=2)


def test_append_without_rotation_and_with_positions(cuda_device):
    dev, gen = cuda_device, torch.Generator().manual_seed(0)
    lens = [33, 5]
    kp, vp, table = make_cache(gen, lens, 2, 64, 16, "fp16", poison=False)
    k, v = randn(gen, "fp16", 2, 2, 64), randn(gen, "fp16", 2, 2, 64)
    gk, gv = kp.to(dev), vp.to(dev)
    args = (k.to(dev), v.to(dev), gk, gv, table.to(dev), _i32(lens, dev))
    assert fa.append_paged(*args) is None
    for b, n in enumerate(lens):
        assert torch.equal(gk[table[b, (n - 1) // 16], :, (n - 1) % 16].cpu(), k[b])
    freqs = freqs_of(64)
    q = randn(gen, "fp16", 2, 6, 64)
    pos = _i32([1000003, -7], dev)
    yq = fa.append_paged(*args, q=q.to(dev), freqs=torch.from_numpy(freqs).to(dev), positions=pos)
    for b, n in enumerate(lens):
        got = gk[table[b, (n - 1) // 16], :, (n - 1) % 16].cpu()
        p = pos[b:b + 1].cpu().numpy()
        check_rotated(got[:, None], k[b][:, None], p, freqs, False, 1.0, False, "k")
        check_rotated(yq[b].cpu()[:, None], q[b][:, None], p, freqs, False, 1.0, False, "q")


def test_append_reports_what_has_no_page(cuda_device):
    """A page outside the pool, and a row past the table: nothing is written, the error word is set."""
    dev, gen = cuda_device, torch.Generator().manual_seed(0)
    k = randn(gen, "bf16", 2, 1, 64).to(dev)
    for table, lens in (([[0], [9]], [1, 1]), ([[0], [-1]], [1, 1]), ([[0], [1]], [1, 17])):
        kp, vp = (torch.zeros(2, 1, 16, 64, dtype=torch.bfloat16, device=dev) for _ in range(2))
        fa.append_paged(k, k, kp, vp, _i32(table, dev), _i32(lens, dev))
        with pytest.raises(fa.FAError) as e:
            fa.check_device_error()
        assert e.value.status == fa.api.FA_ERR_INVALID_ARG
        assert torch.equal(kp[0, 0, 0], k[0, 0]) and (kp[1] == 0).all() and (vp[1] == 0).all()
        assert (kp[0, 0, 1:] == 0).all()
    fa.check_device_error()  # cleared


# ---------------------------------------------------------------- decode

def _decode_case(dev, lens, Hq, Hkv, D, page, dtype, seed, mult=1.0, pool2=False, shared=0, **kw):
    gen = torch.Generator().manual_seed(seed)
    kp, vp, table = make_cache(gen, lens, Hkv, D, page, dtype, shared=shared // page, interleaved=pool2)
    if mult != 1.0:
        kp = kp * mult
    q = randn(gen, dtype, len(lens), Hq, D) * mult
    scale = D ** -0.5
    both = torch.stack([kp, vp], 1).to(dev) if pool2 else None
    gk, gv = (both[:, 0], both[:, 1]) if pool2 else (kp.to(dev), vp.to(dev))
    args = (q.to(dev), gk, gv, table.to(dev), _i32(lens, dev))
    if shared:
        o, lse = fa.decode_prefix(*args, shared, scale=scale, **kw)
    else:
        o, lse = fa.decode_paged(*args, scale=scale, **kw)
    fa.check_device_error()
    ref = op.decode_paged(q, kp, vp, table.numpy(), lens, scale)
    check_decode(o, lse, q, ref, f"lens {lens[:8]} Hq{Hq} Hkv{Hkv} D{D} page {page}")
    return args, o, lse


EDGES = [1, 0, 15, 16, 17, 63, 64, 65, 127, 128, 129, 300]


@pytest.mark.parametrize("page", [16, 32, 64, 256])
@pytest.mark.parametrize("Hq,Hkv,D,dtype", [(8, 2, 128, "bf16"), (4, 4, 64, "fp16"), (16, 1, 128, "fp16"),
                                            (27, 3, 64, "bf16"), (5, 1, 64, "bf16"), (8, 1, 128, "bf16")])
def test_decode_edges(cuda_device, page, Hq, Hkv, D, dtype):
    """Lengths around tiles and pages, empty rows; unused table entries -1 and NaN behind every length."""
    _decode_case(cuda_device, EDGES, Hq, Hkv, D, page, dtype, seed=page + D)


@pytest.mark.parametrize("lens,Hq,Hkv,D,page", [
    ([1], 1, 1, 64, 16),
    ([0, 0, 0], 8, 2, 128, 64),             # nothing at all
    ([9000], 4, 1, 128, 16),                # one unit cut over all SMs
    ([5000, 3], 16, 1, 64, 128),            # the largest group
    ([100] * 90, 8, 4, 128, 32),            # more units than SMs
    ([2, 700, 0, 1500, 64, 64, 1], 12, 3, 64, 64),
    (list(range(0, 300)), 4, 2, 64, 16),    # more sequences than threads find the run with
])
def test_decode_shapes(cuda_device, lens, Hq, Hkv, D, page):
    _decode_case(cuda_device, lens, Hq, Hkv, D, page, "bf16", seed=len(lens), pool2=True)


@pytest.mark.parametrize("Hq,Hkv,D,page", [(8, 4, 128, 64), (16, 1, 128, 16), (2, 2, 64, 128)])
def test_decode_long_runs(cuda_device, Hq, Hkv, D, page):
    """Every CTA's ring goes round several times, over the ends of units too, and call follows call."""
    lens = [16384 // Hkv, 4100, 16384, 8000, 13001]
    args, o, lse = _decode_case(cuda_device, [n * (4 // Hkv + 1) // 2 for n in lens], Hq, Hkv, D, page, "bf16", seed=D + page)
    for _ in range(20):
        again = fa.decode_paged(*args, scale=D ** -0.5)
    fa.check_device_error()
    assert torch.equal(again[0], o) and torch.equal(again[1], lse)


def test_decode_large_scores(cuda_device):
    """Scores of hundreds: the exact maximum keeps every exponent at or below zero."""
    _decode_case(cuda_device, [2000, 77], 8, 2, 128, 64, "bf16", seed=4, mult=8.0)


def test_decode_infinite_scores_drop_out(cuda_device):
    """Keys of the type's lowest value give -inf or huge negative scores: weight zero, the others exact."""
    dev, gen = cuda_device, torch.Generator().manual_seed(3)
    kp, vp, table = make_cache(gen, [100], 1, 64, 64, "fp16")
    q = randn(gen, "fp16", 1, 2, 64).abs()
    kp[table[0, 0], 0, 10:20] = torch.finfo(torch.float16).min
    o, lse = fa.decode_paged(q.to(dev), kp.to(dev), vp.to(dev), table.to(dev), _i32([100], dev), scale=0.125)
    fa.check_device_error()
    keep = [i for i in range(100) if not 10 <= i < 20]
    kk, vv = (op.rows_of(f64(x), table[0].numpy(), 100)[:, keep] for x in (kp, vp))
    s = f64(q)[0] @ kk[0].T * 0.125
    e = np.exp(s - s.max(-1, keepdims=True))
    want = e @ vv[0] / e.sum(-1, keepdims=True)
    # P and O each round by 2^-11, the normaliser too
    assert np.abs(f64(o)[0] - want).max() <= 2.0 ** -11 * np.abs(want).max() + 3 * 2.0 ** -11 * np.abs(vv).max()
    assert np.abs(f64(lse)[0] - (s.max(-1) + np.log(e.sum(-1)))).max() <= 1e-5


def test_decode_matches_the_contiguous_cache(cuda_device):
    """The same cache in one piece through fa.decode, in one order of pages and another."""
    dev, gen = cuda_device, torch.Generator().manual_seed(8)
    B, Hq, Hkv, D, L, page = 3, 8, 2, 128, 512, 64
    lens = _i32([512, 200, 1], dev)
    q = randn(gen, "bf16", B, Hq, D).to(dev)
    k, v = (randn(gen, "bf16", B, Hkv, L, D).to(dev) for _ in range(2))
    o, lse = fa.decode(q, k, v, lens)
    n = L // page
    outs = []
    for order in (torch.arange(B * n), torch.randperm(B * n, generator=gen)):
        pools = []
        for x in (k, v):
            pages = x.view(B, Hkv, n, page, D).transpose(1, 2).reshape(B * n, Hkv, page, D)
            pool = torch.empty_like(pages)
            pool[order.to(dev)] = pages
            pools.append(pool)
        outs.append(fa.decode_paged(q, *pools, order.to(torch.int32).view(B, n).to(dev), lens))
    fa.check_device_error()
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    # both round P and O: 2^-8 of mean |V| twice each, 2^-8 |O| each
    assert (outs[0][0].float() - o.float()).abs().max() <= 8 * 2.0 ** -8 * float(v.float().abs().max())
    assert (outs[0][1] - lse).abs().max() <= 1e-4


def test_decode_reports_a_bad_page(cuda_device):
    dev, gen = cuda_device, torch.Generator().manual_seed(0)
    kp, vp, table = make_cache(gen, [40, 40], 1, 64, 16, "bf16", poison=False)
    table[1, 1] = 1000
    q = randn(gen, "bf16", 2, 2, 64)
    o, lse = fa.decode_paged(q.to(dev), kp.to(dev), vp.to(dev), table.to(dev), _i32([40, 40], dev))
    with pytest.raises(fa.FAError) as e:
        fa.check_device_error()
    assert e.value.status == fa.api.FA_ERR_INVALID_ARG
    ref = op.decode_paged(q[:1], kp, vp, table.numpy(), [40], 64 ** -0.5)
    check_decode(o[:1], lse[:1], q[:1], ref, "the sequence beside it")
    fa.check_device_error()


# ---------------------------------------------------------------- shared prefix

@pytest.mark.parametrize("B,Hq,Hkv,D,page,P,own,dtype", [
    # read for each sequence (up to 24 MB more to read)
    (1, 4, 4, 64, 16, 16, [5], "bf16"),
    (3, 8, 2, 128, 64, 128, [0, 1, 200], "bf16"),
    (5, 5, 1, 64, 16, 272, [7, 0, 64, 65, 33], "fp16"),
    # a pass of their own
    (91, 5, 1, 64, 16, 1072, [i % 71 for i in range(91)], "fp16"),   # group 5: 25 sequences a tile
    (40, 16, 1, 128, 32, 1248, [i for i in range(40)], "fp16"),      # 640 rows: three pairs of tiles
    (70, 4, 2, 128, 256, 512, [3 * i for i in range(70)], "bf16"),
    (140, 2, 2, 64, 16, 1040, [1] * 140, "bf16"),                    # one row a sequence, two tiles
    (4, 1, 1, 128, 64, 16384, [9, 0, 64, 300], "bf16"),              # four query rows, cut over all SMs
    (32, 9, 1, 128, 16, 1600, [0] * 32, "bf16"),                     # nothing of their own; group 9
])
def test_prefix_matches_oracle(cuda_device, B, Hq, Hkv, D, page, P, own, dtype):
    args, o, lse = _decode_case(cuda_device, [P + n for n in own], Hq, Hkv, D, page, dtype, seed=P + B, shared=P)
    po, pl = fa.decode_paged(*args, scale=D ** -0.5)
    fa.check_device_error()
    assert (po.float() - o.float()).abs().max() <= 8 * 2.0 ** -8 * 4  # |V| <= about 4: both within the oracle's bound
    assert (pl - lse).abs().max() <= 1e-4


@pytest.mark.parametrize("many", [1, 9])  # read for each sequence; a pass of their own
def test_prefix_of_short_and_empty_sequences(cuda_device, many):
    """Lengths below the shared part: padding rows and sequences that see part of it."""
    dev, gen = cuda_device, torch.Generator().manual_seed(5)
    P, page, Hq, Hkv, D = 320, 32, 8, 2, 128
    lens = [0, 1, 31, 64, 129, 319, 320, 321, 400] * many
    kp, vp, table = make_cache(gen, lens, Hkv, D, page, "bf16", shared=P // page)
    q = randn(gen, "bf16", len(lens), Hq, D)
    prefix = table[0, :P // page].clone()
    table[0] = -1  # a padding row names no pages: the shared ones are given apart
    o, lse = fa.decode_prefix(q.to(dev), kp.to(dev), vp.to(dev), table.to(dev), _i32(lens, dev), P,
                              prefix_table=prefix.to(dev))
    fa.check_device_error()
    ref = op.decode_paged(q, kp, vp, table.numpy(), lens, D ** -0.5)
    check_decode(o, lse, q, ref, "short sequences")


# ---------------------------------------------------------------- together

ONE_PAGE = np.zeros((1, 1), int)  # a history as the one page of a pool

@pytest.mark.parametrize("dtype,page,shared", [("bf16", 16, 0), ("fp16", 64, 128)])
def test_prompts_then_steps(cuda_device, dtype, page, shared):
    """Prompts of a packed batch: rotated, attended with forward_varlen, appended;
    then decode steps that append and attend.  Every output against attention
    over the whole history in fp64."""
    dev, gen = cuda_device, torch.Generator().manual_seed(21)
    Hq, Hkv, D, R = 4, 2, 64, 32
    G, scale = Hq // Hkv, D ** -0.5
    prompt = [shared + n for n in (37, 0 if shared else 1, 150)]
    B, steps = len(prompt), 3
    lens = [n + steps for n in prompt]
    kp, vp, table = (x.to(dev) for x in make_cache(gen, lens, Hkv, D, page, dtype, shared=shared // page))
    freqs, amp = fa.rope_freqs(R, base=5000.0, scaling="linear", factor=2.0, device=dev)
    F = freqs.cpu().numpy()
    cu = np.concatenate([[0], np.cumsum(prompt)])
    T = int(cu[-1])
    q, k, v = (randn(gen, dtype, h, T, D) for h in (Hq, Hkv, Hkv))
    if shared:  # the same tokens in front of every prompt
        for x in (q, k, v):
            for b in range(1, B):
                x[:, cu[b]:cu[b] + shared] = x[:, :shared]
    cu_dev = _i32(cu, dev)
    fa.append_paged(k.to(dev), v.to(dev), kp, vp, table, _i32(prompt, dev), cu_seqlens=cu_dev, freqs=freqs, amp=amp)
    rq, rk = fa.rope(q.to(dev), k.to(dev), freqs, cu_seqlens=cu_dev, amp=amp)
    o, _ = fa.forward_varlen(rq, rk.repeat_interleave(G, 0).contiguous(),
                             v.to(dev).repeat_interleave(G, 0).contiguous(), cu_dev, max(prompt), True)
    fa.check_device_error()
    # the history as 16-bit rows: keys as rope rounds them
    hist_k = [rk[:, cu[b]:cu[b + 1]].cpu() for b in range(B)]
    hist_v = [v[:, cu[b]:cu[b + 1]] for b in range(B)]
    for b in range(B):
        for t in (0, prompt[b] // 2, prompt[b] - 1):
            qq = rq[:, cu[b] + t].cpu()[None]
            ref = op.decode_paged(qq, hist_k[b][None], hist_v[b][None], ONE_PAGE, [t + 1], scale)
            assert np.abs(f64(o[:, cu[b] + t])[None] - ref[0]).max() <= 1e-2
    for step in range(1, steps + 1):
        q1, k1, v1 = (randn(gen, dtype, B, h, D) for h in (Hq, Hkv, Hkv))
        now = [n + step for n in prompt]
        now_dev = _i32(now, dev)
        yq = fa.append_paged(k1.to(dev), v1.to(dev), kp, vp, table, now_dev, q=q1.to(dev), freqs=freqs, amp=amp)
        o, lse = (fa.decode_prefix(yq, kp, vp, table, now_dev, shared) if shared
                  else fa.decode_paged(yq, kp, vp, table, now_dev))
        fa.check_device_error()
        for b in range(B):
            p = np.array([now[b] - 1])
            check_rotated(yq[b].cpu()[:, None], q1[b][:, None], p, F, False, amp, False, "step q")
            row = kp[table[b, p[0] // page], :, p[0] % page].cpu()
            check_rotated(row[:, None], k1[b][:, None], p, F, False, amp, False, "step k")
            hist_k[b] = torch.cat([hist_k[b], row[:, None]], 1)
            hist_v[b] = torch.cat([hist_v[b], v1[b][:, None]], 1)
            ref = op.decode_paged(yq[b:b + 1].cpu(), hist_k[b][None], hist_v[b][None], ONE_PAGE, [now[b]], scale)
            check_decode(o[b:b + 1], lse[b:b + 1], yq[b:b + 1], ref, f"step {step} sequence {b}")



@pytest.mark.parametrize("dtype,mult", [("bf16", 8.0), ("fp16", 8.0), ("bf16", 64.0)])
def test_prefix_of_large_and_growing_scores(cuda_device, dtype, mult):
    """Scores of hundreds whose maximum grows along the shared rows, in small steps
    and large ones: the lagging maximum and every rescaling of O."""
    dev, gen = cuda_device, torch.Generator().manual_seed(17)
    B, Hq, Hkv, D, page, P = 80, 8, 1, 64, 64, 1344
    lens = [P + 2 * i for i in range(B)]
    kp, vp, table = make_cache(gen, lens, Hkv, D, page, dtype, shared=P // page)
    q = randn(gen, dtype, B, Hq, D)
    grow = torch.linspace(0.02, 1.0, P // page) ** 2 * mult
    for i in range(P // page):
        kp[table[0, i]] *= grow[i]
    args = (q.to(dev), kp.to(dev), vp.to(dev), table.to(dev), _i32(lens, dev))
    o, lse = fa.decode_prefix(*args, P, scale=0.125)
    fa.check_device_error()
    check_decode(o, lse, q, op.decode_paged(q, kp, vp, table.numpy(), lens, 0.125), f"growing scores {dtype} x {mult}")
