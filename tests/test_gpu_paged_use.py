"""How the rotary and paged calls are used: recorded into graphs, on other
streams, side by side, on dirty workspaces, over large pools; and what the
tensor calls refuse."""
import numpy as np
import pytest
import torch

import exact_tiled_attention_31_b200 as fa
from paged_helpers import check_decode, f64, freqs_of, make_cache, randn
from oracle import paged as op

pytestmark = pytest.mark.gpu


def _i32(x, dev):
    return torch.tensor(x, dtype=torch.int32, device=dev)


class Step:
    """A decode step's buffers: append one token a sequence, attend."""

    def __init__(self, dev, B=5, Hq=8, Hkv=2, D=128, page=32, shared=0, room=400, seed=0, dirty=None):
        gen = torch.Generator().manual_seed(seed)
        self.dev, self.shape, self.shared = dev, (B, Hq, Hkv, D), shared
        kp, vp, table = make_cache(gen, [shared + room] * B, Hkv, D, page, "bf16", shared=shared // page, poison=False)
        self.kp, self.vp, self.table = kp.to(dev), vp.to(dev), table.to(dev)
        self.lens = torch.ones(B, dtype=torch.int32, device=dev)
        self.q, self.k, self.v = (torch.zeros(B, h, D, dtype=torch.bfloat16, device=dev) for h in (Hq, Hkv, Hkv))
        self.freqs = torch.from_numpy(freqs_of(D)).to(dev)
        self.rq, self.o = torch.zeros_like(self.q), torch.zeros_like(self.q)
        self.lse = torch.zeros(B, Hq, device=dev)
        size = fa.fa_decode_prefix_workspace_size(B, Hq, Hkv, shared, D)
        self.ws = torch.empty(size, dtype=torch.uint8, device=dev)
        if dirty is not None:
            self.ws.fill_(dirty)

    def set(self, lens, seed):
        gen = torch.Generator().manual_seed(seed)
        self.lens.copy_(_i32(lens, self.dev))
        for x in (self.q, self.k, self.v):
            x.copy_(torch.randn(x.shape, generator=gen).to(x.dtype).to(self.dev))

    def __call__(self, **kw):
        fa.append_paged(self.k, self.v, self.kp, self.vp, self.table, self.lens, q=self.q, freqs=self.freqs,
                        q_out=self.rq, **kw)
        args = (self.rq, self.kp, self.vp, self.table, self.lens)
        if self.shared:
            fa.decode_prefix(*args, self.shared, out=self.o, lse=self.lse, workspace=self.ws, **kw)
        else:
            fa.decode_paged(*args, out=self.o, lse=self.lse, workspace=self.ws, **kw)
        return self.o, self.lse

    def check(self, what):
        fa.check_device_error()
        ref = op.decode_paged(self.rq.cpu(), self.kp.cpu(), self.vp.cpu(), self.table.cpu().numpy(),
                              self.lens.tolist(), self.shape[3] ** -0.5)
        check_decode(self.o, self.lse, self.rq, ref, what)


def _capture(fn):
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            fn()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fn()
    return g


# (shared rows: none; read for each sequence; a pass of their own)
@pytest.mark.parametrize("shared", [0, 128, 6528])
def test_one_graph_serves_all_lengths(cuda_device, shared):
    """A recorded step replayed with other inputs and lengths, padding rows among them."""
    s = Step(cuda_device, shared=shared)
    s.set([shared + 9] * 5, 0)
    g = _capture(s)
    for seed, lens in ((1, [1, 2, 65, 400, 0]), (2, [0, 0, 0, 0, 0]), (3, [300, 299, 64, 0, 33])):
        s.set([shared + n if n else 0 for n in lens], seed)
        g.replay()
        s.check(f"replay {seed}")
        o, lse = s.o.clone(), s.lse.clone()
        s()
        assert torch.equal(s.o, o) and torch.equal(s.lse, lse)


def test_two_graphs_share_a_workspace(cuda_device):
    """Two recorded steps that use one workspace, replayed in turn."""
    a, b = Step(cuda_device, seed=1), Step(cuda_device, Hq=16, Hkv=2, seed=2)
    b.ws = a.ws = b.ws if b.ws.numel() > a.ws.numel() else a.ws
    a.set([50] * 5, 0)
    b.set([50] * 5, 0)
    ga, gb = _capture(a), _capture(b)
    for seed in (3, 4):
        a.set([399, 1, 200, 64, 65], seed)
        b.set([5, 400, 31, 0, 128], seed)
        for g in (ga, gb, ga, gb):
            g.replay()
        a.check("first graph")
        b.check("second graph")


def test_graph_of_rotation_and_attention(cuda_device):
    dev, gen = cuda_device, torch.Generator().manual_seed(0)
    q, k, v, do = (randn(gen, "bf16", 1, 4, 200, 64).to(dev) for _ in range(4))
    freqs = torch.from_numpy(freqs_of(64)).to(dev)
    outs = [torch.empty_like(q) for _ in range(2)]
    grads = [torch.empty_like(q) for _ in range(3)]
    back = [torch.empty_like(q) for _ in range(2)]
    o, lse = torch.empty_like(q), torch.empty(1, 4, 200, device=dev)
    ws = torch.empty(fa.fa_bwd_workspace_size(1, 4, 200, 64), device=dev, dtype=torch.uint8)

    def step():
        fa.rope(q, k, freqs, out=tuple(outs))
        fa.forward(*outs, v, True, out=o, lse=lse)
        fa.backward(*outs, v, o, do, lse, True, deterministic=True, workspace=ws, out=tuple(grads))
        fa.rope_backward(grads[0], grads[1], freqs, out=tuple(back))

    g = _capture(step)
    for x in (q, k, v, do):
        x.copy_(randn(gen, "bf16", 1, 4, 200, 64).to(dev))
    g.replay()
    fa.check_device_error()
    got = [x.clone() for x in back]
    step()
    fa.check_device_error()
    assert torch.equal(got[0], back[0]) and torch.equal(got[1], back[1])


@pytest.mark.parametrize("dirty", [0x00, 0x7F, 0xFF])
@pytest.mark.parametrize("shared", [0, 64, 9024])
def test_any_workspace_contents(cuda_device, dirty, shared):
    s = Step(cuda_device, B=4, shared=shared, dirty=dirty, room=2000)
    s.set([shared + n for n in (1999, 3, 700, 0)], 7)
    s()
    s.check(f"workspace of {dirty:#x}")


def test_other_streams(cuda_device):
    """Given as a stream, as a number, and as the current one; nothing but the given stream's order is relied on."""
    s = Step(cuda_device)
    s.set([10, 20, 30, 40, 50], 1)
    torch.cuda.synchronize()
    s()
    want = s.o.clone()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        s.o.zero_()
        torch.cuda.synchronize()
        torch.cuda._sleep(20_000_000)  # the current stream is busy: the side stream's work does not wait for it
        s(stream=stream)
        side.synchronize()
        assert torch.equal(s.o, want)
        torch.cuda.synchronize()
    o, lse = fa.decode_paged(s.rq, s.kp, s.vp, s.table, s.lens, stream=side)  # outputs and workspace of that stream
    x, _ = fa.rope(s.q[:, :, None], None, s.freqs, stream=side)
    side.synchronize()
    assert torch.equal(o, want) and x.shape == (5, 8, 1, 128)
    s.check("side stream")


def test_two_calls_at_once(cuda_device):
    """Two long calls on two streams, each with its own workspace, give what each gives alone."""
    a, b = Step(cuda_device, B=6, room=6000, seed=1), Step(cuda_device, B=6, room=6000, seed=2, shared=5120)
    a.set([6000, 5999, 1, 0, 3333, 64], 1)
    b.set([5120 + n for n in (6000, 17, 2000, 0, 64, 5000)], 2)
    a(), b()
    torch.cuda.synchronize()
    want = [x.clone() for x in (a.o, a.lse, b.o, b.lse)]
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(10):
        a(stream=sa)
        b(stream=sb)
    torch.cuda.synchronize()
    fa.check_device_error()
    for x, y in zip((a.o, a.lse, b.o, b.lse), want):
        assert torch.equal(x, y)


@pytest.mark.parametrize("B,Hq,Hkv,D,page,shared", [(8, 16, 8, 64, 64, 0), (150, 8, 2, 64, 16, 0), (9, 16, 8, 64, 32, 1536),
                                                    (12, 32, 2, 128, 128, 0)])
def test_handed_out_runs(cuda_device, B, Hq, Hkv, D, page, shared):
    """Enough rows that the CTAs take short runs from the common count: every
    row against the oracle, and the same bits call after call."""
    dev, gen = cuda_device, torch.Generator().manual_seed(B)
    # 48 tiles for each of 2 x 148 CTAs and some more, over ragged lengths
    mean = 50 * 296 * 64 // (B * Hkv)
    lens = [shared + (0 if i == 1 else max(1, 2 * mean * (i + 1) // (B + 1))) for i in range(B)]
    each = -(-max(lens) // page)
    n_pages = shared // page + B * each
    ids = torch.randperm(n_pages, generator=gen).to(torch.int32)
    n0 = shared // page
    table = torch.cat([ids[:n0].expand(B, n0), ids[n0:n0 + B * (each - n0)].view(B, each - n0)], 1).contiguous()
    torch.manual_seed(B)
    kp, vp = (torch.randn(n_pages, Hkv, page, D, device=dev).to(torch.bfloat16) for _ in range(2))
    q = randn(gen, "bf16", B, Hq, D).to(dev)
    args = (q, kp, vp, table.to(dev), _i32(lens, dev))
    call = (lambda: fa.decode_prefix(*args, shared)) if shared else (lambda: fa.decode_paged(*args))
    o, lse = call()
    fa.check_device_error()
    # the oracle's definition in fp64 on the GPU, a sequence at a time
    for b in range(B):
        n = lens[b]
        if n == 0:
            assert (o[b] == 0).all() and torch.isneginf(lse[b]).all()
            continue
        rows = table[b, :-(-n // page)].long().to(dev)
        k, v = (x[rows].transpose(0, 1).reshape(Hkv, -1, D)[:, :n].double() for x in (kp, vp))
        k, v = (x.repeat_interleave(Hq // Hkv, 0) for x in (k, v))
        score = (k @ q[b].double()[:, :, None])[..., 0] * D ** -0.5
        rl = torch.logsumexp(score, -1)
        w = torch.exp(score - rl[:, None])[:, None]
        size = (k.abs() @ q[b].double().abs()[:, :, None])[..., 0].amax(-1) * D ** -0.5
        ref = [x.cpu().numpy()[None] for x in ((w @ v)[:, 0], rl, (w @ v.abs())[:, 0], size)]
        check_decode(o[b:b + 1], lse[b:b + 1], q[b:b + 1], ref, f"sequence {b} of {n}")
    for _ in range(5):
        again = call()
        assert torch.equal(again[0], o) and torch.equal(again[1], lse)
    fa.check_device_error()


def test_pool_beyond_32_bits(cuda_device):
    """Pages whose elements lie past 2^32: appended to and read like any others."""
    dev, gen = cuda_device, torch.Generator().manual_seed(4)
    Hkv, page, D = 8, 64, 128
    n = (1 << 32) // (Hkv * page * D) + 40  # pages of one pool
    kp, vp = (torch.empty(n, Hkv, page, D, dtype=torch.bfloat16, device=dev) for _ in range(2))
    ids = [n - 1, n - 7, 3, n - 20]
    table = _i32([ids[:2], ids[2:]], dev)
    k, v = randn(gen, "bf16", Hkv, 200, D), randn(gen, "bf16", Hkv, 200, D)
    lens = [128, 72]
    fa.append_paged(k.to(dev), v.to(dev), kp, vp, table, _i32(lens, dev), cu_seqlens=_i32([0, 128, 200], dev))
    q = randn(gen, "bf16", 2, 16, D)
    o, lse = fa.decode_paged(q.to(dev), kp, vp, table, _i32(lens, dev))
    fa.check_device_error()
    small = [x[torch.tensor(ids, device=dev)].cpu() for x in (kp, vp)]
    for x, y in zip(small, (k, v)):
        assert torch.equal(x[0, :, :], y[:, :64]) and torch.equal(x[2], y[:, 128:192])
    ref = op.decode_paged(q, *small, np.array([[0, 1], [2, 3]]), lens, D ** -0.5)
    check_decode(o, lse, q, ref, "large pool")


def test_nan_stays_in_its_row(cuda_device):
    """A query or a visible key that is NaN gives NaN in the rows that see it, and in no others."""
    for shared in (0, 64, 8192):
        s = Step(cuda_device, B=4, shared=shared)
        s.set([shared + 40] * 4, 3)
        s()
        clean = s.o.clone()
        s.rq[1, 2] = float("nan")
        s.kp[s.table[3, (shared + 5) // 32], 1, (shared + 5) % 32] = float("nan")
        args = (s.rq, s.kp, s.vp, s.table, s.lens)
        o, lse = fa.decode_prefix(*args, shared) if shared else fa.decode_paged(*args)
        fa.check_device_error()
        bad = torch.zeros(4, 8, dtype=torch.bool, device=o.device)
        bad[1, 2] = True
        bad[3, 4:] = True  # query heads of KV head 1
        assert torch.isnan(o[bad]).all() and torch.isnan(lse[bad]).all()
        assert torch.equal(o[~bad], clean[~bad]) and torch.isfinite(lse[~bad]).all()


# ---------------------------------------------------------------- refusals of the tensor calls

def test_tensor_refusals(cuda_device):
    dev = cuda_device
    bf = dict(dtype=torch.bfloat16, device=dev)
    q, k = torch.zeros(2, 4, 6, 64, **bf), torch.zeros(2, 2, 6, 64, **bf)
    f = torch.ones(16, dtype=torch.float64, device=dev)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device=dev)
    wrong = [
        lambda: fa.rope(q.float(), None, f),
        lambda: fa.rope(q, k.half(), f),
        lambda: fa.rope(q, k[:1], f),
        lambda: fa.rope(q[0, 0], None, f),
        lambda: fa.rope(q[0], None, f),                                     # packed, no positions
        lambda: fa.rope(q, None, f, cu_seqlens=i32(3)),                     # not packed
        lambda: fa.rope(q, None, f.float()),
        lambda: fa.rope(q, None, f.cpu()),
        lambda: fa.rope(q, None, f, positions=i32(5)),
        lambda: fa.rope(q, None, f, positions=i32(3, 6)),
        lambda: fa.rope(q, None, f, positions=i32(6).long()),
        lambda: fa.rope(q[..., ::2], None, f[:8]),                          # rows not contiguous
        lambda: fa.rope(torch.zeros(2, 4, 6, 68, **bf)[..., :64], None, f),  # strides not of 8
        lambda: fa.rope(q, None, f, out=q[:, :, :3]),
        lambda: fa.rope(q, k, f, out=q),
        lambda: fa.rope(q, k, f, out=(q, None)),
        lambda: fa.rope(q[:, :, :5], None, f, out=q[:, :, 1:]),             # overlaps, is not the input
        lambda: fa.rope(k, k, f, out=(k, k)),
        lambda: fa.rope(q, None, f, out=q[:1].expand(2, 4, 6, 64)),
        lambda: fa.rope(q, None, f, stream=object),
    ]
    kp = torch.zeros(5, 2, 16, 64, **bf)
    t, n = i32(2, 3), i32(2)
    k1, q1 = torch.zeros(2, 2, 64, **bf), torch.zeros(2, 4, 64, **bf)
    wrong += [
        lambda: fa.append_paged(k1, k1[:1], kp, kp, t, n),
        lambda: fa.append_paged(k1, k1.half(), kp, kp, t, n),
        lambda: fa.append_paged(k1, k1, kp[:, :1], kp[:, :1], t, n),
        lambda: fa.append_paged(k1, k1, kp, kp[:4], t, n),
        lambda: fa.append_paged(k1, k1, kp.half(), kp.half(), t, n),
        lambda: fa.append_paged(k1, k1, kp, kp, t[:1], n),
        lambda: fa.append_paged(k1, k1, kp, kp, t.long(), n),
        lambda: fa.append_paged(k1, k1, kp, kp, t, n[:1]),
        lambda: fa.append_paged(k1, k1, kp, kp, t, n.cpu()),
        lambda: fa.append_paged(k1, k1, kp, kp, t, n, q=q1),                # q takes freqs
        lambda: fa.append_paged(k1, k1, kp, kp, t, n, q_out=q1),
        lambda: fa.append_paged(k1, k1, kp, kp, t, n, q=q1[:1], freqs=f),
        lambda: fa.append_paged(k1, k1, kp, kp, t, n, freqs=f, positions=i32(3)),
        lambda: fa.append_paged(k1, k1, kp.transpose(1, 2), kp.transpose(1, 2), t, n),
        lambda: fa.decode_paged(q1[:, ::2], kp, kp, t, n),
        lambda: fa.decode_paged(q1[0], kp, kp, t, n),
        lambda: fa.decode_paged(q1, kp, kp, t, n.long()),
        lambda: fa.decode_paged(q1, kp[..., :32], kp[..., :32], t, n),
        lambda: fa.decode_paged(q1, kp, kp, t, n, out=k1),
        lambda: fa.decode_paged(q1, kp, kp, t, n, out=q1.half()),
        lambda: fa.decode_paged(q1, kp, kp, t, n, lse=torch.zeros(2, 4, **bf)),
        lambda: fa.decode_paged(q1, kp, torch.zeros(5, 2, 2, 16, 64, **bf)[:, 0], t, n),
        lambda: fa.decode_prefix(q1, kp, kp, t, n, 32, prefix_table=i32(1)),
        lambda: fa.decode_prefix(q1, kp, kp, t, n, 16, prefix_table=i32(1).long()),
    ]
    for i, call in enumerate(wrong):
        with pytest.raises((ValueError, TypeError)):
            call()
            raise AssertionError(f"call {i} was not refused")
    for call, status in ((lambda: fa.rope(q, None, f[:5]), fa.api.FA_ERR_UNSUPPORTED),
                         (lambda: fa.decode_prefix(q1, kp, kp, t, n, 20), fa.api.FA_ERR_INVALID_ARG),
                         (lambda: fa.decode_prefix(q1, kp, kp, t, n, 64), fa.api.FA_ERR_INVALID_ARG),
                         (lambda: fa.decode_paged(q1[:, :3].contiguous(), kp, kp, t, n), fa.api.FA_ERR_INVALID_ARG),
                         (lambda: fa.decode_paged(q1, kp, kp, t, n, workspace=torch.zeros(512, dtype=torch.uint8, device=dev)),
                          fa.api.FA_ERR_INVALID_ARG),
                         (lambda: fa.decode_paged(q1, kp[:, :, :12].contiguous(), kp[:, :, :12].contiguous(), t, n),
                          fa.api.FA_ERR_UNSUPPORTED)):
        with pytest.raises(fa.FAError) as e:
            call()
        assert e.value.status == status
    fa.check_device_error()


def test_empty_calls(cuda_device):
    bf = dict(dtype=torch.bfloat16, device=cuda_device)
    f = torch.ones(32, dtype=torch.float64, device=cuda_device)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device=cuda_device)
    y, none = fa.rope(torch.zeros(2, 4, 0, 64, **bf), None, f)
    assert y.shape == (2, 4, 0, 64) and none is None
    y, z = fa.rope(torch.zeros(0, 4, 3, 64, **bf), torch.zeros(0, 2, 3, 64, **bf), f)
    assert y.numel() == 0 and z.shape == (0, 2, 3, 64)
    kp = torch.zeros(5, 2, 16, 64, **bf)
    assert fa.append_paged(torch.zeros(0, 2, 64, **bf), torch.zeros(0, 2, 64, **bf), kp, kp, i32(0, 3), i32(0)) is None
    o, lse = fa.decode_paged(torch.zeros(0, 4, 64, **bf), kp, kp, i32(0, 3), i32(0))
    assert o.shape == (0, 4, 64) and lse.shape == (0, 4)
    fa.check_device_error()
