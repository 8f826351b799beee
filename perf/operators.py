"""The workloads on which the rotary, paged-cache and shared-prefix operators are measured.

``listed()`` names the cases, ``draw(rng)`` gives more of the same ranges,
``prepare`` makes the inputs of one, ``run`` does one pass over them: in
elementary torch operations where ``own`` is false, through the library's
public calls where it is true.  ``exact`` gives the result in 64 bits.

Operators:

* ``rope``     rotary positions on q and k (``rope`` / ``rope_backward``)
* ``append``   new keys and values into a paged cache, rotated on the way,
               with the queries of the same tokens rotated too (``append_paged``)
* ``decode``   one new token per sequence against its pages (``decode_paged``)
* ``prefix``   the same for sequences whose first pages are shared (``decode_prefix``)
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # a few tokens of one sequence far into a long context, part of the head rotated: latency
        dict(name="rope few tokens", op="rope", B=1, Hq=32, Hkv=8, S=17, D=128, R=64, dtype="fp16", interleaved=False,
             src="contiguous", pos="far", inverse=False, scaled=False),
        # a training forward: q and k as the projections leave them ([B, S, H, D]), scaled for a longer context
        dict(name="rope training", op="rope", B=1, Hq=32, Hkv=32, S=4096, D=128, R=128, dtype="bf16",
             interleaved=False, src="token-major", pos="index", inverse=False, scaled=True),
        # its backward at the larger training shape: dq and dk of the attention backward, turned back
        dict(name="rope backward large", op="rope", B=4, Hq=16, Hkv=16, S=8192, D=128, R=128, dtype="bf16",
             interleaved=True, src="contiguous", pos="index", inverse=True, scaled=False),
        # one decode step of eight sequences: the new token's q, k, v
        dict(name="append step", op="append", B=8, T=8, Hq=32, Hkv=8, D=128, R=128, L=8192, page=16, dtype="bf16",
             interleaved=False, one=True, with_q=True),
        # a chunk of several prompts on top of cached history, odd lengths
        dict(name="append chunk", op="append", B=5, T=1037, Hq=12, Hkv=3, D=64, R=32, L=2000, page=64, dtype="fp16",
             interleaved=True, one=False, with_q=True),
        # the prompts of a whole packed batch
        dict(name="append prompts", op="append", B=32, T=67000, Hq=32, Hkv=8, D=128, R=128, L=4500, page=64,
             dtype="bf16", interleaved=False, one=False, with_q=False),
        # one short sequence: latency
        dict(name="decode short", op="decode", B=1, Hq=16, Hkv=4, L=301, D=64, page=16, dtype="fp16", fill="full"),
        # the benchmark's decode step, its caches in pages
        dict(name="decode batch", op="decode", B=8, Hq=32, Hkv=8, L=8192, D=128, page=64, dtype="bf16", fill="full"),
        # a large ragged batch, from a padding row to the longest
        dict(name="decode ragged", op="decode", B=64, Hq=32, Hkv=8, L=8192, D=128, page=16, dtype="bf16",
             fill="ragged"),
        # a few answers to one short prompt
        dict(name="prefix few", op="prefix", B=4, Hq=16, Hkv=4, P=1024, L=100, D=64, page=32, dtype="fp16"),
        # a batch of questions over one document
        dict(name="prefix batch", op="prefix", B=64, Hq=32, Hkv=8, P=8192, L=512, D=128, page=64, dtype="bf16"),
        # many samples of one long prompt
        dict(name="prefix many", op="prefix", B=250, Hq=32, Hkv=8, P=32768, L=64, D=128, page=16, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "decode", "prefix"])
    D, dtype = rng.choice([64, 128]), rng.choice(["bf16", "fp16"])
    Hkv, G = rng.choice([1, 2, 3, 4, 8, 16]), rng.choice([1, 2, 3, 4, 5, 8, 16])
    page, R = rng.choice([16, 32, 64, 128, 256]), 16 * rng.randint(1, D // 16)
    inter = rng.random() < 0.5
    if op == "rope":
        Hq, B = Hkv * min(G, 8), _log(rng, 1, 8)
        # at most the elements of the largest listed case
        S = _log(rng, 1, max(1, min(16384, 4 * 32 * 8192 * 128 // (B * (Hq + Hkv) * D))))
        return dict(op="rope", B=B, Hq=Hq, Hkv=Hkv, S=S, D=D, R=R, dtype=dtype, interleaved=inter,
                    src=rng.choice(["contiguous", "token-major", "packed"]), pos=rng.choice(["index", "far"]),
                    inverse=rng.random() < 0.5, scaled=rng.random() < 0.5)
    if op == "append":
        Hkv = min(Hkv, 8)
        one, L = rng.random() < 0.4, _log(rng, 300, 8192)
        B = _log(rng, 1, 256) if one else _log(rng, 1, 32)
        T = B if one else max(B, min(_log(rng, 1, 60000), B * L // 4))
        return dict(op="append", B=B, T=T, Hq=Hkv * min(G, 4), Hkv=Hkv, D=D, R=R, L=L, page=page, dtype=dtype,
                    interleaved=inter, one=one, with_q=rng.random() < 0.5)
    if op == "decode":
        L = _log(rng, 1, 32768)
        B = _log(rng, 1, max(1, min(256, 64 * 8 * 8192 // (2 * Hkv * L))))
        return dict(op="decode", B=B, Hq=Hkv * G, Hkv=Hkv, L=L, D=D, page=page, dtype=dtype,
                    fill=rng.choice(["full", "ragged"]))
    P = -(-_log(rng, 256, 16384) // page) * page
    B = _log(rng, 1, max(1, min(200, 250 * 32 * 16384 // (P * Hkv * G))))
    return dict(op="prefix", B=B, Hq=Hkv * G, Hkv=Hkv, P=P, L=_log(rng, 1, 512), D=D, page=page, dtype=dtype)


def _lens(case):
    """The lengths of the sequences, as a set: which sequence has which goes by the seed."""
    B, L, fill = case["B"], case["L"], case.get("fill", "ragged")
    if fill == "full" or B == 1:
        return [L] * B
    return [L * i // (B - 1) for i in range(B)]  # from an empty row of a padded batch to the longest


def work(case):
    D, Hq, Hkv, B = case["D"], case["Hq"], case["Hkv"], case["B"]
    if case["op"] == "rope":
        n = B * case["S"]
        return {"bytes": 2 * (Hq + Hkv) * n * D * 2 + 4 * n, "flops": 3 * (Hq + Hkv) * n * case["R"]}
    if case["op"] == "append":
        T, hq = case["T"], Hq if case["with_q"] else 0
        return {"bytes": 2 * (hq + 2 * Hkv) * T * D * 2 + 4 * B, "flops": 3 * (hq + Hkv) * T * case["R"]}
    n, P = sum(_lens(case)), case.get("P", 0)
    return {"bytes": 4 * Hkv * D * (P + n) + 4 * Hq * B * D + 4 * Hq * B + 4 * B + 4 * (P + n) // case["page"],
            "flops": 4 * Hq * D * (B * P + n)}


# ---------------------------------------------------------------- inputs

def _inv_freq(R, scaled):
    """Radians a position of each pair, and the amplitude: base 10000, or, scaled by 4 for a context of 16384
    where 4096 was trained, the slow pairs interpolated and the fast ones kept (YaRN, Peng et al. 2023)."""
    f = 10000.0 ** (-torch.arange(R // 2, dtype=torch.float64, device=DEV) * 2.0 / R)
    if not scaled:
        return f, 1.0
    at = [R * math.log(4096 / (beta * 2 * math.pi)) / (2 * math.log(10000.0)) for beta in (32.0, 1.0)]
    lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), R - 1)
    keep = 1 - ((torch.arange(R // 2, dtype=torch.float64, device=DEV) - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
    return f / 4 * (1 - keep) + f * keep, 0.1 * math.log(4.0) + 1.0


def _rand(gen, dtype, *shape):
    return torch.randn(*shape, generator=gen, dtype=torch.float32, device=DEV).to(TYPES[dtype])


def _pieces(T, n):
    """T rows in n ragged pieces, none of them empty: growing, the longest about twice the mean."""
    ends = [j + (T - n) * j * (j + 1) // (n * (n + 1)) for j in range(n + 1)]
    return [b - a for a, b in zip(ends, ends[1:])]


def _cuts(gen, T, n):
    """Offsets of those pieces, in an order that goes by the seed."""
    each = torch.tensor(_pieces(T, n), device=DEV)[torch.randperm(n, generator=gen, device=DEV)]
    return torch.cat([each.new_zeros(1), each.cumsum(0)]).to(torch.int32)


def _pool(case, gen, n_rows_max, shared):
    """Pages in no order, each sequence's table, `shared` first pages the same for all."""
    B, Hkv, D, page = case["B"], case["Hkv"], case["D"], case["page"]
    each = -(-n_rows_max // page)
    n_pages = shared + B * each + 3
    ids = torch.randperm(n_pages, generator=gen, device=DEV).to(torch.int32)
    table = torch.cat([ids[:shared].expand(B, shared), ids[shared : shared + B * each].view(B, each)], 1).contiguous()
    pool = [torch.empty(n_pages, Hkv, page, D, dtype=TYPES[case["dtype"]], device=DEV) for _ in range(2)]
    for x in pool:
        x.normal_(generator=gen)
    return pool[0], pool[1], table


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed * 1000003 + 17)
    s = dict(case)
    B, Hq, Hkv, D, dt, op = (case[x] for x in ("B", "Hq", "Hkv", "D", "dtype", "op"))
    if op == "rope":
        S = case["S"]
        s["freqs"], s["amp"] = _inv_freq(case["R"], case["scaled"])
        s["cu"] = s["positions"] = None
        if case["src"] == "packed":
            s["q"], s["k"] = _rand(gen, dt, Hq, B * S, D), _rand(gen, dt, Hkv, B * S, D)
            s["cu"] = _cuts(gen, B * S, B)
        elif case["src"] == "token-major":
            s["q"] = _rand(gen, dt, B, S, Hq, D).transpose(1, 2)
            s["k"] = _rand(gen, dt, B, S, Hkv, D).transpose(1, 2)
        else:
            s["q"], s["k"] = _rand(gen, dt, B, Hq, S, D), _rand(gen, dt, B, Hkv, S, D)
        if case["pos"] == "far":  # a context that began up to a million tokens earlier
            shape = (B * S,) if case["src"] == "packed" else (B, S)
            start = torch.randint(0, 1 << 20, shape[:-1] + (1,), generator=gen, device=DEV)
            s["positions"] = (start + torch.arange(shape[-1], device=DEV)).to(torch.int32)
        if own:  # the buffers that a training step keeps from step to step
            s["out"] = tuple(torch.empty(x.shape, dtype=x.dtype, device=DEV) for x in (s["q"], s["k"]))
    elif op == "append":
        T, L = case["T"], case["L"]
        s["freqs"], s["amp"] = _inv_freq(case["R"], False)
        if case["one"]:
            new = torch.ones(B, dtype=torch.int32, device=DEV)
            s["cu"] = None
            shape_q, shape_k = (B, Hq, D), (B, Hkv, D)
        else:
            s["cu"] = _cuts(gen, T, B)
            new = s["cu"][1:] - s["cu"][:-1]
            shape_q, shape_k = (Hq, T, D), (Hkv, T, D)
        room = (L - new + 1).clamp(min=1)
        old = (torch.rand(B, generator=gen, device=DEV, dtype=torch.float64) * room).long()
        s["lens"] = (old + new).to(torch.int32)
        rows = L if case["one"] else max(L, *_pieces(T, B))
        s["k_pages"], s["v_pages"], s["table"] = _pool(case, gen, rows, 0)
        s["k"], s["v"] = _rand(gen, dt, *shape_k), _rand(gen, dt, *shape_k)
        s["q"] = _rand(gen, dt, *shape_q) if case["with_q"] else None
        if own:
            s["q_out"] = torch.empty_like(s["q"]) if case["with_q"] else None
    else:
        lens = torch.tensor(_lens(case), device=DEV)[torch.randperm(B, generator=gen, device=DEV)]
        P = case.get("P", 0)
        s["lens"] = (lens + P).to(torch.int32)
        s["k_pages"], s["v_pages"], s["table"] = _pool(case, gen, max(case["L"], 1), P // case["page"])
        s["q"], s["scale"] = _rand(gen, dt, B, Hq, D), 1.0 / math.sqrt(D)
        if own:  # what a serving loop keeps from step to step
            import exact_tiled_attention_31_b200 as fa
            s["out"] = torch.empty_like(s["q"])
            s["lse"] = torch.empty(B, Hq, dtype=torch.float32, device=DEV)
            size = (fa.fa_decode_prefix_workspace_size(B, Hq, Hkv, P, D) if op == "prefix"
                    else fa.fa_decode_paged_workspace_size(B, Hq, Hkv, D))
            s["ws"] = torch.empty(size, dtype=torch.uint8, device=DEV)
    return s


# ---------------------------------------------------------------- one pass

def run(state):
    s = state
    if own:
        import exact_tiled_attention_31_b200 as fa
        if s["op"] == "rope":
            call = fa.rope_backward if s["inverse"] else fa.rope
            return call(s["q"], s["k"], s["freqs"], positions=s["positions"], cu_seqlens=s["cu"],
                        interleaved=s["interleaved"], amp=s["amp"], out=s["out"])
        if s["op"] == "append":
            q = fa.append_paged(s["k"], s["v"], s["k_pages"], s["v_pages"], s["table"], s["lens"], cu_seqlens=s["cu"],
                                q=s["q"], freqs=s["freqs"], interleaved=s["interleaved"], amp=s["amp"],
                                q_out=s["q_out"])
            return s["k_pages"], s["v_pages"], q
        if s["op"] == "decode":
            return fa.decode_paged(s["q"], s["k_pages"], s["v_pages"], s["table"], s["lens"], scale=s["scale"],
                                   out=s["out"], lse=s["lse"], workspace=s["ws"])
        return fa.decode_prefix(s["q"], s["k_pages"], s["v_pages"], s["table"], s["lens"], s["P"], scale=s["scale"],
                                out=s["out"], lse=s["lse"], workspace=s["ws"])
    return {"rope": _plain_rope, "append": _plain_append, "decode": _plain_decode, "prefix": _plain_prefix}[s["op"]](s)


def _plain_rotate(x, positions, s, sign=1.0):
    """x [..., tokens, D] in 32 bits, rotated by positions [..., tokens]; the angles of far positions in 64."""
    R = s["R"]
    angle = positions[..., None].double() * s["freqs"]
    cos, sin = (angle.cos() * s["amp"]).float(), (angle.sin() * (sign * s["amp"])).float()
    rot, rest = x[..., :R].float(), x[..., R:].float()
    if s["interleaved"]:
        a, b = rot[..., 0::2], rot[..., 1::2]
        rot = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = rot[..., : R // 2], rot[..., R // 2 :]
        rot = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([rot, rest], -1)


def _row_positions(s, n):
    """The place of each packed row in its own sequence."""
    t = torch.arange(n, device=DEV)
    which = torch.searchsorted(s["cu"][1:].contiguous(), t.to(torch.int32), right=True)
    return t - s["cu"].long()[which], which


def _plain_rope(s):
    if s["positions"] is not None:
        pos = s["positions"]
    elif s["cu"] is not None:
        pos = _row_positions(s, s["q"].shape[1])[0]
    else:
        pos = torch.arange(s["S"], device=DEV)[None]
    pos = pos if s["cu"] is not None else pos[:, None, :]
    sign = -1.0 if s["inverse"] else 1.0
    return tuple(_plain_rotate(x, pos, s, sign).to(x.dtype) for x in (s["q"], s["k"]))


def _plain_append(s):
    k, v, q, page = s["k"], s["v"], s["q"], s["page"]
    if s["cu"] is None:  # [B, H, D] -> [H, B, D]
        k, v, q = k.transpose(0, 1), v.transpose(0, 1), None if q is None else q.transpose(0, 1)
        which = torch.arange(s["B"], device=DEV)
        pos = s["lens"].long() - 1
    else:
        at, which = _row_positions(s, k.shape[1])
        new = (s["cu"][1:] - s["cu"][:-1]).long()
        pos = at + (s["lens"].long() - new)[which]
    ids = s["table"].long()[which, pos // page]
    s["k_pages"][ids, :, pos % page] = _plain_rotate(k, pos, s).to(k.dtype).transpose(0, 1)
    s["v_pages"][ids, :, pos % page] = v.transpose(0, 1)
    if q is not None:
        q = _plain_rotate(q, pos, s).to(q.dtype)
        q = q.transpose(0, 1).contiguous() if s["cu"] is None else q
    return s["k_pages"], s["v_pages"], q


def _plain_rows(pages, table):
    """[B, Hkv, rows, D] in 32 bits of the pages that the table names."""
    x = pages[table.long()].transpose(1, 2)  # B, Hkv, pages, page, D
    return x.reshape(x.shape[0], x.shape[1], -1, x.shape[-1]).float()


def _plain_softmax(score):
    """Weights and the logarithm of their sum, of rows that may be all -inf."""
    top = score.amax(-1, keepdim=True)
    e = torch.exp(score - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    total = e.sum(-1, keepdim=True)
    return e / total.clamp(min=1e-38), (top + total.log())[..., 0]


def _plain_own_scores(s, start):
    """Scores [B, Hkv, G, rows] of the rows from `start` on, -inf past the length, and the V rows, zero there."""
    first = start // s["page"]
    B, G = s["B"], s["Hq"] // s["Hkv"]
    k, v = (_plain_rows(s[x], s["table"][:, first:]) for x in ("k_pages", "v_pages"))
    live = start + torch.arange(k.shape[2], device=DEV) < s["lens"][:, None].long()
    q = s["q"].float().view(B, s["Hkv"], G, s["D"]) * s["scale"]
    score = (q @ k.transpose(-1, -2)).masked_fill(~live[:, None, None], -math.inf)
    return score, v.masked_fill(~live[:, None, :, None], 0.0)


def _plain_decode(s):
    score, v = _plain_own_scores(s, 0)
    p, lse = _plain_softmax(score)
    return (p @ v).reshape(s["q"].shape).to(s["q"].dtype), lse.reshape(s["B"], s["Hq"])


def _plain_prefix(s):
    B, Hkv, G, D, P = s["B"], s["Hkv"], s["Hq"] // s["Hkv"], s["D"], s["P"]
    score, v = _plain_own_scores(s, P)
    k0, v0 = (_plain_rows(s[x], s["table"][:1, : P // s["page"]])[0] for x in ("k_pages", "v_pages"))
    q = (s["q"].float() * s["scale"]).view(B, Hkv, G, D).transpose(0, 1).reshape(Hkv, B * G, D)
    both = torch.cat([(q @ k0.transpose(-1, -2)).view(Hkv, B, G, P).transpose(0, 1), score], -1)
    p, lse = _plain_softmax(both)
    o = p[..., P:] @ v
    o0 = p[..., :P].transpose(0, 1).reshape(Hkv, B * G, P) @ v0
    o = o + o0.view(Hkv, B, G, D).transpose(0, 1)
    return o.reshape(s["q"].shape).to(s["q"].dtype), lse.reshape(B, s["Hq"])


# ---------------------------------------------------------------- in 64 bits

def _turn(x, pos, s, conj):
    """The first R columns of x [H, tokens, D] as complex numbers, times amp exp(i pos f)."""
    R = s["R"]
    y = x.double().clone()
    z = y[..., :R].reshape(*y.shape[:-1], R // 2, 2) if s["interleaved"] else \
        y[..., :R].reshape(*y.shape[:-1], 2, R // 2).transpose(-1, -2)
    w = torch.polar(torch.full((1,), float(s["amp"]), dtype=torch.float64, device=DEV),
                    torch.outer(pos.double(), s["freqs"]))
    z = torch.view_as_real(torch.view_as_complex(z.contiguous()) * (w.conj() if conj else w))
    y[..., :R] = (z if s["interleaved"] else z.transpose(-1, -2)).reshape(*y.shape[:-1], R)
    return y


def _attend(q, k, v, scale):
    """[G, D] against [n, D] rows, in 64 bits."""
    if k.shape[0] == 0:
        return torch.zeros_like(q), torch.full((q.shape[0],), -math.inf, dtype=torch.float64, device=DEV)
    score = (q @ k.T) * scale
    lse = torch.logsumexp(score, -1)
    return torch.exp(score - lse[:, None]) @ v, lse


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "rope":
        got = []
        for x in (s["q"], s["k"]):
            if s["cu"] is not None:
                cu = s["cu"].tolist()
                pos = s["positions"] if s["positions"] is not None else \
                    torch.cat([torch.arange(b - a, device=DEV) for a, b in zip(cu, cu[1:])])
                got.append(_turn(x, pos, s, s["inverse"]))
            else:
                rows = [s["positions"][b] if s["positions"] is not None else torch.arange(s["S"], device=DEV)
                        for b in range(s["B"])]
                got.append(torch.stack([_turn(x[b], rows[b], s, s["inverse"]) for b in range(s["B"])]))
        return tuple(got)
    lens = s["lens"].tolist()
    page = s["page"]
    if s["op"] == "append":
        k_pages, v_pages = s["k_pages"].double(), s["v_pages"].double()
        cu = list(range(s["B"] + 1)) if s["cu"] is None else s["cu"].tolist()
        heads_first = (lambda x: x.transpose(0, 1)) if s["cu"] is None else (lambda x: x)
        k, v = heads_first(s["k"]), heads_first(s["v"])
        q = None if s["q"] is None else heads_first(s["q"]).double().clone()
        for b in range(s["B"]):
            pos = torch.arange(lens[b] - (cu[b + 1] - cu[b]), lens[b], device=DEV)
            rows = slice(cu[b], cu[b + 1])
            at = s["table"][b].long()[pos // page]
            k_pages[at, :, pos % page] = _turn(k[:, rows], pos, s, False).transpose(0, 1)
            v_pages[at, :, pos % page] = v[:, rows].double().transpose(0, 1)
            if q is not None:
                q[:, rows] = _turn(q[:, rows], pos, s, False)
        if q is not None:
            q = heads_first(q).contiguous()
        return k_pages, v_pages, q
    B, Hkv, D, P = s["B"], s["Hkv"], s["D"], case.get("P", 0)
    q = s["q"].double().view(B, Hkv, -1, D)
    o = torch.empty_like(q)
    lse = torch.empty(q.shape[:3], dtype=torch.float64, device=DEV)
    shared = s["table"][0, : P // page].long()
    for h in range(Hkv):
        k0, v0 = (s[x][shared, h].reshape(-1, D).double() for x in ("k_pages", "v_pages"))
        # the shared rows for all sequences, then each sequence's own, joined by their logarithms
        o0, l0 = _attend(q[:, h].reshape(-1, D), k0, v0, s["scale"])
        o0, l0 = o0.view(B, -1, D), l0.view(B, -1)
        for b in range(B):
            n = lens[b] - P
            own_pages = s["table"][b, P // page : P // page + -(-n // page)].long()
            k, v = (s[x][own_pages, h].reshape(-1, D)[:n].double() for x in ("k_pages", "v_pages"))
            o1, l1 = _attend(q[b, h], k, v, s["scale"])
            both = torch.logaddexp(l0[b], l1)
            w0, w1 = (torch.exp(x - both).nan_to_num(0.0)[:, None] for x in (l0[b], l1))
            o[b, h], lse[b, h] = w0 * o0[b] + w1 * o1, both
    return o.view(B, -1, D), lse.view(B, -1)
