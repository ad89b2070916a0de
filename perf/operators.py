"""The 4-bit paged KV cache and the pages of a cache: what a pass of each costs.

Five operators of a serving loop, each in a plain form (elementary torch
operations) and through the framework's entry points:

  kv_i4      quantise K/V rows into the 4-bit cache at their slots, and read
             them back as BF16 (paged_kv_write_i4, paged_kv_read_i4)
  attention  GQA decode attention over the 4-bit cache
             (paged_decode_attention_i4kv)
  copy       pages copied in every cache of a pool (paged_copy_pages)
  fork       sequences forked: full pages shared, the page in progress copied,
             then pages reserved for the next tokens (paged_fork,
             paged_reserve)
  retire     finished sequences freed, then the live pages moved to the front
             of the pool (paged_free, paged_compact)

The 4-bit form: a row is one KV head's D values of one token, x ~ c s + m with
m the row's smallest value, s = bf16((max - min) / 15) and
c = clamp(rne((x - m) / s), 0, 15); two codes to a byte (element 2j in the low
nibble of byte j), (s, m) beside them as two BF16.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one token of the small test model: the smallest call, latency alone
        dict(name="kv_i4 one token, small heads", op="kv_i4", tokens=1, Hkv=2, D=64, page=16),
        # a 4 x 512-token prefill chunk of the 14B shape entering the cache
        dict(name="kv_i4 prompt chunk", op="kv_i4", tokens=2048, Hkv=8, D=128, page=128),
        # the largest chunk one prefill call takes
        dict(name="kv_i4 longest chunk", op="kv_i4", tokens=16384, Hkv=8, D=128, page=128),
        # a single user's step at a short context
        dict(name="attention batch 1 ctx 256", op="attention", B=1, Hkv=8, G=5, D=128, page=128,
             lo=256, hi=256, empty=0),
        # the batched decode workload: 16 requests, contexts 64 to 4096
        dict(name="attention batch 16 ctx 4096", op="attention", B=16, Hkv=8, G=5, D=128, page=128,
             lo=64, hi=4096, empty=0),
        # small heads and pages, an odd batch with padded rows, odd contexts
        dict(name="attention small heads ragged", op="attention", B=13, Hkv=2, G=2, D=64, page=16,
             lo=1, hi=2111, empty=3),
        # a full server: long contexts over a large pool
        dict(name="attention batch 64 ctx 16384", op="attention", B=64, Hkv=8, G=5, D=128, page=128,
             lo=64, hi=16384, empty=0),
        # one page of one layer's BF16 K and V: the smallest copy
        dict(name="copy one page of one layer", op="copy", kind="bf16", layers=1, Hkv=8, D=128,
             page=128, blocks=64, n=1),
        # sequences duplicated through all 40 layers of the 4-bit pool
        dict(name="copy pages of 40 layers", op="copy", kind="i4", layers=40, Hkv=8, D=128,
             page=128, blocks=256, n=96),
        # four samples of one prompt, and 64 children of 16 sequences
        dict(name="fork one prompt into 4", op="fork", layers=40, Hkv=8, D=128, page=128, rows=8,
             max_blocks=8, blocks=64, parents=1, n=4, grow=128),
        dict(name="fork 64 children", op="fork", layers=40, Hkv=8, D=128, page=128, rows=96,
             max_blocks=32, blocks=448, parents=16, n=64, grow=160),
        # a server's turn: 24 of 64 sequences end, the pool closes up
        dict(name="retire 24 of 64 and compact", op="retire", layers=40, Hkv=8, D=128, page=128,
             rows=64, max_blocks=12, blocks=640, n=24),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["kv_i4", "attention", "attention", "copy", "fork", "retire"])
    D = rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 4, 5, 8, 8])
    page = rng.choice([16, 24, 32, 64, 96, 128, 128])
    if op == "kv_i4":
        return dict(op=op, tokens=_log_int(rng, 1, 16384), Hkv=Hkv, D=D, page=page)
    if op == "attention":
        B = _log_int(rng, 1, 64)
        hi = min(_log_int(rng, 1, 16384), 1 << 20)
        lo = rng.randint(1, min(hi, 64))
        return dict(op=op, B=B, Hkv=Hkv, G=rng.randint(1, 8), D=D, page=page, lo=lo, hi=hi,
                    empty=rng.randint(0, B // 4))
    layers = _log_int(rng, 1, 40)
    if op == "copy":
        blocks = _log_int(rng, 8, 256)
        return dict(op=op, kind=rng.choice(["bf16", "i8", "i4"]) if layers <= 10 else "i4",
                    layers=layers, Hkv=Hkv, D=D, page=page, blocks=blocks,
                    n=rng.randint(1, max(1, blocks * 3 // 8)))
    if op == "fork":
        parents = _log_int(rng, 1, 16)
        n = _log_int(rng, 1, 64)
        max_blocks = rng.randint(4, 32)
        return dict(op=op, layers=layers, Hkv=Hkv, D=D, page=page, rows=parents + n + rng.randint(0, 8),
                    max_blocks=max_blocks, blocks=parents * max_blocks + 3 * n + rng.randint(0, 32),
                    parents=parents, n=n, grow=rng.randint(1, 2 * page))
    rows = _log_int(rng, 2, 64)
    max_blocks = rng.randint(2, 12)
    return dict(op=op, layers=layers, Hkv=Hkv, D=D, page=page, rows=rows, max_blocks=max_blocks,
                blocks=rows * max_blocks * 3 // 4 + 16, n=rng.randint(1, max(1, rows * 3 // 8)))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _gen(seed, k):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 1000 + k)
    return g


def _spread(lo, hi, n, r):
    """n integers spread evenly over [lo, hi] (their sum does not depend on the seed), shuffled."""
    v = [lo + round((hi - lo) * (i + 0.5) / n) for i in range(n)]
    r.shuffle(v)
    return v


def _codes(shape, g):
    """Random packed codes, both nibbles spread about the middle as those of normal rows are."""
    u = torch.randint(0, 256, shape, dtype=torch.uint8, device=DEV, generator=g)
    w = torch.randint(0, 256, shape, dtype=torch.uint8, device=DEV, generator=g)
    lo = (u & 7) + ((u >> 3) & 7) + (u >> 7)
    hi = (w & 7) + ((w >> 3) & 7) + (w >> 7)
    return lo | (hi << 4)


def _meta(shape, g):
    """(s, m) pairs of rows of unit-variance values: a range of about 5 over 15 steps."""
    s = 0.35 * (0.7 + 0.6 * torch.rand(shape, device=DEV, generator=g))
    m = -7.5 * s * (0.85 + 0.3 * torch.rand(shape, device=DEV, generator=g))
    return torch.stack((s, m), dim=-1).to(torch.bfloat16)


def _i4_pool(case, L, g):
    N, page, Hkv, D = case["blocks"], case["page"], case["Hkv"], case["D"]
    codes = torch.randint(0, 256, (2 * L, N, page, Hkv, D // 2), dtype=torch.uint8, device=DEV,
                          generator=g)
    meta = _meta((2 * L, N, page, Hkv), g)
    return [codes, meta]


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _tables(s, bt, ctx, ref, others):
    """The block table, contexts and reference counts in one int32 buffer (each part 16-byte
    aligned), and the buffer that a pass starts from: a pass changes them in place."""
    parts, at = [], 0
    for a in (bt, ctx, ref):
        parts.append((at, a))
        at += (a.numel() + 3) // 4 * 4
    start = torch.zeros(at, dtype=torch.int32, device=DEV)
    for o, a in parts:
        start[o:o + a.numel()] = a.reshape(-1)
    s["start"], s["now"] = start, start.clone()
    for name, (o, a) in zip(("bt", "ctx", "ref"), parts):
        s[name] = s["now"][o:o + a.numel()].view(a.shape)
    s.update(others)


def prepare(case, seed):
    r = random.Random(seed * 77 + 5)
    g = _gen(seed, 1)
    s = dict(case=case)
    op, page = case["op"], case["page"]
    if op == "kv_i4":
        T, Hkv, D = case["tokens"], case["Hkv"], case["D"]
        N = (T + page - 1) // page + 3
        shift = torch.randn((1, Hkv, D), device=DEV, generator=g)   # channels with means of their own
        s["k"] = (torch.randn((T, Hkv, D), device=DEV, generator=g) + shift).to(torch.bfloat16)
        s["v"] = torch.randn((T, Hkv, D), device=DEV, generator=g).to(torch.bfloat16)
        pages = torch.randperm(N, device=DEV, generator=g)
        t = torch.arange(T, device=DEV)
        s["slots"] = (pages[t // page] * page + t % page).to(torch.int32)
        s["kc"] = torch.zeros((N * page, Hkv, D // 2), dtype=torch.uint8, device=DEV)
        s["vc"] = torch.zeros_like(s["kc"])
        s["km"] = torch.zeros((N * page, Hkv, 2), dtype=torch.bfloat16, device=DEV)
        s["vm"] = torch.zeros_like(s["km"])
        return s
    if op == "attention":
        B, Hkv, D = case["B"], case["Hkv"], case["D"]
        ctx = _spread(case["lo"], case["hi"], B - case["empty"], r) + [0] * case["empty"]
        r.shuffle(ctx)
        used = [(c + page - 1) // page for c in ctx]
        M = (case["hi"] + page - 1) // page
        N = sum(used) + 2
        pages = torch.randperm(N, device=DEV, generator=g).to(torch.int32).tolist()
        bt, at = [], 0
        for u in used:
            bt.append(pages[at:at + u] + [-1] * (M - u))
            at += u
        s["bt"], s["ctx"] = _i32(bt), _i32(ctx)
        s["q"] = (1.5 * torch.randn((B, Hkv * case["G"], D), device=DEV, generator=g)).to(torch.bfloat16)
        for n in ("k", "v"):
            s[n + "c"] = _codes((N * page, Hkv, D // 2), g)
            s[n + "m"] = _meta((N * page, Hkv), g)
        return s
    L, N = case["layers"], case["blocks"]
    if op == "copy":
        Hkv, D = case["Hkv"], case["D"]
        if case["kind"] == "i4":
            s["pool"] = _i4_pool(case, L, g)
        elif case["kind"] == "i8":
            s["pool"] = [torch.randint(-127, 128, (2 * L, N, page, Hkv, D), dtype=torch.int8,
                                       device=DEV, generator=g),
                         torch.rand((2 * L, N, page, Hkv), device=DEV, generator=g)]
        else:
            s["pool"] = [torch.randn((2 * L, N, page, Hkv, D), device=DEV, generator=g).to(torch.bfloat16)]
        p = torch.randperm(N, device=DEV, generator=g).to(torch.int32)
        s["src"], s["dst"] = p[:case["n"]].clone(), p[case["n"]:2 * case["n"]].clone()
        return s
    s["pool"] = _i4_pool(case, L, g)
    B, M = case["rows"], case["max_blocks"]
    order = list(range(N))
    r.shuffle(order)
    bt, ctx, ref = [[-1] * M for _ in range(B)], [0] * B, [0] * N
    rows = list(range(B))
    r.shuffle(rows)
    live = rows[:case["parents"]] if op == "fork" else rows
    room = max(1, M - 3) if op == "fork" else M      # forked rows keep room for their next pages
    lens = _spread(1 if len(live) > 1 else page // 2 + (room - 1) * page, room * page, len(live), r)
    at = 0
    for b, c in zip(live, lens):
        if op == "retire":
            c = min(c, (N - 8 - at) * page)
        u = (c + page - 1) // page
        ctx[b] = c
        bt[b][:u] = order[at:at + u]
        for x in order[at:at + u]:
            ref[x] = 1
        at += u
    if op == "fork":
        parents = [live[i % len(live)] for i in range(case["n"])]
        children = rows[case["parents"]:case["parents"] + case["n"]]
        _tables(s, _i32(bt), _i32(ctx), _i32(ref), dict(
            parents=_i32(parents), children=_i32(children),
            tokens=_i32([min(ctx[p] + case["grow"], M * page) for p in parents])))
    else:
        _tables(s, _i32(bt), _i32(ctx), _i32(ref), dict(rows=_i32(rows[:case["n"]])))
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _quant(x):
    """Codes (one to a byte) and (s, m) of rows x [..., D] bf16."""
    f = x.float()
    lo, hi = f.amin(-1, keepdim=True), f.amax(-1, keepdim=True)
    s = ((hi - lo) / torch.full_like(lo, 15.0)).to(torch.bfloat16)
    q = torch.round((f - lo) / s.float())
    c = torch.where(s == 0, torch.zeros_like(q), q).clamp(0, 15).to(torch.uint8)
    return c, torch.cat((s, lo.to(torch.bfloat16)), dim=-1)


def _unpack(codes):
    return torch.stack((codes & 15, codes >> 4), dim=-1).reshape(*codes.shape[:-1], -1)


def _dequant(codes, meta):
    m = meta.float()
    return _unpack(codes).float() * m[..., :1] + m[..., 1:]


def _plain_kv(s):
    at = s["slots"].long()
    out = []
    for x, c, m in ((s["k"], s["kc"], s["km"]), (s["v"], s["vc"], s["vm"])):
        q, meta = _quant(x)
        c[at] = q[..., 0::2] | (q[..., 1::2] << 4)
        m[at] = meta
        out.append(_dequant(c[at], m[at]).to(torch.bfloat16))
    return out


def _plain_attention(s):
    case = s["case"]
    B, Hkv, D, page = case["B"], case["Hkv"], case["D"], case["page"]
    M = s["bt"].shape[1]
    at = s["bt"].long().clamp(min=0)
    pages = lambda c: c.view(-1, page, *c.shape[1:])[at].reshape(B, M * page, *c.shape[1:])  # noqa: E731
    k = _dequant(pages(s["kc"]), pages(s["km"])).permute(0, 2, 3, 1)        # [B, Hkv, D, T]
    q = s["q"].float().view(B, Hkv, case["G"], D)
    x = torch.matmul(q, k) * (1.0 / math.sqrt(D))
    del k
    hidden = torch.arange(M * page, device=DEV)[None] >= s["ctx"][:, None]
    x = x.masked_fill(hidden[:, None, None], -math.inf)
    e = torch.exp(x - x.amax(-1, keepdim=True).clamp(min=-3e38))
    v = _dequant(pages(s["vc"]), pages(s["vm"])).permute(0, 2, 1, 3)        # [B, Hkv, T, D]
    o = torch.matmul(e, v) / e.sum(-1, keepdim=True).clamp(min=1e-30)
    return o.reshape(B, Hkv * case["G"], D).to(torch.bfloat16)


def _bits(pool):
    """The pool's caches as whole numbers: a copy is the same bits."""
    kinds = {2: torch.int16, 4: torch.int32}
    return [c.view(kinds.get(c.element_size(), c.dtype)) for c in pool]


def _plain_copy(s):
    src, dst = s["src"].long(), s["dst"].long()
    for c in s["pool"]:
        c[:, dst] = c[:, src]
    return _bits(s["pool"])


def _plain_reserve(s, rows, tokens):
    page, M = s["case"]["page"], s["bt"].shape[1]
    j = torch.arange(M, device=DEV)
    r = rows.long()
    old = s["bt"][r]
    want = (old < 0) & (j[None] < ((tokens + page - 1) // page)[:, None])
    free = torch.nonzero(s["ref"] == 0)[:, 0]
    rank = torch.cumsum(want.reshape(-1), 0).view(want.shape) - 1
    fresh = free[rank.clamp(min=0)].to(torch.int32)
    s["bt"][r] = torch.where(want, fresh, old)
    s["ref"][fresh[want].long()] = 1


def _plain_fork(s):
    page, M = s["case"]["page"], s["bt"].shape[1]
    s["now"].copy_(s["start"])
    p, c = s["parents"].long(), s["children"].long()
    ctx, old = s["ctx"][p], s["bt"][p]
    full, part = (ctx // page)[:, None], ctx % page
    j = torch.arange(M, device=DEV)[None]
    need = part > 0
    free = torch.nonzero(s["ref"] == 0)[:, 0]
    fresh = free[(torch.cumsum(need, 0) - 1).clamp(min=0)]
    rows = torch.where(j < full, old, torch.full_like(old, -1))
    shared = rows[rows >= 0].long()
    rows = torch.where((j == full) & need[:, None], fresh[:, None].to(torch.int32), rows)
    s["bt"][c], s["ctx"][c] = rows, ctx
    s["ref"].index_add_(0, shared, torch.ones_like(shared, dtype=torch.int32))
    to = fresh[need]
    s["ref"][to] = 1
    frm = old.gather(1, full.clamp(max=M - 1).long())[:, 0][need].long()
    used = torch.arange(page, device=DEV)[None] < part[need][:, None]       # [n, page]
    for x in s["pool"]:
        x[:, to] = torch.where(used[None, :, :, None, None], x[:, frm], x[:, to])
    _plain_reserve(s, s["children"], s["tokens"])
    return [s["bt"], s["ctx"], s["ref"]] + _bits(s["pool"])


def _plain_retire(s):
    s["now"].copy_(s["start"])
    r, ref, bt = s["rows"].long(), s["ref"], s["bt"]
    held = bt[r]
    held = held[held >= 0].long()
    ref.index_add_(0, held, torch.full_like(held, -1, dtype=torch.int32))
    bt[r] = -1
    s["ctx"][r] = 0
    live = ref > 0
    n = live.sum()
    low = torch.arange(ref.numel(), device=DEV) < n
    holes, movers = torch.nonzero(~live & low)[:, 0], torch.nonzero(live & ~low)[:, 0]
    to = torch.arange(ref.numel(), dtype=torch.int32, device=DEV)
    to[movers] = holes.to(torch.int32)
    for x in s["pool"]:
        x[:, holes] = x[:, movers]
    bt.copy_(torch.where(bt >= 0, to[bt.long().clamp(min=0)], bt))
    ref[holes] = ref[movers]
    ref[movers] = 0
    return [bt, s["ctx"], ref, n.to(torch.int32).reshape(1)] + _bits(s["pool"])


# ---------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------

def _handle(s):
    """The handle, workspace and buffers that a program makes once for its pool."""
    import w8a8_quantized_decode_gb300 as a8w8
    if "made" not in s:
        s["made"] = True
        case = s["case"]
        if case["op"] == "attention":
            B, Hkv = case["B"], case["Hkv"]
            need = a8w8.attention_i4_workspace_bytes(B, Hkv * case["G"], Hkv, case["D"],
                                                     s["bt"].shape[1] * case["page"])
            s["ws"] = torch.empty(max(need, 16), dtype=torch.uint8, device=DEV)
        elif case["op"] != "kv_i4":
            caches = [c[i] for i in range(2 * case["layers"]) for c in s["pool"]]
            s["pages"] = a8w8.PagePool(caches, case["blocks"], case["page"])
            need = a8w8.pages_workspace_bytes(case["blocks"], case.get("rows", 1), case["n"])
            s["ws"] = torch.empty(max(need, 16), dtype=torch.uint8, device=DEV)
            s["live"] = torch.empty(1, dtype=torch.int32, device=DEV)
    return a8w8


def _own(s):
    a8w8 = _handle(s)
    case = s["case"]
    op = case["op"]
    if op == "kv_i4":
        a8w8.paged_kv_write_i4(s["k"], s["v"], s["slots"], s["kc"], s["vc"], s["km"], s["vm"],
                               case["page"])
        return list(a8w8.paged_kv_read_i4(s["kc"], s["vc"], s["km"], s["vm"], s["slots"],
                                          case["page"]))
    if op == "attention":
        return a8w8.paged_decode_attention_i4kv(s["q"], s["kc"], s["vc"], s["km"], s["vm"], s["bt"],
                                                s["ctx"], case["page"], ws=s["ws"])
    if op == "copy":
        a8w8.paged_copy_pages(s["pages"], s["src"], s["dst"])
        return _bits(s["pool"])
    s["now"].copy_(s["start"])
    if op == "fork":
        a8w8.paged_fork(s["pages"], s["bt"], s["ctx"], s["ref"], s["parents"], s["children"],
                        ws=s["ws"])
        a8w8.paged_reserve(s["pages"], s["bt"], s["ref"], s["children"], s["tokens"], ws=s["ws"])
        return [s["bt"], s["ctx"], s["ref"]] + _bits(s["pool"])
    a8w8.paged_free(s["pages"], s["bt"], s["ctx"], s["ref"], s["rows"])
    a8w8.paged_compact(s["pages"], s["bt"], s["ref"], num_live=s["live"], ws=s["ws"])
    return [s["bt"], s["ctx"], s["ref"], s["live"]] + _bits(s["pool"])


PLAIN = {"kv_i4": _plain_kv, "attention": _plain_attention, "copy": _plain_copy,
         "fork": _plain_fork, "retire": _plain_retire}


def run(state):
    if own:
        return _own(state)
    return PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# work and exact values
# ---------------------------------------------------------------------------

def _token_bytes(case):
    per = {"bf16": 2 * case["D"], "i8": case["D"] + 4, "i4": case["D"] // 2 + 4}
    return 2 * case["layers"] * case["Hkv"] * per[case.get("kind", "i4")]


def work(case):
    op, page = case["op"], case["page"]
    if op == "kv_i4":
        rows = 2 * case["tokens"] * case["Hkv"]
        one = case["D"] // 2 + 4
        # BF16 rows in, codes out; codes in, BF16 rows out; the slots
        return dict(bytes=rows * (4 * case["D"] + 2 * one) + 4 * case["tokens"],
                    flops=rows * case["D"] * 6)
    if op == "attention":
        Hq, D = case["Hkv"] * case["G"], case["D"]
        ctx = _spread(case["lo"], case["hi"], case["B"] - case["empty"], random.Random(0))
        tokens = sum(ctx)
        pages = sum((c + page - 1) // page for c in ctx)
        return dict(bytes=tokens * case["Hkv"] * (D + 8) + 4 * (pages + case["B"])
                    + 4 * case["B"] * Hq * D, flops=4 * tokens * Hq * D)
    if op == "copy":
        return dict(bytes=2 * case["n"] * page * _token_bytes(case) + 8 * case["n"], flops=0)
    M, B, N = case["max_blocks"], case["rows"], case["blocks"]
    if op == "fork":
        # the partial page of each child, half a page on average, and the tables
        return dict(bytes=case["n"] * page * _token_bytes(case) + 4 * (2 * case["n"] * M + 2 * N),
                    flops=0)
    # the pages behind the last live place, about the share of the rows that end, move forward
    lens = _spread(1 if B > 1 else page // 2 + (M - 1) * page, M * page, B, random.Random(0))
    pages = min(sum((c + page - 1) // page for c in lens), N - 8)
    left = pages * (B - case["n"]) / B
    moved = left * (1 - left / N)
    return dict(bytes=2 * moved * page * _token_bytes(case) + 4 * (2 * B * M + 2 * N), flops=0)


def _exact_kv(s):
    out = []
    for x in (s["k"], s["v"]):
        f = x.cpu().view(torch.int16).numpy().view(np.uint16).astype(np.uint32)
        f = (f << 16).view(np.float32).astype(np.float64)
        lo = f.min(-1, keepdims=True)
        step = ((f.max(-1, keepdims=True) - lo).astype(np.float32) / np.float32(15)).astype(np.float32)
        u = step.view(np.uint32)                            # to BF16, ties to even
        step = ((u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000).view(np.float32).astype(np.float64)
        # the definition rounds the difference and the quotient to 32 bits before the code
        d = (f - lo).astype(np.float32).astype(np.float64)
        q = np.rint(np.divide(d, step, out=np.zeros_like(d), where=step > 0).astype(np.float32))
        out.append(np.clip(q, 0, 15).astype(np.float64) * step + lo)
    return out


def _exact_attention(s):
    case = s["case"]
    Hkv, G, D, page = case["Hkv"], case["G"], case["D"], case["page"]
    out = torch.zeros((case["B"], Hkv * G, D), dtype=torch.float64, device=DEV)
    j = torch.arange(D, device=DEV)
    for b, n in enumerate(s["ctx"].tolist()):
        t = torch.arange(n, device=DEV)
        at = s["bt"][b].long()[t // page] * page + t % page if n else None
        for h in range(Hkv if n else 0):
            kv = []
            for c, m in ((s["kc"], s["km"]), (s["vc"], s["vm"])):
                byte = c[at, h].to(torch.int64)[:, j // 2]
                code = (byte // torch.where(j % 2 == 1, 16, 1)) % 16
                sm = m[at, h].double()
                kv.append(code.double() * sm[:, :1] + sm[:, 1:])
            q = s["q"][b, h * G:(h + 1) * G].double()
            w = torch.softmax((q @ kv[0].T) / math.sqrt(D), dim=-1)
            out[b, h * G:(h + 1) * G] = w @ kv[1]
    return out


def exact(case, seed):
    if case["op"] not in ("kv_i4", "attention"):
        return None      # pages and tables are whole values: nothing is computed
    s = prepare(case, seed)
    return _exact_kv(s) if case["op"] == "kv_i4" else _exact_attention(s)
