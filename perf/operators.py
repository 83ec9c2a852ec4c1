"""Measured cases of the paged key/value cache held in 4 bits, with the operators' plain forms.

A pool holds pages of `page` positions.  A page is [nkv][page / 16][block]; a block holds 16 positions of one head:
the key codes, the value codes, the keys' scales, the values' scales.  A group of 64 dims of one position and head
shares a scale s = bf16(max |x| / 7); a code is n + 8 with n = rint(x / s) in [-8, 7], and stands for n s.
"""
import math
import random

import torch

own = False

GROUP = 64


# ------------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one sequence decoding one token after a short prompt: latency alone
        dict(name="attn_single_token", op="attn", B=1, Q=1, nkv=10, grp=1, d=128, page=64, cap=512, low=300, high=301,
             lens=1),
        # the verify pass: 32 sequences, 3 drafts each, page-shaped contexts (visual tokens and text written so far)
        dict(name="attn_verify_pages", op="attn", B=32, Q=4, nkv=10, grp=1, d=128, page=64, cap=2304, low=360,
             high=2245, lens=2),
        # ragged lengths from one token on, narrow heads, shared key heads, small pages
        dict(name="attn_ragged_grouped", op="attn", B=13, Q=3, nkv=3, grp=5, d=64, page=16, cap=9000, low=3, high=9000,
             lens=3),
        # long documents: 16 sequences near 32K positions, four query heads a key head, 3 drafts
        dict(name="attn_long", op="attn", B=16, Q=4, nkv=8, grp=4, d=128, page=64, cap=32768, low=30000, high=32768,
             lens=4),
        # the verified positions of a step go to the cache
        dict(name="append_verify", op="append", B=32, Q=4, nkv=10, d=128, page=64, cap=2304, low=360, high=2245,
             lens=5),
        # prompts of whole pages go to the cache at once, behind prefixes of any length
        dict(name="append_prompt", op="append", B=8, Q=1156, nkv=10, d=128, page=64, cap=4000, low=1156, high=4000,
             lens=6),
        # between two verify steps: rejected drafts given back, room for the next ones, few pages change
        dict(name="resize_step", op="resize", B=32, M=36, P=1152, layers=11, pb=87040, page=64, low=360, high=2245,
             grow=5, shared=8, lens=7),
        # a scheduler's turn over many sequences: some end, some are admitted, some grow, forked ones separate
        dict(name="resize_turnover", op="resize", B=509, M=1000, P=400000, layers=1, pb=4352, page=16, low=16,
             high=15000, grow=900, shared=64, lens=8),
        # beams of a few sequences
        dict(name="fork_beams", op="fork", B=32, M=36, P=1152, low=6, high=36, lens=9),
        # many beams over long tables
        dict(name="fork_wide", op="fork", B=1000, M=1024, P=700000, low=60, high=1024, lens=10),
        # a small pool of one layer with holes
        dict(name="compact_small", op="compact", B=8, M=40, P=300, layers=1, pb=8704, low=5, high=36, lens=11),
        # every layer's pages after a burst of long documents ended
        dict(name="compact_layers", op="compact", B=48, M=64, P=2048, layers=11, pb=87040, low=4, high=36, lens=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "append", "append", "resize", "fork", "compact"])
    lens = rng.randrange(1, 1 << 30)
    page = rng.choice([16, 32, 64, 128])
    d = rng.choice([64, 128])
    if op == "attn":
        while True:
            B, nkv, cap = _log(rng, 1, 64), _log(rng, 1, 16), _log(rng, 16, 32768)
            Q = rng.randint(1, min(8, cap))
            grp = rng.choice([1, 2, 3, 4, 8] if Q <= 4 else [1, 2, 3, 4])
            if B * nkv * cap * d <= 16 * 8 * 32768 * 128 and Q * grp <= 16:
                break
        low = _log(rng, Q, cap)
        return dict(op=op, B=B, Q=Q, nkv=nkv, grp=grp, d=d, page=page, cap=cap, low=low, high=rng.randint(low, cap),
                    lens=lens)
    if op == "append":
        while True:
            B, Q, nkv = _log(rng, 1, 256), _log(rng, 1, 8000), _log(rng, 1, 16)
            if B * Q * nkv * d <= 8 * 1156 * 10 * 128:
                break
        cap = Q + _log(rng, 1, 4000)
        low = rng.randint(Q, cap)
        return dict(op=op, B=B, Q=Q, nkv=nkv, d=d, page=page, cap=cap, low=low, high=rng.randint(low, cap), lens=lens)
    if op == "resize":
        B, M = _log(rng, 1, 509), _log(rng, 4, 1000)
        layers = rng.choice([1, 2, 11]) if B * M <= 2000 else 1
        low = _log(rng, 1, (M - 1) * page)
        return dict(op=op, B=B, M=M, P=B * M - B * M // 5 + B + 8, layers=layers, pb=page * 272, page=page, low=low,
                    high=rng.randint(low, (M - 1) * page), grow=_log(rng, 1, page * 8), shared=rng.randint(0, B // 2),
                    lens=lens)
    if op == "fork":
        B, M = _log(rng, 1, 1000), _log(rng, 1, 1024)
        low = _log(rng, 1, M)
        return dict(op=op, B=B, M=M, P=B * M - B * M // 4 + B, low=low, high=rng.randint(low, M), lens=lens)
    while True:
        B, M, layers = _log(rng, 1, 48), _log(rng, 2, 64), rng.choice([1, 2, 11])
        P, pb = B * M + rng.randint(0, 200), page * 136 * rng.choice([1, 2, 8])
        if P * layers * pb <= 2048 * 11 * 87040:
            break
    low = _log(rng, 1, M)
    return dict(op=op, B=B, M=M, P=P, layers=layers, pb=pb, low=low, high=rng.randint(low, M), lens=lens)


def _lengths(c):
    """The case's lengths (or page counts), one a sequence: not the seed's, so that every state is the same work."""
    r = random.Random(c["lens"])
    return [r.randint(c["low"], c["high"]) for _ in range(c["B"])]


def _other(c, b):
    """The row whose pages the b-th row from the end was forked from."""
    return b % max(1, c["B"] // 2)


def _turn(c):
    """Lengths before a scheduler's turn, what is kept and what there has to be room for, one a sequence."""
    n, r = _lengths(c), random.Random(c["lens"] + 1)
    # the pool holds what the tables hold and what the turn may take
    room = c["P"] - 2 * c["B"] - c["B"] * -(-c["grow"] // c["page"])
    while sum(-(-x // c["page"]) for x in n) > room and max(n) > 1:
        n = [(x + 1) // 2 for x in n]
    for b in range(c["shared"]):  # forked ones: the same pages as another row's, the last one partly filled
        n[c["B"] - 1 - b] = n[_other(c, b)]
    keep = [max(0, x - r.randint(0, 3)) if r.random() >= 0.05 else 0 for x in n]
    cap = [min(k + c["grow"], c["M"] * c["page"]) if k else 0 for k in keep]
    return n, keep, cap


# ------------------------------------------------------------------------------------------------ layout
def _block(d):
    return 16 * (d + 4 * (d // GROUP))


def _k_byte_dims(d, device):
    """[d / 2] dims of the low nibbles of a position's key bytes; the high nibble's dim is two further."""
    x = torch.arange(d // 2, device=device)
    t, j, i = x // (d // 8), x // 4 % (d // 32), x % 4
    return 32 * j + 8 * t + 4 * (i & 1) + (i >> 1)


def _quantise(x):
    """bf16 [..., d] -> codes 0..15 [..., d] (uint8), scales [..., d / 64] (bf16)."""
    g = x.float().unflatten(-1, (-1, GROUP))
    s = (g.abs().amax(-1) / 7).to(torch.bfloat16)
    f = s.float().unsqueeze(-1)
    n = torch.where(f > 0, torch.round(g / f), torch.zeros_like(g)).clamp(-8, 7)
    return (n + 8).to(torch.uint8).flatten(-2), s


def _pack(kc, ks, vc, vs):
    """Codes [N, 16, d] and scales [N, 16, d / 64] of 16 positions -> blocks [N, bytes]."""
    N, _, d = kc.shape
    lo = _k_byte_dims(d, kc.device)
    kb = kc[..., lo] | (kc[..., lo + 2] << 4)
    # value bytes: [half][g][t][m][position 2t, 2t + 1][2 bytes], byte b of them dims 32 m + 4 g + 2 b (low) and + 1
    vb = vc[..., 0::2] | (vc[..., 1::2] << 4)
    vb = vb.view(N, 2, 4, 2, d // 32, 8, 2).permute(0, 1, 5, 2, 4, 3, 6)
    return torch.cat([kb.reshape(N, -1), vb.reshape(N, -1), ks.contiguous().view(torch.uint8).reshape(N, -1),
                      vs.contiguous().view(torch.uint8).reshape(N, -1)], 1)


def _unpack(blocks, d):
    """Blocks [..., bytes] -> keys, values [..., 16, d] in 32 bits."""
    lead, dev = blocks.shape[:-1], blocks.device
    G, half = d // GROUP, 8 * d
    kb = blocks[..., :half].reshape(*lead, 16, d // 2)
    k = torch.empty(*lead, 16, d, dtype=torch.uint8, device=dev)
    lo = _k_byte_dims(d, dev)
    k[..., lo] = kb & 15
    k[..., lo + 2] = kb >> 4
    n = len(lead)
    vb = blocks[..., half:2 * half].reshape(*lead, 2, 8, 4, d // 32, 2, 2)
    vb = vb.permute(*range(n), n, n + 2, n + 4, n + 3, n + 1, n + 5)
    v = torch.stack([vb & 15, vb >> 4], -1).reshape(*lead, 16, d)
    sc = blocks[..., 2 * half:].contiguous().view(torch.bfloat16).reshape(*lead, 2, 16, G, 1).float()
    k = (k.float() - 8).unflatten(-1, (G, GROUP)) * sc.select(n, 0)
    v = (v.float() - 8).unflatten(-1, (G, GROUP)) * sc.select(n, 1)
    return k.flatten(-2), v.flatten(-2)


# ------------------------------------------------------------------------------------------------ inputs
def _gen(seed, device="cuda"):
    return torch.Generator(device=device).manual_seed(int(seed) * 7919 + 13)


def _pages(c):
    return [-(-n // c["page"]) for n in _lengths(c)]


def _table(c, g, counts, M, P):
    """Every sequence's pages, anywhere in the pool, in any order; -1 behind the last."""
    order = torch.randperm(P, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(counts), M), -1, dtype=torch.int32)
    cnt = torch.tensor(counts)
    used = torch.arange(M)[None, :] < cnt[:, None]
    table[used] = order[:int(cnt.sum())].cpu()
    return table.cuda()


def _rows(g, shape):
    """Projections' outputs: a spread that differs from one position to the next."""
    x = torch.randn(shape, generator=g, device="cuda")
    return (x * (0.5 + torch.rand((*shape[:-1], 1), generator=g, device="cuda"))).to(torch.bfloat16)


def _counts(P, table):
    ref = torch.zeros(P, dtype=torch.int32, device="cuda")
    flat = table[table >= 0].long()
    return ref.index_add_(0, flat, torch.ones_like(flat, dtype=torch.int32))


def prepare(case, seed):
    c, g = case, _gen(seed)
    op = c["op"]
    if op in ("attn", "append"):
        counts = _pages(c) if op == "attn" else [-(-c["cap"] // c["page"])] * c["B"]
        M = -(-c["cap"] // c["page"])
        P = sum(counts) + 3
        per, d = c["nkv"] * (c["page"] // 16), c["d"]
        pool = torch.empty((P, per * _block(d)), dtype=torch.uint8, device="cuda")
        if op == "attn":
            step = max(1, (1 << 26) // (per * 16 * d))
            for p in range(0, P, step):
                n = min(step, P - p) * per
                k, v = _rows(g, (n, 16, d)), _rows(g, (n, 16, d))
                pool[p:p + step] = _pack(*_quantise(k), *_quantise(v)).view(-1, per * _block(d))
        else:
            pool.zero_()
        s = dict(c=c, pool=pool, table=_table(c, g, counts, M, P),
                 ctx=torch.tensor(_lengths(c), dtype=torch.int32).cuda())
        if op == "attn":
            s["q"] = _rows(g, (c["B"], c["Q"], c["nkv"] * c["grp"], d))
            s["out"] = torch.empty_like(s["q"])
        else:
            s["k"], s["v"] = _rows(g, (c["B"], c["Q"], c["nkv"], d)), _rows(g, (c["B"], c["Q"], c["nkv"], d))
        return s
    if op == "fork":
        table = _table(c, g, _lengths(c), c["M"], c["P"])
        # some beams end, some go on in several
        parent = torch.randint(0, c["B"], (c["B"],), generator=g, device="cuda", dtype=torch.int32)
        return dict(c=c, table=table, ref=_counts(c["P"], table), parent=parent, table_out=torch.empty_like(table),
                    ref_out=torch.empty(c["P"], dtype=torch.int32, device="cuda"))
    pool = torch.randint(0, 256, (c["layers"], c["P"], c["pb"]), generator=g, device="cuda", dtype=torch.uint8)
    s = dict(c=c, pool=pool, ref_out=torch.empty(c["P"], dtype=torch.int32, device="cuda"),
             stats=torch.empty(4, dtype=torch.int32, device="cuda"))
    if op == "compact":
        table = _table(c, g, _lengths(c), c["M"], c["P"])
        s |= dict(table=table, ref=_counts(c["P"], table), table_out=torch.empty_like(table),
                  map=torch.empty(c["P"], dtype=torch.int32, device="cuda"))
        return s
    n, keep, cap = _turn(c)
    table = _table(c, g, [-(-x // c["page"]) for x in n], c["M"], c["P"])
    for b in range(c["shared"]):
        table[c["B"] - 1 - b] = table[_other(c, b)]
    keep, cap = torch.tensor(keep, dtype=torch.int32), torch.tensor(cap, dtype=torch.int32)
    s |= dict(table=table, ref=_counts(c["P"], table), keep=keep.cuda(), cap=cap.cuda(),
              table_out=torch.empty_like(table))
    return s


# ------------------------------------------------------------------------------------------------ plain forms
def _plain_attn(s):
    c, q = s["c"], s["q"].float()
    B, Q, nkv, grp, d, page = c["B"], c["Q"], c["nkv"], c["grp"], c["d"], c["page"]
    M = s["table"].shape[1]
    blocks = s["pool"][s["table"].clamp(min=0).long()].view(B, M, nkv, page // 16, _block(d))
    k, v = _unpack(blocks, d)
    T = M * page
    k = k.permute(0, 2, 1, 3, 4, 5).reshape(B, nkv, T, d)
    v = v.permute(0, 2, 1, 3, 4, 5).reshape(B, nkv, T, d)
    t = torch.arange(T, device=q.device)
    n = s["ctx"].long()
    live = (t[None, :] < n[:, None])[:, None, :, None]
    k, v = torch.where(live, k, 0), torch.where(live, v, 0)
    q = q.view(B, Q, nkv, grp, d).permute(0, 2, 1, 3, 4).reshape(B, nkv, Q * grp, d)
    x = (q @ k.transpose(-1, -2) / math.sqrt(d)).view(B, nkv, Q, grp, T)
    seen = t[None, None, :] <= (n[:, None] - Q + torch.arange(Q, device=q.device)[None, :])[:, :, None]
    x = torch.where(seen[:, None, :, None, :], x, -torch.inf)
    p = torch.exp(x - x.amax(-1, keepdim=True))
    o = (p.view(B, nkv, Q * grp, T) @ v).view(B, nkv, Q, grp, d) / p.sum(-1, keepdim=True)
    return o.permute(0, 2, 1, 3, 4).reshape(B, Q, nkv * grp, d).to(torch.bfloat16)


def _places(s):
    """Offset of the block of each new position and head in the pool [B, Q, nkv], and its place in the block [B, Q]."""
    c = s["c"]
    pos = s["ctx"].long()[:, None] - c["Q"] + torch.arange(c["Q"], device=s["ctx"].device)
    pg = torch.gather(s["table"].long(), 1, pos // c["page"])
    head = torch.arange(c["nkv"], device=pos.device)
    blk = (pg[..., None] * c["nkv"] + head) * (c["page"] // 16) + (pos % c["page"] // 16)[..., None]
    return blk * _block(c["d"]), pos % 16


def _plain_append(s):
    c, d = s["c"], s["c"]["d"]
    flat = s["pool"].view(-1)
    base, tk = _places(s)
    base, tk = base[..., None], tk[:, :, None, None]
    (kc, ks), (vc, vs) = _quantise(s["k"]), _quantise(s["v"])
    lo = _k_byte_dims(d, tk.device)
    x = torch.arange(d // 2, device=tk.device)
    y = torch.arange(d // 32, device=tk.device)  # bytes of a position's scales
    # the value byte of dims 2x, 2x + 1: m = x / 16, g = x / 2 % 8, byte x % 2
    vplace = (((tk // 8 * 8 + x // 2 % 8) * 4 + tk % 8 // 2) * (d // 32) + x // 16) * 4 + tk % 2 * 2 + x % 2
    at = [base + tk * (d // 2) + x, base + 8 * d + vplace, base + 16 * d + tk * (d // 32) + y,
          base + 16 * d + 16 * (d // 32) + tk * (d // 32) + y]
    flat[at[0]] = kc[..., lo] | (kc[..., lo + 2] << 4)
    flat[at[1]] = vc[..., 0::2] | (vc[..., 1::2] << 4)
    flat[at[2]], flat[at[3]] = ks.view(torch.uint8), vs.view(torch.uint8)
    # read back
    kb, vb = flat[at[0]], flat[at[1]]
    k = torch.empty(kc.shape, device=kb.device)
    k[..., lo], k[..., lo + 2] = (kb & 15).float(), (kb >> 4).float()
    v = torch.stack([vb & 15, vb >> 4], -1).flatten(-2).float()
    ks, vs = flat[at[2]].view(torch.bfloat16).float(), flat[at[3]].view(torch.bfloat16).float()
    return [((z - 8).unflatten(-1, (-1, GROUP)) * sc.unsqueeze(-1)).flatten(-2).to(torch.bfloat16)
            for z, sc in ((k, ks), (v, vs))]


def _plain_resize(s):
    c, table, ref = s["c"], s["table"].long(), s["ref"].long()
    page, P, M = c["page"], c["P"], s["table"].shape[1]
    keep, cap = s["keep"].long()[:, None], s["cap"].long()[:, None]
    i = torch.arange(M, device=table.device)[None, :]
    held = table >= 0
    shared = held & (ref[table.clamp(min=0)] > 1)
    wanted = i < (cap + page - 1) // page
    tail = (i == keep // page) & (keep % page != 0)
    copied = tail & shared & (cap > keep)
    new = wanted & ((i >= (keep + page - 1) // page) & (~held | shared) | copied | ~held)
    free = ref == 0
    rank = torch.cumsum(free.long(), 0)
    lowest = torch.full((P + 1,), -1, device=table.device)
    lowest[torch.where(free, rank - 1, P)] = torch.arange(P, device=table.device)
    at = torch.cumsum(new.reshape(-1).long(), 0).view_as(table) - 1
    given = lowest[at.clamp(min=0, max=P - 1)]
    table_out = torch.where(new, given, torch.where(wanted, table, -1))
    gone = held & (new | ~wanted)
    ref_out = torch.zeros(P + 1, dtype=torch.int64, device=table.device)
    ref_out[:P] = ref
    ref_out.index_add_(0, torch.where(gone, table, P).view(-1), torch.full_like(table.view(-1), -1))
    ref_out.index_add_(0, torch.where(new, given, P).view(-1), torch.ones_like(table.view(-1)))
    # rows without a copy: a held page onto itself
    src, dst = (torch.where(copied.any(1), torch.where(copied, x, 0).sum(1), (ref > 0).long().argmax())
                for x in (table, given))
    s["pool"][:, dst] = s["pool"][:, src]
    stats = torch.stack([new.sum(), free.sum(), copied.sum(), gone.sum()])
    return [table_out.to(torch.int32), ref_out[:P].to(torch.int32), s["pool"], stats.to(torch.int32)]


def _plain_fork(s):
    table, parent = s["table"], s["parent"].long()
    P = s["c"]["P"]
    out = table[parent]
    children = torch.zeros(table.shape[0], dtype=torch.int64, device=table.device)
    children.index_add_(0, parent, torch.ones_like(parent))
    ref = torch.zeros(P + 1, dtype=torch.int64, device=table.device)
    ref[:P] = s["ref"]
    at = torch.where(table >= 0, table.long(), P)
    ref.index_add_(0, at.view(-1), (children - 1)[:, None].expand_as(table).reshape(-1))
    return [out, ref[:P].to(torch.int32)]


def _plain_compact(s):
    ref, table, P = s["ref"].long(), s["table"].long(), s["c"]["P"]
    ids = torch.arange(P, device=ref.device)
    live = ref > 0
    n = live.sum()
    hole, mover = ~live & (ids < n), live & (ids >= n)
    to = torch.full((P + 1,), -1, device=ref.device)
    to[torch.where(hole, torch.cumsum(hole.long(), 0) - 1, P)] = ids
    new = torch.where(mover, to[(torch.cumsum(mover.long(), 0) - 1).clamp(min=0)], torch.where(live, ids, -1))
    src = ids.clone()
    src = torch.cat([src, src[:1]])
    src[torch.where(mover, new, P)] = ids
    pool = s["pool"][:, src[:P]]
    ref_out = torch.zeros(P + 1, dtype=torch.int64, device=ref.device)
    ref_out[torch.where(live, new, P)] = ref
    table_out = torch.where(table >= 0, new[table.clamp(min=0)], -1)
    return [table_out.to(torch.int32), ref_out[:P].to(torch.int32), new.to(torch.int32), pool,
            torch.stack([n, mover.sum()]).to(torch.int32)]


# ------------------------------------------------------------------------------------------------ one pass
def run(state):
    s, c = state, state["c"]
    op = c["op"]
    if not own:
        if op == "attn":
            return _plain_attn(s)
        if op == "append":
            return _plain_append(s)
        if op == "resize":
            return _plain_resize(s)
        return _plain_fork(s) if op == "fork" else _plain_compact(s)
    from lossless_speculative_verification_gb300 import api
    if op == "attn":
        if "ws" not in s:
            s["ws"] = api.spec_q4_attention_workspace(c["B"], c["Q"], s["table"].shape[1], c["page"],
                                                      c["nkv"] * c["grp"], c["nkv"], c["d"])
        return api.spec_q4_attention(s["q"], s["pool"], s["table"], s["ctx"], c["nkv"], c["page"], s["ws"],
                                     out=s["out"])
    if op == "append":
        api.spec_q4_append(s["k"], s["v"], s["pool"], s["table"], s["ctx"], c["page"])
        return list(api.spec_q4_read(s["pool"], s["table"], s["ctx"], c["Q"], c["nkv"], c["d"], c["page"]))
    if "ws" not in s:
        s["ws"] = api.spec_pages_workspace(c["B"], c["M"], c["P"])
    if op == "resize":
        api.spec_pages_resize(s["pool"], s["table"], s["ref"], s["keep"], s["cap"], c["page"], s["ws"],
                              table_out=s["table_out"], ref_out=s["ref_out"], stats=s["stats"])
        return [s["table_out"], s["ref_out"], s["pool"], s["stats"]]
    if op == "fork":
        api.spec_pages_fork(s["table"], s["ref"], s["parent"], s["ws"], table_out=s["table_out"],
                            ref_out=s["ref_out"])
        return [s["table_out"], s["ref_out"]]
    api.spec_pages_compact(s["pool"], s["table"], s["ref"], s["ws"], table_out=s["table_out"], ref_out=s["ref_out"],
                           map=s["map"], stats=s["stats"])
    return [s["table_out"], s["ref_out"], s["map"], s["pool"], s["stats"][:2]]


def _moves(c):
    """Pages that move, as their expected number: a live one's number is at or above the live count."""
    live = sum(_lengths(c))
    return live * (c["P"] - live) / c["P"]


def work(case):
    c = case
    op = c["op"]
    if op == "attn":
        n = sum(_lengths(c))
        rows = c["B"] * c["Q"] * c["nkv"] * c["grp"]
        cache = n * c["nkv"] * (_block(c["d"]) // 16)
        return {"bytes": cache + 2 * rows * c["d"] * 2 + 4 * (sum(_pages(c)) + c["B"]),
                "flops": 4 * n * c["Q"] * c["nkv"] * c["grp"] * c["d"]}
    if op == "append":
        rows = c["B"] * c["Q"] * c["nkv"]
        # the new rows in, their blocks out; the blocks in, the rows out
        return {"bytes": 2 * rows * (4 * c["d"] + _block(c["d"]) // 16), "flops": 0}
    if op == "fork":
        return {"bytes": 4 * (2 * c["B"] * c["M"] + 2 * c["P"] + c["B"]), "flops": 0}
    if op == "resize":
        forked = {c["B"] - 1 - b for b in range(c["shared"])} | {_other(c, b) for b in range(c["shared"])}
        _, keep, cap = _turn(c)
        # rows that go on writing into a page that another row holds too
        copies = sum(keep[b] % c["page"] != 0 and cap[b] > keep[b] for b in forked)
        return {"bytes": 4 * (2 * c["B"] * c["M"] + 2 * c["P"] + 2 * c["B"]) + copies * 2 * c["layers"] * c["pb"],
                "flops": 0}
    return {"bytes": 4 * (2 * c["B"] * c["M"] + 3 * c["P"]) + _moves(c) * 2 * c["layers"] * c["pb"], "flops": 0}


# ------------------------------------------------------------------------------------------------ in 64 bits
def _exact_attn(s):
    c = s["c"]
    B, Q, nkv, grp, d, page = c["B"], c["Q"], c["nkv"], c["grp"], c["d"], c["page"]
    G, W = d // GROUP, d // 32
    out = torch.zeros((B, Q, nkv * grp, d), dtype=torch.float64, device="cuda")
    pos8 = torch.tensor([0, 4, 1, 5], device="cuda")  # the first dim of eight in byte 0, 1, 2, 3 of a key word
    for b, n in enumerate(_lengths(c)):
        rows = s["pool"][s["table"][b, :-(-n // page)].long()].view(-1, nkv, page // 16, _block(d))
        rows = rows.transpose(0, 1).reshape(nkv, -1, _block(d))
        for h in range(nkv):
            x = rows[h]
            N = x.shape[0]
            kb = x[:, :8 * d].reshape(N, 16, 4, W, 4)
            k = torch.empty((N, 16, W, 4, 8), dtype=torch.float64, device="cuda")
            k[..., pos8] = (kb % 16).double().transpose(2, 3) - 8
            k[..., pos8 + 2] = (kb // 16).double().transpose(2, 3) - 8
            vb = x[:, 8 * d:16 * d].reshape(N, 2, 8, 4, W, 2, 2)
            v = torch.empty((N, 2, 4, 2, W, 8, 2, 2), dtype=torch.float64, device="cuda")
            v[..., 0] = (vb % 16).double().permute(0, 1, 3, 5, 4, 2, 6) - 8
            v[..., 1] = (vb // 16).double().permute(0, 1, 3, 5, 4, 2, 6) - 8
            sc = x[:, 16 * d:].contiguous().view(torch.bfloat16).double().view(N, 2, 16, G, 1)
            k = (k.reshape(N, 16, G, GROUP) * sc[:, 0]).reshape(N * 16, d)[:n]
            v = (v.reshape(N, 16, G, GROUP) * sc[:, 1]).reshape(N * 16, d)[:n]
            q = s["q"][b, :, h * grp:(h + 1) * grp].double()
            x = torch.einsum("jgd,td->jgt", q, k) * d ** -0.5
            after = torch.arange(n, device="cuda")[None, :] > (n - Q + torch.arange(Q, device="cuda"))[:, None]
            x.masked_fill_(after[:, None, :], -torch.inf)
            out[b, :, h * grp:(h + 1) * grp] = torch.einsum("jgt,td->jgd", torch.softmax(x, -1), v)
    return out


def exact(case, seed):
    if case["op"] == "attn":
        return _exact_attn(prepare(case, seed))
    if case["op"] == "append":
        s = prepare(case, seed)
        got = []
        for x in (s["k"], s["v"]):
            g = x.double().reshape(*x.shape[:-1], -1, GROUP)
            sc = (g.abs().amax(-1, keepdim=True) / 7).to(torch.bfloat16).double()
            n = torch.where(sc > 0, torch.round(g / torch.where(sc > 0, sc, 1)), 0)
            got.append((n.clamp(-8, 7) * sc).reshape(x.shape))
        return got
    return None
