"""Plain numpy definitions of the paged 4-bit key/value cache and of its page calls.

Everything is written from the definitions: codes and scales in float64, one position at a time; the page calls one
table entry at a time, in order.
"""
from __future__ import annotations

import numpy as np

GROUP = 64
BLOCK = 16


def bf16_f64(bits):
    return (np.asarray(bits, np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def bf16_round(x):
    """float64 -> bf16 bits, nearest even (finite values)."""
    f = np.asarray(x, np.float64)
    m, e = np.frexp(f)
    q = np.rint(np.ldexp(m, 8))                       # 8 significant bits
    low = e < -125                                    # subnormal: a multiple of 2^-133
    v = np.where(low, np.ldexp(np.rint(np.ldexp(f, 133)), -133), np.ldexp(q, e - 8))
    return (v.astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)


def quantise(bits):
    """bf16 bits [..., d] -> nibbles n + 8 [..., d] uint8, scale bits [..., d / 64] uint16."""
    x = bf16_f64(bits)
    g = x.reshape(*x.shape[:-1], -1, GROUP)
    amax = np.abs(g).max(-1)
    bad = ~np.isfinite(g).all(-1)
    s = np.where(bad, np.uint16(0x7FC0), bf16_round(np.where(bad, 0.0, amax) / 7))
    f = np.where(bad, 0.0, bf16_f64(s))[..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        n = np.where(f > 0, np.rint(np.where(f > 0, g, 0) / np.where(f > 0, f, 1)), 0)
    n = np.clip(n, -8, 7)
    return (n + 8).astype(np.uint8).reshape(x.shape), s.astype(np.uint16)


def value(nib, s):
    """What codes [..., d] and scale bits [..., d / 64] stand for, float64."""
    g = (nib.astype(np.float64) - 8).reshape(*s.shape, GROUP)
    return (g * bf16_f64(s)[..., None]).reshape(nib.shape)


def block_bytes(d):
    return BLOCK * (d + 4 * (d // GROUP))


def put(block, d, tk, kn, ks, vn, vs):
    """One position's codes and scales into a block (uint8 [block bytes]) at place tk."""
    W, G = d // 32, d // GROUP
    for dim in range(d):
        # keys: word j of lane t, nibble r / 2 + 4 (r % 2)
        j, t, r = dim // 32, dim % 32 // 8, dim % 8
        nib = r // 2 + 4 * (r % 2)
        at = tk * (d // 2) + (t * W + j) * 4 + nib // 2
        block[at] = (block[at] & (0xF0 if nib % 2 == 0 else 0x0F)) | (int(kn[dim]) << (4 * (nib % 2)))
        # values: word m of lane (g, t) of the half, 16 bits a position, nibble c
        m, g, c = dim // 32, dim % 32 // 4, dim % 4
        half, t, e = tk // 8, tk % 8 // 2, tk % 2
        at = BLOCK * d // 2 + (((half * 8 + g) * 4 + t) * W + m) * 4 + 2 * e + c // 2
        block[at] = (block[at] & (0xF0 if c % 2 == 0 else 0x0F)) | (int(vn[dim]) << (4 * (c % 2)))
    for g in range(G):
        for base, s in ((BLOCK * d, ks), (BLOCK * d + BLOCK * G * 2, vs)):
            at = base + (tk * G + g) * 2
            block[at], block[at + 1] = int(s[g]) & 255, int(s[g]) >> 8


def append(pool, table, ctx_len, page, k_new, v_new):
    """k_new, v_new bf16 bits [B, Q, nkv, d] into pool [P, page bytes] uint8 (in place)."""
    B, Q, nkv, d = k_new.shape
    blk = pool.reshape(pool.shape[0], nkv, page // BLOCK, block_bytes(d))
    (kn, ks), (vn, vs) = quantise(k_new), quantise(v_new)
    for b in range(B):
        for j in range(Q):
            pos = int(ctx_len[b]) - Q + j
            if pos < 0:
                continue
            pg = table[b, pos // page]
            for h in range(nkv):
                put(blk[pg, h, pos % page // BLOCK], d, pos % BLOCK, kn[b, j, h], ks[b, j, h], vn[b, j, h], vs[b, j, h])


def attention(q, k, v, ctx_len, scale):
    """q [B, Q, nh, d] and cached values k, v [B, T, nkv, d] float64 -> out, and for every element the weighted
    mean of |v| (what rounding the weights can move it by)."""
    B, Q, nh, d = q.shape
    nkv = k.shape[2]
    out, mag = np.zeros(q.shape), np.zeros(q.shape)
    for b in range(B):
        for j in range(Q):
            n = int(ctx_len[b]) - Q + j + 1
            if n <= 0:
                continue
            for h in range(nh):
                kk, vv = k[b, :n, h // (nh // nkv)], v[b, :n, h // (nh // nkv)]
                x = kk @ q[b, j, h] * scale
                p = np.exp(x - x.max())
                p /= p.sum()
                out[b, j, h], mag[b, j, h] = p @ vv, p @ np.abs(vv)
    return out, mag


# ------------------------------------------------------------------------------------------------ pages
def resize(table, ref, keep, cap, page, pool=None):
    """(table, ref, stats, ok); pool [layers, P, ...] (optional) gets the copies in place."""
    B, M = table.shape
    out, new_ref = table.copy(), ref.copy()
    free = [p for p in range(len(ref)) if ref[p] <= 0]
    nfree, taken, copied, gone = len(free), 0, 0, 0
    copies = []
    for b in range(B):
        if not (0 <= keep[b] <= cap[b] <= M * page):
            continue
        kept, wanted = -(-keep[b] // page), -(-cap[b] // page)
        for i in range(M):
            p = table[b, i]
            held = 0 <= p < len(ref)
            shared = held and ref[p] > 1
            if i >= wanted:
                act = "drop"
            elif not held:
                act = "new"
            elif i >= kept:
                act = "new" if shared else "keep"
            elif i == keep[b] // page and keep[b] % page and shared and cap[b] > keep[b]:
                act = "copy"
            else:
                act = "keep"
            if act == "keep":
                continue
            if held:
                gone += 1
                new_ref[p] -= 1
            out[b, i] = -1
            if act != "drop":
                to = free[taken] if taken < nfree else -1
                taken += 1
                if to >= 0:
                    out[b, i] = to
                    new_ref[to] += 1
                    if act == "copy":
                        copies.append((p, to))
                        copied += 1
    if taken > nfree:
        return table.copy(), ref.copy(), [taken, nfree, 0, 0], False
    if pool is not None:
        for s, t in copies:
            pool[:, t] = pool[:, s]
    return out, new_ref, [taken, nfree, copied, gone], True


def fork(table, ref, parent):
    out = np.full_like(table, -1)
    new_ref = ref.copy()
    for row in table:
        for p in row:
            if p >= 0:
                new_ref[p] -= 1
    for b, a in enumerate(parent):
        if a < 0:
            continue
        out[b] = table[a]
        for p in out[b]:
            if p >= 0:
                new_ref[p] += 1
    return out, new_ref


def compact(table, ref, pool=None):
    """(table, ref, map, stats); pool [layers, P, ...] (optional) moves in place."""
    n = int((ref > 0).sum())
    to = np.full(len(ref), -1, np.int32)
    holes = [p for p in range(n) if ref[p] <= 0]
    for p in range(n):
        if ref[p] > 0:
            to[p] = p
    movers = [p for p in range(n, len(ref)) if ref[p] > 0]
    for p, h in zip(movers, holes):
        to[p] = h
        if pool is not None:
            pool[:, h] = pool[:, p]
    new_ref = np.zeros_like(ref)
    for p in range(len(ref)):
        if to[p] >= 0:
            new_ref[to[p]] = ref[p]
    out = np.where(table >= 0, to[np.clip(table, 0, None)], -1).astype(table.dtype)
    return out, new_ref, to, [n, len(movers)]
