"""The 4-bit paged cache without a GPU: the plain definitions of oracle/q4.py against other formulations, and the
calls' refusals, which are decided on the host."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import q4


def bits(x):
    return torch.from_numpy(np.asarray(x, np.float32)).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)


def test_bf16_round_is_torchs():
    rs = np.random.default_rng(0)
    x = np.concatenate([rs.normal(size=2000) * 10.0 ** rs.integers(-40, 38, 2000), [0.0, 1.0, 2.0 ** -133, 3e-41]])
    # float64 -> bf16 through float32 differs only at double roundings, which random values do not meet
    np.testing.assert_array_equal(q4.bf16_round(x), bits(x))


def test_quantise_is_within_half_a_step_and_hits_the_ends():
    rs = np.random.default_rng(1)
    x = bits(rs.normal(size=(50, 128)) * 2.0 ** rs.integers(-20, 20, (50, 1)))
    n, s = q4.quantise(x)
    v = q4.bf16_f64(x)
    step = np.repeat(q4.bf16_f64(s), q4.GROUP, -1)
    # the scale is bf16(amax / 7): at most 2^-8 off, so the largest value is at most 7 (1 + 2^-8) steps
    assert np.all(np.abs(q4.value(n, s) - v) <= step * (0.5 + 7 * 2.0 ** -8))
    assert n.max() <= 15 and n.min() >= 1
    g = np.abs(n.astype(int) - 8).reshape(50, 2, 64).max(-1)
    assert np.all(g == 7)


def test_quantise_special_groups():
    x = np.zeros((4, 128), np.float32)
    x[1, 5] = np.inf
    x[2, 70] = np.nan
    x[3, :64] = 3.5 * np.arange(64) / 9.0                      # 3.5 / .5 = 7: halves are exact
    x[3, 63] = 3.5 * 7
    n, s = q4.quantise(bits(x))
    assert s[0].tolist() == [0, 0] and np.all(n[0] == 8)
    assert s[1].tolist() == [0x7FC0, 0] and s[2].tolist() == [0, 0x7FC0]
    assert np.isnan(q4.value(n, s)[1, :64]).all() and (q4.value(n, s)[1, 64:] == 0).all()


def test_ties_go_to_the_even_code():
    x = np.full((1, 64), 7.0, np.float32)
    x[0, :6] = [0.5, 1.5, 2.5, -0.5, -1.5, -2.5]                # s = 1
    n, _ = q4.quantise(bits(x))
    assert (n[0, :6].astype(int) - 8).tolist() == [0, 2, 2, 0, -2, -2]


@pytest.mark.parametrize("d", [64, 128])
def test_every_nibble_has_a_place_of_its_own(d):
    seen = set()
    for tk in range(16):
        for dim in range(d):
            for which in range(2):
                kn, vn = np.zeros(d, int), np.zeros(d, int)
                (kn if which == 0 else vn)[dim] = 15
                blk = np.zeros(q4.block_bytes(d), np.uint8)
                q4.put(blk, d, tk, kn, [0] * (d // 64), vn, [0] * (d // 64))
                at = np.flatnonzero(blk)
                assert len(at) == 1 and blk[at[0]] in (15, 240)
                seen.add((int(at[0]), int(blk[at[0]])))
    assert len(seen) == 2 * 16 * d and max(a for a, _ in seen) < 16 * d


def test_attention_is_torchs():
    rs = np.random.default_rng(3)
    B, Q, nkv, grp, d, T = 2, 3, 2, 2, 64, 40
    q, k, v = rs.normal(size=(B, Q, nkv * grp, d)), rs.normal(size=(B, T, nkv, d)), rs.normal(size=(B, T, nkv, d))
    n = np.array([40, 2])
    out, mag = q4.attention(q, k, v, n, 0.3)
    t = [torch.from_numpy(a).transpose(1, 2) for a in (q, k, v)]
    for b in range(B):
        L = n[b]
        mask = torch.arange(L)[None, :] <= (L - Q + torch.arange(Q))[:, None]
        ref = torch.nn.functional.scaled_dot_product_attention(
            t[0][b:b + 1], t[1][b:b + 1, :, :L].repeat_interleave(grp, 1), t[2][b:b + 1, :, :L].repeat_interleave(grp, 1),
            attn_mask=mask, scale=0.3)[0].transpose(0, 1).numpy()
        seen = mask.any(1).numpy()
        np.testing.assert_allclose(out[b][seen], ref[seen], rtol=1e-12, atol=1e-13)
        assert (out[b][~seen] == 0).all()
    assert np.all(mag >= np.abs(out) - 1e-15)


def counts(table, P):
    return np.bincount(table[table >= 0], minlength=P).astype(np.int32)


def random_state(rs, B, M, P, page, shared):
    table = np.full((B, M), -1, np.int32)
    order = rs.permutation(P)
    n = rs.integers(0, M * page + 1, B)
    while sum(-(-x // page) for x in n) > P * 2 // 3:
        n = n // 2
    at = 0
    for b in range(B):
        c = -(-int(n[b]) // page)
        table[b, :c] = order[at:at + c]
        at += c
    for _ in range(shared):
        a, b = rs.integers(0, B, 2)
        table[b], n[b] = table[a], n[a]
    return table, counts(table, P), n


@pytest.mark.parametrize("seed", range(6))
def test_page_calls_keep_the_counts(seed):
    """After any sequence of calls the counts are the entries', no page has two contents, and a sequence's kept
    contents are what they were."""
    rs = np.random.default_rng(seed)
    B, M, page, P = 6, 7, 4, 60
    table, ref, n = random_state(rs, B, M, P, page, 3)
    pool = rs.integers(0, 1 << 30, (2, P))

    def contents(tb):
        return [[pool[:, p].tolist() for p in row if p >= 0] for row in tb]

    for _ in range(12):
        before = contents(table)
        kind = rs.integers(0, 3)
        if kind == 0:
            keep = np.array([rs.integers(0, x + 1) for x in n])
            cap = np.minimum(keep + rs.integers(0, 9, B), M * page)
            out, new_ref, stats, ok = q4.resize(table, ref, keep, cap, page, pool)
            if ok:
                for b in range(B):
                    k = -(-keep[b] // page)
                    assert contents(out)[b][:k] == before[b][:k]
                    assert (out[b] >= 0).sum() == -(-cap[b] // page)
                    # what will be written is the row's own
                    for i in range(keep[b] // page, -(-cap[b] // page)):
                        if cap[b] > keep[b] and (i >= k or keep[b] % page):
                            assert new_ref[out[b, i]] == 1
                assert stats[0] - stats[3] == counts(out, P).sum() - counts(table, P).sum()
                n = cap
            table, ref = out, new_ref
        elif kind == 1:
            parent = rs.integers(-1, B, B)
            table, ref = q4.fork(table, ref, parent)
            n = np.where(parent >= 0, n[parent], 0)
            assert contents(table) == [before[a] if a >= 0 else [] for a in parent]
        else:
            table, ref, to, (live, _) = q4.compact(table, ref, pool)
            assert contents(table) == before
            assert (ref[:live] > 0).all() and (ref[live:] == 0).all()
        np.testing.assert_array_equal(ref, counts(table, P))


@pytest.fixture(scope="module")
def lib():
    from lossless_speculative_verification_gb300 import _build, _ffi
    _build.build()
    return _ffi.load()


p16, odd = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10008)


def test_page_bytes(lib):
    assert lib.spec_q4_page_bytes(10, 128, 64) == 10 * 4 * 2176 == 10 * 4 * q4.block_bytes(128)
    assert lib.spec_q4_page_bytes(3, 64, 16) == 3 * q4.block_bytes(64)
    for bad in [(0, 128, 64), (1025, 128, 64), (4, 96, 64), (4, 256, 64), (4, 128, 8), (4, 128, 48), (4, 128, 512)]:
        assert lib.spec_q4_page_bytes(*bad) == 0


def test_append_and_read_refuse(lib):
    def app(k=p16, v=p16, pool=p16, tb=p16, n=p16, B=2, Q=3, nkv=4, d=128, page=64, M=5, P=10):
        return lib.spec_q4_append(k, v, pool, tb, n, B, Q, nkv, d, page, M, P, None)

    def read(k=p16, v=p16, pool=p16, tb=p16, n=p16, B=2, Q=3, nkv=4, d=128, page=64, M=5, P=10):
        return lib.spec_q4_read(pool, tb, n, B, Q, nkv, d, page, M, P, k, v, None)

    for f in (app, read):
        for none in ("k", "v", "pool", "tb", "n"):
            assert f(**{none: None}) == 1
            assert f(**{none: odd}) == 3
        for bad in (dict(B=-1), dict(Q=-1), dict(nkv=0), dict(d=0), dict(page=0), dict(M=0), dict(P=0)):
            assert f(**bad) == 1
        for bad in (dict(d=96), dict(page=24), dict(nkv=2000), dict(M=1 << 25), dict(B=1 << 20, M=1 << 12),
                    dict(B=1 << 20, Q=1 << 20)):
            assert f(**bad) == 2
        assert f(None, None, None, None, None, B=0) == 0
        assert f(None, None, None, None, None, Q=0) == 0


def test_attention_refuses(lib):
    size = lib.spec_q4_attention_workspace_size
    need = size(4, 4, 36, 64, 10, 10, 128)
    assert need > 0
    for bad in [(-1, 4, 36, 64, 10, 10, 128), (65536, 4, 36, 64, 10, 10, 128), (4, 0, 36, 64, 10, 10, 128),
                (4, 9, 36, 64, 10, 10, 128), (4, 4, 0, 64, 10, 10, 128), (4, 4, 36, 63, 10, 10, 128),
                (4, 4, 36, 64, 10, 3, 128), (4, 4, 36, 64, 34, 2, 128), (4, 4, 36, 64, 10, 10, 96),
                (4, 4, 36, 64, 2, 10, 128), (4, 4, 1 << 19, 64, 10, 10, 128), (60000, 4, 36, 64, 10, 10, 128)]:
        assert size(*bad) == 0, bad

    def att(q=p16, pool=p16, tb=p16, n=p16, out=p16, ws=p16, B=4, Q=4, nh=10, nkv=10, d=128, page=64, M=36, P=99,
            scale=0.1, ws_bytes=need):
        return lib.spec_q4_attention(q, pool, tb, n, B, Q, nh, nkv, d, page, M, P, scale, out, ws, ws_bytes, None)

    for none in ("q", "pool", "tb", "n", "out"):
        assert att(**{none: None}) == 1
        assert att(**{none: odd}) == 3
    assert att(ws=None) == 4 and att(ws_bytes=need - 1) == 4 and att(ws=odd) == 3
    for s in (0.0, -1.0, float("nan"), float("inf")):
        assert att(scale=s) == 1
    assert att(Q=9) == 2 and att(nkv=3) == 2 and att(d=32) == 2 and att(page=20) == 2
    assert att(Q=0) == 1 and att(P=0) == 1 and att(M=0) == 1
    assert att(None, None, None, None, None, None, B=0, ws_bytes=0) == 0


def test_page_calls_refuse(lib):
    need = lib.spec_pages_workspace_size(4, 9, 100)
    assert need > 0
    for bad in [(-1, 9, 100), (4, 0, 100), (4, 9, 0), (65537, 9, 100), (4, 9, (1 << 24) + 1), (65536, 32768, 100)]:
        assert lib.spec_pages_workspace_size(*bad) == 0

    def resize(pool=p16, tb=p16, ref=p16, keep=p16, cap=p16, to=p16, ro=p16, st=None, ws=p16, layers=2, pb=1088, B=4,
               M=9, P=100, page=16, ws_bytes=need):
        return lib.spec_pages_resize(pool, layers, pb, tb, ref, keep, cap, B, M, P, page, to, ro, st, ws, ws_bytes, None)

    def fork(tb=p16, ref=p16, parent=p16, to=p16, ro=p16, ws=p16, B=4, M=9, P=100, ws_bytes=need):
        return lib.spec_pages_fork(tb, ref, parent, B, M, P, to, ro, ws, ws_bytes, None)

    def compact(pool=p16, tb=p16, ref=p16, to=p16, ro=p16, mp=None, st=None, ws=p16, layers=2, pb=1088, B=4, M=9,
                P=100, ws_bytes=need):
        return lib.spec_pages_compact(pool, layers, pb, tb, ref, B, M, P, to, ro, mp, st, ws, ws_bytes, None)

    for f, args in ((resize, ("pool", "tb", "ref", "keep", "cap", "to", "ro")), (fork, ("tb", "ref", "parent", "to", "ro")),
                    (compact, ("pool", "tb", "ref", "to", "ro"))):
        for a in args:
            assert f(**{a: None}) == 1
            assert f(**{a: odd}) == 3
        assert f(ws=None) == 4 and f(ws_bytes=need - 1) == 4 and f(ws=odd) == 3
        assert f(B=-1) == 1 and f(M=0) == 1 and f(P=0) == 1 and f(B=70000) == 2 and f(P=1 << 25) == 2
    for f in (resize, compact):
        assert f(layers=0) == 1 and f(pb=0) == 1 and f(pb=24) == 2 and f(pb=1 << 32) == 2 and f(st=odd) == 3
    assert resize(page=0) == 1 and resize(page=1 << 30) == 2 and compact(mp=odd) == 3


def test_status_names_the_empty_pool(lib):
    assert lib.lsv_status_string(8) == b"too few free pages"


def test_the_launch_count_is_of_the_bf16_cache():
    from lossless_speculative_verification_gb300 import synth
    from lossless_speculative_verification_gb300.decoder import Decoder

    dec = Decoder.__new__(Decoder)
    dec.layers, dec.prob = [None] * 2, synth.decoder_problem(1, synth.MoeDims(0, 256, 8, 2, 1, 128), V=64, nh=2, I_draft=256)
    dec.cache = "bf16"
    assert dec.launches_per_verify(4, 2) == 1 + 2 * (1 + 3 + 1 + 2 + 1 + 1 + 3) + 1 + 2
    dec.cache = "q4"
    with pytest.raises(ValueError):
        dec.launches_per_verify(4, 2)
