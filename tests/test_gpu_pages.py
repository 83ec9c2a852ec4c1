"""The page calls of a paged cache on the GPU against oracle/q4.py, entry by entry: whole numbers and moved bytes,
all exact."""
import numpy as np
import pytest
import torch

from oracle import q4
from lossless_speculative_verification_gb300 import api

from gpu_util import need_gpu
from test_q4_cpu import counts, random_state

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()
    yield
    torch.cuda.synchronize()
    assert api.get_device_error() == 0


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()


def host(t):
    return t.cpu().numpy()


def outputs(table, ref, place):
    """The tensors of a call in place, or apart from its inputs (filled with what must not stay)."""
    t, r = i32(table), i32(ref)
    if place:
        return t, r, {}
    return t, r, dict(table_out=torch.full_like(t, -7), ref_out=torch.full_like(r, -7))


SIZES = [(1, 1, 1, 1), (3, 5, 40, 16), (7, 9, 130, 5), (33, 64, 3000, 3), (70, 300, 9000, 16), (5, 1000, 5000, 1)]


@pytest.mark.parametrize("place", [True, False])
@pytest.mark.parametrize("B,M,P,page", SIZES + [(64, 64, 4096, 4), (241, 17, 4095, 2), (9, 40, 4097, 8)])
def test_resize(B, M, P, page, place):
    rs = np.random.default_rng(B * M)
    for turn in range(3):
        table, ref, n = random_state(rs, B, M, P, page, B // 3)
        keep = np.array([max(0, x - rs.integers(0, 2 * page)) if rs.random() < 0.8 else 0 for x in n])
        cap = np.minimum(keep + rs.integers(0, 3 * page, B) * (rs.random(B) < 0.8), M * page)
        pool = rs.integers(0, 256, (3, P, 48)).astype(np.uint8)
        want_pool = pool.copy()
        out, new_ref, stats, ok = q4.resize(table, ref, keep, cap, page, want_pool)
        t, r, kw = outputs(table, ref, place)
        dp, st = torch.from_numpy(pool).cuda(), torch.full((4,), -7, dtype=torch.int32, device="cuda")
        ws = api.spec_pages_workspace(B, M, P).fill_(255)
        got, got_ref = api.spec_pages_resize(dp, t, r, i32(keep), i32(cap), page, ws, stats=st, **kw)
        assert api.get_device_error() == (0 if ok else 8)
        np.testing.assert_array_equal(host(got), out)
        np.testing.assert_array_equal(host(got_ref), new_ref)
        np.testing.assert_array_equal(host(dp), want_pool)
        assert host(st).tolist() == stats
        if not place:
            np.testing.assert_array_equal(host(t), table)
            np.testing.assert_array_equal(host(r), ref)


@pytest.mark.parametrize("place", [True, False])
def test_resize_with_too_few_pages_changes_nothing(place):
    table = np.array([[0, 1, -1, -1], [2, -1, -1, -1]], np.int32)
    ref = counts(table, 5)
    pool = torch.randint(0, 256, (1, 5, 16), dtype=torch.uint8, device="cuda")
    before = pool.clone()
    t, r, kw = outputs(table, ref, place)
    st = torch.zeros(4, dtype=torch.int32, device="cuda")
    got, got_ref = api.spec_pages_resize(pool, t, r, i32([0, 3]), i32([32, 16]), 8, api.spec_pages_workspace(2, 4, 5),
                                         stats=st, **kw)
    assert api.get_device_error() == 8
    np.testing.assert_array_equal(host(got), table)
    np.testing.assert_array_equal(host(got_ref), ref)
    assert host(st).tolist() == [3, 2, 0, 0] and torch.equal(pool, before)
    # exactly enough
    got, got_ref = api.spec_pages_resize(pool, t, r, i32([0, 3]), i32([24, 16]), 8, api.spec_pages_workspace(2, 4, 5), **kw)
    assert api.get_device_error() == 0
    assert host(got).tolist() == [[0, 1, 3, -1], [2, 4, -1, -1]] and host(got_ref).tolist() == [1] * 5


@pytest.mark.parametrize("place", [True, False])
@pytest.mark.parametrize("extra", [0, 4096])                    # both forms of the call
def test_too_few_pages_are_reported_whatever_else_is_wrong(extra, place):
    good = np.array([[0, 1, -1, -1], [2, -1, -1, -1]], np.int32)
    P = 5 + extra
    for table, keep, cap in ((good, [-1, 3], [32, 32]), (good, [0, 9], [32, 32]),
                             (np.where(good == 1, P, good), [0, 3], [32, 32]),
                             (np.where(good == 1, 3, good), [16, 3], [32, 32])):   # page 3 is counted free
        ref = np.r_[1, 1, 1, 0, 0, np.ones(extra)].astype(np.int32)
        t, r, kw = outputs(table, ref, place)
        pool = torch.zeros((1, P, 16), dtype=torch.uint8, device="cuda")
        st = torch.zeros(4, dtype=torch.int32, device="cuda")
        a, b = api.spec_pages_resize(pool, t, r, i32(keep), i32(cap), 8, api.spec_pages_workspace(2, 4, P), stats=st, **kw)
        needed, free = host(st).tolist()[:2]
        assert needed > free == 2 and host(st).tolist()[2:] == [0, 0]
        assert api.get_device_error() == 8
        np.testing.assert_array_equal(host(a), table)
        np.testing.assert_array_equal(host(b), ref)
        # the same with pages enough: what is wrong is reported
        small = np.maximum(keep, 0) if keep[0] < 0 else keep
        a, b = api.spec_pages_resize(pool, i32(table), r, i32(keep), i32(np.maximum(small, 0)), 8,
                                     api.spec_pages_workspace(2, 4, P))
        assert api.get_device_error() == 7


def test_resize_many_pages_of_many_chunks():
    # every fourth page is free: ranks that reach over chunks of pages and rows that need thousands
    B, M, P, page = 4, 30000, 200000, 16
    ref = np.where(np.arange(P) % 4 == 1, 0, 1).astype(np.int32)
    table = np.full((B, M), -1, np.int32)
    cap = np.array([page * 11, page * 20000, 0, page * 29990 - 3])
    out, new_ref, stats, ok = q4.resize(table, ref, np.zeros(B, int), cap, page)
    assert not ok and stats[0] == 50001                         # one too many
    cap = np.array([page * 11, page * 20000, 0, page * 29000 - 3])
    out, new_ref, stats, ok = q4.resize(table, ref, np.zeros(B, int), cap, page)
    assert ok
    pool = torch.zeros((1, P, 16), dtype=torch.uint8, device="cuda")
    t, r = i32(table), i32(ref)
    api.spec_pages_resize(pool, t, r, i32(np.zeros(B)), i32(cap), page, api.spec_pages_workspace(B, M, P))
    np.testing.assert_array_equal(host(t), out)
    np.testing.assert_array_equal(host(r), new_ref)


def test_resize_copies_on_write_in_every_layer_of_a_large_page():
    # forked rows: the page that both will write is copied for each, the full ones stay shared, an idle fork stays
    page, pb = 8, 16 * 1031 * 5
    table = np.array([[4, 2, 7, -1], [4, 2, 7, -1], [4, 2, 7, -1], [5, -1, -1, -1]], np.int32)
    ref = counts(table, 12)
    pool = torch.randint(0, 256, (3, 12, pb), dtype=torch.uint8, device="cuda")
    before = host(pool)
    t, r = i32(table), i32(ref)
    api.spec_pages_resize(pool, t, r, i32([18, 18, 18, 3]), i32([20, 25, 18, 8]), page, api.spec_pages_workspace(4, 4, 12))
    assert host(t).tolist() == [[4, 2, 0, -1], [4, 2, 1, 3], [4, 2, 7, -1], [5, -1, -1, -1]]
    assert host(r).tolist() == [1, 1, 3, 1, 3, 1, 0, 1, 0, 0, 0, 0]
    want = before.copy()
    want[:, 0] = want[:, 1] = before[:, 7]
    np.testing.assert_array_equal(host(pool), want)


def test_resize_out_of_range_is_reported():
    table = np.array([[0, -1], [1, -1], [9, -1], [-2, 2], [3, -1]], np.int32)
    ref = np.array([1, 1, 1, 0, 0, 0, 0, 0, 0], np.int32)
    pool = torch.zeros((1, 9, 16), dtype=torch.uint8, device="cuda")
    ws = api.spec_pages_workspace(5, 2, 9)
    for keep, cap in (([5, 0, 0, 0, 0], [4, 8, 8, 8, 0]), ([-1, 0, 0, 0, 0], [4, 8, 8, 8, 0]),
                      ([0, 0, 0, 0, 0], [17, 8, 8, 8, 0])):
        t, r = i32(table), i32(ref)
        api.spec_pages_resize(pool, t, r, i32(keep), i32(cap), 8, ws)
        assert api.get_device_error() == 7
        assert host(t)[0].tolist() == [0, -1] and host(t)[1].tolist() == [1, -1]
        assert host(t)[2].tolist() == [3, -1]                   # an entry out of range is none
    # a held page that counts as free, and a kept position without a page
    t, r = i32([[0, -1]]), i32([0, 0, 0])
    api.spec_pages_resize(pool[:, :3].contiguous(), t, r, i32([8]), i32([8]), 8, api.spec_pages_workspace(1, 2, 3))
    assert api.get_device_error() == 7
    t, r = i32([[-1, -1]]), i32([1, 0, 0])
    api.spec_pages_resize(pool[:, :3].contiguous(), t, r, i32([8]), i32([8]), 8, api.spec_pages_workspace(1, 2, 3))
    assert api.get_device_error() == 7 and host(t).tolist() == [[1, -1]]


@pytest.mark.parametrize("place", [True, False])
@pytest.mark.parametrize("B,M,P,page", SIZES)
def test_fork(B, M, P, page, place):
    rs = np.random.default_rng(B + M)
    table, ref, _ = random_state(rs, B, M, P, page, B // 4)
    for parent in (rs.integers(-1, B, B), np.zeros(B, int), np.arange(B), np.full(B, -1), np.arange(B)[::-1]):
        out, new_ref = q4.fork(table, ref, parent)
        t, r, kw = outputs(table, ref, place)
        got, got_ref = api.spec_pages_fork(t, r, i32(parent), api.spec_pages_workspace(B, M, P).fill_(255), **kw)
        np.testing.assert_array_equal(host(got), out)
        np.testing.assert_array_equal(host(got_ref), new_ref)


def test_fork_out_of_range_is_reported():
    t, r = i32([[0, 1], [2, -1]]), i32([1, 1, 1])
    api.spec_pages_fork(t, r, i32([2, 0]), api.spec_pages_workspace(2, 2, 3))
    assert api.get_device_error() == 7
    assert host(t).tolist() == [[-1, -1], [0, 1]] and host(r).tolist() == [1, 1, 0]


@pytest.mark.parametrize("place", [True, False])
@pytest.mark.parametrize("B,M,P,page", SIZES + [(8, 40, 250, 16), (8, 40, 300, 16), (64, 64, 4096, 4)])
def test_compact(B, M, P, page, place):
    rs = np.random.default_rng(B + P)
    table, ref, _ = random_state(rs, B, M, P, page, B // 4)
    layers, pb = (11, 16) if B % 2 else (1, 16 * 1025)
    pool = rs.integers(0, 256, (layers, P, pb)).astype(np.uint8)
    want = pool.copy()
    out, new_ref, to, stats = q4.compact(table, ref, want)
    t, r, kw = outputs(table, ref, place)
    dp = torch.from_numpy(pool).cuda()
    mp, st = torch.full((P,), -7, dtype=torch.int32, device="cuda"), torch.full((4,), -7, dtype=torch.int32, device="cuda")
    got, got_ref = api.spec_pages_compact(dp, t, r, api.spec_pages_workspace(B, M, P).fill_(255), map=mp, stats=st, **kw)
    np.testing.assert_array_equal(host(got), out)
    np.testing.assert_array_equal(host(got_ref), new_ref)
    np.testing.assert_array_equal(host(mp), to)
    np.testing.assert_array_equal(host(dp), want)
    assert host(st).tolist() == stats + [0, 0]


@pytest.mark.parametrize("P", [31, 4096, 4097, 8192, 20000])
@pytest.mark.parametrize("kind", ["none", "all", "low", "high", "odd"])
def test_compact_of_counts_of_every_shape(P, kind):
    i = np.arange(P)
    live = {"none": i < 0, "all": i >= 0, "low": i < P // 2, "high": i >= P // 2, "odd": i % 2 == 1}[kind]
    ref = np.where(live, 1 + i % 3, 0).astype(np.int32)
    table = np.where(live, i, -1).astype(np.int32)[None]
    pool = torch.arange(P, device="cuda").to(torch.int64)[None, :, None].expand(2, P, 2).contiguous()
    want = host(pool).copy()
    out, new_ref, to, stats = q4.compact(table, ref, want)
    t, r, mp = i32(table), i32(ref), torch.empty(P, dtype=torch.int32, device="cuda")
    api.spec_pages_compact(pool, t, r, api.spec_pages_workspace(1, P, P), map=mp)
    for a, b in ((t, out), (r, new_ref), (mp, to), (pool, want)):
        np.testing.assert_array_equal(host(a), b)


def test_compact_of_an_entry_without_a_live_page_is_reported():
    t, r = i32([[0, 3, 7, -3]]), i32([1, 0, 0, 0, 1])
    pool = torch.zeros((1, 5, 16), dtype=torch.uint8, device="cuda")
    api.spec_pages_compact(pool, t, r, api.spec_pages_workspace(1, 4, 5))
    assert api.get_device_error() == 7
    assert host(t).tolist() == [[0, -1, -1, -1]] and host(r).tolist() == [1, 1, 0, 0, 0]


@pytest.mark.parametrize("place", [True, False])
def test_the_forms_of_a_call_agree_on_what_is_wrong(place):
    # small tables and pools take one launch; with pages or rows added that change nothing, the other form
    rs = np.random.default_rng(5)
    for turn in range(8):
        B, M, P, page, more = 20, 30, 500, 8, 4096
        table, ref, n = random_state(rs, B, M, P, page, B // 3)
        keep = np.maximum(n - rs.integers(0, 2 * page, B), 0)
        cap = np.minimum(keep + rs.integers(0, 3 * page, B), M * page)
        if turn:
            wrong = rs.random((B, M)) < 0.03
            table = np.where(wrong, rs.choice([-2, 1 << 20, -1], (B, M)), table).astype(np.int32)
            ref[rs.random(P) < 0.03] = 0                        # held pages that count as free
            keep[rs.integers(0, B, 2)] = -1, M * page + 1
            cap[rs.integers(0, B, 2)] = 0, M * page + 3
        pool = rs.integers(0, 256, (2, P, 32)).astype(np.uint8)

        def resize(extra):
            t, r, kw = outputs(table, np.r_[ref, np.ones(extra, np.int32)], place)
            dp = torch.from_numpy(np.concatenate([pool, np.zeros((2, extra, 32), np.uint8)], 1)).cuda()
            st = torch.full((4,), -7, dtype=torch.int32, device="cuda")
            a, b = api.spec_pages_resize(dp, t, r, i32(keep), i32(cap), page, api.spec_pages_workspace(B, M, P + extra),
                                         stats=st, **kw)
            return host(a), host(b)[:P], host(st), host(dp)[:, :P], api.get_device_error()

        def compact(extra):
            t, r, kw = outputs(table, np.r_[ref, np.zeros(extra, np.int32)], place)
            dp = torch.from_numpy(np.concatenate([pool, np.zeros((2, extra, 32), np.uint8)], 1)).cuda()
            mp = torch.full((P + extra,), -7, dtype=torch.int32, device="cuda")
            a, b = api.spec_pages_compact(dp, t, r, api.spec_pages_workspace(B, M, P + extra), map=mp, **kw)
            return host(a), host(b)[:P], host(mp)[:P], host(dp)[:, :int((ref > 0).sum())], api.get_device_error()

        def fork(extra):
            t, r, kw = outputs(np.r_[table, np.full((extra, M), -1, np.int32)], ref, place)
            parent = np.r_[rs_parent, np.full(extra, -1)]
            a, b = api.spec_pages_fork(t, r, i32(parent), api.spec_pages_workspace(B + extra, M, P), **kw)
            return host(a)[:B], host(b), api.get_device_error()

        rs_parent = rs.integers(-1, B, B)
        if turn % 2:
            rs_parent[3] = -4
        for call, extra in ((resize, more), (compact, more), (fork, 50)):
            for x, y in zip(call(0), call(extra)):
                np.testing.assert_array_equal(x, y)


def test_page_moves_beyond_4_gb():
    pb, P = 1 << 20, 5000
    pool = torch.empty((1, P, pb), dtype=torch.uint8, device="cuda")
    t, r = i32([[4990, 4999, 4997]]), torch.zeros(P, dtype=torch.int32, device="cuda")
    for p in (4990, 4999, 4997):
        pool[0, p] = p % 251
        r[p] = 1
    api.spec_pages_compact(pool, t, r, api.spec_pages_workspace(1, 3, P))
    assert host(t).tolist() == [[0, 2, 1]]
    for p, x in ((0, 4990), (1, 4997), (2, 4999)):
        assert bool((pool[0, p] == x % 251).all())


def test_no_rows():
    ws = api.spec_pages_workspace(0, 3, 10)
    none, e = i32(np.zeros((0, 3))), i32([])
    pool, r = torch.zeros((1, 10, 16), dtype=torch.uint8, device="cuda"), i32([0] * 9 + [2])
    out = torch.full((10,), -7, dtype=torch.int32, device="cuda")
    st = torch.full((4,), -7, dtype=torch.int32, device="cuda")
    api.spec_pages_resize(pool, none, r, e, e, 4, ws, ref_out=out, stats=st)
    assert torch.equal(out, r) and host(st).tolist() == [0, 9, 0, 0]
    out.fill_(-7)
    api.spec_pages_fork(none, r, e, ws, ref_out=out)
    assert torch.equal(out, r)
    api.spec_pages_compact(pool, none, r, ws, ref_out=out)
    assert host(out).tolist() == [2] + [0] * 9


def test_as_many_rows_as_there_may_be():
    B, M, P, page = 65536, 2, 150000, 8
    rs = np.random.default_rng(11)
    table, ref, n = random_state(rs, B, M, P, page, 1000)
    keep = np.maximum(n - rs.integers(0, 4, B), 0)
    cap = np.minimum(keep + rs.integers(0, 4, B), M * page)
    pool = rs.integers(0, 256, (1, P, 16)).astype(np.uint8)
    ws = api.spec_pages_workspace(B, M, P)
    t, r, dp = i32(table), i32(ref), torch.from_numpy(pool).cuda()
    st = torch.zeros(4, dtype=torch.int32, device="cuda")
    api.spec_pages_resize(dp, t, r, i32(keep), i32(cap), page, ws, stats=st)
    table, ref, stats, ok = q4.resize(table, ref, keep, cap, page, pool)
    assert ok and host(st).tolist() == stats
    parent = rs.integers(-1, B, B)
    parent[:2000] = 7
    steps = [lambda: None, lambda: api.spec_pages_fork(t, r, i32(parent), ws), lambda: api.spec_pages_compact(dp, t, r, ws)]
    for i, step in enumerate(steps):
        step()
        if i == 1:
            table, ref = q4.fork(table, ref, parent)
        if i == 2:
            table, ref, _, stats = q4.compact(table, ref, pool)
            pool = pool[:, :stats[0]]
        np.testing.assert_array_equal(host(t), table)
        np.testing.assert_array_equal(host(r), ref)
        np.testing.assert_array_equal(host(dp)[:, :pool.shape[1]], pool)


def test_turns_of_two_tables_at_once():
    rs = np.random.default_rng(12)
    sides = []
    for B, M, P, page in ((20, 30, 900, 8), (90, 200, 9000, 8)):
        table, ref, n = random_state(rs, B, M, P, page, B // 3)
        keep, cap = n, np.minimum(n + 9, M * page)
        pool = rs.integers(0, 256, (2, P, 64)).astype(np.uint8)
        sides.append([i32(table), i32(ref), torch.from_numpy(pool).cuda(), i32(keep), i32(cap), i32(rs.integers(-1, B, B)),
                      api.spec_pages_workspace(B, M, P), page, torch.cuda.Stream(), (table, ref, keep, cap, pool)])
    torch.cuda.synchronize()
    for turn in range(4):
        for t, r, dp, kp, cp, pa, ws, page, stream, _ in sides:
            api.spec_pages_resize(dp, t, r, kp, cp, page, ws, stream=stream)
            api.spec_pages_fork(t, r, pa, ws, stream=stream)
            api.spec_pages_compact(dp, t, r, ws, stream=stream)
    torch.cuda.synchronize()
    api.get_device_error()                                      # (a forked row may keep more than its parent had)
    for t, r, dp, kp, cp, pa, ws, page, stream, (table, ref, keep, cap, pool) in sides:
        alone = [i32(table), i32(ref), torch.from_numpy(pool).cuda()]
        for turn in range(4):
            api.spec_pages_resize(alone[2], *alone[:2], kp, cp, page, ws)
            api.spec_pages_fork(*alone[:2], pa, ws)
            api.spec_pages_compact(alone[2], *alone[:2], ws)
        torch.cuda.synchronize()
        api.get_device_error()
        live = int((alone[1] > 0).sum())
        assert torch.equal(t, alone[0]) and torch.equal(r, alone[1]) and torch.equal(dp[:, :live], alone[2][:, :live])


def test_captured_turns():
    """A turn's resize and the fork after it in one graph, replayed on its own outputs."""
    rs = np.random.default_rng(3)
    B, M, P, page = 5, 6, 80, 4
    table, ref, n = random_state(rs, B, M, P, page, 1)
    t, r = i32(table), i32(ref)
    keep, cap, parent = i32(n), i32(n), i32(np.arange(B))
    pool = torch.randint(0, 256, (2, P, 32), dtype=torch.uint8, device="cuda")
    ws = api.spec_pages_workspace(B, M, P)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.spec_pages_fork(t, r, parent, ws)
        api.spec_pages_resize(pool, t, r, keep, cap, page, ws)
    want = host(pool).copy()
    for _ in range(5):
        pa = rs.integers(0, B, B)
        n = n[pa]
        kp = np.array([rs.integers(0, x + 1) for x in n])
        cp = np.minimum(kp + rs.integers(0, 6, B), M * page)
        parent.copy_(i32(pa)); keep.copy_(i32(kp)); cap.copy_(i32(cp))
        graph.replay()
        table, ref = q4.fork(table, ref, pa)
        table, ref, _, ok = q4.resize(table, ref, kp, cp, page, want)
        assert ok
        n = cp
        np.testing.assert_array_equal(host(t), table)
        np.testing.assert_array_equal(host(r), ref)
        np.testing.assert_array_equal(host(pool), want)


def test_wrappers_refuse():
    t, r, ws = i32([[0, -1]]), i32([1, 0]), api.spec_pages_workspace(1, 2, 2)
    pool, k = torch.zeros((2, 16), dtype=torch.uint8, device="cuda"), i32([0])
    bad = [
        lambda: api.spec_pages_resize(pool[:1], t, r, k, k, 4, ws),
        lambda: api.spec_pages_resize(pool, t, r.long(), k, k, 4, ws),
        lambda: api.spec_pages_resize(pool, t, r, i32([0, 0]), k, 4, ws),
        lambda: api.spec_pages_resize(pool, t, r, k, k, 4, ws, stats=k),
        lambda: api.spec_pages_resize(pool.cpu(), t, r, k, k, 4, ws),
        lambda: api.spec_pages_fork(t, r, i32([0, 0]), ws),
        lambda: api.spec_pages_fork(t, r, k, ws, table_out=t[:, :1].contiguous()),
        lambda: api.spec_pages_compact(pool, t, r, ws, map=k),
        lambda: api.spec_pages_compact(pool, t, r, ws.cpu()),
        lambda: api.spec_pages_workspace(1, 0, 2),
    ]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    with pytest.raises(RuntimeError):
        api.spec_pages_fork(t, r, k, ws[:16])
