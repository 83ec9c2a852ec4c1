"""The 4-bit paged cache on the GPU (spec_q4_append, spec_q4_read, spec_q4_attention) against oracle/q4.py in 64 bits.

Codes, scales and their places are exact (bytes are compared).  The attention's tolerance, element by element, from
what the kernel rounds (A = sum p |v|, S = sum p s, the weights' mean of |v| and of the scales):
  the output to bf16                                     2^-8 |out|
  the weights P s to f16 (half a step, 2^-11)            2^-11 A
  the fp32 sums over codes 0..15 from which 8 S are taken: at most 64 MMAs in a row in a warp, each adding its
  16 products and its accumulator at 2^-23 of the largest       64 * 2^-23 * (15 + 8) S < 2^-12 S
  scores in fp32, of size X = scale sum |q k|: d + 8 roundings at 2^-23, twice (numerator and sum): 2 * 136 * 2^-23 X A
"""
import numpy as np
import pytest
import torch

from oracle import q4
from lossless_speculative_verification_gb300 import api

from gpu_util import need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()
    yield
    torch.cuda.synchronize()
    assert api.get_device_error() == 0


def bits(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)


def dev(b):
    return torch.from_numpy(np.ascontiguousarray(b).view(np.int16)).cuda().view(torch.bfloat16)


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()


class Cache:
    """Sequences of the given lengths in scattered pages; what no position covers is 0xFF (NaN scales)."""

    def __init__(self, lens, nkv, d, page, seed=0, k=None, v=None, extra=2, M=None):
        rs = np.random.default_rng(seed)
        self.lens, self.nkv, self.d, self.page = np.asarray(lens, np.int32), nkv, d, page
        B, T = len(lens), max(1, int(max(lens))) if k is None and v is None else (v if k is None else k).shape[1]
        self.B, self.T = B, T
        self.M = -(-T // page) if M is None else M
        used = [-(-int(n) // page) for n in lens]
        self.P = sum(used) + extra
        order = rs.permutation(self.P)
        self.tb = np.full((B, self.M), -1, np.int32)
        at = 0
        for b in range(B):
            self.tb[b, :used[b]] = order[at:at + used[b]]
            at += used[b]
        spread = 0.25 + rs.random((B, T, nkv, 1))
        self.k = bits(rs.normal(size=(B, T, nkv, d)) * spread if k is None else k)
        self.v = bits(rs.normal(size=(B, T, nkv, d)) * spread if v is None else v)
        self.pool = torch.full((self.P, api.spec_q4_page_bytes(nkv, d, page)), 255, dtype=torch.uint8, device="cuda")
        self.table, self.ctx = i32(self.tb), i32(self.lens)
        # position t of sequence b is row T - lens[b] + t of the last T rows
        kr, vr = np.zeros_like(self.k), np.zeros_like(self.v)
        for b, n in enumerate(lens):
            kr[b, T - n:], vr[b, T - n:] = self.k[b, :n], self.v[b, :n]
        api.spec_q4_append(dev(kr), dev(vr), self.pool, self.table, self.ctx, page)

    def values(self):
        return q4.value(*q4.quantise(self.k)), q4.value(*q4.quantise(self.v))

    def attend(self, q, scale=None, ws=None, **kw):
        B, Q, nh, d = q.shape
        ws = api.spec_q4_attention_workspace(B, Q, self.M, self.page, nh, self.nkv, d) if ws is None else ws
        out = api.spec_q4_attention(dev(q), self.pool, self.table, self.ctx, self.nkv, self.page, ws, scale=scale, **kw)
        torch.cuda.synchronize()
        return out.float().cpu().numpy().astype(np.float64)


def check(c, q, scale=None, got=None, what=""):
    scale = 1 / np.sqrt(c.d) if scale is None else scale
    k, v = c.values()
    qf = q4.bf16_f64(q)
    ref, A = q4.attention(qf, k, v, c.lens, scale)
    s = np.repeat(q4.bf16_f64(q4.quantise(c.v)[1]), 64, -1)
    _, S = q4.attention(qf, k, s, c.lens, scale)
    X = np.zeros(ref.shape[:3] + (1,))
    grp = q.shape[2] // c.nkv
    for b, n in enumerate(c.lens):
        if n:
            x = np.einsum("jhd,thd->jht", np.abs(qf[b]), np.abs(np.repeat(k[b, :n], grp, 1)))
            X[b, ..., 0] = x.max(-1) * scale
    tol = 2.0 ** -8 * np.abs(ref) + 2.0 ** -11 * A + 2.0 ** -12 * S + 272 * 2.0 ** -23 * X * A
    got = c.attend(q, scale) if got is None else got
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), "%s: %d of %d off, worst %.3g of its tolerance" % (
        what, bad.sum(), bad.size, np.nanmax(np.abs(got - ref) / np.maximum(tol, 1e-300)))
    return got


def queries(c, Q, grp, seed=1, std=1.0):
    return bits(np.random.default_rng(seed).normal(size=(c.B, Q, c.nkv * grp, c.d)) * std)


# ---------------------------------------------------------------------------------------------- append, read
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page,nkv,Q,lens", [
    (16, 2, 1, (1, 16, 17, 48)),
    (16, 3, 5, (5, 18, 33, 20)),           # rows across blocks and pages
    (64, 1, 37, (37, 100, 64, 101)),       # ragged blocks at both ends
    (32, 2, 8, (3, 0, 8, 70)),             # sequences shorter than Q, and a slot without one
    (256, 1, 2, (255, 256, 257, 300)),
])
def test_append_writes_its_bytes_and_no_others(d, page, nkv, Q, lens):
    rs = np.random.default_rng(d + page + Q)
    B, M = len(lens), -(-max(lens) // page) + 1
    P = B * M + 3
    tb = rs.permutation(P)[:B * M].reshape(B, M).astype(np.int32)
    k, v = (bits(rs.normal(size=(B, Q, nkv, d)) * 2.0 ** rs.integers(-12, 12, (B, Q, nkv, 1))) for _ in range(2))
    start = rs.integers(0, 256, (P, api.spec_q4_page_bytes(nkv, d, page))).astype(np.uint8)
    want = start.copy()
    q4.append(want, tb, lens, page, k, v)
    pool = torch.from_numpy(start).cuda()
    api.spec_q4_append(dev(k), dev(v), pool, i32(tb), i32(lens), page)
    np.testing.assert_array_equal(pool.cpu().numpy(), want)
    got = api.spec_q4_read(pool, i32(tb), i32(lens), Q, nkv, d, page)
    for x, y in zip(got, (k, v)):
        n, s = q4.quantise(y)
        ref = torch.from_numpy(q4.value(n, s)).to(torch.bfloat16).float().numpy()   # 12 bits at most: one rounding
        for b in range(B):
            ref[b, :max(0, Q - lens[b])] = 0
        np.testing.assert_array_equal(x.float().cpu().numpy(), ref)


def test_append_of_ends_and_of_what_is_no_number():
    x = np.zeros((1, 7, 1, 128), np.float32)
    x[0, 1, 0, :64] = 3.38e38                                   # the largest: the scale stays finite
    x[0, 2, 0, :64] = np.arange(64) * 2.0 ** -133               # subnormals: a scale of few bits
    x[0, 3, 0, 3], x[0, 3, 0, 100] = np.nan, np.inf
    x[0, 4, 0, 0] = -np.inf
    x[0, 5, 0, :8] = [7, .5, 1.5, 2.5, 3.5, -.5, -1.5, -6.5]    # ties
    x[0, 6, 0, 64:] = -0.0
    k, v = bits(x), bits(x[..., ::-1])
    start = np.zeros((1, api.spec_q4_page_bytes(1, 128, 16)), np.uint8)
    want = start.copy()
    tb = np.zeros((1, 1), np.int32)
    q4.append(want, tb, [7], 16, k, v)
    pool = torch.from_numpy(start).cuda()
    api.spec_q4_append(dev(k), dev(v), pool, i32(tb), i32([7]), 16)
    np.testing.assert_array_equal(pool.cpu().numpy(), want)
    got = api.spec_q4_read(pool, i32(tb), i32([7]), 7, 1, 128, 16)[0].float().cpu().numpy()
    assert np.isnan(got[0, 3]).all() and np.isnan(got[0, 4, 0, :64]).all() and np.isfinite(got[0, 4, 0, 64:]).all()


def test_every_code_of_every_scale_rounds_as_defined():
    # all bf16 significands against all scales' significands: x = any 8-bit significand, the group's largest any other
    m = np.arange(128, 256)
    k = np.zeros((1, 128 * 4, 1, 128), np.float32)
    for j in range(4):
        k[0, j * 128:(j + 1) * 128, 0, :64] = np.where(np.arange(64) % 2, -1, 1) * m[None, (j % 2) * 64:(j % 2) * 64 + 64] * 2.0 ** -(j // 2)
        k[0, j * 128:(j + 1) * 128, 0, 64:] = k[0, j * 128:(j + 1) * 128, 0, :64] / 8
    k[0, :, 0, 0] = k[0, :, 0, 64] = np.tile(m * 2.0, 4)
    c = Cache([512], 1, 128, 64, k=k, v=k[:, ::-1])
    kr, vr = api.spec_q4_read(c.pool, c.table, c.ctx, 512, 1, 128, 64)
    for got, ref in zip((kr, vr), c.values()):
        np.testing.assert_array_equal(got.float().cpu().numpy(), torch.from_numpy(ref).to(torch.bfloat16).float().numpy())


def test_append_out_of_range_is_reported_and_writes_nothing_there():
    k = bits(np.ones((3, 2, 1, 64)))
    pool = torch.zeros((4, api.spec_q4_page_bytes(1, 64, 16)), dtype=torch.uint8, device="cuda")
    tb = i32([[0, 4], [1, -1], [2, 3]])
    for lens, err in (([18, 5, 33], 7), ([4, 17, 5], 7), ([-1, 0, 0], 7), ([2, 2, 2], 0)):
        pool.zero_()
        api.spec_q4_append(dev(k), dev(k), pool, tb, i32(lens), 16)
        assert api.get_device_error() == err
    got = api.spec_q4_read(pool, tb, i32([17, 2, 99]), 1, 1, 64, 16)[0]
    assert api.get_device_error() == 7
    assert float(got[0].abs().max()) == 0 and float(got[2].abs().max()) == 0 and float(got[1].min()) == 1


# ---------------------------------------------------------------------------------------------- attention
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 64, 128])
@pytest.mark.parametrize("Q,nkv,grp", [(1, 2, 1), (3, 1, 5), (8, 2, 1), (2, 1, 16), (8, 1, 7), (5, 3, 2)])
def test_attention_lengths(d, page, Q, nkv, grp):
    # from nothing and one position over the ends of blocks, pages and chunks (128 positions)
    lens = [0, 1, Q, 15, 16, 17, 63, 64, 65, 127, 128, 129, 256, 300]
    c = Cache(lens, nkv, d, page, seed=Q)
    got = check(c, queries(c, Q, grp), what="d %d page %d" % (d, page))
    assert (got[0] == 0).all()
    if Q > 1:
        assert (got[1, :Q - 1] == 0).all()                      # rows before position 0


@pytest.mark.parametrize("d,Q,nkv,grp,n", [(128, 4, 1, 4, 9000), (64, 1, 2, 1, 20011), (128, 2, 1, 1, 4097)])
def test_attention_long(d, Q, nkv, grp, n):
    c = Cache([n], nkv, d, 64)
    check(c, queries(c, Q, grp))


# how a sequence's chunks meet goes by the batch, the key heads and the capacity: one chunk; a cluster; two or four groups
# of a CTA or the last CTA of several rounds of them; a second kernel
@pytest.mark.parametrize("lens,nkv,page,M", [
    ((100, 0, 128), 2, 32, 4),
    ((900, 1024, 1, 0, 517), 2, 64, 16),
    (tuple(range(30, 1230, 40)), 10, 64, 20),
    ((3000, 17, 9000, 6000), 1, 128, 80),
    ((3000, 17, 9000, 0, 5000, 1) + (200,) * 20, 2, 128, 80),
    ((20000, 30000), 2, 256, 128),
    (tuple(range(30, 2200, 70)), 10, 64, 36),
    (tuple(range(0, 1920, 80)), 10, 64, 36),
    (tuple(range(1, 2100, 131)), 10, 64, 64),
])
@pytest.mark.parametrize("d,Q,grp", [(64, 2, 1), (64, 3, 4), (128, 1, 2), (128, 1, 9)])
def test_attention_however_the_chunks_meet(lens, nkv, page, M, d, Q, grp):
    c = Cache(lens, nkv, d, page, M=M)
    q = queries(c, Q, grp)
    got = check(c, q)
    ws = api.spec_q4_attention_workspace(c.B, Q, M, page, nkv * grp, nkv, d)
    for _ in range(3):                                          # the order in which CTAs end does not show
        np.testing.assert_array_equal(c.attend(q, ws=ws), got)
    assert int(ws[:65536].count_nonzero()) == 0


# more CTAs than the GPU has room for take the sequences by length (up to 128 of them); chunks that lie one behind the
# other, and chunks by turns over the whole sequence
@pytest.mark.parametrize("B,nkv,page,M,top", [(70, 10, 16, 4, 64), (128, 6, 16, 4, 60), (129, 6, 16, 4, 60),
                                              (20, 8, 128, 32, 2500), (16, 8, 256, 128, 1700),
                                              (36, 10, 64, 36, 2304)])
@pytest.mark.parametrize("Q,grp", [(2, 1), (3, 3)])
def test_attention_by_length(B, nkv, page, M, top, Q, grp):
    rs = np.random.default_rng(B)
    lens = rs.integers(0, top + 1, B)
    lens[:6] = 0, top, 1, top, 0, 17
    lens[-3:] = 17, top, 2
    c = Cache(lens, nkv, 64, page, M=M)
    q = queries(c, Q, grp)
    got = check(c, q)
    np.testing.assert_array_equal(c.attend(q), got)
    wrong = c.lens.copy()                                       # lengths out of range, in the first and the last place
    wrong[[0, B // 2, -1]] = M * page + 1, -1, np.iinfo(np.int32).max
    c.ctx = i32(wrong)
    ref = got.copy()
    ref[[0, B // 2, -1]] = 0
    np.testing.assert_array_equal(c.attend(q), ref)
    assert api.get_device_error() == 7


@pytest.mark.parametrize("lens,nkv,page,M", [((2100, 900, 0, 517), 64, 64, 36), ((3000, 17, 2049), 80, 128, 72)])
def test_a_row_does_not_depend_on_the_others_in_any_cut(lens, nkv, page, M):
    c = Cache(lens, nkv, 64, page, M=M)                         # two chunks or more of 9 and of 18 steps or so
    q = queries(c, 8, 2)
    all_rows = c.attend(q)
    for j in (0, 6):
        c.ctx = i32(np.maximum(c.lens - 7 + j, 0))
        np.testing.assert_array_equal(c.attend(q[:, j:j + 1])[c.lens > 7, 0], all_rows[c.lens > 7, j])


@pytest.mark.parametrize("B", [57, 1200])
@pytest.mark.parametrize("Q,grp", [(1, 1), (3, 5)])
def test_sums_over_the_longest_chunk(Q, grp, B):
    # 9600 (sequence, key head) pairs: one chunk each, of 32768 positions (456: a few); flat weights over values of mean
    # 0, where a sum that loses its low bits shows.  32 MMAs between two times that the 8 S are taken off (32 * 2^-23 * 23 S),
    # 512 MMAs into an accumulator that has them off (512 * 2^-23 A)
    lens = [0] * (B - 1) + [32768]
    rs = np.random.default_rng(0)
    k, v = (rs.normal(size=(1, 32768, 8, 64)) for _ in range(2))
    one = Cache([32768], 8, 64, 128, k=k, v=v)
    q = np.zeros((B, Q, 8 * grp, 64), np.uint16)
    q[-1] = bits(rs.normal(size=(Q, 8 * grp, 64)) * 0.05)
    table = np.full((B, one.M), -1, np.int32)
    table[-1] = one.tb
    ws = api.spec_q4_attention_workspace(B, Q, one.M, 128, 8 * grp, 8, 64)
    got = api.spec_q4_attention(dev(q), one.pool, i32(table), i32(lens), 8, 128, ws).float().cpu().numpy().astype(np.float64)
    assert (got[:-1] == 0).all()
    kf, vf = one.values()
    ref, A = q4.attention(q4.bf16_f64(q[-1:]), kf, vf, one.lens, 1 / 8)
    S = np.repeat(q4.bf16_f64(q4.quantise(one.v)[1]), 64, -1).max()
    tol = 2.0 ** -8 * np.abs(ref) + 2.0 ** -11 * A + 32 * 2.0 ** -23 * 23 * S + (512 + 272) * 2.0 ** -23 * A
    assert (np.abs(got[-1:] - ref) <= tol).all()
    # over all elements little more than the rounding of the output, whose steps' rms is 2^-8 / sqrt(3) of the power of
    # two below a value, and so at most that of the value
    assert np.linalg.norm(got[-1:] - ref) <= 2.0 ** -8 / np.sqrt(3) * np.linalg.norm(ref)


def test_attention_peaked_and_scaled():
    c = Cache([700, 333], 2, 128, 32, seed=4)
    check(c, queries(c, 4, 2, std=6.0), what="peaked")
    check(c, queries(c, 4, 2, std=2.0 ** -70), scale=2.0 ** 60, what="small queries")
    check(c, queries(c, 4, 2, std=2.0 ** 60), scale=2.0 ** -62, what="large queries")


@pytest.mark.parametrize("grp", [1, 3])
def test_attention_of_values_of_any_size(grp):
    # value scales from 2^-100 to 2^100 in one sequence, also behind what a row sees; keys that make the largest count
    rs = np.random.default_rng(7)
    for lo, hi in ((-100, -80), (80, 100), (-20, 20), (-60, 60)):
        e = rs.integers(lo, hi, (1, 400, 2, 1))
        v = rs.normal(size=(1, 400, 2, 128)) * 2.0 ** e
        c = Cache([400], 2, 128, 64, v=v)
        check(c, queries(c, 8, grp), what="2^%d .. 2^%d" % (lo, hi))
    v = rs.normal(size=(1, 70, 1, 64))
    v[0, -1] *= 2.0 ** 90                                       # only the last row sees it
    c = Cache([70], 1, 64, 16, v=v)
    got = check(c, queries(c, 6, grp))
    assert np.abs(got[0, :5]).max() < 8


@pytest.mark.parametrize("d,grp", [(128, 1), (128, 2), (64, 1), (64, 3)])
def test_what_is_no_number_reaches_only_the_rows_that_see_it(d, grp):
    rs = np.random.default_rng(8)
    k, v = rs.normal(size=(2, 1, 150, 2, d))
    base = Cache([150], 2, d, 64, k=k, v=v)
    q = queries(base, 5, grp)
    ref = base.attend(q)
    for which in (0, 1):
        for x in (np.nan, np.inf, -np.inf):
            k2, v2 = k.copy(), v.copy()
            (k2, v2)[which][0, 147, 1, 9] = x                   # rows 2, 3, 4 see position 147; key head 1's heads
            got = Cache([150], 2, d, 64, k=k2, v=v2).attend(q)
            np.testing.assert_array_equal(got[0, :2], ref[0, :2])
            np.testing.assert_array_equal(got[0, :, :grp], ref[0, :, :grp])
            assert np.isnan(got[0, 2:, grp:, :64]).all()
            if which == 0:
                assert np.isnan(got[0, 2:, grp:, 64:]).all()
            else:                                               # the values' other group is what it was
                np.testing.assert_allclose(got[0, 2:, grp:, 64:], ref[0, 2:, grp:, 64:], rtol=2.0 ** -7, atol=1e-4)
    for x in (np.nan, np.inf):
        q2 = q4.bf16_f64(q)
        q2[0, 1, -1, 7] = x
        got = base.attend(bits(q2))
        assert np.isnan(got[0, 1, -1]).all()
        got[0, 1, -1] = ref[0, 1, -1]
        np.testing.assert_array_equal(got, ref)


def test_a_row_does_not_depend_on_the_others():
    c = Cache([517, 130, 64, 1000], 2, 128, 16, seed=5)
    q = queries(c, 8, 8)
    all_rows = c.attend(q)
    for j in (0, 3, 7):
        part = Cache(c.lens - 7 + j, 2, 128, 16, seed=5, k=q4.bf16_f64(c.k)[:, :c.T], v=q4.bf16_f64(c.v)[:, :c.T], M=c.M)
        np.testing.assert_array_equal(part.attend(q[:, j:j + 1])[:, 0], all_rows[:, j])
    some = np.concatenate([q[:, 2:5, h:h + 1] for h in (5, 13)], 2)
    at3 = Cache(c.lens - 3, 2, 128, 16, seed=5, k=q4.bf16_f64(c.k), v=q4.bf16_f64(c.v), M=c.M)
    np.testing.assert_array_equal(at3.attend(some), all_rows[:, 2:5][:, :, [5, 13]])
    np.testing.assert_array_equal(c.attend(q), all_rows)        # and from run to run


def test_pages_in_any_place_of_a_pool_beyond_4_gb():
    nkv, d, page = 8, 128, 128
    nbytes = api.spec_q4_page_bytes(nkv, d, page)
    P = (5 << 30) // nbytes
    c = Cache([300, 200], nkv, d, page)
    q = queries(c, 2, 1)
    ref = c.attend(q)
    big = torch.empty((P, nbytes), dtype=torch.uint8, device="cuda")
    far = np.where(c.tb >= 0, P - 1 - c.tb * 7, -1)
    assert (far[far >= 0].astype(np.int64) * nbytes > 1 << 32).all()
    kr, vr = np.zeros_like(c.k), np.zeros_like(c.v)
    for b, n in enumerate(c.lens):
        kr[b, c.T - n:], vr[b, c.T - n:] = c.k[b, :n], c.v[b, :n]
    api.spec_q4_append(dev(kr), dev(vr), big, i32(far), c.ctx, page)
    c.pool, c.table = big, i32(far)
    np.testing.assert_array_equal(c.attend(q), ref)
    k, v = c.values()
    got = api.spec_q4_read(big, c.table, c.ctx, 50, nkv, d, page)[0].float().cpu().numpy()
    np.testing.assert_array_equal(got[0], torch.from_numpy(k[0, 250:300]).to(torch.bfloat16).float().numpy())


@pytest.mark.parametrize("lens,nkv,M", [(tuple(range(5, 2165, 60)), 10, 36), (tuple(range(0, 1920, 80)), 10, 36),
                                        ((4000,), 2, 64), ((900, 4000, 30), 80, 72), (tuple(range(70)), 10, 2)])
@pytest.mark.parametrize("Q,grp", [(2, 1), (2, 5)])
def test_a_captured_call_follows_the_lengths(lens, nkv, M, Q, grp):
    c = Cache(lens, nkv, 64, 64, M=M)
    q = dev(queries(c, Q, grp))
    ws = api.spec_q4_attention_workspace(c.B, Q, M, 64, nkv * grp, nkv, 64)
    out = torch.empty_like(q)

    def call():
        return api.spec_q4_attention(q, c.pool, c.table, c.ctx, nkv, 64, ws, out=out)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for turn in range(3):
        c.ctx.copy_(i32(np.maximum(c.lens - 37 * turn * (np.arange(c.B) % 3), 0)))
        graph.replay()
        got = out.clone()
        out.fill_(-7.0)
        assert torch.equal(call(), got) and int(ws[:65536].count_nonzero()) == 0


def test_attention_out_of_range_is_reported():
    c = Cache([100, 100, 100], 1, 64, 32)
    q = queries(c, 2, 1)
    ref = c.attend(q)
    c.ctx = i32([100, 129, -5])
    got = c.attend(q)
    assert api.get_device_error() == 7
    np.testing.assert_array_equal(got[0], ref[0])
    assert (got[1:] == 0).all()
    # a page out of range: its positions are left out
    c.ctx = i32([100, 100, 100])
    for wrong in (-1, c.P, 1 << 30):
        tb = c.tb.copy()
        tb[1, 1] = wrong
        c.table = i32(tb)
        got = c.attend(q)
        assert api.get_device_error() == 7
        np.testing.assert_array_equal(got[[0, 2]], ref[[0, 2]])
        keep = np.r_[0:32, 64:100]
        k, v = c.values()
        x = np.exp(k[1, keep, 0] @ q4.bf16_f64(q)[1, 1, 0] / 8)
        np.testing.assert_allclose(got[1, 1, 0], (x / x.sum()) @ v[1, keep, 0], atol=2e-2)


def test_empty_batch_streams_graphs_and_one_workspace_for_all():
    q = torch.empty((0, 2, 2, 64), dtype=torch.bfloat16, device="cuda")
    c = Cache([200, 700], 2, 64, 16)
    ws = api.spec_q4_attention_workspace(2, 8, c.M, 16, 4, 2, 64)
    none = i32(np.zeros((0, 3)))
    assert api.spec_q4_attention(q, c.pool, none, i32([]), 2, 16, ws).shape == (0, 2, 2, 64)
    a, b = queries(c, 1, 2), queries(c, 8, 1, seed=2)
    ra, rb = c.attend(a), c.attend(b)
    ws[65536:].fill_(255)                                       # behind the counters nothing is wanted
    for _ in range(2):
        np.testing.assert_array_equal(c.attend(a, ws=ws), ra)
        np.testing.assert_array_equal(c.attend(b, ws=ws), rb)
    assert int(ws[:65536].count_nonzero()) == 0
    side = torch.cuda.Stream()
    out = torch.empty((2, 8, 2, 64), dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    np.testing.assert_array_equal(c.attend(b, ws=ws, out=out, stream=side), rb)
    # captured: append, attend; replayed with other lengths and other rows
    k, v = torch.zeros((2, 8, 2, 64), dtype=torch.bfloat16, device="cuda"), torch.zeros((2, 8, 2, 64), dtype=torch.bfloat16, device="cuda")
    qd, ctx = dev(b), c.ctx.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.spec_q4_append(k, v, c.pool, c.table, ctx, 16)
        api.spec_q4_attention(qd, c.pool, c.table, ctx, 2, 16, ws, out=out)
    for lens in ([200, 700], [77, 699], [8, 16]):
        ctx.copy_(i32(lens))
        kn, vn = (bits(np.random.default_rng(lens[0] + i).normal(size=(2, 8, 2, 64))) for i in range(2))
        k.copy_(dev(kn)); v.copy_(dev(vn))
        graph.replay()
        torch.cuda.synchronize()
        for s, n in enumerate(lens):
            c.k[s, n - 8:n], c.v[s, n - 8:n] = kn[s], vn[s]
        c.lens = np.array(lens, np.int32)
        check(c, b, got=out.float().cpu().numpy().astype(np.float64), what=str(lens))


def test_two_calls_at_once():
    shapes = (((900, 1024, 1, 0, 517), 2, 64, 16, 1), (tuple(range(30, 2200, 70)), 10, 64, 36, 1),
              (tuple(range(0, 1920, 80)), 10, 64, 36, 1), ((20000, 30000), 2, 256, 128, 9))
    calls = []
    for lens, nkv, page, M, grp in shapes:
        c = Cache(lens, nkv, 64, page, M=M)
        q = dev(queries(c, 1, grp))
        ws = [api.spec_q4_attention_workspace(c.B, 1, M, page, nkv * grp, nkv, 64) for _ in range(2)]
        ref = api.spec_q4_attention(q, c.pool, c.table, c.ctx, nkv, page, ws[0])
        calls.append((c, q, ws, ref, [torch.empty_like(q) for _ in range(2)]))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, q, ws, ref, out in calls:
            for i, s in enumerate(streams):
                api.spec_q4_attention(q, c.pool, c.table, c.ctx, c.nkv, c.page, ws[i], out=out[i], stream=s)
    torch.cuda.synchronize()
    for c, q, ws, ref, out in calls:
        assert torch.equal(out[0], ref) and torch.equal(out[1], ref)
        assert not any(int(w[:65536].count_nonzero()) for w in ws)


def test_wrappers_refuse():
    c = Cache([20, 30], 2, 64, 16)
    q, ws = dev(queries(c, 2, 1)), api.spec_q4_attention_workspace(2, 2, c.M, 16, 2, 2, 64)
    k = torch.zeros((2, 2, 2, 64), dtype=torch.bfloat16, device="cuda")
    bad = [
        lambda: api.spec_q4_append(k.float(), k, c.pool, c.table, c.ctx, 16),
        lambda: api.spec_q4_append(k, k[:, :1], c.pool, c.table, c.ctx, 16),
        lambda: api.spec_q4_append(k, k, c.pool, c.table, c.ctx, 32),
        lambda: api.spec_q4_append(k, k, c.pool, c.table.long(), c.ctx, 16),
        lambda: api.spec_q4_append(k, k, c.pool, c.table, c.ctx[:1], 16),
        lambda: api.spec_q4_append(k, k, c.pool.cpu(), c.table, c.ctx, 16),
        lambda: api.spec_q4_append(k.transpose(1, 2), k.transpose(1, 2), c.pool, c.table, c.ctx, 16),
        lambda: api.spec_q4_read(c.pool, c.table, c.ctx, 4, 2, 64, 16, k=k, v=k),
        lambda: api.spec_q4_attention(q, c.pool, c.table, c.ctx, 1, 16, ws),
        lambda: api.spec_q4_attention(q, c.pool, c.table, c.ctx, 2, 16, ws, out=q[:1]),
        lambda: api.spec_q4_attention(q[0], c.pool, c.table, c.ctx, 2, 16, ws),
        lambda: api.spec_q4_attention_workspace(2, 9, c.M, 16, 2, 2, 64),
        lambda: api.spec_q4_page_bytes(2, 96, 16),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
    with pytest.raises(RuntimeError):
        api.spec_q4_attention(q, c.pool, c.table, c.ctx, 2, 16, ws[:16])


# as above: one chunk, a cluster, two and four groups of a CTA, the last CTA of several, a second kernel
# (On a GB300 a try of a wait lasts as long as the load; with tries that return at once the limit ran out in every call, and
# these held as well.)
@pytest.mark.parametrize("lens,nkv,page,M", [
    ((100, 0, 128), 2, 32, 4),
    ((3000, 17, 9000, 6000), 1, 128, 80),
    (tuple(range(30, 2200, 70)), 10, 64, 36),
    (tuple(range(1, 2100, 131)), 10, 64, 64),
    (tuple(range(0, 1920, 80)), 10, 64, 36),
    ((20000, 30000), 2, 256, 128),
])
@pytest.mark.parametrize("grp", [1, 9])
def test_a_wait_that_runs_out_is_reported_and_the_workspace_serves_the_next_call(lens, nkv, page, M, grp):
    c = Cache(lens, nkv, 128, page, M=M)
    q = queries(c, 1, grp)
    ws = api.spec_q4_attention_workspace(c.B, 1, M, page, nkv * grp, nkv, 128)
    ref = c.attend(q, ws=ws)
    flush = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    try:
        api.set_wait_limit_ns(1)
        for turn in range(3):
            flush.fill_(turn)                                   # the pages come from memory again
            got = c.attend(q, ws=ws)
            err = api.get_device_error()
            assert err in (0, 6)                                # a wait may end before anyone looks at the time
            if err == 0:
                np.testing.assert_array_equal(got, ref)
            assert int(ws[:65536].count_nonzero()) == 0
    finally:
        api.set_wait_limit_ns(2000000000)
    np.testing.assert_array_equal(c.attend(q, ws=ws), ref)
