"""The attention over the 4-bit cache where value scales and scores differ far: groups of a head, positions of a step,
chunks of a sequence.  An output element is held to its own size: the tolerance of test_gpu_q4 (bf16 output 2^-8 |out|,
f16 weights 2^-11 A, sums over codes 2^-12 S, scores 272 * 2^-23 X A, with A and S the weighted means of that dim's |v|
and of that group's scale), and 2^-134 for outputs below the smallest normal bf16."""
import numpy as np
import pytest
import torch

from oracle import q4
from lossless_speculative_verification_gb300 import api

from gpu_util import need_gpu
from test_gpu_q4 import Cache, bits, i32, queries

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()
    yield
    torch.cuda.synchronize()
    assert api.get_device_error() == 0


def check(c, q, what=""):
    scale = 1 / np.sqrt(c.d)
    k, v = c.values()
    qf = q4.bf16_f64(q)
    ref, A = q4.attention(qf, k, v, c.lens, scale)
    _, S = q4.attention(qf, k, np.repeat(q4.bf16_f64(q4.quantise(c.v)[1]), 64, -1), c.lens, scale)
    X = np.zeros(ref.shape[:3] + (1,))
    for b, n in enumerate(c.lens):
        if n:
            kk = np.abs(np.repeat(k[b, :n], q.shape[2] // c.nkv, 1))
            X[b, ..., 0] = np.einsum("jhd,thd->jht", np.abs(qf[b]), kk).max(-1) * scale
    tol = 2.0 ** -8 * np.abs(ref) + 2.0 ** -11 * A + 2.0 ** -12 * S + 272 * 2.0 ** -23 * X * A + 2.0 ** -134
    got = c.attend(q)
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), "%s: %d of %d off, worst %.3g of its tolerance" % (
        what, bad.sum(), bad.size, np.nanmax(np.abs(got - ref) / tol))
    return got


FORMS = [1, 3]                                                  # query heads a key head: up to eight rows, nine and more


@pytest.mark.parametrize("grp", FORMS)
@pytest.mark.parametrize("r", [6, 9, 20, 28, 36, 60, 100])
def test_groups_of_a_head_of_different_size(r, grp):
    rs = np.random.default_rng(r)
    for half in (slice(0, 64), slice(64, 128)):
        v = rs.normal(size=(2, 300, 2, 128))
        v[..., half] *= 2.0 ** -r
        v[1, 150:, 1] *= 2.0 ** -r                              # and smaller from some position on
        c = Cache([300, 290], 2, 128, 64, v=v)
        check(c, queries(c, 4, grp), what="2^-%d" % r)


def leaning(rs, T, d, at, lean):
    """Keys [1, T, 1, d] whose scores with leaning_queries are lower by `lean` (log2 units) at the positions `at`."""
    k = rs.normal(size=(1, T, 1, d))
    k[..., 0] = 0
    k[0, at, 0, 0] = -lean * np.log(2) * np.sqrt(d) / 16
    return k


def leaning_queries(rs, Q, nh, d):
    q = rs.normal(size=(1, Q, nh, d))
    q[..., 0] = 16
    return bits(q)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("grp", FORMS)
@pytest.mark.parametrize("r", [7, 16, 24, 28, 32, 40, 80])
def test_large_values_of_negligible_weight(r, grp, d):
    rs = np.random.default_rng(r)
    for at in ([5], [299], [2, 40, 77, 130, 200, 255]):
        v = rs.normal(size=(1, 300, 1, d))
        v[0, at] *= 2.0 ** r
        c = Cache([300], 1, d, 64, k=leaning(rs, 300, d, at, r + 20), v=v)
        check(c, leaning_queries(rs, 4, grp, d), what="%s" % at)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("grp", FORMS)
@pytest.mark.parametrize("size", [0.0, 2.0 ** -34, 2.0 ** -7])
@pytest.mark.parametrize("a", [8, 24, 28, 34, 40, 90])
def test_small_values_of_the_largest_weights(a, size, grp, d):
    rs = np.random.default_rng(a)
    for at in ([150], list(range(7, 300, 32))):
        v = rs.normal(size=(1, 300, 1, d))
        v[0, at] *= size
        c = Cache([300], 1, d, 16, k=leaning(rs, 300, d, at, -a), v=v)
        check(c, leaning_queries(rs, 4, grp, d), what="%s" % at)


@pytest.mark.parametrize("grp", FORMS)
@pytest.mark.parametrize("lo,hi", [(-124, -124), (-112, -112), (-96, -96), (-70, -58), (58, 70), (100, 100), (118, 120),
                                   (-4, 4), (-5, 4), (-3, 5), (-118, 118)])
def test_scales_at_the_ends_of_what_there_is(lo, hi, grp):
    rs = np.random.default_rng(200 + hi)
    for d in (64, 128):
        v = rs.normal(size=(2, 400, 1, d)) * 2.0 ** rs.integers(lo, hi + 1, (2, 400, 1, 1))
        c = Cache([400, 333], 1, d, 64, v=v)
        check(c, queries(c, 6, grp), what="2^%d .. 2^%d" % (lo, hi))


def mixed(rs, B, T, nkv, d):
    """Values of one size for a stretch of positions, of any size for the next, one group zero or small here and there."""
    v = rs.normal(size=(B, T, nkv, d))
    e = np.repeat(rs.integers(-40, 40, (B, -(-T // 96), nkv, 1)), 96, 1)[:, :T].astype(float)
    e += np.where(rs.random((B, T, 1, 1)) < 0.1, rs.integers(-60, 60, (B, T, nkv, 1)), 0)
    v *= 2.0 ** e
    v[..., :64] *= np.where(rs.random((B, T, nkv, 1)) < 0.1, 0, 1) * np.where(rs.random((B, 1, nkv, 1)) < 0.5, 2.0 ** -30, 1)
    return v


# one chunk, a cluster, groups of a CTA, the last CTA of several, a second kernel
@pytest.mark.parametrize("lens,nkv,page,M", [
    ((100, 0, 128), 2, 32, 4),
    ((900, 1024, 1, 0, 517), 2, 64, 16),
    ((3000, 17, 2500), 1, 128, 80),
    (tuple(range(30, 2200, 70)), 10, 64, 36),
    (tuple(range(0, 1920, 80)), 10, 64, 36),
    (tuple(range(1, 2100, 131)), 10, 64, 64),
    ((3000, 17, 1000, 0, 500, 1) + (200,) * 20, 2, 128, 80),
])
@pytest.mark.parametrize("d,Q,grp", [(64, 3, 4), (128, 3, 1), (128, 1, 9), (64, 2, 1)])
def test_mixed_sizes_however_the_chunks_meet(lens, nkv, page, M, d, Q, grp):
    rs = np.random.default_rng(len(lens))
    c = Cache(lens, nkv, d, page, M=M, v=mixed(rs, len(lens), max(lens), nkv, d))
    q = queries(c, Q, grp, std=2.0)
    got = check(c, q)
    np.testing.assert_array_equal(c.attend(q), got)


@pytest.mark.parametrize("d", [64, 128])
def test_a_row_of_mixed_sizes_does_not_depend_on_the_others(d):
    rs = np.random.default_rng(d)
    lens = np.array([517, 130, 64, 1000])
    c = Cache(lens, 2, d, 16, v=mixed(rs, 4, 1000, 2, d))
    q = queries(c, 8, 8, std=2.0)
    all_rows = c.attend(q)
    for j in range(8):
        c.ctx = i32(lens - 7 + j)
        np.testing.assert_array_equal(c.attend(q[:, j:j + 1])[:, 0], all_rows[:, j])
        some = np.concatenate([q[:, max(0, j - 2):j + 1, h:h + 1] for h in (3, 13)], 2)
        np.testing.assert_array_equal(c.attend(some), all_rows[:, max(0, j - 2):j + 1][:, :, [3, 13]])


@pytest.mark.parametrize("d,grp", [(128, 1), (128, 2), (64, 3)])
def test_what_is_no_number_among_mixed_sizes(d, grp):
    rs = np.random.default_rng(9)
    k, v = rs.normal(size=(1, 150, 2, d)), mixed(rs, 1, 150, 2, d)
    base = Cache([150], 2, d, 64, k=k, v=v)
    q = queries(base, 5, grp)
    ref = base.attend(q)
    assert np.isfinite(ref).all()
    for which in (0, 1):
        k2, v2 = k.copy(), v.copy()
        (k2, v2)[which][0, 147, 1, 9] = np.nan                  # rows 2, 3, 4 see position 147; key head 1's heads
        got = Cache([150], 2, d, 64, k=k2, v=v2).attend(q)
        np.testing.assert_array_equal(got[0, :2], ref[0, :2])
        np.testing.assert_array_equal(got[0, :, :grp], ref[0, :, :grp])
        assert np.isnan(got[0, 2:, grp:, :64]).all()
        if which == 0:
            assert np.isnan(got[0, 2:, grp:, 64:]).all()
        else:
            assert np.isfinite(got[0, 2:, grp:, 64:]).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("factor", [0.0, 2.0 ** -40, 2.0 ** -12, 2.0 ** 12, 2.0 ** 40])
def test_a_few_positions_of_another_size(d, factor):
    """Steps of one size behind steps of several: the sums have one base again."""
    rs = np.random.default_rng(3)
    lens = np.array([1500, 1400, 700])
    for both in (True, False):
        v = rs.normal(size=(3, 1500, 2, d))
        at = [0, 1, 33, 64, 100, 129, 640, 1390]
        if both:
            v[:, at] *= factor
        else:
            v[:, at, :, :64] *= factor
        c = Cache(lens, 2, d, 64, v=v)
        q = queries(c, 4, 4, std=3.0)
        all_rows = check(c, q, what="both %s" % both)
        for j in (0, 3):
            c.ctx = i32(lens - 3 + j)
            np.testing.assert_array_equal(c.attend(q[:, j:j + 1])[:, 0], all_rows[:, j])
            np.testing.assert_array_equal(c.attend(q[:, j:j + 1, [1, 6]])[:, 0], all_rows[:, j][:, [1, 6]])
