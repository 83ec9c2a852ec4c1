"""Log probabilities, entropies and the most likely tokens (spec_logprobs) on the GPU against oracle/q8.py in 64 bits.

Tokens are exact.  The tolerance of the numbers: a logit's e^(x - m) is off by 2^-22 (the exponential), by the rounding of
x - m where it has one and of its product with log2 e, 2^-23 |x - m| together, and by a rescaling where a maximum
rose, 2^-22 and 2^-23 of its exponent again: as a share of S = sum e^(x - m), 2^-21 + 2^-22 D with D = sum p (m - x).
The sums are of at most n = V / 512 + 40 roundings of 2^-24 (a thread adds every other logit that it takes).  With
r = 2^-21 + 2^-22 D + n 2^-24 the logarithm of S is off by r and its own rounding; a log probability by that and its
roundings, 2^-23 (|x - m| + log S); the entropy log S - D by r (1 + 2 D) and 2^-23 (log S + D).
"""
import numpy as np
import pytest
import torch

from oracle import q8
from lossless_speculative_verification_gb300 import api

from gpu_util import need_gpu

pytestmark = pytest.mark.gpu

LOWEST = {torch.bfloat16: float(torch.finfo(torch.bfloat16).min), torch.float32: float(torch.finfo(torch.float32).min)}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()
    yield
    torch.cuda.synchronize()
    assert api.get_device_error() == 0


def check(x, n, tokens=None, what=""):
    """x [R, V] on the host, of the type to test."""
    R, V = x.shape
    rs = np.random.default_rng(V)
    if tokens is None:
        tokens = rs.integers(-1, V, R)
    got = api.spec_logprobs(x.cuda(), torch.from_numpy(tokens.astype(np.int32)).cuda(), n)
    lp, ent, ids, tops = (t.cpu().numpy().astype(np.float64) for t in got)
    f = x.double().numpy()
    rlp, rent, rids, rtops = q8.logprobs(f, tokens, n)
    np.testing.assert_array_equal(ids, rids, err_msg=what)
    with np.errstate(invalid="ignore", over="ignore"):
        m = f.max(1)
        e = np.exp(f - m[:, None])
        log_s = np.log(e.sum(1))
        D = np.nansum(np.where(e > 0, e * (m[:, None] - f), 0), 1) / e.sum(1)
        r = 2.0 ** -21 + 2.0 ** -22 * D + (V / 512 + 40) * 2.0 ** -24
        size = lambda v: np.where(np.isfinite(v), np.abs(v), 0) + 2 * np.abs(log_s).reshape((-1,) + (1,) * (v.ndim - 1))
        tol = {"lp": r + 2.0 ** -23 * size(rlp), "tops": r[:, None] + 2.0 ** -23 * size(rtops),
               "ent": r * (1 + 2 * D) + 2.0 ** -23 * (np.abs(log_s) + D)}
    for name, g, w in (("lp", lp, rlp), ("ent", ent, rent), ("tops", tops, rtops)):
        fine = np.isfinite(w)
        np.testing.assert_array_equal(np.isnan(g), np.isnan(w), err_msg=what + name)
        np.testing.assert_array_equal(g[~fine & ~np.isnan(w)], w[~fine & ~np.isnan(w)], err_msg=what + name)
        off, most = np.abs(g[fine] - w[fine]), np.nan_to_num(tol[name][fine], nan=0.0)   # (nothing allowed: exact)
        assert (off <= most).all(), "%s %s: worst %.3g of its tolerance" % (what, name, np.max(off / np.maximum(most, 1e-300)))
    return got


def logits(seed, R, V, dtype, spread=3.0, peaks=5):
    g = torch.Generator().manual_seed(seed)
    x = spread * torch.randn((R, V), generator=g)
    x[torch.arange(R)[:, None], torch.randint(0, V, (R, peaks), generator=g)] += 8
    return x.to(dtype)


TYPES = [torch.bfloat16, torch.float32]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V", [1, 2, 3, 7, 8, 9, 16, 31, 63, 64, 65, 100, 255, 513, 1000, 2049, 8191, 8193, 40007])
def test_vocabularies_of_every_end(V, dtype):
    # odd ones begin rows on every byte that a value may
    for n in (0, 1, 5, 32):
        check(logits(V, 5, V, dtype), n, what="V %d n %d " % (V, n))


# the forms: clusters of 16, 8, 4, 2 narrow CTAs, of wide ones, one wide, middle, narrow or tiny CTA a row; rows of one batch
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("R,V", [(1, 129280), (2, 70001), (4, 32000), (16, 129280), (37, 20000), (50, 60001), (60, 129280),
                                 (100, 33333), (152, 30000), (200, 40001), (304, 20000), (700, 9001), (3000, 257), (320, 3999), (1300, 7001), (1220, 15000)])
def test_every_form(R, V, dtype):
    check(logits(R, R, V, dtype), 20, what="%d x %d " % (R, V))


@pytest.mark.parametrize("R,V", [(1, 129280), (70, 9001), (400, 3001)])
def test_logits_of_any_size(R, V):
    # what the sums are relative to is a product with log2 e: rows around and beyond the size where its rounding counts
    for k, at in enumerate((0.0, 700.0, -65000.0, 65535.5, -65536.0, 65536.0, 1e5, -3e6, 1e7, -1e9, 1e12, 3e38, -3e38)):
        x = logits(k, R, V, torch.float32, spread=1.0)
        step = float(np.spacing(np.float32(abs(at) + 32)))      # so that logits there are not all the same
        check((x * max(1.0, step) + at).clamp(-3.3e38, 3.3e38), 7, what="around %g " % at)
    # half of a row around each size
    x = logits(9, R, V, torch.float32, spread=1.0)
    x[:, V // 2:] += 65530.0
    x[:, :V // 2] += 65538.0
    check(x, 7, what="around 2^16 ")
    check(torch.cat([x[:, V // 2:], x[:, :V // 2]], 1), 7, what="around 2^16, rising ")
    check(logits(10, R, V, torch.bfloat16, spread=900.0), 7, what="wide ")
    check(logits(11, R, V, torch.bfloat16, spread=1e6), 7, what="far ")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("R,V", [(1, 129280), (40, 30001), (130, 17000), (310, 4001), (3, 200)])
def test_rows_that_are_no_ordinary_ones(R, V, dtype):
    g = torch.Generator().manual_seed(R)
    x = logits(1, R, V, dtype)
    kinds = [
        ("equal", lambda: torch.zeros(V)),
        ("few values", lambda: torch.randint(0, 3, (V,), generator=g).float()),
        ("rising", lambda: torch.arange(V) * 1e-3),
        ("falling", lambda: -torch.arange(V) * 1e-3),
        ("nothing allowed", lambda: torch.full((V,), -torch.inf)),
        ("one allowed", lambda: torch.where(torch.arange(V) == V // 2, 1.5, -torch.inf)),
        ("three allowed", lambda: torch.where(torch.arange(V) % (V // 3) == 7, 2.0, -torch.inf)),
        ("all of the lowest", lambda: torch.full((V,), LOWEST[dtype])),
        ("lowest but two", lambda: torch.where(torch.arange(V) < 2, 0.25, LOWEST[dtype])),
        ("lowest and -inf", lambda: torch.where(torch.arange(V) % 3 == 0, LOWEST[dtype], -torch.inf)),
        ("zeros of both signs", lambda: torch.where(torch.arange(V) % 2 == 0, -0.0, 0.0)),
        ("far apart", lambda: torch.where(torch.arange(V) % 7 == 0, 3e4, -3e4)),
        ("a peak of certainty", lambda: torch.where(torch.arange(V) == V - 1, 60.0, 0.0)),
        ("a NaN", lambda: torch.where(torch.arange(V) == V // 3, torch.nan, 1.0)),
        ("an infinity", lambda: torch.where(torch.arange(V) == V - 2, torch.inf, 1.0)),
        ("largest values", lambda: torch.where(torch.arange(V) % 5 == 0, -LOWEST[dtype], 0.0)),
    ]
    for k, (name, make) in enumerate(kinds):
        y = x.clone()
        y[k % R] = make().to(dtype)          # beside rows that are
        for n in (1, 32):
            check(y, n, what=name + " ")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("R,V", [(64, 1000), (3, 129280), (400, 9001)])
def test_log_probabilities_are_never_above_0_and_entropies_never_below(R, V, dtype):
    # one allowed token, and one that outweighs the others by far: log S is 0 but for roundings
    g = torch.Generator().manual_seed(V)
    at = torch.randint(0, V, (R,), generator=g)
    peak = 5 * torch.randn(R, generator=g)
    for rest, more in ((-torch.inf, 0.0), (0.0, 60.0), (-900.0, 40.0)):
        x = torch.full((R, V), rest)
        x[torch.arange(R), at] = peak + more
        lp, ent, ids, tops = check(x.to(dtype), 2, at.numpy(), what="rest %g " % rest)
        assert bool((lp <= 0).all()) and bool((tops <= 0).all()) and bool((ent >= 0).all())
        assert torch.equal(ids[:, 0].cpu(), at.int()) and torch.equal(lp, tops[:, 0])


def test_more_vectors_than_there_is_room_for():
    # every vector's largest above all before it: each is collected, until there is no room
    for R, V in ((1, 262144), (130, 120000), (400, 100000)):
        x = (torch.arange(V).float() * 1e-4).expand(R, V).contiguous()
        check(x, 32)
    x = torch.arange(120000).flip(0).float().expand(2, -1).contiguous() * 1e-4
    check(x, 32)


def behind(m, what, low):
    """Logits whose first m a mask has set to `low`."""
    return torch.where(torch.arange(what.shape[-1]) < m, torch.tensor(low), what)


# a row in one wide CTA, in middle, narrow and tiny ones, in clusters of both; pieces of less than one batch of vectors, of
# a whole number of periods and of more
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("R,V", [(1, 262144), (3, 129280), (30, 60001), (130, 129280), (200, 70001), (330, 65536), (1300, 16384)])
def test_first_logits_far_below_the_rest(R, V, dtype):
    x = logits(R, R, V, dtype)
    steps = torch.arange(V)
    kinds = [behind(m, 3 * torch.randn(V), low)
             for m in (V // 40, V // 8, V // 4 + 3, V // 2, V - 700) for low in (-torch.inf, LOWEST[dtype], -1e9, -1e4, -999.0, -30.0)]
    kinds += [
        behind(V // 4, torch.full((V,), 2.5), -torch.inf),              # as many equal ones as there are
        behind(V // 4, torch.full((V,), 2.5), -30.0),
        behind(V // 4, (steps % 97).float(), -30.0),
        behind(V // 3, steps * 1e-3, -30.0),                            # rising behind the mask
        torch.floor(steps / 4096) + torch.randn(V) * 0.1,               # each stretch above the one before it
        # all of what rises in a few threads' vectors, of either type: few groups have any of it
        torch.where(steps // 8 % 128 == 5, steps * 1e-3, -30.0),
        torch.where(steps // 4 % 512 == 5, steps * 1e-3, -30.0),
        torch.where(steps // 2048 % 2 == 0, steps * 1e-3, -torch.inf),
    ]
    at = np.random.default_rng(V).permutation(max(R, len(kinds)))[:len(kinds)] % R
    for n in (1, 20, 32) if R <= 3 else (32,):
        for part in range(0, len(kinds), max(1, R // 2)):               # some beside rows that are ordinary
            y = x[:min(R, 40)].clone()
            for r, k in zip(at[part:], kinds[part:part + max(1, R // 2)]):
                y[r % len(y)] = k.to(dtype)
            check(y if R <= 40 else torch.cat([y] * (R // len(y) + 1))[:R], n, what="kinds from %d " % part)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("R,V", [(1, 262144), (130, 129280), (330, 65536), (1300, 16384)])
def test_what_is_no_number_in_a_row_that_is_collected_again(R, V, dtype):
    steps = torch.arange(V) * 1e-3
    kinds = [behind(V // 4, 3 * torch.randn(V), -30.0), steps]
    x = logits(3, R, V, dtype)
    t = torch.zeros(R, dtype=torch.int32, device="cuda")
    bad = []
    for k, (kind, what, at) in enumerate((kind, what, at) for kind in kinds for what in (torch.nan, torch.inf)
                                         for at in (0, V // 4 + 1, V - 1)):
        r = (7 * k) % R
        x[r] = kind.to(dtype)
        x[r, at] = what
        bad.append(r)
        got = api.spec_logprobs(x.cuda(), t, 32)
        rows = sorted(set(bad))
        assert bool(torch.isnan(got[0][rows]).all()) and bool(torch.isnan(got[1][rows]).all())
        assert bool((got[2][rows] == -1).all()) and bool(torch.isnan(got[3][rows]).all())
        if R > len(rows):
            well = [r for r in range(R) if r not in rows]
            assert bool(torch.isfinite(got[3][well]).all()) and bool(torch.isfinite(got[1][well]).all())


def test_first_logits_far_below_the_rest_cost_no_more_than_a_second_look():
    def us(x, n):
        t = torch.zeros(x.shape[0], dtype=torch.int32, device="cuda")
        outs = api.spec_logprobs(x, t, n)
        times = []
        for _ in range(7):
            torch.cuda.synchronize()
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            for _ in range(20):
                api.spec_logprobs(x, t, n, *outs)
            b.record()
            b.synchronize()
            times.append(a.elapsed_time(b) / 20 * 1e3)
        return min(times)

    for R, V, dtype, n in ((128, 129280, torch.bfloat16, 20), (400, 50000, torch.bfloat16, 32), (1000, 100277, torch.float32, 5)):
        x = logits(R, 1, V, dtype).cuda().expand(R, V).contiguous()
        ordinary = us(x, n)
        for low in (-torch.inf, -1e9, -30.0):
            x[:, :V // 4] = low
            # read once or twice more, without sums; a pass for each of the n largest took 7 to 22 times as long
            assert us(x, n) < 4 * ordinary, (R, V, low)
    # fewer allowed than are asked for: those that are not take no ranking of hundreds (9 times as long)
    x = logits(1, 100, 9001, torch.bfloat16).cuda()
    ordinary = us(x, 20)
    for low in (-torch.inf, LOWEST[torch.bfloat16]):
        assert us(torch.where(torch.arange(9001, device="cuda") % 900 == 7, x, low), 20) < 3 * ordinary, low


def test_the_largest_in_one_place():
    # the n largest side by side, in one thread's vectors, at the ends, in the elements outside vectors
    for V in (129283, 4099):
        x = torch.randn((6, V), generator=torch.Generator().manual_seed(3))
        for r, at in enumerate((0, V - 40, 8 * 256, V // 2, 5, V - 33)):
            x[r, at:at + 33] = 10 + torch.randperm(33).float() / 8
        for dtype in TYPES:
            check(x.to(dtype), 32)


@pytest.mark.parametrize("dtype", TYPES)
def test_tokens(dtype):
    x = logits(4, 4, 1000, dtype)
    lp = check(x, 3, np.array([-1, 0, 999, -1]))[0]
    assert float(lp[0]) == 0 and float(lp[3]) == 0
    got = api.spec_logprobs(x.cuda(), torch.tensor([0, 1000, -2, 5], dtype=torch.int32, device="cuda"), 0)
    assert api.get_device_error() == 7
    assert torch.isnan(got[0]).tolist() == [False, True, True, False] and bool(torch.isfinite(got[1]).all())
    x3 = x.view(2, 2, 1000)
    got = api.spec_logprobs(x3.cuda(), torch.zeros((2, 2), dtype=torch.int32, device="cuda"), 4)
    assert [tuple(t.shape) for t in got] == [(2, 2), (2, 2), (2, 2, 4), (2, 2, 4)]


def test_committed_tokens_add_up():
    B, K, V = 5, 3, 5000
    x = logits(6, B * (K + 1), V, torch.bfloat16).view(B, K + 1, V).cuda()
    drafts = x[:, :K].argmax(-1).to(torch.int32)
    drafts[1, 1] = (drafts[1, 1] + 1) % V
    drafts[4, 0] = (drafts[4, 0] + 1) % V
    alen, comm = api.spec_verify_accept(x, drafts.contiguous(), api.spec_verify_workspace(B, K, V))
    assert alen.tolist() == [3, 1, 3, 3, 0]
    lp, _, ids, tops = api.spec_logprobs(x, comm, 1)
    want = torch.log_softmax(x.double(), -1).amax(-1)
    live = torch.arange(K + 1, device="cuda")[None] <= alen[:, None]
    assert bool((ids[..., 0][live] == comm[live]).all()) and torch.equal(tops[..., 0][live], lp[live])
    torch.testing.assert_close(lp.double(), torch.where(live, want, 0), rtol=0, atol=2e-5)
    assert bool((lp[~live] == 0).all())


def test_the_same_twice_and_at_once_and_replayed():
    x = logits(7, 128, 129280, torch.bfloat16).cuda()
    t = torch.arange(128, dtype=torch.int32, device="cuda")
    ref = api.spec_logprobs(x, t, 20)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        a = api.spec_logprobs(x, t, 20)
        b = api.spec_logprobs(x, t, 20, stream=s)
        torch.cuda.synchronize()
        for p, q, r in zip(a, b, ref):
            assert torch.equal(p.view(torch.int32), r.view(torch.int32)) and torch.equal(q.view(torch.int32), r.view(torch.int32))
    outs = dict(zip(("logprob", "entropy", "top_ids", "top_logprobs"), [torch.zeros_like(r) for r in ref]))
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            api.spec_logprobs(x, t, 20, **outs)
        for _ in range(2):
            x.copy_(logits(8, 128, 129280, torch.bfloat16))
            g.replay()
            for p, q in zip(outs.values(), api.spec_logprobs(x, t, 20)):
                assert torch.equal(p.view(torch.int32), q.view(torch.int32))
    s.synchronize()


@pytest.mark.parametrize("R,V,dtype", [(1, 262144, torch.bfloat16), (128, 129280, torch.bfloat16), (400, 50000, torch.float32)])
def test_rows_that_are_collected_again_are_the_same_twice_and_at_once_and_replayed(R, V, dtype):
    # which vectors find room first differs from run to run
    x = torch.stack([behind(V // 4, 3 * torch.randn(V), -30.0), torch.arange(V) * 1e-3]).to(dtype)
    x = torch.cat([x] * ((R + 1) // 2))[:R].cuda()
    t = torch.arange(R, dtype=torch.int32, device="cuda")
    ref = api.spec_logprobs(x, t, 32)
    same = lambda got: all(torch.equal(p.view(torch.int32), r.view(torch.int32)) for p, r in zip(got, ref))
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(8):
        a, b = api.spec_logprobs(x, t, 32), api.spec_logprobs(x, t, 32, stream=s)
        torch.cuda.synchronize()
        assert same(a) and same(b)
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            outs = [api.spec_logprobs(x, t, 32) for _ in range(3)]
        for _ in range(4):
            g.replay()
    s.synchronize()
    assert all(same(o) for o in outs)


def test_places_past_32_bits():
    R, V = 17000, 129280
    x = torch.empty((R, V), dtype=torch.bfloat16, device="cuda").fill_(-5.0)
    last = logits(9, 3, V, torch.bfloat16)
    x[-3:] = last.cuda()
    t = torch.full((R,), 17, dtype=torch.int32, device="cuda")
    got = api.spec_logprobs(x, t, 4)
    want = api.spec_logprobs(last.cuda(), t[-3:].clone(), 4)
    assert torch.equal(got[2][-3:], want[2])
    assert torch.allclose(got[0][-3:], want[0], rtol=0, atol=1e-4) and torch.allclose(got[3][-3:], want[3], rtol=0, atol=1e-4)
    assert bool((got[2][:-3] == torch.arange(4, dtype=torch.int32, device="cuda")).all())
    assert torch.allclose(got[1][:-3], torch.full_like(got[1][:-3], float(np.log(V))), rtol=0, atol=1e-4)


def test_refusals():
    x = torch.zeros((2, 100), dtype=torch.bfloat16, device="cuda")
    t = torch.zeros(2, dtype=torch.int32, device="cuda")
    for bad in (x.half(), x.cpu(), x.t(), x[:, :50]):
        with pytest.raises(ValueError):
            api.spec_logprobs(bad, t, 3)
    for bad in (t.long(), t[:1], t.cpu()):
        with pytest.raises(ValueError):
            api.spec_logprobs(x, bad, 3)
    with pytest.raises(api._ffi.LsvError):
        api.spec_logprobs(x, t, 33)
    with pytest.raises(ValueError):
        api.spec_logprobs(x, t, 3, top_ids=torch.zeros((2, 4), dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        api.spec_logprobs(x, t, 3, entropy=torch.zeros(2, dtype=torch.float64, device="cuda"))
    got = api.spec_logprobs(x[:0], t[:0], 3)
    assert [tuple(o.shape) for o in got] == [(0,), (0,), (0, 3), (0, 3)]
