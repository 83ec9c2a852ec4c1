"""The 8-bit path on the GPU (quantize_q8_rows, quantize_q8_weight, dequantize_q8, rmsnorm_residual_q8,
dense_matmul_q8) against oracle/q8.py in 64 bits.

Codes and scales of what is quantised as it stands are exact: bytes are compared.  Behind the norm a value h is off by
its roundings, 2^-24 each: at most 24 additions of a row's squares, whose root counts half, the division and the root,
two for the product with the correction and one for the gain: 2^-20 |h| bounds them.  A code then lies between those of
h (1 - 2^-20) and h (1 + 2^-20), and the scale is one of theirs.

Products, element by element, with A the sum of the terms' sizes: the output's rounding to bf16 2^-8 |y|; a group's
products are added in four steps of 32 to fp32 accumulators, each step off by at most 2^-23 of what the accumulator
holds and 32 * 2^-25 of its largest product: 4 (2^-23 + 2^-20) A < 2^-17 A; the groups' sums by an FMA a group and the
product of the two scales: (G + 8) 2^-24 A.
"""
import numpy as np
import pytest
import torch

from oracle import q4, q8
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


def host(t):
    """Codes as bytes, scales and values as float64."""
    if t.dtype == torch.float8_e4m3fn:
        return t.view(torch.uint8).cpu().numpy()
    return t.float().cpu().numpy().astype(np.float64)


def same_but_nan(got, want):
    """Bytes of groups whose scale is a number, and scales."""
    (gc, gs), (wc, ws) = got, want
    np.testing.assert_array_equal(gs, ws)
    live = np.isfinite(q8.spread(ws, *wc.shape))
    np.testing.assert_array_equal(np.where(live, gc, 0), np.where(live, wc, 0))


def rows(seed, R, C):
    rs = np.random.default_rng(seed)
    return bits(rs.normal(size=(R, C)) * 2.0 ** rs.integers(-12, 12, (R, 1)) * np.where(rs.random(C) < 0.02, 50, 1))


SHAPES = [(1, 16), (3, 128), (5, 144), (2, 1280), (129, 272), (130, 1296), (4, 2064), (2, 16384), (257, 16)]


# ---------------------------------------------------------------------------------------------- quantising, back
@pytest.mark.parametrize("R,C", SHAPES)
def test_quantised_bytes(R, C):
    x = rows(R + C, R, C)
    for f, by in ((api.quantize_q8_rows, 1), (api.quantize_q8_weight, 128)):
        c, s = f(dev(x))
        want = q8.quantise(q4.bf16_f64(x), by)
        same_but_nan((host(c), host(s)), want)
        # values of four bits times a power of two are exact in bf16
        np.testing.assert_array_equal(host(api.dequantize_q8(c, s)), q8.value(*want))


def test_every_significand_and_tie_and_end():
    # all 8-bit significands, against all others as a group's largest, over the format's whole range and below
    m = np.arange(128, 256)
    x = np.zeros((128 * 3, 128), np.float32)
    for j in range(3):
        x[128 * j:128 * j + 128] = m[None, :] * np.where(m % 2, -1, 1)[None, :] * 2.0 ** (-8 * j)
        x[128 * j:128 * j + 128, 0] = m * 2.0 ** (1 + j)
    x = np.concatenate([x, x * 2.0 ** -130, x * 2.0 ** 100])        # (the smallest become subnormal, or nothing)
    b = bits(x)
    c, s = api.quantize_q8_rows(dev(b))
    same_but_nan((host(c), host(s)), q8.quantise(q4.bf16_f64(b)))


def test_what_is_no_number_and_what_is_nothing():
    x = np.ones((6, 272), np.float32)
    x[0] = 0
    x[1, 3], x[1, 271] = np.nan, np.inf
    x[2, 130] = -np.inf
    x[3, :128] = 3.3895e38
    x[4, :128] = 1e-40
    x[5, 256:] = -0.0
    b = bits(x)
    c, s = api.quantize_q8_rows(dev(b))
    same_but_nan((host(c), host(s)), q8.quantise(q4.bf16_f64(b)))
    v = host(api.dequantize_q8(c, s))
    assert np.isnan(v[1, :128]).all() and np.isnan(v[1, 256:]).all() and (v[1, 128:256] == 1).all()
    assert np.isnan(v[2, 128:256]).all() and (v[2, :128] == 1).all()
    c, s = api.quantize_q8_weight(dev(b))
    assert np.isnan(host(s)).tolist() == [[True, True, True]]
    assert np.isnan(host(api.dequantize_q8(c, s))).all()
    # a NaN in a row, or in a block, and nowhere else
    y = host(api.dense_matmul_q8(*api.quantize_q8_rows(dev(b)), *api.quantize_q8_weight(dev(bits(np.ones((5, 272)))))))
    assert np.isnan(y).all(1).tolist() == [False, True, True, False, False, False] and not np.isnan(y[[0, 3, 4, 5]]).any()


@pytest.mark.parametrize("R,C,by", [(3, 144, 1), (130, 400, 128), (1, 16, 1), (300, 8192, 128)])
def test_read_back_of_any_scales(R, C, by):
    rs = np.random.default_rng(R)
    c = rs.integers(0, 256, (R, C)).astype(np.uint8)
    c[(c & 127) == 127] = 0
    s = rs.integers(1, 1 << 16, (-(-R // by), -(-C // 128))).astype(np.float32) * np.float32(2.0 ** -13)   # 16 bits: exact products
    got = api.dequantize_q8(torch.from_numpy(c).cuda().view(torch.float8_e4m3fn), torch.from_numpy(s).cuda())
    np.testing.assert_array_equal(host(got), q4.bf16_f64(q4.bf16_round(q8.value(c, s))))


# ---------------------------------------------------------------------------------------------- the norm
def check_norm(x, y, gain, eps=1e-6, in_place=False):
    want, h = q8.rmsnorm(x, y, gain, eps)
    xd = dev(x)
    out = xd if in_place or y is None else torch.empty_like(xd)
    c, s = api.rmsnorm_residual_q8(xd, None if y is None else dev(y), gain=None if gain is None else dev(gain),
                                   x_out=None if in_place else out, eps=eps)
    np.testing.assert_array_equal(host(out), q4.bf16_f64(want))
    if not in_place:
        np.testing.assert_array_equal(host(xd), q4.bf16_f64(x))          # the input stays
    c, s = host(c), host(s)
    v = q8.value(c, s)
    lo, hi = h - np.abs(h) * 2.0 ** -20, h + np.abs(h) * 2.0 ** -20
    R, C = h.shape
    for g in range(s.shape[1]):
        at = np.s_[:, 128 * g:128 * g + 128]
        small, large = (np.array([q8.scale(a) for a in np.abs(h[at]).max(1) * (1 + e * 2.0 ** -20)]) for e in (-1, 1))
        assert ((s[:, g] == small) | (s[:, g] == large)).all()
        each = s[:, g:g + 1]
        ends = [np.where(np.signbit(q), -1, 1) * q8.VALUES[q8.nearest(q) & 127] * each for q in (lo[at] / each, hi[at] / each)]
        assert ((v[at] >= ends[0]) & (v[at] <= ends[1])).all()


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("res,gain", [(False, False), (True, True)])
def test_norm(T, H, res, gain):
    rs = np.random.default_rng(T * H)
    check_norm(rows(T, T, H), rows(T + 1, T, H) if res else None, bits(1 + rs.normal(size=H)) if gain else None)


def test_norm_in_place_and_of_nothing():
    check_norm(rows(1, 7, 400), rows(2, 7, 400), None, in_place=True)
    check_norm(np.zeros((3, 272), np.uint16), np.zeros((3, 272), np.uint16), None, eps=1e-3)    # rows of zeros
    check_norm(rows(3, 5, 144), None, None, eps=0.0)
    x = rows(4, 2, 272)
    x[1, 7] = 0x7FC0
    c, s = api.rmsnorm_residual_q8(dev(x))
    assert np.isfinite(host(s)[0]).all() and np.isnan(host(s)[1]).all()     # a NaN takes its row, and no other


# ---------------------------------------------------------------------------------------------- products
def operands(seed, M, N, K, scales="any"):
    """Codes of all sizes, scales that are no powers of two."""
    rs = np.random.default_rng(seed)

    def codes(R):
        c = q8.nearest(rs.normal(size=(R, K)) * 2.0 ** rs.integers(-6, 7, (R, 1)))
        return c

    def some(R):
        s = (0.5 + rs.random((R, -(-K // 128)))) * 2.0 ** rs.integers(-9, 9, (R, 1))
        return (s if scales == "any" else 2.0 ** np.round(np.log2(s))).astype(np.float32)

    return codes(M), some(M), codes(N), some(-(-N // 128))


def cuda(xc, xs, wc, ws):
    e4m3 = lambda c: torch.from_numpy(c).cuda().view(torch.float8_e4m3fn)
    return e4m3(xc), torch.from_numpy(xs).cuda(), e4m3(wc), torch.from_numpy(ws).cuda()


def check_product(ops, got, what=""):
    ref, A = q8.matmul(*ops)
    G = ops[1].shape[1]
    tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -17 + (G + 8) * 2.0 ** -24) * A
    bad = ~(np.abs(host(got) - ref) <= tol)
    assert not bad.any(), "%s: %d of %d off, worst %.3g of its tolerance" % (
        what, bad.sum(), bad.size, np.nanmax(np.abs(host(got) - ref) / tol))


@pytest.mark.parametrize("M", [1, 7, 8, 31, 33, 127, 128, 129, 200, 257])
@pytest.mark.parametrize("N,K", [(1, 16), (8, 128), (127, 144), (128, 1280), (129, 272), (200, 2064), (1001, 400)])
def test_products(M, N, K):
    ops = operands(M * N + K, M, N, K)
    check_product(ops, api.dense_matmul_q8(*cuda(*ops)), "%d x %d x %d" % (M, N, K))


# the forms: a cluster for a tile's groups (1, 2, 4, 8 CTAs), persistent CTAs, pairs of CTAs; rows of y that TMA takes
# and others
@pytest.mark.parametrize("M,N,K", [
    (5, 19500, 128), (100, 9000, 400), (64, 5000, 640), (3, 130, 16384), (128, 2048, 4112),
    (130, 10000, 400), (4000, 300, 272), (512, 9728, 144), (700, 9729, 400), (2049, 4104, 272), (2560, 2048, 1296),
    (257, 19456, 16), (300, 40000, 128), (5, 1001, 3088), (128, 1280, 7168), (300, 2304, 2576), (300, 2301, 2576),
    (500, 1100, 1552), (300, 40000, 144), (600, 13000, 400), (600, 13001, 1680), (640, 13000, 1680),
])
def test_products_of_every_form(M, N, K):
    ops = operands(N, M, N, K)
    check_product(ops, api.dense_matmul_q8(*cuda(*ops)), "%d x %d x %d" % (M, N, K))


def test_products_write_their_rows_alone():
    for M, N, K in ((3, 13, 144), (129, 264, 272), (2050, 2056, 144)):
        ops = operands(1, M, N, K)
        room = torch.full((M * N + 4096,), 7.0, dtype=torch.bfloat16, device="cuda")
        got = api.dense_matmul_q8(*cuda(*ops), out=room[2048:2048 + M * N].view(M, N))
        check_product(ops, got)
        assert bool((room[:2048] == 7).all()) and bool((room[2048 + M * N:] == 7).all())


# rows of every alignment, out of persistent CTAs, of pairs and of a split's CTAs; the values beside them stay
@pytest.mark.parametrize("M,N,K", [(100, 19456, 144), (600, 9728, 144), (77, 1000, 1296), (77, 1000, 1552), (4000, 16, 144)])
def test_rows_that_begin_anywhere(M, N, K):
    for more in (1, 2, 3, 4, 5, 6, 7):
        ops = operands(more, M, N + more, K)
        room = torch.full((M * (N + more) + 4096,), 7.0, dtype=torch.bfloat16, device="cuda")
        got = api.dense_matmul_q8(*cuda(*ops), out=room[2048:2048 + M * (N + more)].view(M, N + more))
        check_product(ops, got, "N %d " % (N + more))
        assert bool((room[:2048] == 7).all()) and bool((room[2048 + M * (N + more):] == 7).all())


@pytest.mark.parametrize("N,K", [(1280, 1280), (1001, 2064), (20000, 400), (130, 7168), (8000, 2576)])
def test_a_rows_bits_do_not_depend_on_the_others(N, K):
    x, xs, w, ws = cuda(*operands(3, 128, N, K))
    whole = api.dense_matmul_q8(x, xs, w, ws)
    for M in (1, 4, 16, 65):
        at = slice(128 - M, 128)
        part = api.dense_matmul_q8(x[at].clone(), xs[at].clone(), w, ws)
        assert torch.equal(part.view(torch.int16), whole[at].view(torch.int16))
    assert torch.equal(api.dense_matmul_q8(x, xs, w, ws).view(torch.int16), whole.view(torch.int16))


# K over eight, four and two CTAs (where clusters of them for two row tiles fit at once and where not), whole, and pairs of
# CTAs; short last groups, weight tiles and rows of y that TMA does not take
@pytest.mark.parametrize("N,K", [(1280, 7168), (1001, 3088), (640, 4096), (2048, 2048), (4096, 4096), (4099, 1552), (2304, 2576),
                                 (5120, 5120), (7168, 2576), (8000, 2000), (12000, 1424), (20000, 2048), (1280, 1280)])
def test_a_rows_bits_do_not_depend_on_the_others_up_to_256(N, K):
    ops = operands(3, 256, N, K)
    x, xs, w, ws = cuda(*ops)
    whole = api.dense_matmul_q8(x, xs, w, ws)
    check_product(ops, whole)
    for M in (1, 65, 128, 129, 160, 200, 255):
        at = slice(256 - M, 256)
        part = api.dense_matmul_q8(x[at].clone(), xs[at].clone(), w, ws)
        assert torch.equal(part.view(torch.int16), whole[at].view(torch.int16)), M


def test_of_codes_and_powers_of_two_small_products_are_exact():
    # whole numbers whose sums fit 24 bits, outputs that fit 8
    rs = np.random.default_rng(5)
    xc, wc = q8.nearest(rs.integers(-2, 3, (70, 272)).astype(float)), q8.nearest(rs.integers(0, 2, (140, 272)).astype(float))
    wc[:, 40:] = 0
    ops = xc, np.full((70, 3), 0.25, np.float32), wc, np.full((2, 3), 4.0, np.float32)
    np.testing.assert_array_equal(host(api.dense_matmul_q8(*cuda(*ops))), q8.matmul(*ops)[0])


# ---------------------------------------------------------------------------------------------- a run of them
def test_quantised_normed_multiplied_and_read_in_a_graph():
    T, H, V = 24, 272, 2000
    rs = np.random.default_rng(8)
    x, y, w = dev(rows(1, T, H)), dev(rows(2, T, H)), dev(bits(rs.normal(size=(V, H)) * 0.1))
    tokens = torch.arange(T, dtype=torch.int32, device="cuda")
    wq = api.quantize_q8_weight(w)

    def run():
        h = api.rmsnorm_residual_q8(x, y, x_out=xo)
        logits = api.dense_matmul_q8(*h, *wq)
        return (*h, logits, *api.spec_logprobs(logits, tokens, 5))

    xo = torch.empty_like(x)
    eager = [t.clone() for t in run()]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            out = run()
        for seed in (1, 11, 12):
            x.copy_(dev(rows(seed, T, H)))
            g.replay()
            got = [t.clone() for t in out]
            want = run()
            for a, b in zip(got, want):
                assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
            if seed == 1:
                for a, b in zip(got, eager):
                    assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    s.synchronize()


# many calls without a wait between them, each of whose CTAs begin as those of the one before end
@pytest.mark.parametrize("M,N,K", [(128, 129280, 1280), (100, 20000, 400), (1, 1280, 1280), (1, 1280, 4096), (200, 4096, 2560), (700, 9728, 1296)])
def test_call_behind_call(M, N, K):
    x, xs, w, ws = cuda(*operands(4, M, N, K))
    want = api.dense_matmul_q8(x, xs, w, ws)
    out = [torch.empty_like(want) for _ in range(3)]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            for i in range(24):
                api.dense_matmul_q8(x, xs, w, ws, out=out[i % 3])
        for _ in range(4):
            g.replay()
    s.synchronize()
    for o in out:
        assert torch.equal(o.view(torch.int16), want.view(torch.int16))


# One CTA a tile, splits over eight and two CTAs, persistent CTAs, and pairs whose last tiles are short.  (On a GB300 a try of a
# wait lasts as long as the load; with tries that return at once the limit ran out in every call, and these held as well.)
@pytest.mark.parametrize("M,N,K", [(5, 1280, 1296), (5, 1280, 3088), (300, 2301, 2576), (1, 129280, 1280), (128, 40000, 656), (700, 9728, 1296), (129, 40001, 400)])
def test_a_product_whose_waits_run_out_says_so_and_the_next_call_is_right(M, N, K):
    ops = cuda(*operands(M + N, M, N, K))
    ref = api.dense_matmul_q8(*ops).view(torch.int16).clone()
    flush = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    try:
        api.set_wait_limit_ns(1)
        for turn in range(4):
            flush.fill_(turn)                                   # the operands come from memory again
            got = api.dense_matmul_q8(*ops)
            err = api.get_device_error()
            assert err in (0, 6)                                # a wait may end before anyone looks at the time
            if err == 0:
                assert torch.equal(got.view(torch.int16), ref)
    finally:
        api.set_wait_limit_ns(2000000000)
    assert torch.equal(api.dense_matmul_q8(*ops).view(torch.int16), ref)


# the same forms, and two shares a CTA (of a split, and whole): a limit far below a load from memory does run out, in every
# one, and the call behind it in the stream is right, as are those after it
@pytest.mark.parametrize("M,N,K", [(5, 1280, 1296), (5, 1280, 3088), (300, 2301, 2576), (1, 129280, 1280), (128, 40000, 656),
                                   (700, 9728, 1296), (129, 40001, 400), (200, 4096, 2560), (256, 5120, 5120), (1, 16, 16)])
def test_a_limit_below_a_load_runs_out(M, N, K):
    ops = cuda(*operands(M + N, M, N, K))
    ref = api.dense_matmul_q8(*ops).view(torch.int16).clone()
    flush = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    seen = []
    try:
        for turn in range(4):
            flush.fill_(turn)
            api.set_wait_limit_ns((1, 100)[turn % 2])
            api.dense_matmul_q8(*ops)
            api.set_wait_limit_ns(2000000000)
            behind = api.dense_matmul_q8(*ops)
            seen.append(api.get_device_error())
            assert torch.equal(behind.view(torch.int16), ref)
    finally:
        api.set_wait_limit_ns(2000000000)
    assert 6 in seen and set(seen) <= {0, 6}, seen
    for _ in range(3):
        assert torch.equal(api.dense_matmul_q8(*ops).view(torch.int16), ref)
    assert api.get_device_error() == 0


def test_two_calls_at_once():
    a, b = (cuda(*operands(k, 128, 30000, 1280)) for k in (1, 2))
    ra, rb = api.dense_matmul_q8(*a), api.dense_matmul_q8(*b)
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        with torch.cuda.stream(s):
            oa = api.dense_matmul_q8(*a)
        ob = api.dense_matmul_q8(*b, stream=t)
        torch.cuda.synchronize()
        assert torch.equal(oa, ra) and torch.equal(ob, rb)


# clusters of both, two shares a CTA and one, beside each other
@pytest.mark.parametrize("M,N,K", [(256, 4096, 4096), (200, 1280, 7168), (256, 5120, 5120), (128, 1280, 7168)])
def test_two_split_calls_at_once(M, N, K):
    a, b = cuda(*operands(1, M, N, K)), cuda(*operands(2, 128, 1280, 4096))
    ra, rb = api.dense_matmul_q8(*a), api.dense_matmul_q8(*b)
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(10):
        with torch.cuda.stream(s):
            oa = [api.dense_matmul_q8(*a) for _ in range(3)]
        ob = [api.dense_matmul_q8(*b, stream=t) for _ in range(3)]
        torch.cuda.synchronize()
        assert all(torch.equal(o.view(torch.int16), ra.view(torch.int16)) for o in oa)
        assert all(torch.equal(o.view(torch.int16), rb.view(torch.int16)) for o in ob)


# ---------------------------------------------------------------------------------------------- large
def test_places_past_32_bits():
    R, C = 140000, 16384                                             # 2.3e9 values
    x = torch.empty((R, C), dtype=torch.bfloat16, device="cuda").fill_(0.5)
    last = rows(6, 3, C)
    x[-3:] = dev(last)
    for f, by in ((api.quantize_q8_rows, 1), (api.quantize_q8_weight, 128)):
        c, s = f(x)
        if by == 1:
            same_but_nan((host(c[-3:]), host(s[-3:])), q8.quantise(q4.bf16_f64(last)))
        v = api.dequantize_q8(c, s)
        assert torch.equal(v[-3:], api.dequantize_q8(c[-3:].clone(), s[-3:].clone() if by == 1 else s[-1:].clone()))
        assert bool((v[1000] == 0.5).all())
        del c, s, v
    del x
    torch.cuda.empty_cache()
    M, N, K = 17000, 129280, 16                                      # 2.2e9 outputs
    ops = operands(7, 300, N, K)
    xc, xs, w, ws = cuda(*ops)
    x, sx = xc.view(torch.uint8).repeat(57, 1)[:M].view(torch.float8_e4m3fn), xs.repeat(57, 1)[:M].contiguous()
    y = api.dense_matmul_q8(x, sx, w, ws)
    at = np.arange(M - 200, M)
    ref, A = q8.matmul(ops[0][at % 300], ops[1][at % 300], *ops[2:])
    assert (np.abs(host(y[M - 200:]) - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -16 * A).all()


# ---------------------------------------------------------------------------------------------- refusals
def test_refusals():
    x = torch.zeros((4, 128), dtype=torch.bfloat16, device="cuda")
    c, s = api.quantize_q8_rows(x)
    w = api.quantize_q8_weight(x)
    assert c.shape == (4, 128) and s.shape == (4, 1) and w[1].shape == (1, 1)
    for bad in (x.float(), x.cpu(), x.t(), x[:, :120], x[0]):
        with pytest.raises((ValueError, api._ffi.LsvError)):
            api.quantize_q8_rows(bad)
        with pytest.raises((ValueError, api._ffi.LsvError)):
            api.rmsnorm_residual_q8(bad)
    with pytest.raises(ValueError):
        api.quantize_q8_rows(x, scales=torch.zeros((4, 2), device="cuda"))
    with pytest.raises(ValueError):
        api.quantize_q8_rows(x, codes=torch.zeros((4, 128), dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        api.rmsnorm_residual_q8(x, x[:2])
    with pytest.raises(ValueError):
        api.rmsnorm_residual_q8(x, gain=x)
    with pytest.raises(ValueError):
        api.rmsnorm_residual_q8(x, x, x_out=x[:2])
    with pytest.raises(ValueError):
        api.dequantize_q8(c, torch.zeros((2, 1), device="cuda"))
    with pytest.raises(ValueError):
        api.dense_matmul_q8(c, s, w[0][:, :64], w[1])
    with pytest.raises(ValueError):
        api.dense_matmul_q8(c, w[1], w[0], w[1])
    with pytest.raises(ValueError):
        api.dense_matmul_q8(c, s, *w, out=x)
    with pytest.raises(ValueError):
        api.dense_matmul_q8(c.view(torch.uint8), s, *w)
    with pytest.raises(api._ffi.LsvError):
        api.dense_matmul_q8(c.flatten()[8:8 + 256].view(2, 128), s[:2].clone(), *w)      # not 16-byte aligned
    for empty in (torch.empty((0, 128), dtype=torch.bfloat16, device="cuda"),):
        ec, es = api.quantize_q8_rows(empty)
        assert api.dense_matmul_q8(ec, es, *w).shape == (0, 4)
        assert api.dequantize_q8(ec, es).shape == (0, 128)
