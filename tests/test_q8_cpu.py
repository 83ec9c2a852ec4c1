"""The 8-bit path without a GPU: the plain definitions of oracle/q8.py against other formulations, and the calls'
refusals, which are decided on the host."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import q8
from oracle.q4 import bf16_f64


def bits(x):
    return torch.from_numpy(np.asarray(x, np.float32)).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)


def test_the_formats_values_are_torchs():
    b = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(q8.VALUES[:127], b)


def test_nearest_is_torchs_with_every_tie():
    mid = (q8.VALUES[1:127] + q8.VALUES[:126]) / 2
    rs = np.random.default_rng(0)
    q = np.concatenate([mid, -mid, mid * (1 + 2.0 ** -20), mid * (1 - 2.0 ** -20), q8.VALUES[:127], [0.0, -0.0],
                        rs.normal(size=4000) * 2.0 ** rs.integers(-14, 8, 4000)]).clip(-448, 448)
    q = q.astype(np.float32)
    want = torch.from_numpy(q).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(q8.nearest(q.astype(np.float64)), want)


def test_scale_is_the_least_power_of_two():
    for a in (0.0, 1e-40, 448 * 2.0 ** -126, 447.0, 448.0, 448.0001, 449.0, 3.39e38, 1.0, 1.75, 1.7500001):
        s = q8.scale(a)
        assert np.log2(s) == np.round(np.log2(s)) and s >= 2.0 ** -126 and a <= 448 * s
        assert s == 2.0 ** -126 or a > 448 * s / 2
    assert np.isnan(q8.scale(np.inf)) and np.isnan(q8.scale(np.nan))


@pytest.mark.parametrize("R,C,by", [(3, 272, 1), (130, 144, 128), (1, 16, 1), (5, 16, 128)])
def test_quantise_is_within_half_a_step(R, C, by):
    rs = np.random.default_rng(R)
    x = bf16_f64(bits(rs.normal(size=(R, C)) * 2.0 ** rs.integers(-9, 9, (R, 1))))
    c, s = q8.quantise(x, by)
    assert s.shape == (-(-R // by), -(-C // 128))
    v, each = q8.value(c, s), q8.spread(s, R, C)
    # half a step: 2^-4 of the value's power of two, 2^-10 of the scale at least
    assert np.all(np.abs(v - x) <= np.maximum(np.abs(x) * 2.0 ** -4, each * 2.0 ** -10))


def test_logprobs_of_distributions_that_are_known():
    lp, ent, ids, tops = q8.logprobs(np.zeros((1, 8)), np.array([3]), 2)
    assert abs(lp[0] + np.log(8)) < 1e-15 and abs(ent[0] - np.log(8)) < 1e-15 and ids[0].tolist() == [0, 1]
    x = np.log(np.array([[0.5, 0.25, 0.125, 0.125, 0.0]]) + 0.0, where=np.array([[1, 1, 1, 1, 0]], bool),
               out=np.full((1, 5), -np.inf))
    lp, ent, ids, tops = q8.logprobs(x, np.array([4]), 7)
    assert lp[0] == -np.inf and abs(ent[0] - 1.75 * np.log(2)) < 1e-15
    assert ids[0].tolist() == [0, 1, 2, 3, 4, -1, -1] and tops[0, 4] == -np.inf
    rs = np.random.default_rng(1)
    x = rs.normal(size=(6, 300)) * 4
    lp, ent, ids, tops = q8.logprobs(x, np.arange(6), 5)
    want = torch.log_softmax(torch.from_numpy(x), -1)
    np.testing.assert_allclose(lp, want[torch.arange(6), torch.arange(6)].numpy(), rtol=0, atol=1e-13)
    np.testing.assert_allclose(ent, torch.distributions.Categorical(logits=torch.from_numpy(x)).entropy().numpy(), rtol=1e-12)
    np.testing.assert_array_equal(ids, torch.topk(want, 5).indices.numpy())


def test_the_product_is_the_sum_of_scaled_groups():
    rs = np.random.default_rng(2)
    xc, wc = rs.integers(0, 127, (3, 144)).astype(np.uint8), rs.integers(0, 127, (130, 144)).astype(np.uint8)
    xs, ws = rs.random((3, 2)), rs.random((2, 2))
    y, size = q8.matmul(xc, xs, wc, ws)
    for m, n in ((0, 0), (2, 127), (1, 128), (2, 129)):
        want = sum(xs[m, g] * ws[n // 128, g] * sum(q8.VALUES[xc[m, k]] * q8.VALUES[wc[n, k]]
                                                  for k in range(128 * g, min(144, 128 * g + 128))) for g in (0, 1))
        assert abs(y[m, n] - want) < 1e-12 * abs(want) and size[m, n] >= abs(want) * (1 - 1e-12)


@pytest.fixture(scope="module")
def lib():
    from lossless_speculative_verification_gb300 import _build, _ffi
    _build.build()
    return _ffi.load()


def test_refusals(lib):
    p, odd = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10008)
    for f in (lib.quantize_q8_rows, lib.quantize_q8_weight):
        assert f(p, 4, 24, p, p, None) == 2                     # columns not a multiple of 16
        assert f(p, 4, 16400, p, p, None) == 2
        assert f(p, -1, 128, p, p, None) == 1
        assert f(p, 4, 0, p, p, None) == 1
        assert f(None, 4, 128, p, p, None) == 1
        assert f(p, 4, 128, p, None, None) == 1
        assert f(odd, 4, 128, p, p, None) == 3
        assert f(p, 4, 128, odd, p, None) == 3
        assert f(p, 2 ** 31 - 1, 16384, p, p, None) == 2        # 2^45 values
        assert f(p, 2 ** 26 + 1, 16, p, p, None) == 2
        assert f(None, 0, 128, None, None, None) == 0
    assert lib.dequantize_q8(p, p, 4, 128, 2, p, None) == 1     # rows of a scale: 1 or 128
    assert lib.dequantize_q8(p, p, 4, 100, 1, p, None) == 2
    assert lib.dequantize_q8(p, odd, 4, 128, 1, p, None) == 3
    assert lib.dequantize_q8(None, None, 0, 128, 128, None, None) == 0
    norm = lib.rmsnorm_residual_q8
    assert norm(p, p, None, None, p, p, 4, 128, 1e-6, None) == 1   # a residual wants somewhere to go
    assert norm(p, p, None, p, p, p, 4, 128, -1.0, None) == 1
    assert norm(p, p, None, p, p, p, 4, 128, float("nan"), None) == 1
    assert norm(p, p, None, p, p, p, 4, 120, 1e-6, None) == 2
    assert norm(p, p, odd, p, p, p, 4, 128, 1e-6, None) == 3
    assert norm(None, None, None, None, None, None, 0, 128, 1e-6, None) == 0
    mm = lib.dense_matmul_q8
    assert mm(p, p, p, p, p, 4, 8, 100, None) == 2
    assert mm(p, p, p, p, p, 4, 8, 16400, None) == 2
    assert mm(p, p, p, p, p, 4, -1, 128, None) == 1
    assert mm(p, p, p, p, p, 4, 8, 0, None) == 1
    assert mm(p, None, p, p, p, 4, 8, 128, None) == 1
    assert mm(p, p, odd, p, p, 4, 8, 128, None) == 3
    assert mm(p, p, p, p, p, 2 ** 31 - 1, 2 ** 31 - 1, 128, None) == 2
    assert mm(p, p, p, p, p, 2 ** 31 - 1, 1, 16, None) == 2
    assert mm(p, p, p, p, p, 1, 2 ** 31 - 1, 16, None) == 2
    assert mm(None, None, None, None, None, 0, 8, 128, None) == 0
    assert mm(None, None, None, None, None, 4, 0, 128, None) == 0
    lp = lib.spec_logprobs
    assert lp(p, 0, p, 4, 100, 33, p, p, p, p, None) == 2
    assert lp(p, 0, p, 4, 2 ** 30 + 1, 3, p, p, p, p, None) == 2
    assert lp(p, 0, p, 4, 0, 3, p, p, p, p, None) == 1
    assert lp(p, 0, p, 4, 100, -1, p, p, p, p, None) == 1
    assert lp(p, 0, None, 4, 100, 3, p, p, p, p, None) == 1     # log probabilities of which tokens?
    assert lp(p, 0, p, 4, 100, 3, p, p, None, p, None) == 1
    assert lp(odd, 0, p, 4, 100, 3, p, p, p, p, None) == 3
    assert lp(p, 1, p, 4, 100, 3, p, odd, p, p, None) == 3
    assert lp(None, 0, None, 0, 100, 3, None, None, None, None, None) == 0
