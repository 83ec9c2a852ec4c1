"""The speculative loop with 8-bit projections and output layer (Decoder(weights="q8")): the committed stream equals plain
greedy decoding with the same weights, token for token, over both caches (a row's products do not depend on the rows
beside it); and the log probabilities that a pass adds."""
import ctypes

import numpy as np
import pytest
import torch

from lossless_speculative_verification_gb300 import api, synth
from lossless_speculative_verification_gb300.decoder import Decoder

from gpu_util import need_gpu
import test_gpu_q4_loop as q4loop
import test_gpu_spec_loop as loop

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()
    yield
    torch.cuda.synchronize()
    assert api.get_device_error() == 0


def problem(seed, out_scale):
    dims = synth.MoeDims(0, 256, 8, 2, 1, 128)
    return synth.decoder_problem(2, dims, V=2048, nh=2, I_draft=256, seed=seed, out_scale=out_scale, mimic_draft=True)


@pytest.mark.parametrize("seed", [0, 1])
def test_speculative_loop_commits_the_greedy_sequence(seed):
    seen = set()
    for out_scale in (0.05, 0.6):
        prob = problem(seed, out_scale)
        dec = Decoder(prob, loop.B, L=loop.P + 4 * loop.N_NEW + 32, weights="q8")
        prompt = torch.from_numpy(np.random.default_rng(seed + 7).integers(0, prob.V, (loop.B, loop.P)).astype(np.int32)).cuda()
        ref = loop.greedy(dec, prompt)
        for K in (1, 2, 3):
            got, lengths = loop.speculative(dec, prompt, K)
            np.testing.assert_array_equal(got, ref, err_msg="K=%d, out_scale %g" % (K, out_scale))
            seen |= {(K, int(n)) for n in lengths}
    assert (3, 3) in seen and any(n < K for K, n in seen), sorted(seen)


def test_passes_over_pages_and_contiguous_caches():
    # one token at a time and four, over 4-bit pages
    prob = problem(2, 0.3)
    B, L, n = 3, 64, 12
    tokens = torch.from_numpy(np.random.default_rng(3).integers(0, prob.V, (B, n)).astype(np.int32)).cuda()
    none = torch.zeros((B, 0), dtype=torch.int32, device="cuda")
    seen = []
    for Q in (1, 4):
        dec = Decoder(prob, B, L, cache="q4", page=16, weights="q8")
        rows = []
        for i in range(0, n, Q):
            dec.reserve(q4loop.i32([i] * B), q4loop.i32([i + Q] * B))
            part = tokens[:, i:i + Q].contiguous()
            b = dec.verify(part, q4loop.i32([i + Q] * B), part[:, 1:].contiguous() if Q > 1 else none)
            rows.append(b["argmax"].clone())
        seen.append(torch.cat(rows, 1))
    assert torch.equal(*seen)


def test_passes_of_many_rows():
    # projections whose K is split over CTAs, two shares a CTA where there are more than 128 rows: a pass of two positions
    # of 96 sequences gives what two of one position give
    dims = synth.MoeDims(0, 2560, 8, 2, 1, 128)
    prob = synth.decoder_problem(1, dims, V=2048, nh=20, I_draft=256, seed=10, out_scale=0.3)
    B, Q = 96, 2
    tokens = torch.from_numpy(np.random.default_rng(11).integers(0, prob.V, (B, Q)).astype(np.int32)).cuda()
    none = torch.zeros((B, 0), dtype=torch.int32, device="cuda")
    at = lambda n: torch.full((B,), n, dtype=torch.int32, device="cuda")
    one, two = (Decoder(prob, B, 16, weights="q8") for _ in range(2))
    b = two.verify(tokens, at(Q), tokens[:, 1:].contiguous())
    for i in range(Q):
        a = one.verify(tokens[:, i:i + 1].contiguous(), at(i + 1), none)
        for n in ("q", "k", "v", "o"):
            assert torch.equal(a[n].view(B, -1), b[n].view(B, Q, -1)[:, i]), n
        assert torch.equal(a["logits"][:, 0], b["logits"][:, i])
        assert torch.equal(a["argmax"][:, 0], b["argmax"][:, i])


@pytest.mark.parametrize("weights", ["bf16", "q8"])
def test_log_probabilities_of_a_pass(weights):
    prob = problem(4, 0.6)
    B, Q, n = 4, 4, 6
    dec = Decoder(prob, B, 64, weights=weights)
    tokens = torch.from_numpy(np.random.default_rng(5).integers(0, prob.V, (B, Q)).astype(np.int32)).cuda()
    after = torch.full((B,), Q, dtype=torch.int32, device="cuda")
    drafts = tokens[:, 1:].contiguous()
    plain = {k: v.clone() for k, v in dec.verify(tokens, after, drafts).items() if k in ("argmax", "alen", "comm")}
    b = dec.verify(tokens, after, drafts, logprobs=n)
    for k, v in plain.items():
        assert torch.equal(b[k], v)
    logp = torch.log_softmax(b["logits"].double(), -1)
    live = b["comm"] >= 0
    want = torch.gather(logp, 2, b["comm"].clamp(min=0).long()[..., None])[..., 0]
    # of the logits that are rounded to bf16: the numbers to fp32's roundings
    torch.testing.assert_close(b["logprob"].double(), torch.where(live, want, 0), rtol=0, atol=2e-5)
    torch.testing.assert_close(b["entropy"].double(), -(logp.exp() * logp).sum(-1), rtol=0, atol=5e-5)
    top = torch.gather(logp, 2, b["top_ids"].long())
    torch.testing.assert_close(b["top_logprobs"].double(), top, rtol=0, atol=2e-5)
    assert b["top_ids"].shape == (B, Q, n)
    if weights == "q8":
        assert torch.equal(b["top_ids"][..., 0], b["argmax"])
        # the norm and the product in 8 bits, as an output layer does them: the pass's logits are the calls'
        h = api.rmsnorm_residual_q8(b["x"])
        again = api.dense_matmul_q8(*h, *dec.vocab_q8).view(B, Q, -1)
        assert torch.equal(again, b["logits"])
    first = {k: b[k].data_ptr() for k in ("logprob", "top_ids")}
    again = dec.verify(tokens, after, drafts, logprobs=n)
    assert {k: again[k].data_ptr() for k in first} == first         # a pass's buffers are kept
    assert dec.verify(tokens, after, drafts, logprobs=0)["top_ids"].shape == (B, Q, 0)


@pytest.mark.parametrize("weights", ["bf16", "q8"])
def test_a_pass_returns_its_own_numbers_alone(weights):
    prob = problem(8, 0.6)
    B, Q = 2, 3
    dec = Decoder(prob, B, 64, weights=weights)
    rs = np.random.default_rng(9)
    tokens = [torch.from_numpy(rs.integers(0, prob.V, (B, Q)).astype(np.int32)).cuda() for _ in range(2)]
    after = torch.full((B,), Q, dtype=torch.int32, device="cuda")
    keys = {"logprob", "entropy", "top_ids", "top_logprobs"}
    before = set(dec.verify(tokens[0], after, tokens[0][:, 1:].contiguous()))
    assert not keys & before
    first = dec.verify(tokens[0], after, tokens[0][:, 1:].contiguous(), logprobs=4)
    assert keys | {"logits"} <= set(first)
    # a pass without them returns none, of an earlier pass's neither, nor the earlier pass's logits
    assert set(dec.verify(tokens[1], after, tokens[1][:, 1:].contiguous())) == before
    # and what the earlier pass returned still has its own, of its n
    other = dec.verify(tokens[1], after, tokens[1][:, 1:].contiguous(), logprobs=2)
    assert first["top_ids"].shape == (B, Q, 4) and other["top_ids"].shape == (B, Q, 2)


@pytest.mark.parametrize("weights", ["bf16", "q8"])
@pytest.mark.parametrize("B,Q", [(2, 3), (1, 1)])
def test_launches_of_a_pass(weights, B, Q):
    # the kernels of a captured pass, which has nothing else in it, are as many as the decoder says
    dec = Decoder(problem(12, 0.3), B, 64, weights=weights)
    tokens = torch.zeros((B, Q), dtype=torch.int32, device="cuda")
    after = torch.full((B,), Q, dtype=torch.int32, device="cuda")
    drafts = torch.zeros((B, Q - 1), dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        dec.verify(tokens, after, drafts)
        g = torch.cuda.CUDAGraph(keep_graph=True)
        with torch.cuda.graph(g, stream=s):
            dec.verify(tokens, after, drafts)
    n = ctypes.c_size_t(0)
    runtime = ctypes.CDLL("libcudart.so.13")
    assert runtime.cudaGraphGetNodes(ctypes.c_void_p(g.raw_cuda_graph()), None, ctypes.byref(n)) == 0
    assert n.value == dec.launches_per_verify(B, Q)
    s.synchronize()


def test_a_pass_replayed():
    prob = problem(6, 0.6)
    dec = Decoder(prob, 2, 64, weights="q8")
    tokens = torch.zeros((2, 3), dtype=torch.int32, device="cuda")
    after = torch.full((2,), 3, dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()
    rs = np.random.default_rng(7)
    with torch.cuda.stream(s):
        dec.verify(tokens, after, tokens[:, 1:].contiguous(), logprobs=3)
        drafts = torch.zeros((2, 2), dtype=torch.int32, device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            b = dec.verify(tokens, after, drafts, logprobs=3)
        for _ in range(2):
            tokens.copy_(torch.from_numpy(rs.integers(0, prob.V, (2, 3)).astype(np.int32)))
            drafts.copy_(tokens[:, 1:])
            g.replay()
            got = {k: b[k].clone() for k in ("argmax", "comm", "logprob", "entropy", "top_ids", "top_logprobs")}
            want = dec.verify(tokens, after, drafts, logprobs=3)
            for k, v in got.items():
                assert torch.equal(v, want[k]), k
    s.synchronize()


def test_refusals():
    with pytest.raises(ValueError):
        Decoder(problem(0, 0.5), 1, 16, weights="fp8")
