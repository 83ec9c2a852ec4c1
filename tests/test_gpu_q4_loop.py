"""The speculative loop over the paged 4-bit cache: prompts, forks, drafts, verify passes that append to and read the
pages, rejected drafts given back, compactions in between.  The committed stream must equal plain greedy decoding one
token at a time over the same kind of cache, token for token: a row's attention does not depend on the rows beside
it, so the verifier's greedy token after a prefix is the same in both."""
import numpy as np
import pytest
import torch

from lossless_speculative_verification_gb300 import api, synth
from lossless_speculative_verification_gb300.decoder import Decoder

from gpu_util import need_gpu

pytestmark = pytest.mark.gpu

B, PROMPT, N_NEW, PAGE = 4, 21, 30, 16
L = PROMPT + 4 * N_NEW + 32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()
    yield
    torch.cuda.synchronize()
    assert api.get_device_error() == 0


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()


def decoder(prob, pages=None):
    return Decoder(prob, B, L, cache="q4", page=PAGE, pages=pages)


def step(dec, ctx, tokens, drafts):
    """One verify pass over tokens [B, Q] behind ctx positions; the pages are there for exactly those."""
    after = np.where(ctx < 0, 0, ctx + tokens.shape[1])
    dec.reserve(i32(np.maximum(ctx, 0)), i32(after))
    return dec.verify(tokens, i32(after), drafts)


def prefill(dec, prompt, rows):
    """The prompts of the given rows, seven positions a pass; the other rows are slots without a sequence."""
    on = np.isin(np.arange(B), rows)
    for i in range(0, PROMPT, 7):
        part = prompt[:, i:i + 7].contiguous()
        b = step(dec, np.where(on, i, -1), part, part[:, 1:].contiguous())
    return b["argmax"][:, 6].clone(), b["x"].view(B, 7, dec.H)[:, 6].clone()


def greedy(prob, prompt):
    dec = decoder(prob)
    t, _ = prefill(dec, prompt, range(B))
    out = [t.cpu().numpy()]
    none = torch.zeros((B, 0), dtype=torch.int32, device="cuda")
    for i in range(N_NEW - 1):
        b = step(dec, np.full(B, PROMPT + i), t.view(B, 1).contiguous(), none)
        t = b["argmax"][:, 0].clone()
        out.append(t.cpu().numpy())
    return np.stack(out, 1)


@pytest.mark.parametrize("K", [1, 3])
@pytest.mark.parametrize("out_scale", [0.05, 0.6])
def test_speculative_loop_over_pages_commits_the_greedy_sequence(K, out_scale):
    dims = synth.MoeDims(0, 256, 8, 2, 1, 128)
    prob = synth.decoder_problem(2, dims, V=2048, nh=2, I_draft=256, seed=K, out_scale=out_scale, mimic_draft=True)
    two = np.random.default_rng(K).integers(0, prob.V, size=(2, PROMPT)).astype(np.int32)
    prompt = i32(two[[0, 0, 1, 1]])
    ref = greedy(prob, prompt)
    np.testing.assert_array_equal(ref[0], ref[1])

    # rows 0 and 2 read the prompts, 1 and 3 are forked from them; a pool that just holds what is live
    dec = decoder(prob, pages=3 * B * (-(-L // PAGE)) // 4)
    t, h = prefill(dec, prompt, [0, 2])
    held = int((dec.table >= 0).sum())
    dec.fork(i32([0, 0, 2, 2]))
    assert int((dec.ref > 0).sum()) == held and int(dec.ref.sum()) == 2 * held
    t, h = t[[0, 0, 2, 2]].contiguous(), h[[0, 0, 2, 2]].contiguous()
    ctx = np.full(B, PROMPT)
    committed = [[int(v)] for v in t.cpu().numpy()]
    g = torch.Generator(device="cuda").manual_seed(3)
    dk, dv = (torch.randn((B, L, dec.nh, dec.hd), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    dws = api.spec_draft_workspace(B, dec.H, dec.nh, prob.I_draft, dec.V, L)
    lengths, turn = [], 0
    stats = torch.zeros(4, dtype=torch.int32, device="cuda")
    while min(len(c) for c in committed) < N_NEW:
        drafts = api.spec_draft_loop(dec.draft_w, h, t, dk, dv, i32(ctx), K, dws)
        tokens = torch.cat([t.view(B, 1), drafts], 1).contiguous()
        b = step(dec, ctx, tokens, drafts)
        if turn == 0:                                           # what was shared and is written now is each row's own
            dec_ref = dec.ref[dec.table[:, PROMPT // PAGE].long()]
            assert (dec_ref == 1).all() and (dec.ref[dec.table[:, 0].long()] == 2).all()
        alen, comm = b["alen"].cpu().numpy(), b["comm"].cpu().numpy()
        for s in range(B):
            committed[s].extend(int(c) for c in comm[s, :alen[s] + 1])
        lengths.extend(alen.tolist())
        ctx = ctx + alen + 1
        idx = torch.from_numpy(alen.astype(np.int64)).cuda()
        t = b["comm"].gather(1, idx.view(B, 1)).view(B).contiguous()
        h = b["x"].view(B, K + 1, dec.H)[torch.arange(B, device="cuda"), idx].contiguous()
        if turn % 3 == 2:                                       # the rejected drafts' pages, then all live ones together
            dec.reserve(i32(ctx), i32(ctx))
            assert ((dec.table >= 0).sum(1).cpu().numpy() == -(-ctx // PAGE)).all()
            dec.compact(stats)
            live = int(stats[0])
            assert live == int((dec.ref > 0).sum()) and (dec.ref[:live] > 0).all()
        turn += 1
    np.testing.assert_array_equal(np.array([c[:N_NEW] for c in committed]), ref)
    assert 0 <= min(lengths) and max(lengths) <= K
    dec.reserve(i32(np.zeros(B)), i32(np.zeros(B)), stats)      # every sequence ends
    assert int(dec.ref.abs().sum()) == 0 and bool((dec.table == -1).all())


def test_a_captured_step_over_pages():
    """Reserve and verify in one graph, replayed at other lengths, against the calls one by one."""
    dims = synth.MoeDims(0, 256, 8, 2, 1, 128)
    prob = synth.decoder_problem(2, dims, V=2048, nh=2, I_draft=256, seed=5, out_scale=0.3, mimic_draft=True)
    prompt = i32(np.random.default_rng(1).integers(0, prob.V, size=(B, PROMPT)))
    plain, graphed = decoder(prob), decoder(prob)
    t, _ = prefill(plain, prompt, range(B))
    prefill(graphed, prompt, range(B))
    tokens, drafts = torch.zeros((B, 3), dtype=torch.int32, device="cuda"), torch.zeros((B, 2), dtype=torch.int32, device="cuda")
    keep, after = i32(np.full(B, PROMPT)), i32(np.full(B, PROMPT))
    graphed.verify(tokens, i32(np.zeros(B)), drafts)            # the buffers are made before the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        graphed.reserve(keep, after)
        out = graphed.verify(tokens, after, drafts)
    ctx = np.full(B, PROMPT)
    for i in range(12):
        rs = np.random.default_rng(i)
        tk = rs.integers(0, prob.V, (B, 3))
        tokens.copy_(i32(tk)); drafts.copy_(i32(tk[:, 1:]))
        keep.copy_(i32(ctx)); after.copy_(i32(ctx + 3))
        graph.replay()
        ref = step(plain, ctx, i32(tk), i32(tk[:, 1:]))
        for n in ("argmax", "alen", "comm", "x"):
            assert torch.equal(out[n], ref[n]), n
        assert torch.equal(graphed.table, plain.table) and torch.equal(graphed.ref, plain.ref)
        ctx = ctx + rs.integers(0, 4, B)


@pytest.mark.parametrize("captured", [False, True])
def test_a_pass_without_room_writes_nothing(captured):
    """Four sequences share a prefix in a pool with no page left for their copies: the pass behind the failed reserve must
    not write to what they share; once a sequence has ended the others go on as if nothing had been."""
    dims = synth.MoeDims(0, 256, 8, 2, 1, 128)
    prob = synth.decoder_problem(2, dims, V=2048, nh=2, I_draft=256, seed=7, out_scale=0.3, mimic_draft=True)
    prompt = i32(np.random.default_rng(2).integers(0, prob.V, size=(1, PROMPT)).repeat(B, 0))
    tk = np.random.default_rng(3).integers(0, prob.V, (B, 3))
    tokens, drafts = i32(tk), i32(tk[:, 1:])
    held = -(-PROMPT // PAGE)
    room, tight = decoder(prob), decoder(prob, pages=held + 2)      # two copies of the last page, where four are wanted
    for dec in (room, tight):
        prefill(dec, prompt, [0])
        dec.fork(i32([0] * B))
        dec.verify(tokens, i32(np.zeros(B)), drafts)                # the buffers are made before the capture
    keep, cap = i32(np.full(B, PROMPT)), i32(np.full(B, PROMPT + 3))
    torch.cuda.synchronize()
    before = [x.clone() for x in (tight.pool, tight.table, tight.ref)]
    stats = torch.full((4,), -7, dtype=torch.int32, device="cuda")

    def turn():
        tight.reserve(keep, cap, stats)
        return tight.verify(tokens, cap, drafts)

    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = turn()
        graph.replay()
    else:
        out = turn()
    assert api.get_device_error() == 8 and stats.tolist() == [4, 2, 0, 0]
    for x, y in zip((tight.pool, tight.table, tight.ref), before):
        assert torch.equal(x, y)
    for n in (2, 3):                                                # those two sequences end
        keep[n] = cap[n] = 0
    graph.replay() if captured else turn()
    assert api.get_device_error() == 0 and stats.tolist()[:2] == [2, 2]
    room.reserve(keep, cap)
    ref = room.verify(tokens, cap, drafts)
    for n in ("argmax", "alen", "comm"):
        assert torch.equal(out[n][:2], ref[n][:2])


def test_the_decoder_refuses_lengths_and_counts_of_another_kind():
    dims = synth.MoeDims(0, 256, 8, 2, 1, 128)
    dec = decoder(synth.decoder_problem(1, dims, V=512, nh=2, I_draft=256, seed=6))
    tokens, drafts = torch.zeros((B, 2), dtype=torch.int32, device="cuda"), torch.zeros((B, 1), dtype=torch.int32, device="cuda")
    n = i32(np.full(B, 2))
    for bad in (n[:1], n.long(), n[0], n.cpu(), i32(np.zeros((B, 2)))[:, 0]):
        with pytest.raises(ValueError):
            dec.verify(tokens, bad, drafts)
    for bad in (n[:3], n.long(), i32(np.zeros((2, 4))), n.cpu()):
        with pytest.raises(ValueError):
            dec.reserve(n, n, bad)
    assert bool((dec.table == -1).all()) and int(dec.pool.count_nonzero()) == 0


def test_filled_caches():
    dims = synth.MoeDims(0, 256, 8, 2, 1, 128)
    prob = synth.decoder_problem(2, dims, V=512, nh=2, I_draft=256, seed=6)
    dec = decoder(prob)
    dec.fill_caches(1)
    k, v = api.spec_q4_read(dec.pool[1], dec.table, i32(np.full(B, L)), L, 2, 128, PAGE)
    assert abs(float(k.float().std()) - 1) < 0.02 and abs(float(v.float().std()) - 1) < 0.02
    with pytest.raises(ValueError):
        Decoder(prob, B, L, cache="fp8")
