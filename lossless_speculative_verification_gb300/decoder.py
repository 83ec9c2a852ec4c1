"""A verify pass of an n-layer decoder, composed from the library's entry points.

The FastMTP verify step runs the drafted positions of every sequence through
the main decoder in one pass and keeps the longest prefix that greedy
decoding would have produced (kg.zhiyong.dev, "The speed comes from three
layers working together" and "Why FastMTP fits OCR particularly well").  The
pages give the decoder as an MoE decoder; the plainest reading is a stack of
pre-norm layers, each an attention block and the MoE FFN on the residual
stream x:

    h = RMSNorm(x);  q, k, v = h W_q^T, h W_k^T, h W_v^T   (the Q new keys and values appended)
    x = x + attention(q, caches) W_o^T;  h = RMSNorm(x);  x = x + MoE(h)

followed by the output layer fused with the greedy search and the acceptance
rule on RMSNorm(x).  Every step runs in the library's kernels
(lsv_gather_rows, rmsnorm_residual, dense_matmul, spec_cache_append,
spec_verify_attention, moe_verify_layer, spec_verify_lmhead); this module only
orders the calls and owns the buffers, so that a verify pass (and a draft +
verify step) can be replayed as one CUDA graph.

The keys and values stand in contiguous bf16 caches, or, with cache="q4", in the
paged 4-bit cache: one pool of pages for every layer, one page table for all of
them (spec_q4_append, spec_q4_attention).  Then reserve() gives every sequence
its pages before a pass and takes the rejected drafts' pages back after it,
fork() lets sequences go on from one prefix, and compact() moves the live pages
together (spec_pages_resize, spec_pages_fork, spec_pages_compact).  Where the pool
has too few free pages for a reserve(), the pages that a pass would write may still be
other sequences' too, so verify() appends nothing until a reserve() succeeds: it looks
at that call's counts on the device, also inside one graph with it.

With weights="q8" the projections and the output layer are held in 8 bits: the norms
before them write 8-bit rows (rmsnorm_residual_q8), the attention's output is quantised
(quantize_q8_rows), the products are dense_matmul_q8, and the greedy tokens come from the
output layer's logits (spec_verify_accept), which are rounded to bf16 before that search: of
equal ones the lower token, where bf16 weights compare the unrounded sums.  A row's products
are the same in passes of up to 256 positions (B * Q), as the loop's equality with greedy
decoding needs; in larger ones, from a hidden size of 1424 on, their last bits may differ.
The experts and the draft block stay as they are.  verify(logprobs=n) adds the committed
tokens' log probabilities, the entropies and the n most likely tokens of every position
(spec_logprobs).
"""
from __future__ import annotations

import math

import numpy as np
import torch

from . import api


def _dev(bits, device):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).view(torch.bfloat16).to(device)


class Decoder:
    """Device weights and per-layer key/value caches of a synthetic decoder (synth.DecoderProblem):
    [B, L, nh, d] bf16, or with cache="q4" pages of `page` positions, `pages` of them (as many as B
    sequences of L positions need unless given), all free at first.  weights="q8": projections and output
    layer in 8 bits.  verify() runs one verify pass over Q positions per sequence, for the first
    tokens.shape[0] <= B sequences."""

    weights = "bf16"

    def __init__(self, prob, B: int, L: int, device="cuda", cache: str = "bf16", page: int = 64, pages: int | None = None,
                 weights: str = "bf16"):
        if cache not in ("bf16", "q4"):
            raise ValueError("cache must be 'bf16' or 'q4'")
        if weights not in ("bf16", "q8"):
            raise ValueError("weights must be 'bf16' or 'q8'")
        self.prob, self.B, self.L, self.device = prob, B, L, device
        self.cache, self.page, self.weights = cache, page, weights
        d = prob.dims
        self.H, self.nh = d.H, prob.nh
        self.hd = d.H // prob.nh
        self.V = prob.V
        self.emb = _dev(prob.emb, device)
        self.w_vocab = _dev(prob.w_vocab, device)
        self.layers = []
        for lw in prob.layers:
            t = {n: _dev(lw[n], device) for n in ("w_q", "w_k", "w_v", "w_o")}
            if weights == "q8":
                t = {n: api.quantize_q8_weight(w) for n, w in t.items()}
            t["moe"] = api.weights(*[_dev(lw[n], device) for n in ("w_router", "w_gate_up", "w_down", "ws_gate_up",
                                                                    "ws_down")])
            if cache == "bf16":
                t["kc"] = torch.zeros((B, L, self.nh, self.hd), dtype=torch.bfloat16, device=device)
                t["vc"] = torch.zeros_like(t["kc"])
            self.layers.append(t)
        if cache == "q4":
            M = -(-L // page)
            P = B * M if pages is None else pages
            self.pool = torch.zeros((len(self.layers), P, api.spec_q4_page_bytes(self.nh, self.hd, page)),
                                    dtype=torch.uint8, device=device)
            self.table = torch.full((B, M), -1, dtype=torch.int32, device=device)
            self.ref = torch.zeros(P, dtype=torch.int32, device=device)
            self.pws = api.spec_pages_workspace(B, M, P, device)
            self.room = torch.zeros(4, dtype=torch.int32, device=device)   # the last reserve()'s counts
        self.vocab_q8 = api.quantize_q8_weight(self.w_vocab) if weights == "q8" else None
        dw = dict(prob.draft)
        dw["emb"], dw["w_vocab"] = prob.emb, prob.w_vocab
        self.draft_w = {n: (self.emb if n == "emb" else self.w_vocab if n == "w_vocab" else _dev(dw[n], device))
                        for n in api.DRAFT_WEIGHTS}
        self._bufs = {}
        self._read = {}   # what logprobs=n reads off a pass of (B, Q), by n

    def fill_caches(self, seed: int):
        """N(0, 1) keys and values everywhere (the entries of a prefix that is not replayed)."""
        g = torch.Generator(device=self.device).manual_seed(seed)
        if self.cache == "q4":
            full = torch.full((self.B,), self.L, dtype=torch.int32, device=self.device)
            self.reserve(torch.zeros_like(full), full)
            for pool in self.pool:
                k, v = (torch.randn((self.B, self.L, self.nh, self.hd), generator=g, device=self.device).to(torch.bfloat16)
                        for _ in range(2))
                api.spec_q4_append(k, v, pool, self.table, full, self.page)
            return
        for t in self.layers:
            t["kc"].copy_(torch.randn(t["kc"].shape, generator=g, device=self.device).to(torch.bfloat16))
            t["vc"].copy_(torch.randn(t["vc"].shape, generator=g, device=self.device).to(torch.bfloat16))

    def reserve(self, keep, cap, stats=None):
        """Pages for the positions 0..cap[b]-1 of every sequence, of which keep[b] are kept (int32 [B]); see
        spec_pages_resize.  With too few free pages nothing changes, LSV_ERR_PAGES is in the error word
        (api.get_device_error), room[0] (pages needed) is above room[1] (pages free), and verify() takes every
        sequence for a slot without one until a reserve() succeeds.  stats [4] int32: a copy of room."""
        if stats is not None:
            api.check_lengths(stats, 4, "stats")
        api.spec_pages_resize(self.pool, self.table, self.ref, keep, cap, self.page, self.pws, stats=self.room)
        if stats is not None:
            stats.copy_(self.room)

    def fork(self, parent):
        """Sequence b goes on from sequence parent[b] (-1: none); int32 [B]."""
        api.spec_pages_fork(self.table, self.ref, parent, self.pws)

    def compact(self, stats=None):
        """The live pages to the lowest numbers of the pool."""
        api.spec_pages_compact(self.pool, self.table, self.ref, self.pws, stats=stats)

    def buffers(self, B: int, Q: int):
        """The activations, workspaces and outputs of a pass over Q positions of B sequences."""
        if (B, Q) not in self._bufs:
            H, dev = self.H, self.device
            T = B * Q
            d = self.prob.dims
            b = {n: torch.zeros((T, H), dtype=torch.bfloat16, device=dev) for n in ("x", "h", "zero", "q", "k", "v",
                                                                                     "a", "o", "y")}
            b["sh"] = api.shape(T, H, d.E, d.k, d.S, d.I)
            b["mws"] = api.workspace(b["sh"], dev)
            if self.cache == "q4":
                b["aws"] = api.spec_q4_attention_workspace(B, Q, self.table.shape[1], self.page, self.nh, self.nh, self.hd,
                                                           dev)
                b["none"], b["len"] = (torch.zeros(B, dtype=torch.int32, device=dev) for _ in range(2))
            else:
                b["aws"] = api.spec_verify_attention_workspace(B, Q, self.L, self.nh, self.hd, dev)
            if self.weights == "q8":
                for n in ("hq", "aq"):   # 8-bit rows: the norm's, the attention's
                    b[n] = (torch.zeros((T, H), dtype=torch.float8_e4m3fn, device=dev),
                            torch.zeros(api.q8_scales_shape(T, H), device=dev))
                b["lws"] = api.spec_verify_workspace(B, Q - 1, self.V, dev)
            else:
                b["lws"] = api.spec_verify_lmhead_workspace(B, Q - 1, self.V, H, dev)
            b["argmax"] = torch.zeros((B, Q), dtype=torch.int32, device=dev)
            b["alen"] = torch.zeros(B, dtype=torch.int32, device=dev)
            b["comm"] = torch.zeros((B, Q), dtype=torch.int32, device=dev)
            self._bufs[(B, Q)] = b
            self._read[(B, Q)] = {}
        return self._bufs[(B, Q)]

    def _logits(self, buffers, B, Q):
        """Logits [B, Q, V] among these buffers, made when they are first asked for."""
        if "logits" not in buffers:
            buffers["logits"] = torch.empty((B, Q, self.V), dtype=torch.bfloat16, device=self.device)
        return buffers["logits"]

    def verify(self, tokens, ctx_after, drafts, logprobs: int | None = None):
        """One verify pass.  tokens [B, Q] int32: input 0 is each sequence's last committed token,
        inputs 1..Q-1 its drafts (drafts [B, Q-1] int32, the same tokens); ctx_after [B] int32: the
        cache lengths once the Q positions are appended (with the 4-bit cache reserve() comes before, and 0
        stands for a slot without a sequence, as every length does where that call found too few pages: then
        no page is written, and the outputs are of no use).  Returns the pass's buffers: argmax [B, Q]
        (the greedy token after each input), alen [B], comm [B, Q] (the rule's outputs), x [B*Q, H]
        (the last residual stream, the draft block's next input state), with 8-bit weights logits
        [B, Q, V].  logprobs=n returns beside them logprob [B, Q] (of comm's tokens; 0 behind the last),
        entropy [B, Q], top_ids and top_logprobs [B, Q, n], of the bf16 logits after each input, and these
        (with bf16 weights a second product with the output layer, whose logits the greedy search does not
        round; V a multiple of 8).  They are kept apart for each n: a pass without them returns none."""
        B, Q = tokens.shape
        b = self.buffers(B, Q)
        nh, hd = self.nh, self.hd
        api.gather_rows(self.emb, tokens.reshape(-1), out=b["x"])
        y = b["zero"]
        if self.cache == "q4":
            api.check_lengths(ctx_after, B, "ctx_after")
            torch.where(self.room[0] <= self.room[1], ctx_after, b["none"], out=b["len"])
            ctx_after = b["len"]
        for i, t in enumerate(self.layers):
            if self.weights == "q8":
                api.rmsnorm_residual_q8(b["x"], y if i else None, codes=b["hq"][0], scales=b["hq"][1])
                for n in ("q", "k", "v"):
                    api.dense_matmul_q8(*b["hq"], *t["w_" + n], out=b[n])
            else:
                api.rmsnorm_residual(b["x"], y, h=b["h"])
                for n in ("q", "k", "v"):
                    api.dense_matmul(b["h"], t["w_" + n], out=b[n])
            if self.cache == "q4":
                api.spec_q4_append(b["k"].view(B, Q, nh, hd), b["v"].view(B, Q, nh, hd), self.pool[i], self.table[:B],
                                   ctx_after, self.page)
                api.spec_q4_attention(b["q"].view(B, Q, nh, hd), self.pool[i], self.table[:B], ctx_after, nh, self.page,
                                      b["aws"], out=b["a"].view(B, Q, nh, hd))
            else:
                kc, vc = t["kc"][:B], t["vc"][:B]
                api.spec_cache_append(b["k"].view(B, Q, nh, hd), b["v"].view(B, Q, nh, hd), kc, vc, ctx_after)
                api.spec_verify_attention(b["q"].view(B, Q, nh, hd), kc, vc, ctx_after, b["aws"],
                                          out=b["a"].view(B, Q, nh, hd))
            if self.weights == "q8":
                api.quantize_q8_rows(b["a"], *b["aq"])
                api.dense_matmul_q8(*b["aq"], *t["w_o"], out=b["o"])
            else:
                api.dense_matmul(b["a"], t["w_o"], out=b["o"])
            api.rmsnorm_residual(b["x"], b["o"], h=b["h"])
            api.moe_verify_layer(b["h"], t["moe"], b["sh"], b["mws"], out=b["y"])
            y = b["y"]
        if self.weights == "q8":
            logits = self._logits(b, B, Q)
            api.rmsnorm_residual_q8(b["x"], y if self.layers else None, codes=b["hq"][0], scales=b["hq"][1])
            api.dense_matmul_q8(*b["hq"], *self.vocab_q8, out=logits.view(B * Q, self.V))
            api.spec_verify_accept(logits, drafts, b["lws"], argmax=b["argmax"], accept_len=b["alen"], committed=b["comm"])
        else:
            api.rmsnorm_residual(b["x"], y, h=b["h"])
            api.spec_verify_lmhead(b["h"], self.w_vocab, drafts, b["lws"], Q - 1, argmax=b["argmax"],
                                   accept_len=b["alen"], committed=b["comm"])
        if logprobs is None:
            return b
        read = self._read[(B, Q)]
        if self.weights != "q8":
            logits = self._logits(read, B, Q)
            api.dense_matmul(b["h"], self.w_vocab, out=logits.view(B * Q, self.V))
        outs = read.setdefault(logprobs, {})
        outs.update(zip(("logprob", "entropy", "top_ids", "top_logprobs"),
                        api.spec_logprobs(logits, b["comm"], logprobs, **outs)))
        return {**b, "logits": logits, **outs}

    def launches_per_verify(self, B: int, Q: int) -> int:
        """Library kernel launches of one verify pass over the bf16 caches, without log probabilities (the MoE layer:
        3 up to 256 tokens).  Over 4-bit pages the attention is one launch or two, as the library cuts the sequences, and
        no count is given."""
        if self.cache != "bf16":
            raise ValueError("launches_per_verify counts the pass over bf16 caches")
        T = B * Q
        moe = 3 if T <= 256 else (4 if T * self.prob.dims.k <= 8192 else 6)
        q8 = 1 if self.weights == "q8" else 0    # the attention's rows quantised; the output layer apart from the search
        return 1 + len(self.layers) * (1 + 3 + 1 + 2 + q8 + 1 + 1 + moe) + 1 + q8 + 2
