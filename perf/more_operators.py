"""Measured cases of the 8-bit path of a verify pass and of what is read off its logits, with the operators' plain forms.

In the 8-bit form, 128 consecutive columns of a row, or a block of 128 x 128 of a weight, share a scale s: the smallest
power of two, 2^-126 at least, with max |x| <= 448 s.  A code is e4m3(x / s), nearest, ties to even, and stands for
code * s.  The last group of a row, and the last blocks of a weight, may be short.
"""
import math
import random

import torch

own = False

GROUP = 128
LARGEST = 448.0


# ------------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one sequence decoding one token: the norm before a projection, latency alone
        dict(name="norm_token", op="norm", T=1, H=1280, res=True, gain=False),
        # a wide model's rows, a batch that is no round number, the last group short
        dict(name="norm_wide_odd", op="norm", T=733, H=7120, res=True, gain=True),
        # eight pages' prompts at once
        dict(name="norm_prompt", op="norm", T=9760, H=1280, res=True, gain=False),
        # a model's output layer brought to 8 bits when it is loaded
        dict(name="weight_head", op="weight", N=129280, K=1280),
        # attention's output to 8 bits for the projection behind it, a ragged prompt
        dict(name="rows_prompt", op="rows", T=4879, H=1280),
        # one projection of one token: latency alone
        dict(name="mm_token", op="mm", M=1, N=1280, K=1280),
        # the output layer on the verified positions: the weights' bytes
        dict(name="mm_head_verify", op="mm", M=128, N=129280, K=1280),
        # a wide feed-forward layer's second half over a ragged prompt
        dict(name="mm_down_prompt", op="mm", M=4879, N=1280, K=7168),
        # the output layer over two prompts, for their tokens' probabilities: the tensor cores
        dict(name="mm_head_prompt", op="mm", M=2440, N=129280, K=1280),
        # the probability of one sequence's next token: latency alone
        dict(name="logprobs_token", op="logprobs", R=1, V=129280, n=5, dtype="bf16", masked=0.0),
        # probabilities of a verify pass's tokens (32 sequences, 3 drafts each), with the alternatives that an API returns
        dict(name="logprobs_verify", op="logprobs", R=128, V=129280, n=20, dtype="bf16", masked=0.0),
        # the same over two prompts in 32 bits, a vocabulary that is odd, a grammar that allows few tokens in some rows
        dict(name="logprobs_prompt", op="logprobs", R=2440, V=100277, n=5, dtype="fp32", masked=0.25),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "rows", "weight", "mm", "mm", "mm", "logprobs", "logprobs", "logprobs"])
    while True:
        if op in ("norm", "rows"):
            c = dict(op=op, T=_log(rng, 1, 9760), H=16 * _log(rng, 1, 1024))
            if c["T"] * c["H"] > 9760 * 1280:
                continue
            return c | dict(res=rng.random() < 0.8, gain=rng.random() < 0.5) if op == "norm" else c
        if op == "weight":
            c = dict(op=op, N=_log(rng, 1, 129280), K=16 * _log(rng, 1, 1024))
            if c["N"] * c["K"] > 129280 * 1280:
                continue
            return c
        if op == "mm":
            c = dict(op=op, M=_log(rng, 1, 9760), N=_log(rng, 1, 129280), K=16 * _log(rng, 1, 1024))
            if c["M"] * c["N"] * c["K"] > 2440 * 129280 * 1280 or c["N"] * c["K"] > 129280 * 1280 or \
                    c["M"] * c["N"] > 2440 * 129280:
                continue
            return c
        c = dict(op=op, R=_log(rng, 1, 2440), V=_log(rng, 100, 262144), n=rng.randint(1, 32),
                 dtype=rng.choice(["bf16", "bf16", "fp32"]), masked=rng.choice([0.0, 0.0, 0.25]))
        if c["R"] * c["V"] <= 2440 * 100277:
            return c


# ------------------------------------------------------------------------------------------------ the 8-bit form
def _groups(n):
    return -(-n // GROUP)


def _spread(s, rows, cols, by):
    """Scales [groups of `by` rows, groups of columns] as one a value [rows, cols]."""
    return s.repeat_interleave(by, 0)[:rows].repeat_interleave(GROUP, 1)[:, :cols]


def _power(top):
    """The smallest power of two, 2^-126 at least, that 448 times is not below top; in 32 bits."""
    m, e = torch.frexp(top)
    e = torch.where(m > 0.875, e - 8, e - 9)  # 448 = 0.875 * 2^9
    return ((torch.where(top > 0, e, -126).clamp(min=-126) + 127).to(torch.int32) << 23).view(torch.float32)


def _quantise(x, by):
    """[R, C] in 32 bits -> codes (e4m3) and scales (fp32) of groups of `by` rows x 128 columns; quotients are exact."""
    R, C = x.shape
    a = torch.nn.functional.pad(x.abs(), (0, -C % GROUP, 0, -R % by))
    s = _power(a.view(a.shape[0] // by, by, a.shape[1] // GROUP, GROUP).amax((1, 3)))
    return (x * (1 / _spread(s, R, C, by))).to(torch.float8_e4m3fn), s


def _values(codes, s, by):
    return codes.float() * _spread(s, *codes.shape, by)


# ------------------------------------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 13)


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _rand(g, *shape):
    return torch.rand(shape, generator=g, device="cuda")


def _stream_rows(g, T, H):
    """Rows of a residual stream: sizes that differ from row to row, and some dims far larger than the others."""
    dims = torch.where(_rand(g, H) < 0.01, 20.0, 1.0) * (0.5 + _rand(g, H))
    return (_randn(g, T, H) * dims * (0.5 + 2 * _rand(g, T, 1))).to(torch.bfloat16)


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = dict(c=c)
    if c["op"] in ("norm", "rows"):
        T, H = c["T"], c["H"]
        s["x"] = _stream_rows(g, T, H)
        if c["op"] == "norm":
            s["y"] = _randn(g, T, H).to(torch.bfloat16) if c["res"] else None
            s["gain"] = (1 + 0.2 * _randn(g, H)).to(torch.bfloat16) if c["gain"] else None
            s["sum"] = torch.empty_like(s["x"]) if c["res"] else None
        s["by"], shape = 1, (T, H)
    elif c["op"] == "weight":
        shape = (c["N"], c["K"])
        s["x"] = (_randn(g, *shape) * 0.02 * (0.5 + _rand(g, shape[0], 1))).to(torch.bfloat16)
        s["by"] = GROUP
    elif c["op"] == "mm":
        M, N, K = c["M"], c["N"], c["K"]
        s["x"], s["sx"] = _quantise(_stream_rows(g, M, K).float(), 1)
        s["w"], s["sw"] = _quantise(_randn(g, N, K) * 0.02 * (0.5 + _rand(g, N, 1)), GROUP)
        s["out"] = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
        return s
    else:
        R, V, n = c["R"], c["V"], c["n"]
        # most tokens far below a few that a model holds for likely
        x = 2.0 * _randn(g, R, V)
        step = V // 24  # one of them in each 24th of the vocabulary, in any order
        some = torch.randint(0, step, (R, 24), generator=g, device="cuda")
        some += step * _rand(g, R, 24).argsort(-1)
        x.scatter_(1, some, 6 + 4 * _rand(g, R, 24) + 4 * _rand(g, R, 1))
        if c["masked"]:
            # rows where a grammar allows one token in fifty, one of them at least
            few = (_rand(g, R, 1) < c["masked"]) & (_rand(g, R, V) >= 0.02)
            few.scatter_(1, some[:, :1], False)
            x.masked_fill_(few, -torch.inf)
        s["x"] = x.to(torch.bfloat16) if c["dtype"] == "bf16" else x
        # tokens: likely ones, some that are not, none behind the last committed one
        t = torch.where(_rand(g, R) < 0.7, some[:, 0], torch.randint(0, V, (R,), generator=g, device="cuda"))
        s["tokens"] = torch.where(_rand(g, R) < 0.15, -1, t).to(torch.int32)
        f32 = dict(dtype=torch.float32, device="cuda")
        s["out"] = (torch.empty(R, **f32), torch.empty(R, **f32),
                    torch.empty((R, n), dtype=torch.int32, device="cuda"), torch.empty((R, n), **f32))
        return s
    s["codes"] = torch.empty(shape, dtype=torch.float8_e4m3fn, device="cuda")
    s["scales"] = torch.empty((-(-shape[0] // s["by"]), _groups(shape[1])), device="cuda")
    s["values"] = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    return s


# ------------------------------------------------------------------------------------------------ plain forms
def _plain_norm(s):
    x = s["x"] if s["y"] is None else (s["x"].float() + s["y"].float()).to(torch.bfloat16)
    f = x.float()
    h = f / torch.sqrt((f * f).mean(-1, keepdim=True) + 1e-6)
    if s["gain"] is not None:
        h = h * s["gain"].float()
    codes, scales = _quantise(h, 1)
    values = _values(codes, scales, 1).to(torch.bfloat16)
    return values if s["y"] is None else [values, x]


def _plain_quantise(s):
    codes, scales = _quantise(s["x"].float(), s["by"])
    return _values(codes, scales, s["by"]).to(torch.bfloat16)


def _plain_mm(s):
    return (_values(s["x"], s["sx"], 1) @ _values(s["w"], s["sw"], GROUP).T).to(torch.bfloat16)


def _plain_logprobs(s):
    x, t, n = s["x"].float(), s["tokens"].long(), s["c"]["n"]
    V = x.shape[1]
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - m)
    S = e.sum(-1)
    logS = torch.log(S)
    entropy = logS - torch.where(e > 0, e * (x - m), 0).sum(-1) / S
    at = torch.gather(x, 1, t.clamp(min=0)[:, None])
    logprob = torch.where(t >= 0, (at - m)[:, 0] - logS, 0)
    # whole numbers in the order of the values, equal ones by falling index
    b = (x + 0.0).view(torch.int32)
    b = torch.where(b >= 0, b, b ^ 0x7FFFFFFF).long()
    key = (b << 32) + (0xFFFFFFFF - torch.arange(V, device=x.device))
    ids = 0xFFFFFFFF - (torch.topk(key, n, -1).values & 0xFFFFFFFF)
    return [logprob, entropy, ids.to(torch.int32), torch.gather(x, 1, ids) - m - logS[:, None]]


# ------------------------------------------------------------------------------------------------ one pass
def run(state):
    s, op = state, state["c"]["op"]
    if not own:
        if op == "norm":
            return _plain_norm(s)
        if op == "mm":
            return _plain_mm(s)
        return _plain_logprobs(s) if op == "logprobs" else _plain_quantise(s)
    from lossless_speculative_verification_gb300 import api
    if op == "mm":
        return api.dense_matmul_q8(s["x"], s["sx"], s["w"], s["sw"], out=s["out"])
    if op == "logprobs":
        logprob, entropy, ids, tops = s["out"]
        return list(api.spec_logprobs(s["x"], s["tokens"], s["c"]["n"], logprob=logprob, entropy=entropy, top_ids=ids,
                                      top_logprobs=tops))
    if op == "norm":
        api.rmsnorm_residual_q8(s["x"], s["y"], gain=s["gain"], x_out=s["sum"], codes=s["codes"], scales=s["scales"])
    elif op == "rows":
        api.quantize_q8_rows(s["x"], codes=s["codes"], scales=s["scales"])
    else:
        api.quantize_q8_weight(s["x"], codes=s["codes"], scales=s["scales"])
    values = api.dequantize_q8(s["codes"], s["scales"], out=s["values"])
    return [values, s["sum"]] if op == "norm" and s["y"] is not None else values


def work(case):
    c = case
    if c["op"] == "mm":
        M, N, K = c["M"], c["N"], c["K"]
        return {"bytes": M * K + N * K + 4 * _groups(K) * (M + _groups(N)) + 2 * M * N, "flops": 2 * M * N * K}
    if c["op"] == "logprobs":
        R, V, n = c["R"], c["V"], c["n"]
        # a difference, an exponential and two sums a logit
        return {"bytes": R * V * (2 if c["dtype"] == "bf16" else 4) + R * (12 + 8 * n), "flops": 5 * R * V}
    rows, cols = (c["N"], c["K"]) if c["op"] == "weight" else (c["T"], c["H"])
    n, scales = rows * cols, 4 * _groups(cols) * (_groups(rows) if c["op"] == "weight" else rows)
    # the rows in, codes and scales out, codes and scales in, the values out
    moved = 2 * n + 2 * (n + scales) + 2 * n
    if c["op"] == "norm":
        moved += (4 * n if c["res"] else 0) + (2 * cols if c["gain"] else 0)
    return {"bytes": moved, "flops": (8 if c["op"] == "norm" else 4) * n}


# ------------------------------------------------------------------------------------------------ in 64 bits
def _nearest(q):
    """q (|q| <= 448) to the nearest value of the 8-bit format, ties to the even one: by its table of values."""
    e, m = torch.arange(16, device=q.device)[:, None].double(), torch.arange(8, device=q.device)[None, :].double()
    table = torch.where(e > 0, (8 + m) * torch.exp2(e - 10), m * 2.0 ** -9).reshape(-1)[:-1]
    up = torch.bucketize(q.abs(), (table[1:] + table[:-1]) / 2)  # at a middle: the lower one
    low = table[up]
    high = table[(up + 1).clamp(max=126)]
    tie = (q.abs() - low == high - q.abs()) & (up % 2 == 1)
    return torch.where(tie, high, low).copysign(q)


def _exact_q8(h, by):
    R, C = h.shape
    values = torch.empty_like(h)
    powers = torch.exp2(torch.arange(-126, 128, device=h.device).double())
    for k in range(_groups(C)):
        x = h[:, GROUP * k:GROUP * (k + 1)]
        top = torch.nn.functional.pad(x.abs().amax(1), (0, -R % by)).view(-1, by).amax(1)
        each = powers[torch.searchsorted(LARGEST * powers, top)].repeat_interleave(by)[:R, None]
        values[:, GROUP * k:GROUP * (k + 1)] = _nearest(x / each) * each
    return values


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "norm":
        x = s["x"].double()
        if s["y"] is not None:
            x = (x + s["y"].double()).to(torch.bfloat16).double()
        h = x * torch.rsqrt(x.square().sum(1, keepdim=True) / x.shape[1] + 1e-6)
        if s["gain"] is not None:
            h = h * s["gain"].double()
        return _exact_q8(h, 1) if s["y"] is None else [_exact_q8(h, 1), x]
    if c["op"] in ("rows", "weight"):
        return _exact_q8(s["x"].double(), s["by"])
    if c["op"] == "mm":
        out = torch.zeros((c["M"], c["N"]), dtype=torch.float64, device="cuda")
        for n in range(0, c["N"], 4096):
            m = min(c["N"], n + 4096)
            by = s["sw"][n // GROUP:_groups(m)].double().repeat_interleave(GROUP, 0)[:m - n]
            for k in range(_groups(c["K"])):
                at = slice(GROUP * k, GROUP * (k + 1))
                part = s["x"][:, at].double() @ s["w"][n:m, at].double().T
                out[:, n:m] += part * s["sx"][:, k:k + 1].double() * by[:, k]
        return out
    n = c["n"]
    logprob, entropy = (torch.zeros(c["R"], dtype=torch.float64, device="cuda") for _ in range(2))
    tops = torch.empty((c["R"], n), dtype=torch.float64, device="cuda")
    for r in range(0, c["R"], 256):
        at = slice(r, r + 256)
        logp = torch.log_softmax(s["x"][at].double(), -1)
        p = logp.exp()
        entropy[at] = -torch.where(p > 0, p * logp, 0).sum(-1)
        tops[at] = logp.sort(-1, descending=True).values[:, :n]
        t = s["tokens"][at].long()
        logprob[at] = torch.where(t >= 0, logp.gather(1, t.clamp(min=0)[:, None])[:, 0], 0)
    return [logprob, entropy, None, tops]
