"""ssc_sample_rows on the GPU against the definition in 64 bits. Tokens and
kept counts are equal. Logprobs are off by the rounding to fp32, half a step,
and by the sum of the weights. A weight is at most 1 and its fp64 value off by
7e-15 (the series' last term) and some steps of 2^-53 of itself, together
under 2^-46; it is rounded to an integer multiple of 2^-bits, half of that off.
The sum over V logits is 1 at least, so it is off by at most V * 2^-(bits + 1)
+ 2^-46 of itself, equal weights all the same way, and its logarithm by as
much. The chosen weight's own logarithm is taken from the logit."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import scan_stream_compaction_amd as ssc
from tests.sample_reference import sample

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = [torch.float32, torch.bfloat16, torch.float16]


def _np(t):
    return None if t is None else t.double().cpu().numpy()


def _check(logits, u, temperature=None, top_k=None, top_p=None, min_p=None):
    got = ssc.sample_rows(logits, u, temperature, top_k, top_p, min_p)
    torch.cuda.synchronize()
    tokens, kept, logprobs = sample(_np(logits), _np(u), _np(temperature), _np(top_k), _np(top_p), _np(min_p))
    assert np.array_equal(got[1].cpu().numpy(), kept), np.flatnonzero(got[1].cpu().numpy() != kept)
    assert np.array_equal(got[0].cpu().numpy(), tokens), np.flatnonzero(got[0].cpu().numpy() != tokens)
    lp = got[2].double().cpu().numpy()
    none = tokens < 0
    assert np.all(lp[none] == -np.inf)
    vocab = logits.shape[1]
    bits = min(62 - vocab.bit_length(), 50)
    tol = 2.0 ** -24 * np.abs(logprobs[~none]) + vocab * 2.0 ** -(bits + 1) + 2.0 ** -45
    assert np.all(np.abs(lp[~none] - logprobs[~none]) <= tol)
    return got


def _inputs(seed, rows, vocab, dtype, spread=2.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    rand = lambda *s: torch.rand(*s, device=DEV, generator=g)  # noqa: E731
    logits = (torch.randn(rows, vocab, device=DEV, generator=g) * spread).to(dtype)
    return logits, rand(rows), rand


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("vocab", [1, 2, 7, 9, 63, 1000, 4095, 4097, 16384, 16385, 50_001, 131_072])
def test_settings_of_each_kind(dtype, vocab):
    rows = 9
    logits, u, rand = _inputs(vocab, rows, vocab, dtype)
    t = 0.4 + rand(rows)
    k = (1 + rand(rows) * min(vocab, 300)).int()
    p = 0.3 + 0.69 * rand(rows)
    m = 0.2 * rand(rows)
    _check(logits, u)
    _check(logits, u, t)
    _check(logits, u, top_k=k)
    _check(logits, u, t, None, p)
    _check(logits, u, t, None, None, m)
    _check(logits, u, t, k, p)
    t[0] = 0.0
    k[1] = 0
    p[2] = 1.0
    _check(logits, u, t, k, p, m)


@pytest.mark.parametrize("dtype", TYPES)
def test_many_rows(dtype):
    logits, u, rand = _inputs(77, 130, 5003, dtype, 4.0)
    _check(logits, u, 0.2 + 2 * rand(130), (rand(130) * 100).int(), rand(130), 0.1 * rand(130))


@pytest.mark.parametrize("dtype", TYPES)
def test_ties_and_borders(dtype):
    """Rows of few values: the cut falls among equal logits, and the ones
    with the lowest indexes are kept; powers of two as weights make every
    border exact on both sides."""
    vocab, rows = 9001, 12
    g = torch.Generator(device=DEV)
    g.manual_seed(4)
    logits = torch.randint(0, 3, (rows, vocab), device=DEV, generator=g).to(dtype)
    u = torch.rand(rows, device=DEV, generator=g)
    k = torch.tensor([1, 2, 100, 2999, 3000, 3001, 5000, 8999, 9000, 9001, 9002, 0], device=DEV, dtype=torch.int32)
    p = torch.linspace(0.05, 1.0, rows, device=DEV)
    _check(logits, u, top_k=k)
    _check(logits, u, top_p=p)
    _check(logits, u, None, k, p)
    flat = torch.zeros(rows, vocab, device=DEV, dtype=dtype)
    _check(flat, u, None, k, p)
    _check(flat, u, top_p=torch.full((rows,), 0.5, device=DEV))
    _check(flat, u, min_p=torch.ones(rows, device=DEV))
    _check(flat, torch.linspace(0, 1, rows, device=DEV), top_k=k)
    signed = torch.where(torch.rand(rows, vocab, device=DEV, generator=g) < 0.5, -0.0, 0.0).to(dtype)
    _check(signed, u, top_k=k)


@pytest.mark.parametrize("dtype", TYPES)
def test_masked_and_special_logits(dtype):
    vocab = 5000
    logits, u, _ = _inputs(9, 14, vocab, dtype)
    inf = float("inf")
    logits[0] = -inf                        # nothing left
    logits[1] = float("nan")
    logits[2, 1:] = -inf                    # one token
    logits[3, :-1] = -inf
    logits[4, ::2] = float("nan")
    logits[5, 17] = inf
    logits[6, [5, 4999, 1234]] = inf
    logits[7] = torch.finfo(dtype).min      # a mask of the lowest finite value, everywhere
    logits[8, 100:] = torch.finfo(dtype).min
    logits[9, :4990] = -inf
    logits[10] = inf
    logits[11] = torch.finfo(dtype).max
    for kw in ({}, {"top_k": 3}, {"top_k": 40}, {"top_p": 0.9}, {"min_p": 0.05}, {"temperature": 0.0},
               {"temperature": 1e-3}, {"temperature": 1e30}, {"temperature": inf}, {"temperature": float("nan")},
               {"temperature": -1.0}, {"top_k": 2, "top_p": 0.5, "min_p": 0.3},
               {"temperature": 1e-40, "top_p": 0.9}):
        args = {k: torch.full((14,), v, device=DEV, dtype=torch.int32 if k == "top_k" else torch.float32)
                for k, v in kw.items()}
        _check(logits, u, **args)


def test_settings_out_of_range():
    logits, u, _ = _inputs(3, 6, 1000, torch.float32)
    nan, inf = float("nan"), float("inf")
    f = lambda *v: torch.tensor(v, device=DEV)  # noqa: E731
    _check(logits, f(-1.0, 1.0, 2.0, nan, inf, -inf))
    _check(logits, u, top_p=f(0.0, -1.0, nan, 1.0, 2.0, inf))
    _check(logits, u, min_p=f(0.0, -1.0, nan, 1.0, 2.0, inf))
    _check(logits, u, top_k=torch.tensor([0, -1, -2 ** 31, 2 ** 31 - 1, 1000, 999], device=DEV, dtype=torch.int32))
    _check(logits, torch.full((6,), 1 - 2.0 ** -24, device=DEV))
    _check(logits, torch.zeros(6, device=DEV), top_p=torch.full((6,), 2.0 ** -24, device=DEV))


@pytest.mark.parametrize("dtype", TYPES)
def test_concentrated_logits(dtype):
    """All logits in a few bins of the first histogram, and one bin alone."""
    logits, u, rand = _inputs(5, 8, 40_000, dtype, 1e-3)
    logits = logits + 1.0
    _check(logits, u, None, (rand(8) * 20_000).int(), 0.1 + 0.8 * rand(8))
    _check(logits.abs() * 1e4, u, None, (rand(8) * 20_000).int(), 0.1 + 0.8 * rand(8))


def test_strided_rows_and_unaligned():
    """The last position's logits of (batch, length, vocab), and rows that
    start at odd elements."""
    g = torch.Generator(device=DEV)
    g.manual_seed(2)
    full = torch.randn(5, 3, 1003, device=DEV, generator=g).to(torch.bfloat16)
    u = torch.rand(5, device=DEV, generator=g)
    p = torch.full((5,), 0.8, device=DEV)
    last = full[:, -1]
    assert not last.is_contiguous()
    got = _check(last, u, top_p=p)
    again = ssc.sample_rows(last.contiguous(), u, top_p=p)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    _check(full[0, :, 1:1000], u[:3], top_p=p[:3])


def test_the_distribution_of_the_tokens():
    """Over evenly spread u the tokens come as often as their weights say:
    each cumulative share is met within one step of u."""
    g = torch.Generator(device=DEV)
    g.manual_seed(11)
    n, vocab = 4096, 40
    row = torch.randn(vocab, device=DEV, generator=g)
    logits = row.expand(n, vocab).contiguous()
    u = (torch.arange(n, device=DEV) / n).float()
    tokens, _, _ = ssc.sample_rows(logits, u)
    share = torch.softmax(row.double(), 0)
    freq = torch.bincount(tokens.long(), minlength=vocab).double() / n
    assert bool(((freq.cumsum(0) - share.cumsum(0)).abs() <= 1.01 / n).all())


def test_outputs_repeat_and_stay_in_place():
    logits, u, rand = _inputs(13, 20, 70_000, torch.float32)
    t, k, p = 0.5 + rand(20), (rand(20) * 1000).int(), rand(20)
    buf = torch.full((3, 32), -9, dtype=torch.int32, device=DEV)
    first = None
    scratch = torch.full((ssc.sample_scratch_bytes(20, 70_000),), 255, dtype=torch.uint8, device=DEV)
    for _ in range(5):
        lp = buf[2, 6:26].view(torch.float32)
        got = ssc.sample_rows(logits, u, t, k, p, tokens=buf[0, 6:26], kept=buf[1, 6:26], logprobs=lp, scratch=scratch)
        now = [x.clone() for x in got]
        first = first or now
        assert all(torch.equal(a, b) for a, b in zip(first, now))
    assert bool((buf[:, :6] == -9).all()) and bool((buf[:, 26:] == -9).all())


def test_graph_replays_and_streams():
    logits, u, rand = _inputs(14, 8, 33_000, torch.bfloat16)
    t, k, p, m = 0.5 + rand(8), (rand(8) * 50).int(), rand(8), 0.01 * rand(8)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ssc.sample_rows(logits, u, t, k, p, m)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = ssc.sample_rows(logits, u, t, k, p, m)
    for i in range(4):
        logits.copy_(logits.roll(i + 1, 1))
        u.copy_(u.flip(0))
        graph.replay()
        torch.cuda.synchronize()
        eager = _check(logits, u, t, k, p, m)
        assert all(torch.equal(a, b) for a, b in zip(captured, eager))


@pytest.mark.parametrize("dtype", TYPES)
def test_equal_small_weights(dtype):
    """Thousands of weights that are all rounded alike, beside one of 1: the
    logprob of the large one is as small as their sum."""
    for vocab, low in ((131_072, -25.0), (36_917, -20.0), (4097, -30.0)):
        logits = torch.full((2, vocab), low, device=DEV, dtype=dtype)
        logits[0, 7] = 0.0
        logits[1, vocab - 1] = 0.0
        u = torch.tensor([0.5, 0.5], device=DEV)
        _check(logits, u)
        _check(logits, u, top_p=torch.tensor([1.0, 0.999], device=DEV))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_largest_vocabulary(dtype):
    vocab = 2 ** 22
    logits, u, rand = _inputs(22, 2, vocab, dtype, 1.5)
    _check(logits, u)
    _check(logits, u, top_k=torch.tensor([100, 3_000_000], dtype=torch.int32, device=DEV))
    _check(logits, u, 0.5 + rand(2), None, torch.tensor([0.3, 0.95], device=DEV), torch.tensor([0.0, 1e-4], device=DEV))


def test_most_rows():
    """65,535 rows, more than 2^32 logits in all, against some of the rows alone."""
    rows, vocab = 65_535, 66_001
    if torch.cuda.mem_get_info()[0] < 40 * 2 ** 30:
        pytest.skip("needs 40 GB of device memory")
    logits, u, rand = _inputs(23, rows, vocab, torch.bfloat16)
    t, k, p = 0.5 + rand(rows), (rand(rows) * 100).int(), 0.5 + 0.6 * rand(rows)
    tokens, kept, logprobs = ssc.sample_rows(logits, u, t, k, p)
    some = torch.tensor([0, 1, 32_767, 65_074, 65_075, 65_533, 65_534], device=DEV)
    got = _check(logits[some], u[some], t[some], k[some], p[some])
    assert torch.equal(got[0], tokens[some]) and torch.equal(got[1], kept[some]) and torch.equal(got[2], logprobs[some])
    assert bool(((tokens >= 0) & (tokens < vocab)).all())


def test_two_calls_at_once():
    """Calls in flight on two streams, each with a scratch of its own."""
    inputs, want = [], []
    for i in range(2):
        logits, u, rand = _inputs(40 + i, 24, 70_001, torch.bfloat16)
        inputs.append((logits, u, 0.5 + rand(24), (rand(24) * 90).int(), 0.5 + 0.6 * rand(24)))
        want.append([x.clone() for x in _check(*inputs[i])])
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    scratch = [torch.empty(ssc.sample_scratch_bytes(24, 70_001), dtype=torch.uint8, device=DEV) for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(8):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(ssc.sample_rows(*inputs[i], scratch=scratch[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(g, want[i]))


def test_sampled_tokens_feed_the_lookup():
    """A decoding step: the sampled ids, -1 for a row without tokens, go
    straight into the embedding lookup."""
    logits, u, _ = _inputs(15, 6, 300, torch.float32)
    logits[3] = -float("inf")
    tokens, kept, _ = ssc.sample_rows(logits, u)
    table = torch.randn(300, 64, device=DEV)
    out = ssc.embed_rows(table, tokens)
    assert int(tokens[3]) == -1 and int(kept[3]) == 0 and bool((out[3] == 0).all())
    live = [0, 1, 2, 4, 5]
    assert torch.equal(out[live], table[tokens[live].long()])


def test_refusals_on_the_gpu():
    x = torch.zeros(4, 100, device=DEV)
    u = torch.zeros(4, device=DEV)
    with pytest.raises(TypeError):
        ssc.sample_rows(x.double(), u)
    with pytest.raises(ValueError):
        ssc.sample_rows(x.t(), u)
    with pytest.raises(ValueError):
        ssc.sample_rows(x[:1].expand(4, 100), u)  # rows over one another
    with pytest.raises(ValueError):
        ssc.sample_rows(x, u[:3])
    with pytest.raises(TypeError):
        ssc.sample_rows(x, u, top_k=u)
    with pytest.raises(TypeError):
        ssc.sample_rows(x, u, 0.7)
    with pytest.raises(ssc.SSCError):
        ssc.sample_rows(torch.zeros(4, 0, device=DEV), u)
    with pytest.raises(ssc.SSCError):
        ssc.sample_rows(x, u, logprobs=u)
    with pytest.raises(ssc.SSCError):
        ssc.sample_rows(torch.zeros(1, 2 ** 22 + 1, device=DEV), u[:1])
    assert ssc.sample_rows(x[:0], u[:0])[0].numel() == 0


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("seed", range(4))
def test_rows_of_few_values(dtype, seed):
    """More equal logits at the border than are collected, beside settings that cut them."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    rows, vocab = 5, (9000, 20_001, 60_000)[seed % 3]
    logits = (torch.randint(-4, 3, (rows, vocab), device=DEV, generator=g) * (1.0, 0.37, 3.1)[seed % 3]).to(dtype)
    u, t, p = (torch.rand(rows, device=DEV, generator=g) for _ in range(3))
    k = torch.randint(0, vocab, (rows,), device=DEV, generator=g).int()
    _check(logits, u, top_k=k)
    _check(logits, u, top_p=p)
    _check(logits, u, 0.3 + t, k, p)
