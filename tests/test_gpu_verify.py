"""ssc_verify_rows on the GPU against the definition in 64 bits. Results are
whole numbers and equal: products of two fp32 values and differences of values
whose exponents lie within 29 bits of each other are exact in fp64, and sums of
both sides differ by some 2^-50, which a random u lies within of one of 131,072
borders once in 2^32 rows."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import scan_stream_compaction_amd as ssc

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = [torch.float32, torch.bfloat16, torch.float16]


def reference(probs, drafted, u, draft_probs=None, lengths=None):
    p = probs.double().cpu().numpy()
    x = drafted.cpu().numpy().astype(np.int64)
    r = np.nan_to_num(u.double().cpu().numpy(), nan=0.0, posinf=2.0, neginf=-1.0).clip(0.0, 1.0 - 2.0 ** -24)
    q = None if draft_probs is None else draft_probs.double().cpu().numpy()
    rows, places, vocab = p.shape
    drafts = places - 1
    tokens = np.full((rows, places), -1, np.int64)
    accepted = np.zeros(rows, np.int64)
    weigh = lambda w: np.where((w > 0) & np.isfinite(w), w, 0.0)  # noqa: E731
    for b in range(rows):
        length = drafts if lengths is None else min(max(int(lengths[b]), 0), drafts)
        a = 0
        while a < length:
            t = x[b, a]
            if not (0 <= t < vocab and r[b, a] * (1.0 if q is None else q[b, a, t]) < p[b, a, t]):
                break
            tokens[b, a] = t
            a += 1
        w = weigh(p[b, a])
        if a < length:
            with np.errstate(invalid="ignore"):
                if q is not None:
                    rest = weigh(p[b, a] - q[b, a])
                else:
                    rest = w.copy()
                    if 0 <= x[b, a] < vocab:
                        rest[x[b, a]] = 0.0
            if rest.sum() > 0:
                w = rest
        run = np.cumsum(w)
        if run[-1] > 0:
            at = int(np.searchsorted(run, r[b, drafts] * run[-1], side="right"))
            tokens[b, a] = min(at, np.flatnonzero(w > 0)[-1])
        accepted[b] = a
    return tokens, accepted


def check(probs, drafted, u, draft_probs=None, lengths=None):
    got = ssc.verify_rows(probs, drafted, u, draft_probs, lengths=lengths)
    torch.cuda.synchronize()
    tokens, accepted = reference(probs, drafted, u, draft_probs, lengths)
    assert np.array_equal(got[1].cpu().numpy(), accepted)
    assert np.array_equal(got[0].cpu().numpy(), tokens), np.argwhere(got[0].cpu().numpy() != tokens)[:5]
    return got


def inputs(seed, rows, drafts, vocab, dtype, near=0.5, ids=torch.int32):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    logits = torch.randn(rows, drafts + 1, vocab, device=DEV, generator=g) * 2
    q = torch.softmax(logits[:, :drafts], 2)
    race = -torch.log(torch.rand(rows, drafts, vocab, device=DEV, generator=g).clamp_(1e-20, 1 - 1e-7))
    drafted = (q / race).argmax(2).to(ids)
    p = torch.softmax(logits + near * torch.randn(logits.shape, device=DEV, generator=g), 2)
    u = torch.rand(rows, drafts + 1, device=DEV, generator=g)
    return p.to(dtype), drafted, u, q.to(dtype), g


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("vocab", [1, 2, 7, 9, 1000, 1023, 1024, 1025, 4097, 50_001, 65_536, 65_537, 131_072])
@pytest.mark.parametrize("drafts", [1, 4])
def test_sizes(drafts, vocab, dtype):
    p, x, u, q, g = inputs(vocab + drafts, 13, drafts, vocab, dtype, ids=torch.int64 if vocab % 2 else torch.int32)
    check(p, x, u, q)
    check(p, x, u)
    lengths = torch.randint(-1, drafts + 2, (13,), device=DEV, generator=g).int()
    check(p, x, u, q, lengths)
    check(p, x, u, None, lengths)


@pytest.mark.parametrize("drafts", [0, 2, 63, 64, 65, 200])
def test_numbers_of_drafts(drafts):
    """p and q alike, so that many drafts stand."""
    p, x, u, q, _ = inputs(drafts, 9, drafts, 50, torch.float32, near=0.02)
    got = check(p, x, u, q if drafts else None)
    assert drafts == 0 or int(got[1].max()) > 0
    u[:, :-1] = 0
    assert bool((check(p, x, u, q if drafts else None)[1] == drafts).all())


@pytest.mark.parametrize("dtype", TYPES)
def test_the_largest_vocabulary(dtype):
    p, x, u, q, _ = inputs(3, 2, 1, 2 ** 22, dtype)
    check(p, x, u, q)


@pytest.mark.parametrize("rows,vocab", [(65_535, 5), (159, 70_000), (160, 70_000)])
def test_many_rows(rows, vocab):
    p, x, u, q, _ = inputs(4, rows, 2, vocab, torch.float32)
    check(p, x, u, q)


def test_borders_met_exactly():
    """Equal weights of powers of two, u on each of their borders: the next token."""
    vocab, n = 4096, 64
    p = torch.full((n, 2, vocab), 1.0 / vocab, device=DEV)
    q = torch.zeros(n, 1, vocab, device=DEV)
    x = torch.zeros(n, 1, dtype=torch.int32, device=DEV)
    q[:, 0, 0] = 1.0
    u = torch.stack([torch.full((n,), 0.5, device=DEV), torch.arange(n, device=DEV) / n], 1)
    got = check(p, x, u)  # drafted without chance: 1/4096 > u fails
    assert bool((got[1] == 0).all())
    u[:, 0] = 0.0
    got = check(p, x, u, q)
    assert torch.equal(got[0][:, 1], torch.arange(n, device=DEV).int() * (vocab // n))
    # u q = p falls, a step below stands
    p2, q2 = torch.full((2, 2, 4), 0.25, device=DEV), torch.full((2, 1, 4), 0.5, device=DEV)
    u2 = torch.tensor([[0.5, 0.3], [0.5 - 2.0 ** -25, 0.3]], device=DEV)
    assert check(p2, x[:2], u2, q2)[1].tolist() == [0, 1]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("vocab", [3000, 70_000])
def test_rows_that_leave_nothing_and_special_values(vocab, dtype):
    inf, nan = float("inf"), float("nan")
    p, x, u, q, _ = inputs(5, 16, 2, vocab, dtype)
    u[:, 0] = 0.9999999
    p[0] = 0
    p[1] = nan
    p[2] = q[2, :1]                       # nothing left above q, the draft falls: p draws
    x[2, 0] = int(p[2, 0].argmin())
    q[3] = 1.0                            # q covers p
    p[4, :, ::2] = nan
    p[5, :, 7] = inf
    p[6] = -1.0
    q[7, :, 100:] = nan
    q[8] = inf
    x[9] = -1
    x[10] = vocab
    x[11] = 2 ** 31 - 1
    x[12] = -2 ** 31
    p[13, :, :-1] = 0
    p[14, :, 1:] = 0
    for given in (q, None):
        check(p, x, u, given)
        check(p, x, torch.zeros_like(u), given)
    u[:6, 0] = torch.tensor([nan, inf, -inf, -1.0, 1.0, 2.0], device=DEV)
    u[6:12, 2] = torch.tensor([nan, inf, -inf, -1.0, 1.0, 2.0], device=DEV)
    check(p, x, u, q)
    check(p, x, u, q, torch.zeros(16, dtype=torch.int32, device=DEV))


def test_the_distribution_of_the_tokens():
    """Every draft by its share of q, u over an even grid: the first token comes as p says."""
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    vocab, m = 6, 128
    p, q = (torch.softmax(torch.randn(vocab, device=DEV, generator=g), 0) for _ in range(2))
    grid = (torch.arange(m, device=DEV) + 0.5) / m
    share = torch.zeros(vocab, dtype=torch.float64, device=DEV)
    for x in range(vocab):
        n = m * m
        u = torch.stack([grid.repeat_interleave(m), grid.repeat(m)], 1).contiguous()
        tokens, _ = ssc.verify_rows(p.expand(n, 2, vocab), torch.full((n, 1), x, device=DEV), u, q.expand(n, 1, vocab))
        share += q[x].double() * torch.bincount(tokens[:, 0].long(), minlength=vocab).double() / n
    # each of the two borders of a draft is met within one step of its grid
    assert bool(((share - p.double()).abs() <= 2.0 / m).all())


@pytest.mark.parametrize("vocab", [1003, 66_001])
def test_strides_outputs_and_repeats(vocab):
    p, x, u, q, g = inputs(6, 7, 3, vocab, torch.bfloat16)
    wide = torch.zeros(7, 9, vocab + 97, device=DEV, dtype=torch.bfloat16)
    wide[:, 1:8:2, 13:vocab + 13] = p
    qt = torch.zeros(3, 7, vocab, device=DEV, dtype=torch.bfloat16).copy_(q.transpose(0, 1)).transpose(0, 1)
    view = wide[:, 1:8:2, 13:vocab + 13]
    assert not view.is_contiguous() and not qt.is_contiguous()
    want = check(p, x, u, q)
    buf = torch.full((2, 40), -9, dtype=torch.int32, device=DEV)
    scratch = torch.full((ssc.verify_scratch_bytes(7, vocab),), 255, dtype=torch.uint8, device=DEV)
    for _ in range(3):
        got = ssc.verify_rows(view, x, u, qt, tokens=buf[0, 5:33], accepted=buf[1, 5:12], scratch=scratch)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert bool((buf[0, :5] == -9).all()) and bool((buf[0, 33:] == -9).all()) and bool((buf[1, 12:] == -9).all())
    empty = ssc.verify_rows(p[:0], x[:0], u[:0], q[:0])
    assert empty[0].shape == (0, 4) and empty[1].shape == (0,)


@pytest.mark.parametrize("vocab", [5000, 70_000])
def test_graph_replays_and_streams(vocab):
    p, x, u, q, g = inputs(7, 20, 4, vocab, torch.float32)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ssc.verify_rows(p, x, u, q)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = ssc.verify_rows(p, x, u, q)
    for _ in range(4):
        u.copy_(torch.rand(20, 5, device=DEV, generator=g))
        graph.replay()
        torch.cuda.synchronize()
        eager = check(p, x, u, q)
        assert torch.equal(got[0], eager[0]) and torch.equal(got[1], eager[1])


def test_two_calls_at_once():
    ins = [inputs(40 + i, 30, 3, 70_000, torch.bfloat16)[:4] for i in range(2)]
    want = [ssc.verify_rows(*a) for a in ins]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ins]
    got = []
    for _ in range(5):
        for a, s in zip(ins, streams):
            with torch.cuda.stream(s):
                got.append(ssc.verify_rows(*a))
    torch.cuda.synchronize()
    for i, r in enumerate(got):
        assert torch.equal(r[0], want[i % 2][0]) and torch.equal(r[1], want[i % 2][1])
