"""Edges of the token-path calls on the GPU: what include/ssc.h says of
settings, positions and buffers that ordinary programs do not meet."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import scan_stream_compaction_amd as ssc
from tests.token_inputs import BLOCK_CASES, BLOCK_WIDTH, EQUAL_ROWS, block_case, group_sums

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = [torch.float32, torch.bfloat16, torch.float16]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("vocab", [2, 100, 9001, 40_000])
def test_min_p_above_one_keeps_the_first_alone(dtype, vocab):
    """No weight reaches a min_p above 1, and the first of the order is always
    kept: one token, also where many logits equal the largest (more than are
    collected, in the longer rows). A min_p of 1 keeps all of those."""
    inf = float("inf")
    logits = torch.zeros(5, vocab, device=DEV, dtype=dtype)
    logits[1, 0] = -1.0
    logits[2, : vocab - 2] = -3.0
    logits[3, vocab // 2:] = inf
    logits[4, 0] = float("nan")
    first = torch.tensor([0, 1, vocab - 2, vocab // 2, 1], device=DEV)
    equal = torch.tensor([vocab, vocab - 1, 2, vocab - vocab // 2, vocab - 1], device=DEV)
    u = torch.tensor([0.99, 0.99, 0.6, 0.99, 0.99], device=DEV)
    def row(v, dt=torch.float32):
        return torch.full((5,), v, device=DEV, dtype=dt)
    for extra in ({}, {"temperature": row(0.7)}, {"top_k": row(3000, torch.int32)}, {"top_k": row(50, torch.int32)},
                  {"top_p": row(0.9)}, {"temperature": row(inf), "top_k": row(2500, torch.int32), "top_p": row(0.5)}):
        for min_p in (float(np.nextafter(np.float32(1), np.float32(2))), 1.5, inf):
            tokens, kept, logprobs = ssc.sample_rows(logits, u, min_p=row(min_p), **extra)
            assert torch.equal(tokens.long(), first) and bool((kept == 1).all()) and bool((logprobs == 0).all())
    tokens, kept, logprobs = ssc.sample_rows(logits, u, min_p=row(1.0))
    assert torch.equal(kept.long(), equal)


def _small_integers(g, *shape, dtype=torch.float32):
    """Whole numbers of [-3, 3], whose sums are exact in fp32 up to 2^24."""
    return torch.randint(-3, 4, shape, device=DEV, generator=g).to(dtype)


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


@pytest.mark.parametrize("fill", [0, 7, -1, 2 ** 31 - 1])
def test_larger_buffers_for_a_grouping(fill):
    """order, ranks and offsets in buffers that are larger than needed, filled
    with anything: what is returned is the result alone, in its shape, and the
    calls that take it on do not meet the rest."""
    g = _gen(51)
    n, vocab, width = 5000, 300, 24
    ids = torch.randint(-1, vocab, (n // 4, 4), device=DEV, generator=g)
    dout = _small_integers(g, n // 4, 4, width, dtype=torch.bfloat16)
    want = torch.zeros(vocab + 1, width, device=DEV).index_add_(0, ids.view(-1) % (vocab + 1), dout.view(n, width).float())[:-1]
    worder, wranks, woffsets = ssc.group_by_key(ids, vocab)

    def buffer(size):
        return torch.full((size,), fill, dtype=torch.int32, device=DEV)
    buf = buffer(2000)
    order, ranks, offsets = ssc.group_by_key(ids, vocab, order=buffer(9000), ranks=buffer(9000), offsets=buf)
    assert order.shape == (n,) and ranks.shape == ids.shape and offsets.shape == (vocab + 1,)
    kept = int(offsets[-1])
    assert torch.equal(order[:kept], worder[:kept]) and torch.equal(ranks, wranks) and torch.equal(offsets, woffsets)
    assert bool((buf[vocab + 1:] == fill).all()) and offsets.data_ptr() == buf.data_ptr()
    for kw in ({"offsets": offsets}, {"offsets": buf, "vocab": vocab}):
        grad = ssc.embed_rows_grad(dout, ids, order, dtype=torch.float32, **kw)
        assert grad.shape == (vocab, width) and torch.equal(grad, want)
    # rows there and back by ranks out of a larger buffer
    x = _small_integers(g, n // 4, width)
    back = ssc.dispatch_rows_grad(ssc.dispatch_rows(x, ranks), ranks)
    assert torch.equal(back, x * (ids >= 0).sum(1, keepdim=True))
    # a tensor of the right shape is returned as it is
    assert ssc.group_by_key(ids, vocab, offsets=offsets)[2] is offsets
    with pytest.raises(ValueError):
        ssc.embed_rows_grad(dout, ids, order, offsets, vocab=vocab + 1)
    with pytest.raises(ValueError):
        ssc.embed_rows_grad(dout, ids, order, offsets, vocab=0)


def test_larger_buffers_for_rows_and_tokens():
    """Outputs in larger buffers come back as the result alone, in its shape:
    the tokens of a step, say, that the lookup takes next."""
    g = _gen(52)
    rows, vocab, width, experts, per = 5, 200, 16, 6, 2
    logits = _small_integers(g, rows, vocab)
    u = torch.rand(rows, device=DEV, generator=g)
    table = _small_integers(g, vocab, width)

    def buffer(dtype):
        return torch.full((4000,), 3, dtype=dtype, device=DEV)
    i32, f32 = torch.int32, torch.float32
    bufs = [buffer(i32), buffer(i32), buffer(f32)]
    got = ssc.sample_rows(logits, u, tokens=bufs[0], kept=bufs[1], logprobs=bufs[2])
    for a, b, buf in zip(got, ssc.sample_rows(logits, u), bufs):
        assert torch.equal(a, b) and a.data_ptr() == buf.data_ptr() and bool((buf[rows:] == 3).all())
    tokens = got[0]
    out = buffer(f32)
    x = ssc.embed_rows(table, tokens.view(rows, 1), out=out)
    assert x.shape == (rows, 1, width) and torch.equal(x[:, 0], table[tokens.long()]) and bool((out[x.numel():] == 3).all())
    x = x.view(rows, width)
    _, ranks, _ = ssc.group_by_key(torch.randint(0, experts, (rows, per), device=DEV, generator=g), experts)
    y = ssc.dispatch_rows(x, ranks)
    w = _small_integers(g, rows, per)
    back = ssc.combine_rows(y, ranks, w, out=buffer(f32))
    assert back.shape == (rows, width) and torch.equal(back, x * w.sum(1, keepdim=True))
    dy, dw = ssc.combine_rows_grad(x, y, ranks, w, dy=buffer(f32), dweights=buffer(f32))
    want = ssc.combine_rows_grad(x, y, ranks, w)
    assert dy.shape == y.shape and dw.shape == w.shape and torch.equal(dy, want[0]) and torch.equal(dw, want[1])
    order, _, offsets = ssc.group_by_key(tokens, vocab)
    grad = ssc.embed_rows_grad(x, tokens, order, offsets, out=buffer(f32))
    assert grad.shape == (vocab, width) and torch.equal(grad, ssc.embed_rows_grad(x, tokens, order, offsets))
    # a tensor of the right shape is returned as it is
    assert ssc.embed_rows(table, tokens, out=x) is x and ssc.combine_rows(y, ranks, w, out=back) is back


@pytest.mark.parametrize("n,vocab", [(256, 1), (4999, 3), (70_001, 2), (300_007, 3)])
def test_embed_grad_of_positions_outside(n, vocab):
    """Positions outside [0, n) add nothing, also where they begin or end a
    block of 16, 256 or 4096 sorted tokens whose sum is made first; and where
    the last offset cuts ranges short, nothing is taken from sums that were
    not made. The scratch holds NaN before each call."""
    g = _gen(n)
    width = 24
    ids = torch.randint(0, vocab, (n,), device=DEV, generator=g)
    dout = _small_integers(g, n, width, dtype=torch.bfloat16)
    order, _, offsets = ssc.group_by_key(ids, vocab, ranks=False)
    size = ssc.lib().ssc_embed_grad_scratch_bytes(n, width)

    def check(order, offsets):
        group = torch.bucketize(torch.arange(n, device=DEV), offsets[1:].long(), right=True).clamp(max=vocab)
        inside = (order >= 0) & (order < n) & (group < vocab)
        rows = dout.float()[order.long().clamp(0, n - 1)] * inside[:, None]
        want = torch.zeros(vocab + 1, width, device=DEV).index_add_(0, group, rows)[:-1]
        scratch = torch.full((size,), 255, dtype=torch.uint8, device=DEV)
        got = ssc.embed_rows_grad(dout, ids, order, offsets, 0.5, dtype=torch.float32, scratch=scratch)
        assert torch.equal(got, want * 0.5)
    check(order, offsets)
    for outside in (-1, n, 2 ** 31 - 1, -2 ** 31):
        for at in (torch.arange(0, n, 16), torch.arange(15, n, 16), torch.arange(0, n, 4096), torch.arange(255, n, 256),
                   torch.randint(0, n, (n // 5,))):
            bad = order.clone()
            bad[at.to(DEV)] = outside
            check(bad, offsets)
    check(torch.full_like(order, n), offsets)
    for last in (0, int(offsets[-1]) - 100):
        cut = offsets.clamp(max=last)
        check(order, cut)
        if vocab > 1:  # the last offset alone: earlier rows reach past it
            cut = offsets.clone()
            cut[-1] = last
            scratch = torch.full((size,), 255, dtype=torch.uint8, device=DEV)
            got = ssc.embed_rows_grad(dout, ids, order, cut, 0.5, dtype=torch.float32, scratch=scratch)
            assert torch.equal(got, ssc.embed_rows_grad(dout, ids, order, cut.clamp(max=last), 0.5, dtype=torch.float32))


@pytest.mark.parametrize("n,vocab,hot", BLOCK_CASES)
def test_embed_grad_block_sums_exactly(n, vocab, hot):
    """Sums through every level of blocks, of whole numbers that fp32 holds:
    equal to the last bit, whatever the order, with a power of two as scale."""
    ids, rows = block_case(n, vocab, hot)
    want = torch.from_numpy(group_sums(ids, rows, vocab)).to(DEV).double() * 0.25
    ids = torch.from_numpy(ids).to(DEV)
    order, _, offsets = ssc.group_by_key(ids, vocab, ranks=False)
    for dtype in TYPES:
        dout = torch.from_numpy(rows).to(DEV).to(dtype)
        grad = ssc.embed_rows_grad(dout, ids, order, offsets, 0.25, dtype=torch.float32)
        assert torch.equal(grad.double(), want)
        if dtype is not torch.float16:  # whose range the sums may leave
            base = torch.ones(vocab, BLOCK_WIDTH, dtype=torch.float32, device=DEV)
            assert torch.equal(ssc.embed_rows_grad(dout, ids, order, offsets, 0.25), want.to(dtype))
            ssc.embed_rows_grad(dout, ids, order, offsets, 0.25, out=base, accumulate=True)
            assert torch.equal(base.double(), want + 1)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("vocab", sorted({c[0] for c in EQUAL_ROWS}))
def test_equal_weights_meet_the_border(dtype, vocab):
    """top_p times the sum is met exactly by the running weight of equal
    logits: the token at the border is not kept, in rows whose border logits
    are collected and in rows that have more of them. u at exact borders, too."""
    cases = [c for c in EQUAL_ROWS if c[0] == vocab]
    logits = torch.full((len(cases), vocab), 0.5, device=DEV, dtype=dtype)
    for r, (_, step, *_) in enumerate(cases):
        logits[r, torch.arange(vocab, device=DEV) % step != 0] = float("-inf")
    step, k, p, kept = (torch.tensor([c[i] for c in cases], device=DEV) for i in (1, 2, 3, 4))
    p = p.float()
    for j in (torch.zeros_like(kept), torch.ones_like(kept), kept // 2, kept - 1):
        # u in fp32 may lie below j / kept by a step: the token before is then the first past it
        u = (j.double() / kept).float()
        want = (u.double() * kept).floor().long() * step
        tokens, count, logprobs = ssc.sample_rows(logits, u, top_k=k.int(), top_p=p)
        assert torch.equal(count.long(), kept) and torch.equal(tokens.long(), want)
        lp = -kept.double().log()
        assert bool(((logprobs.double() - lp).abs() <= 2.0 ** -24 * lp.abs() + 2.0 ** -45).all())
    up = torch.nextafter(p, torch.ones_like(p))
    _, count, _ = ssc.sample_rows(logits, torch.zeros(len(cases), device=DEV), top_k=k.int(), top_p=up)
    assert torch.equal(count.long(), kept + 1)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("chunks,extra", [(65, 0), (65, 1), (129, 3), (200, 0), (256, 0), (256, 1)])
@pytest.mark.parametrize("vocab", [65_535, 65_536])
def test_embed_grad_of_larger_tables(vocab, dtype, chunks, extra):
    """Tables on both sides of the size from which half the threads take two
    chunks of a row each, with a last chunk that starts early; ids that occur
    often, once and never, and rows added to what is there."""
    width = chunks * (16 // torch.empty(0, dtype=dtype).element_size()) - extra
    g = _gen(width)
    n = 1500
    ids = (torch.rand(n, device=DEV, generator=g) ** 8 * (vocab + 1)).long() - 1
    ids[::50] = vocab - 1
    dout = _small_integers(g, n, width, dtype=dtype)
    order, _, offsets = ssc.group_by_key(ids, vocab, ranks=False)
    inside = ids >= 0
    want = torch.zeros(vocab, width, device=DEV).index_add_(0, ids[inside], dout[inside].float())
    assert torch.equal(ssc.embed_rows_grad(dout, ids, order, offsets, dtype=torch.float32), want)
    assert torch.equal(ssc.embed_rows_grad(dout, ids, order, offsets, 0.5), (want * 0.5).to(dtype))
    base = torch.ones(vocab, width, device=DEV)
    assert torch.equal(ssc.embed_rows_grad(dout, ids, order, offsets, out=base, accumulate=True), want + 1)
