"""Edges of the token-path calls on the GPU: what include/ssc.h says of
settings, positions and buffers that ordinary programs do not meet."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import scan_stream_compaction_amd as ssc

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
