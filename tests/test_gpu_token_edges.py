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
