"""Host-side checks of the token-path calls, without a GPU: every refusal
comes before HIP is touched (the addresses here are never read), the scratch
sizes, the binding's refusal of CPU tensors, and the sampling reference."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import scan_stream_compaction_amd as ssc
from tests.sample_reference import sample_row

ARG, SIZE, ALIAS, SCRATCH = 1, 2, 3, 4
A, B, C, D, E, F, S = (0x7F0000000000 + i * 0x10000000000 for i in range(7))
BIG = 2 ** 31


def _call(name, defaults, **kw):
    assert not set(kw) - set(defaults)
    return getattr(ssc.lib(), name)(*{**defaults, **kw}.values())


@pytest.mark.parametrize("name", ["ssc_group_by_key_i32", "ssc_group_by_key_i64"])
def test_group_refusals(name):
    d = dict(keys=A, n=1000, groups=10, order=B, ranks=C, offsets=D, scratch=S, sbytes=1 << 24, stream=None)
    assert _call(name, d, n=-1) == ARG
    assert _call(name, d, groups=0) == ARG
    assert _call(name, d, n=BIG) == SIZE
    assert _call(name, d, groups=BIG - 1) == SIZE
    assert _call(name, d, keys=None) == ARG
    assert _call(name, d, offsets=None) == ARG
    assert _call(name, d, keys=A + 2) == ARG
    assert _call(name, d, order=B + 1) == ARG
    assert _call(name, d, order=A + 400) == ALIAS
    assert _call(name, d, ranks=B + 3996) == ALIAS
    assert _call(name, d, offsets=C) == ALIAS
    assert _call(name, d, n=20_000, scratch=None) == SCRATCH
    assert _call(name, d, n=20_000, scratch=S + 8) == SCRATCH
    assert _call(name, d, n=20_000, sbytes=ssc.group_scratch_bytes(20_000, 10) - 1) == SCRATCH
    assert _call(name, d, n=20_000, scratch=A) == ALIAS


def test_scratch_sizes():
    assert ssc.group_scratch_bytes(8192, 4096) == 0
    assert ssc.group_scratch_bytes(1000, 4097) == 4000  # the sorted keys, to find many offsets in
    # 17 spans of 1024 keys x 128 digits of 7 bits (100 groups and one more)
    assert ssc.group_scratch_bytes(16_385, 100) == 17 * 128 * 4
    # two passes of 9 bits: the table, (key, position) once, sorted keys
    assert ssc.group_scratch_bytes(65_536, 131_072) == 64 * 512 * 4 + 3 * 4 * 65_536
    # at most 256 spans
    assert ssc.group_scratch_bytes(2 ** 20 + 1, 100) == 205 * 128 * 4
    assert ssc.group_scratch_bytes(-1, 5) == 0 and ssc.group_scratch_bytes(5, 0) == 0
    L = ssc.lib()
    assert L.ssc_embed_grad_scratch_bytes(255, 64) == 0
    assert L.ssc_embed_grad_scratch_bytes(256, 64) == 16 * 64 * 4
    assert L.ssc_embed_grad_scratch_bytes(4096, 64) == (256 + 16) * 64 * 4
    assert L.ssc_embed_grad_scratch_bytes(65_536, 64) == (4096 + 256) * 64 * 4
    assert L.ssc_embed_grad_scratch_bytes(2 ** 18, 64) == (16_384 + 1024 + 64) * 64 * 4
    assert ssc.sample_scratch_bytes(0, 100) == 0 and ssc.sample_scratch_bytes(4, 0) == 0
    assert ssc.sample_scratch_bytes(4, 100_000) > 0


@pytest.mark.parametrize("name", ["ssc_embed_rows_i32", "ssc_embed_rows_i64"])
def test_embed_refusals(name):
    d = dict(table=A, dtype=1, vocab=100, width=64, ids=B, n=50, scale=1.0, out=C, stream=None)
    assert _call(name, d, dtype=3) == ARG
    assert _call(name, d, width=0) == ARG
    assert _call(name, d, width=2 ** 28 + 1) == SIZE
    assert _call(name, d, n=-1) == ARG
    assert _call(name, d, n=BIG) == SIZE
    assert _call(name, d, vocab=BIG) == SIZE
    assert _call(name, d, table=None) == ARG
    assert _call(name, d, ids=None) == ARG
    assert _call(name, d, out=None) == ARG
    assert _call(name, d, table=A + 1) == ARG
    assert _call(name, d, ids=B + 2) == ARG
    assert _call(name, d, out=A + 100 * 128 - 2) == ALIAS
    assert _call(name, d, out=B) == ALIAS


@pytest.mark.parametrize("name", ["ssc_embed_rows_grad_i32", "ssc_embed_rows_grad_i64"])
def test_embed_grad_refusals(name):
    d = dict(dout=A, dtype=1, n=1000, width=64, ids=B, order=C, offsets=D, vocab=100, scale=1.0, grad=E,
             gdtype=1, accumulate=0, scratch=S, sbytes=1 << 24, stream=None)
    assert _call(name, d, gdtype=2) == ARG       # neither dout's type nor fp32
    assert _call(name, d, dtype=0, gdtype=1) == ARG
    assert _call(name, d, vocab=0) == ARG
    assert _call(name, d, vocab=BIG - 1) == SIZE
    assert _call(name, d, dout=None) == ARG
    assert _call(name, d, order=None) == ARG
    assert _call(name, d, offsets=None) == ARG
    assert _call(name, d, grad=None) == ARG
    assert _call(name, d, grad=E + 1) == ARG
    assert _call(name, d, grad=A + 64) == ALIAS
    assert _call(name, d, grad=D) == ALIAS
    assert _call(name, d, scratch=None) == SCRATCH
    assert _call(name, d, sbytes=100) == SCRATCH
    assert _call(name, d, scratch=E) == ALIAS
    assert _call(name, d, scratch=C) == ALIAS


def test_routed_refusals():
    d = dict(x=A, dtype=0, tokens=100, per=4, width=16, ranks=B, rows=400, out=C, stream=None)
    for name in ("ssc_dispatch_rows",):
        assert _call(name, d, per=0) == ARG
        assert _call(name, d, tokens=2 ** 30) == SIZE  # 2^32 assignments
        assert _call(name, d, rows=-1) == ARG
        assert _call(name, d, x=None) == ARG
        assert _call(name, d, out=None) == ARG
        assert _call(name, d, ranks=B + 2) == ARG
        assert _call(name, d, out=A) == ALIAS
        assert _call(name, d, out=B + 1596) == ALIAS
    d = dict(y=A, dtype=1, rows=400, width=16, ranks=B, weights=C, tokens=100, per=4, out=D, stream=None)
    assert _call("ssc_combine_rows", d, y=None) == ARG
    assert _call("ssc_combine_rows", d, ranks=None) == ARG
    assert _call("ssc_combine_rows", d, weights=C + 2) == ARG
    assert _call("ssc_combine_rows", d, dtype=-1) == ARG
    assert _call("ssc_combine_rows", d, rows=BIG) == SIZE
    assert _call("ssc_combine_rows", d, out=A + 32) == ALIAS
    assert _call("ssc_combine_rows", d, out=C) == ALIAS
    d = dict(dout=A, y=B, dtype=1, rows=400, width=16, ranks=C, weights=D, tokens=100, per=4, dy=E, dweights=F,
             stream=None)
    assert _call("ssc_combine_rows_grad", d, weights=None) == ARG
    assert _call("ssc_combine_rows_grad", d, dweights=None) == ARG
    assert _call("ssc_combine_rows_grad", d, dy=None) == ARG
    assert _call("ssc_combine_rows_grad", d, dy=B) == ALIAS
    assert _call("ssc_combine_rows_grad", d, dweights=E + 16) == ALIAS
    assert _call("ssc_combine_rows_grad", d, dweights=D) == ALIAS


def test_sample_refusals():
    d = dict(logits=A, dtype=0, rows=4, vocab=1000, stride=1000, u=B, t=None, k=None, p=None, m=None, tokens=C,
             kept=None, logprobs=None, scratch=S, sbytes=1 << 24, stream=None)
    name = "ssc_sample_rows"
    assert _call(name, d, dtype=9) == ARG
    assert _call(name, d, rows=-1) == ARG
    assert _call(name, d, rows=65_536) == SIZE
    assert _call(name, d, vocab=0) == ARG
    assert _call(name, d, vocab=2 ** 22 + 1, stride=2 ** 23) == SIZE
    assert _call(name, d, stride=999) == ARG
    assert _call(name, d, logits=None) == ARG
    assert _call(name, d, u=None) == ARG
    assert _call(name, d, tokens=None) == ARG
    assert _call(name, d, logits=A + 2) == ARG
    assert _call(name, d, p=D + 1) == ARG
    assert _call(name, d, tokens=A + 15_996) == ALIAS
    assert _call(name, d, tokens=B) == ALIAS
    assert _call(name, d, kept=C) == ALIAS
    assert _call(name, d, scratch=None) == SCRATCH
    assert _call(name, d, sbytes=1000) == SCRATCH
    assert _call(name, d, scratch=A) == ALIAS


def test_binding_refuses_cpu_tensors():
    x, ids = torch.zeros(4, 8), torch.zeros(4, dtype=torch.int64)
    ranks, f = torch.zeros(4, 1, dtype=torch.int32), torch.zeros(4)
    for call in (lambda: ssc.group_by_key(ids, 4), lambda: ssc.embed_rows(x, ids),
                 lambda: ssc.embed_rows_grad(x, ids, ranks, ranks), lambda: ssc.dispatch_rows(x, ranks),
                 lambda: ssc.combine_rows(x, ranks), lambda: ssc.dispatch_rows_grad(x, ranks),
                 lambda: ssc.combine_rows_grad(x, x, ranks, f), lambda: ssc.sample_rows(x, f)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        ssc.sample_rows([[1.0]], f)
    with pytest.raises(TypeError):
        ssc.group_by_key([1, 2], 4)


def test_dtype_numbering():
    assert ssc.DTYPE == {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}


def test_sampling_reference_by_hand():
    """Rows small enough to work out: weights 4, 2, 1, 1 (of 8)."""
    x = np.log([2.0, 4.0, 1.0, 1.0])
    assert [sample_row(x, u)[0] for u in (0.0, 0.24, 0.26, 0.74, 0.76, 0.86, 0.88, 0.99)] == [0, 0, 1, 1, 2, 2, 3, 3]
    assert sample_row(x, 0.5)[1:] == (4, pytest.approx(np.log(0.5)))
    assert [sample_row(x, 0.99, k=k)[:2] for k in (1, 2, 3, 4, 9)] == [(1, 1), (1, 2), (2, 3), (3, 4), (3, 4)]
    assert [sample_row(x, 0.0, p=p)[1] for p in (0.1, 0.49, 0.51, 0.76, 0.9, 1.0)] == [1, 1, 2, 3, 4, 4]
    assert [sample_row(x, 0.0, m=m)[1] for m in (0.0, 0.2, 0.3, 0.6, 2.0)] == [4, 4, 2, 1, 1]
    assert sample_row(x, 0.9, t=0.0)[:2] == (1, 1)
    assert sample_row(np.array([-np.inf, np.nan]), 0.5) == (-1, 0, -np.inf)
    assert sample_row(np.array([1.0, np.inf, 0.0, np.inf]), 0.6, p=0.9)[0] == 3
