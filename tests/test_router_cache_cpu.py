"""Host-side checks of the router, the verification of drafts and the cache
calls, without a GPU: every refusal comes before HIP is touched (the addresses
here are never read), the scratch sizes, and the binding's refusal of CPU
tensors."""
from __future__ import annotations

import pytest
import torch

import scan_stream_compaction_amd as ssc

ARG, SIZE, ALIAS, SCRATCH = 1, 2, 3, 4
A, B, C, D, E, F, G, S = (0x7F0000000000 + i * 0x10000000000 for i in range(8))
BIG = 2 ** 31


def _call(name, defaults, **kw):
    assert not set(kw) - set(defaults)
    return getattr(ssc.lib(), name)(*{**defaults, **kw}.values())


def test_scratch_sizes():
    # one count of workgroups done, a loss for each 16 experts, shares and counts of each workgroup
    assert ssc.route_scratch_bytes(0, 8) == ssc.route_scratch_bytes(512, 128) == ssc.route_scratch_bytes(64, 1024) == 0
    assert ssc.route_scratch_bytes(513, 128) == 16 + 8 * 8 + 5 * (128 + 129) * 4
    assert ssc.route_scratch_bytes(65_536, 128) == 16 + 8 * 8 + 256 * (128 + 129) * 4
    # at most 64 rows of a lane: 32 rows of 512 experts to a workgroup at a time
    assert ssc.route_scratch_bytes(2 ** 20, 512) == 16 + 8 * 32 + 512 * (512 + 513) * 4
    assert ssc.route_scratch_bytes(-1, 8) == ssc.route_scratch_bytes(8, 0) == ssc.route_scratch_bytes(8, 1025) == 0
    assert ssc.route_scratch_bytes(BIG, 8) == 0
    assert ssc.verify_scratch_bytes(0, 100) == ssc.verify_scratch_bytes(4, 0) == 0
    assert ssc.verify_scratch_bytes(65_536, 10) == ssc.verify_scratch_bytes(1, 2 ** 22 + 1) == 0
    assert ssc.verify_scratch_bytes(3, 65_536) == ssc.verify_scratch_bytes(160, 131_072) == 0
    assert ssc.verify_scratch_bytes(3, 65_537) == 32 + 3 * 65 * 8
    assert ssc.verify_scratch_bytes(160, 131_073) == 160 * 8 + 160 * 129 * 8
    # sums of each part: one for each 128 rows, up to 4096 wavefronts
    assert ssc.accumulate_scratch_bytes(2, 3, 4, 100, 90, torch.bfloat16) == 4 * 6 * 90 * 4
    assert ssc.accumulate_scratch_bytes(1, 1, 4, 10_000, 90, torch.float32) == 313 * 90 * 4
    assert ssc.accumulate_scratch_bytes(8, 8, 4, 10_000, 1025, torch.bfloat16) == 3 * 64 * 1025 * 4
    assert ssc.accumulate_scratch_bytes(8, 8, 4, 32, 90, torch.bfloat16) == ssc.accumulate_scratch_bytes(32, 8, 8, 100, 90, torch.float16) == 0
    # up to 128 rows take none, however few the heads
    assert ssc.accumulate_scratch_bytes(1, 1, 4, 32, 90, torch.float32) == 0
    assert ssc.accumulate_scratch_bytes(1, 1, 1, 129, 90, torch.float32) == 2 * 90 * 4
    # two tables of 2048 counts a split, a threshold a head, two numbers a split, a list of its positions
    assert ssc.evict_scratch_bytes(1, 8, 16_384) == ssc.evict_scratch_bytes(40, 8, 32_768) == 0
    assert ssc.evict_scratch_bytes(1, 8, 131_072) == 8 * 16 * (16_384 + 8 + 4 * 8192) + 8 * 16
    assert ssc.evict_scratch_bytes(40, 8, 131_072) == 320 * (4 * (16_384 + 8 + 4 * 32_768) + 16)
    assert ssc.evict_scratch_bytes(1, 1, 2 ** 24) == 64 * (16_384 + 8 + 4 * 2 ** 18) + 16
    assert ssc.evict_scratch_bytes(1, 0, 100) == ssc.evict_scratch_bytes(-1, 1, 100) == ssc.evict_scratch_bytes(0, 1, 2 ** 20) == 0


def test_route_refusals():
    d = dict(logits=A, dtype=0, tokens=100, experts=16, stride=16, live=None, per=4, normalize=1, ids=B, weights=C,
             counts=D, share=E, loss=F, scratch=S, sbytes=1 << 24, stream=None)
    name = "ssc_route_rows"
    assert _call(name, d, dtype=3) == ARG
    assert _call(name, d, tokens=-1) == ARG
    assert _call(name, d, experts=0) == ARG
    assert _call(name, d, stride=15) == ARG
    assert _call(name, d, per=0) == ARG
    assert _call(name, d, per=17) == ARG
    assert _call(name, d, tokens=BIG) == SIZE
    assert _call(name, d, tokens=2 ** 30) == SIZE              # 2^32 assignments
    assert _call(name, d, experts=1025, stride=1025) == SIZE
    assert _call(name, d, experts=100, stride=100, per=65) == SIZE
    assert _call(name, d, stride=2 ** 30 + 1) == SIZE
    for key in ("logits", "ids", "weights", "counts", "share", "loss"):
        assert _call(name, d, **{key: None}) == ARG
    for key in ("logits", "ids", "weights", "counts", "share", "loss"):
        assert _call(name, d, **{key: d[key] + 2}) == ARG
    many = dict(d, tokens=1000, ids=B, weights=C)
    assert _call(name, many, scratch=None) == SCRATCH
    assert _call(name, many, scratch=S + 8) == SCRATCH
    assert _call(name, many, sbytes=ssc.route_scratch_bytes(1000, 16) - 1) == SCRATCH
    assert _call(name, many, scratch=A) == ALIAS
    assert _call(name, d, ids=A + 6396) == ALIAS
    assert _call(name, d, weights=B + 1596) == ALIAS
    assert _call(name, d, live=C, ) == ALIAS
    assert _call(name, d, share=D + 64) == ALIAS
    assert _call(name, d, loss=E) == ALIAS


def test_route_grad_refusals():
    d = dict(logits=A, dtype=1, tokens=100, experts=16, stride=20, live=None, ids=B, per=4, normalize=0, dweights=C,
             counts=D, dloss=E, dlogits=F, stream=None)
    name = "ssc_route_rows_grad"
    assert _call(name, d, dtype=-1) == ARG
    assert _call(name, d, per=17) == ARG
    assert _call(name, d, logits=None) == ARG
    assert _call(name, d, dlogits=None) == ARG
    assert _call(name, d, ids=None) == ARG
    assert _call(name, d, counts=None) == ARG
    assert _call(name, d, dloss=None) == ARG
    assert _call(name, d, dlogits=F + 1) == ARG
    assert _call(name, d, dweights=C + 2) == ARG
    assert _call(name, d, dlogits=A + 99 * 40 + 30) == ALIAS    # the last row's last element
    assert _call(name, d, dlogits=B) == ALIAS
    assert _call(name, d, dlogits=C + 1596) == ALIAS
    assert _call(name, d, dlogits=D + 64) == ALIAS
    assert _call(name, d, dlogits=E) == ALIAS
    assert _call(name, d, live=F + 10) == ALIAS


@pytest.mark.parametrize("name", ["ssc_verify_rows_i32", "ssc_verify_rows_i64"])
def test_verify_refusals(name):
    d = dict(probs=A, dtype=1, rows=5, drafts=3, vocab=1000, row=4000, place=1000, drafted=B, draft_probs=C,
             drow=3000, dplace=1000, u=D, lengths=E, tokens=F, accepted=G, scratch=S, sbytes=1 << 24, stream=None)
    assert _call(name, d, dtype=3) == ARG
    assert _call(name, d, rows=-1) == ARG
    assert _call(name, d, drafts=-1) == ARG
    assert _call(name, d, vocab=0) == ARG
    assert _call(name, d, rows=65_536) == SIZE
    assert _call(name, d, vocab=2 ** 22 + 1) == SIZE
    assert _call(name, d, drafts=2 ** 20 + 1) == SIZE
    assert _call(name, d, row=-1) == ARG
    assert _call(name, d, dplace=-1) == ARG
    for key in ("probs", "drafted", "u", "tokens", "accepted"):
        assert _call(name, d, **{key: None}) == ARG
    assert _call(name, d, probs=A + 1) == ARG
    assert _call(name, d, drafted=B + 2) == ARG
    assert _call(name, d, u=D + 1) == ARG
    long = dict(d, vocab=70_000, place=70_000, row=280_000, dplace=70_000, drow=210_000)
    assert _call(name, long, scratch=None) == SCRATCH
    assert _call(name, long, scratch=S + 8) == SCRATCH
    assert _call(name, long, sbytes=ssc.verify_scratch_bytes(5, 70_000) - 1) == SCRATCH
    assert _call(name, long, scratch=C) == ALIAS
    assert _call(name, d, tokens=A + 39_996) == ALIAS
    assert _call(name, d, tokens=C + 29_996) == ALIAS
    assert _call(name, d, accepted=F + 76) == ALIAS
    assert _call(name, d, accepted=B) == ALIAS
    assert _call(name, d, tokens=D) == ALIAS
    assert _call(name, d, accepted=E + 16) == ALIAS


def test_accumulate_refusals():
    d = dict(scores=A, batch=2, heads=3, capacity=100, sb=300, sh=100, weights=B, dtype=1, group=4, queries=2,
             length=90, wb=12 * 180, wh=180, wq=90, lengths=C, fresh=1, decay=1.0,
             scratch=S, sbytes=1 << 24, stream=None)
    name = "ssc_accumulate_weights"
    assert _call(name, d, batch=-1) == ARG
    assert _call(name, d, heads=0) == ARG
    assert _call(name, d, capacity=0) == ARG
    assert _call(name, d, dtype=5) == ARG
    assert _call(name, d, group=0) == ARG
    assert _call(name, d, queries=-1) == ARG
    assert _call(name, d, length=101) == ARG
    assert _call(name, d, fresh=-1) == ARG
    assert _call(name, d, batch=2 ** 16) == SIZE
    assert _call(name, d, capacity=BIG) == SIZE
    assert _call(name, d, group=2 ** 30) == SIZE      # 2^31 rows a head
    assert _call(name, d, sh=99) == ARG              # heads that share scores
    assert _call(name, d, sb=0) == ARG
    assert _call(name, d, wq=-1) == ARG
    assert _call(name, d, scores=None) == ARG
    assert _call(name, d, weights=None) == ARG
    assert _call(name, d, scores=A + 2) == ARG
    assert _call(name, d, weights=B + 1) == ARG
    assert _call(name, d, weights=A + 2396) == ALIAS
    assert _call(name, d, lengths=A) == ALIAS
    many = dict(d, queries=100, wh=9000, wb=12 * 9000)
    assert _call(name, many, scratch=None) == SCRATCH
    assert _call(name, many, scratch=S + 8) == SCRATCH
    assert _call(name, many, sbytes=ssc.accumulate_scratch_bytes(2, 3, 4, 100, 90, torch.bfloat16) - 1) == SCRATCH
    assert _call(name, many, scratch=A + 16) == ALIAS
    assert _call(name, many, scratch=B) == ALIAS


def test_evict_refusals():
    d = dict(scores=A, batch=2, heads=3, capacity=100, sb=300, sh=100, lengths=B, keep=50, first=4, recent=10, kept=C,
             counts=D, scratch=S, sbytes=1 << 24, stream=None)
    name = "ssc_evict_rows"
    assert _call(name, d, keep=0) == ARG
    assert _call(name, d, keep=101) == ARG
    assert _call(name, d, first=-1) == ARG
    assert _call(name, d, recent=-1) == ARG
    assert _call(name, d, first=41) == ARG
    assert _call(name, d, recent=2 ** 62, first=3) == ARG
    assert _call(name, d, batch=30_000) == SIZE
    assert _call(name, d, capacity=BIG - 1, keep=5, first=0, recent=0) == SIZE
    assert _call(name, d, sb=-1) == ARG
    for key in ("scores", "kept", "counts"):
        assert _call(name, d, **{key: None}) == ARG
        assert _call(name, d, **{key: d[key] + 2}) == ARG
    assert _call(name, d, kept=A + 2396) == ALIAS
    assert _call(name, d, counts=B + 4) == ALIAS
    assert _call(name, d, counts=C + 1196) == ALIAS
    long = dict(d, capacity=40_000, sh=40_000, sb=120_000)
    assert _call(name, long, scratch=None) == SCRATCH
    assert _call(name, long, scratch=S + 8) == SCRATCH
    assert _call(name, long, sbytes=ssc.evict_scratch_bytes(2, 3, 40_000) - 1) == SCRATCH
    assert _call(name, long, scratch=A + 112) == ALIAS


def test_move_refusals():
    d = dict(cache=A, es=2, batch=2, heads=3, capacity=100, width=16, cb=4800, ch=1600, cr=16, kept=B, keep=50, out=C,
             ob=2400, oh=800, orow=16, scratch=None, sbytes=0, stream=None)
    name = "ssc_move_rows"
    for es in (0, 3, 16):
        assert _call(name, d, es=es) == ARG
    assert _call(name, d, width=0) == ARG
    assert _call(name, d, keep=0) == ARG
    assert _call(name, d, keep=101) == ARG
    assert _call(name, d, width=2 ** 24 + 1) == SIZE
    assert _call(name, d, batch=30_000) == SIZE
    assert _call(name, d, cr=-1) == ARG
    assert _call(name, d, orow=15) == ARG            # rows of the result that share elements
    assert _call(name, d, oh=799) == ARG
    for key in ("cache", "kept", "out"):
        assert _call(name, d, **{key: None}) == ARG
        assert _call(name, d, **{key: d[key] + 1}) == ARG
    assert _call(name, d, out=A + 2 * 9600 - 2) == ALIAS
    assert _call(name, d, out=A) == ALIAS            # the same address, other strides
    assert _call(name, d, kept=C + 2 * 4800 - 4) == ALIAS
    # in place the whole cache is written to
    place = dict(d, out=A, ob=4800, oh=1600)
    assert _call(name, place, kept=A + 2 * 9600 - 4) == ALIAS
    # few long heads go by way of scratch
    assert ssc.move_scratch_bytes(2, 1, 2, 20_000, 64) == 2 * 20_000 * 128 and ssc.move_scratch_bytes(2, 2, 3, 50, 16) == 0
    long = dict(place, capacity=40_000, width=64, keep=20_000, ch=40_000 * 64, oh=40_000 * 64, cb=120_000 * 64,
                ob=120_000 * 64, cr=64, orow=64)
    need = ssc.move_scratch_bytes(2, 2, 3, 20_000, 64)
    assert need == 6 * 20_000 * 128
    assert _call(name, long) == SCRATCH
    assert _call(name, long, scratch=S + 8, sbytes=need) == SCRATCH
    assert _call(name, long, scratch=S, sbytes=need - 1) == SCRATCH
    assert _call(name, long, scratch=A + 64, sbytes=need) == ALIAS
    assert _call(name, long, scratch=B, sbytes=need) == ALIAS
    # positions before heads, keys beside values: strides that interleave are no overlap of the cache with itself
    assert _call(name, d, cache=A, cb=100 * 96, ch=32, cr=96, out=A + 32, ob=100 * 96, oh=32, orow=96) == ALIAS


def test_the_binding_refuses_cpu_tensors_and_wrong_shapes():
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="GPU"):
        ssc.route_rows(x, 2)
    with pytest.raises(ValueError, match="GPU"):
        ssc.route_rows_grad(x, None, None)
    with pytest.raises(ValueError, match="GPU"):
        ssc.verify_rows(torch.zeros(2, 3, 5), torch.zeros(2, 2).int(), torch.zeros(2, 3))
    with pytest.raises(ValueError, match="GPU"):
        ssc.accumulate_weights(torch.zeros(1, 1, 4), torch.zeros(1, 1, 1, 4))
    with pytest.raises(ValueError, match="GPU"):
        ssc.evict_rows(torch.zeros(1, 1, 4), 2)
    with pytest.raises(ValueError, match="GPU"):
        ssc.move_rows(torch.zeros(1, 1, 4, 2), torch.zeros(1, 1, 2).int())
    for f in (ssc.route_rows, ssc.evict_rows):
        with pytest.raises(TypeError):
            f([1.0], 1)


def test_outputs_in_the_gaps_of_views_are_refused():
    """Rows that are apart are one span where overlaps are checked."""
    route = dict(logits=A, dtype=0, tokens=100, experts=16, stride=32, live=None, per=4, normalize=1, ids=A + 64, weights=C,
                 counts=None, share=None, loss=None, scratch=None, sbytes=0, stream=None)
    assert _call("ssc_route_rows", route) == ALIAS
    grad = dict(logits=A, dtype=0, tokens=100, experts=16, stride=32, live=None, ids=B, per=4, normalize=0, dweights=C,
                counts=None, dloss=None, dlogits=A + 64, stream=None)
    assert _call("ssc_route_rows_grad", grad) == ALIAS
    # keys and values in one buffer, moved from the one half to the other
    move = dict(cache=A, es=2, batch=1, heads=3, capacity=100, width=16, cb=9600, ch=32, cr=96, kept=B, keep=50, out=A + 32,
                ob=9600, oh=32, orow=96, scratch=None, sbytes=0, stream=None)
    assert _call("ssc_move_rows", move) == ALIAS
