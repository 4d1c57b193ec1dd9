"""Calls large enough that a workgroup takes further rows, a lane further batches
of rows, a wavefront further segments, or a head several tiles or parts; and the
form of a head in one workgroup that only many long heads take. The references are
those of the operators' own tests, with their tolerances unless stated."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import scan_stream_compaction_amd as ssc
from tests import test_gpu_cache as cache
from tests import test_gpu_route as route
from tests import test_gpu_verify as verify

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = [torch.float32, torch.bfloat16, torch.float16]
STEP = 2.0 ** -24  # half a step of fp32


# ---- accumulate_weights: sums over many rows ----
#
# Sixteen rows at most are added up in fp32, 15 roundings; such sums are added in
# fp64 and rounded once a wavefront; eight wavefronts are joined by 7 additions, parts
# in fp64 and one rounding, and the earlier score by one: 25 half steps of the sum of
# the magnitudes at most, and under one for the additions in fp64, for any number of rows.
ACCUMULATE_STEPS = 26


def check_sums(scores, weights, added, size, decay=1.0):
    """scores' new values against old * decay + added, both given in 64 bits."""
    want = scores.double().cpu() * float(np.float32(decay)) + added
    bound = ACCUMULATE_STEPS * STEP * (scores.double().abs().cpu() * abs(decay) + size)
    got = ssc.accumulate_weights(scores.clone(), weights, decay=decay).double().cpu()
    err = (got - want).abs()
    assert bool((err <= bound).all()), float((err / bound.clamp(min=1e-300)).max())


@pytest.mark.parametrize("value", [0.1, 1.0 / 3.0, 0.7])
def test_accumulate_one_weight_added_often(value):
    """Roundings of equal additions all go one way: 262,144 of one weight, so many heads that their rows are in one part."""
    heads, group, queries = 256, 8, 32_768
    assert ssc.accumulate_scratch_bytes(1, heads, group, queries, 3, torch.float32) == 0
    weights = torch.full((1, 1, 1, 3), value, device=DEV).expand(1, heads * group, queries, 3)
    scores = torch.rand(1, heads, 3, device=DEV, generator=cache.gen(1))
    total = float(np.float32(value)) * group * queries
    check_sums(scores, weights, total, total)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("batch,heads,group,queries,length", [
    (64, 4, 1, 129, 5), (32, 8, 3, 700, 3), (16, 16, 1, 2063, 9), (1, 1, 1, 65_600, 9), (2, 1, 8, 57, 1390), (1, 2, 2, 3000, 33)])
def test_accumulate_many_rows(batch, heads, group, queries, length, dtype):
    g = cache.gen(queries)
    weights = torch.rand(batch, heads * group, queries, length, device=DEV, generator=g).to(dtype)
    scores = torch.rand(batch, heads, length, device=DEV, generator=g)
    added = weights.double().view(batch, heads, group * queries, length).sum(2).cpu()
    check_sums(scores, weights, added, added)
    check_sums(scores, weights, added, added, decay=0.9)
    weights = weights - 0.5  # of both signs
    grouped = weights.double().view(batch, heads, group * queries, length)
    check_sums(scores, weights, grouped.sum(2).cpu(), grouped.abs().sum(2).cpu())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("batch,heads,group,queries,length", [
    (1, 1, 1, 1, 5), (2, 3, 4, 16, 1025), (1, 2, 4, 17, 300), (3, 2, 1, 128, 511), (1, 1, 1, 129, 90), (2, 1, 8, 57, 1390),
    (1, 2, 3, 700, 513), (1, 1, 2, 3000, 33), (1, 1, 1, 65_600, 9), (1, 1, 1, 65_599, 8), (64, 4, 8, 37, 5), (16, 16, 1, 2063, 9)])
def test_accumulate_each_row_once(batch, heads, group, queries, length, dtype):
    """Whole weights of 1 to 7, whose sums below 2^24 are exact: a row that is lost or added twice changes every column."""
    g = cache.gen(queries + length)
    weights = torch.randint(1, 8, (batch, heads * group, queries, length), device=DEV, generator=g).to(dtype)
    scores = torch.randint(0, 100, (batch, heads, length), device=DEV, generator=g).float()
    added = weights.double().view(batch, heads, group * queries, length).sum(2)
    assert float(added.max()) + 100 < 2 ** 24
    want = scores.double() + added
    assert torch.equal(ssc.accumulate_weights(scores, weights).double(), want)
    # the queries before the heads: rows that lie unevenly apart
    apart = weights.transpose(1, 2).contiguous().transpose(1, 2)
    assert torch.equal(ssc.accumulate_weights(scores, apart, decay=0.5).double(), 0.5 * want + added)


@pytest.mark.parametrize("queries", [40, 300, 5000])
def test_accumulate_infinities_among_many_rows(queries):
    """As a sum of plain additions: infinities of one sign give it, of both no number; NaN adds nothing."""
    inf, nan = float("inf"), float("nan")
    for heads in (1, 256):
        weights = torch.rand(1, heads, queries, 4, device=DEV, generator=cache.gen(queries))
        weights[:, :, queries // 2, 0] = inf
        weights[:, :, 1, 1] = -inf
        weights[:, :, [0, queries - 1], 2] = torch.tensor([inf, -inf], device=DEV)
        weights[:, :, ::3, 3] = nan
        got = ssc.accumulate_weights(torch.zeros(1, heads, 4, device=DEV), weights)
        assert bool((got[..., 0] == inf).all()) and bool((got[..., 1] == -inf).all()) and bool(torch.isnan(got[..., 2]).all())
        want = torch.nan_to_num(weights[..., 3].double(), nan=0.0).sum(2)
        assert bool(((got[..., 3] - want).abs() <= ACCUMULATE_STEPS * STEP * want).all())


# ---- route_rows_grad: further rows of a workgroup ----


@pytest.mark.parametrize("n,experts,per,dtype", [
    (40_001, 11, 2, torch.float32), (70_000, 24, 9, torch.bfloat16), (33_000, 160, 6, torch.bfloat16), (33_000, 128, 8, torch.float32),
    (40_001, 60, 20, torch.float16), (17_000, 250, 5, torch.float32), (8300, 300, 8, torch.float16), (4200, 600, 4, torch.bfloat16),
    (13_000, 1000, 3, torch.float32)])
def test_gradient_of_many_tokens(n, experts, per, dtype):
    """A workgroup takes two rows or more; what a row added in LDS must be gone when the next one begins."""
    x, g = route.inputs(n + experts, n, experts, dtype)
    live = torch.rand(n, device=DEV, generator=g) < 0.8
    dw = torch.randn(n, per, device=DEV, generator=g)
    dloss = torch.full((1,), 0.5 * n, device=DEV)
    for normalize in (True, False):
        ids, _, counts, _, _ = ssc.route_rows(x, per, normalize=normalize, live=live, balance=True)
        route.check_gradient(x, ids, dw, normalize, live, counts, dloss)
    any_ids = torch.randint(-1, experts + 1, (n, per), device=DEV, generator=g).int()
    any_ids[::7, -1] = any_ids[::7, 0]
    # few rows name an expert: what the row before left would show in the others
    any_ids[:, 1:] = torch.where(torch.rand(n, 1, device=DEV, generator=g) < 0.5, -1, any_ids[:, 1:])
    # of one sign, so that what one expert is named for twice does not cancel
    route.check_gradient(x, any_ids, dw.abs(), False, live)


# ---- route_rows: more workgroups than one a compute unit, so that no lane adds over 64 rows ----


def test_balance_of_two_million_tokens():
    n = 64 * 256 * 128 + 1
    assert ssc.route_scratch_bytes(n, 8) == 16 + 8 + 257 * (8 + 9) * 4
    x, g = route.inputs(2, n, 8, torch.bfloat16)
    route.check_forward(x, 2, live=torch.rand(n, device=DEV, generator=g) < 0.9)


def test_balance_of_many_tokens_and_experts():
    """262,200 of 520 experts, the definition in 64 bits by parts on the GPU."""
    n, experts, per = 262_200, 520, 10
    assert ssc.route_scratch_bytes(n, experts) > ssc.route_scratch_bytes(262_144, experts)
    x, _ = route.inputs(3, n, experts, torch.bfloat16)
    ids, weights, counts, share, loss = ssc.route_rows(x, per, balance=True)
    tol = (60 + 2 * 30) * STEP  # logits of a normal distribution lie within 30 of the row's largest
    total = torch.zeros(experts, dtype=torch.float64, device=DEV)
    many = torch.zeros(experts, dtype=torch.int64, device=DEV)
    for part, i, w in zip(x.split(20_000), ids.split(20_000), weights.split(20_000)):
        p = torch.softmax(part.double(), 1)
        assert float((part.amax(1) - part.amin(1)).max()) < 30
        at = torch.sort(part, dim=1, descending=True, stable=True)[1][:, :per]
        assert torch.equal(i.long(), at)
        want = p.gather(1, at)
        want = want / want.sum(1, keepdim=True)
        assert bool(((w - want).abs() <= want * tol).all())
        total += p.sum(0)
        many += torch.bincount(at.reshape(-1), minlength=experts)
    assert torch.equal(counts.long(), torch.cat([many, torch.tensor([n], device=DEV)]))
    want = total / n
    tol += 75 * STEP
    assert bool(((share - want).abs() <= want * tol).all())
    want = experts * float((many / (per * n) * want).sum())
    assert abs(float(loss) - want) <= want * tol


# ---- verify_rows: several segments to a wavefront, in two launches ----


@pytest.mark.parametrize("rows,vocab,dtype", [
    (159, 131_072, torch.bfloat16), (160, 131_073, torch.float16), (200, 140_000, torch.bfloat16), (100, 200_704, torch.float32),
    (16, 2 ** 22 - 5, torch.bfloat16), (12, 2 ** 22, torch.float16)])
def test_drafts_of_long_vocabularies(rows, vocab, dtype):
    assert rows * -(-vocab // 1024) >= 2 * 6144 and ssc.verify_scratch_bytes(rows, vocab) > 0
    p, x, u, q, g = verify.inputs(rows, rows, 1, vocab, dtype)
    verify.check(p, x, u, q)
    lengths = torch.randint(0, 2, (rows,), device=DEV, generator=g).int()
    verify.check(p, x, u, None, lengths)
    # q covers p: p draws
    p[::3] = 0.5 * p[::3]
    x[::3] = 0
    u[::3, 0] = 0.9999999
    q[::3] = 1.0
    verify.check(p, x, u, q)


# ---- evict_rows: heads of up to 32,768 by one workgroup where there are many, and splits of several tiles ----


def check_cut(scores, keep, first=0, recent=0, lengths=None):
    """Against a stable sort on the GPU in 64 bits, NaN below -infinity."""
    kept, counts = ssc.evict_rows(scores, keep, first=first, recent=recent, lengths=lengths)
    batch, heads, capacity = scores.shape
    for b in range(batch):
        n = capacity if lengths is None else int(lengths[b])
        want = torch.arange(min(n, keep), device=DEV).expand(heads, -1)
        if n > keep:
            x = scores[b, :, first:n - recent].double() + 0.0  # -0 as 0
            x = torch.where(x == -float("inf"), -1e300, x)
            x = torch.where(torch.isnan(x), -float("inf"), x)
            best = torch.sort(x, dim=1, descending=True, stable=True)[1][:, :keep - first - recent].sort(1)[0]
            want = torch.cat([want[:, :first], first + best, torch.arange(n - recent, n, device=DEV).expand(heads, -1)], 1)
        assert bool((counts[b] == want.shape[1]).all())
        assert torch.equal(kept[b, :, :want.shape[1]].long(), want) and bool((kept[b, :, want.shape[1]:] == -1).all())


@pytest.mark.parametrize("batch,heads,capacity,splits,tiles", [
    (26, 8, 16_385, 1, 0), (26, 8, 20_001, 1, 0), (130, 1, 32_768, 1, 0), (130, 1, 32_769, 2, 4), (13, 10, 40_000, 2, 4),
    (27, 3, 66_000, 3, 4), (1, 1, 524_289, 33, 2), (1, 1, 2 ** 20, 64, 2), (2, 2, 1_100_000, 34, 4)])
def test_evict_many_and_longest_heads(batch, heads, capacity, splits, tiles):
    """Tiles of 8192 positions: over 512 in all, or over 64 a head."""
    rows = batch * heads
    table = rows * splits * (16_384 + 8 + 4 * 8192 * tiles) + 16 * rows
    assert ssc.evict_scratch_bytes(batch, heads, capacity) == (table if splits > 1 else 0)
    g = cache.gen(capacity)
    s = torch.exp(2.5 * torch.randn(batch, heads, capacity, device=DEV, generator=g))
    s = torch.where(torch.rand(s.shape, device=DEV, generator=g) < 0.1, 0.0, s)
    lengths = torch.randint(0, capacity + 1, (batch,), device=DEV, generator=g).int()
    lengths[0] = capacity
    check_cut(s, capacity // 2, 4, 256)
    check_cut(s, capacity // 8, 4, capacity // 100, lengths)
    check_cut(s, capacity - 1, 0, 1, lengths)
    check_cut(s, 1)
    # few values: the border falls among equal scores of every tile
    few = torch.randint(0, 4, s.shape, device=DEV, generator=g).float()
    few[0, :, ::3] = float("nan")
    few[-1, :, 1::5] = -float("inf")
    check_cut(few, capacity // 3, 3, 1000, lengths)
    check_cut(few, capacity - 7)
    # neighbours that share their first 11 or 22 bits
    one = torch.full((1,), 1.0, device=DEV).view(torch.int32)
    for spread in (2 ** 9, 2 ** 20):
        near = (one + torch.randint(0, spread, s.shape, device=DEV, generator=g)).int().view(torch.float32)
        check_cut(near, capacity // 3, 1, 3, lengths)
    nan = torch.full(s.shape, float("nan"), device=DEV)
    nan[..., ::2] = -float("inf")
    check_cut(nan, capacity // 2 + 3)


# ---- views whose offsets pass 2^32 elements ----


def far(shape, strides, dtype, values):
    """A view of `shape` with its first dimensions far apart, holding `values`."""
    span = sum((n - 1) * s for n, s in zip(shape, strides)) + 1
    view = torch.empty(span, dtype=dtype, device=DEV).as_strided(shape, strides)
    view.copy_(values)
    return view


def test_rows_far_apart():
    """Results equal those of the same values side by side."""
    g = cache.gen(9)
    x = torch.randn(9, 40, device=DEV, generator=g).to(torch.bfloat16)
    away = far(x.shape, (2 ** 30, 1), x.dtype, x)
    want = ssc.route_rows(x, 4, balance=True)
    assert all(torch.equal(a, b) for a, b in zip(ssc.route_rows(away, 4, balance=True), want))
    dw = torch.randn(9, 4, device=DEV, generator=g)
    assert torch.equal(ssc.route_rows_grad(away, want[0], dw), ssc.route_rows_grad(x, want[0], dw))
    del away
    for vocab in (3000, 70_000):
        p, ids, u, q, _ = verify.inputs(9, 3, 2, vocab, torch.bfloat16)
        want = ssc.verify_rows(p, ids, u, q)
        # the places of a sequence side by side, and the sequences of a place
        got = ssc.verify_rows(far(p.shape, (2 ** 32, 2 ** 30, 1), p.dtype, p), ids, u, far(q.shape, (2 ** 30, 2 ** 32, 1), q.dtype, q))
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_heads_far_apart():
    g = cache.gen(10)
    for queries in (1, 200):
        w = torch.rand(2, 4, queries, 300, device=DEV, generator=g).to(torch.bfloat16)
        s = torch.rand(2, 2, 300, device=DEV, generator=g)
        away = far(w.shape, (2 ** 32, 2 ** 30, 2 ** 20, 1), w.dtype, w)
        to = far(s.shape, (2 ** 32 + 2 ** 20, 2 ** 31, 1), s.dtype, s)
        ssc.accumulate_weights(to, away)
        assert torch.equal(to, ssc.accumulate_weights(s, w))
        del away, to
    for capacity in (900, 20_000):
        s = torch.rand(2, 2, capacity, device=DEV, generator=g)
        away = far(s.shape, (2 ** 32 + 2 ** 20, 2 ** 31, 1), s.dtype, s)
        want = ssc.evict_rows(s, capacity // 2, first=2, recent=100)
        assert all(torch.equal(a, b) for a, b in zip(ssc.evict_rows(away, capacity // 2, first=2, recent=100), want))
        del away
    rows = torch.randn(2, 2, 50, 24, device=DEV, generator=g).to(torch.bfloat16)
    kept = cache.positions(g, 2, 2, 50, 20)
    away = far(rows.shape, (2 ** 33, 2 ** 32, 2 ** 25, 1), rows.dtype, rows)
    ssc.move_rows(away, kept)
    assert torch.equal(away, ssc.move_rows(rows, kept))


# ---- one scratch buffer of two captured graphs ----


def test_graphs_that_share_scratch():
    """Replayed in turn, over changed inputs: each graph writes what it reads of the scratch."""
    g = cache.gen(11)
    scratch = torch.full((2 ** 22,), 255, dtype=torch.uint8, device=DEV)

    def inputs_of(n):
        return dict(logits=torch.randn(900 * n, 60, device=DEV, generator=g), scores=torch.rand(1, n, 17_000 * n, device=DEV, generator=g),
                    weights=torch.rand(1, n, 300, 900, device=DEV, generator=g), sums=torch.rand(1, n, 900, device=DEV, generator=g),
                    rows=torch.randn(1, n, 9000, 16, device=DEV, generator=g), kept=cache.positions(g, 1, n, 9000, 8000),
                    drafts=verify.inputs(n, 3 * n, 2, 70_000, torch.float32)[:4])

    def step(s, scratch):
        routed = ssc.route_rows(s["logits"], 4, balance=True, scratch=scratch)
        ssc.accumulate_weights(s["sums"], s["weights"], scratch=scratch)
        ssc.move_rows(s["rows"], s["kept"], scratch=scratch)
        return (*routed, *ssc.evict_rows(s["scores"], 5000, first=3, recent=50, scratch=scratch),
                *ssc.verify_rows(*s["drafts"], scratch=scratch), s["sums"], s["rows"])

    def copy_of(s):
        return {k: v.clone() if isinstance(v, torch.Tensor) else tuple(x.clone() for x in v) for k, v in s.items()}

    sets = [inputs_of(1), inputs_of(2)]
    assert ssc.accumulate_scratch_bytes(1, 1, 1, 300, 900, torch.float32) > 0 and ssc.move_scratch_bytes(4, 1, 1, 8000, 16) > 0
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for s in sets:
            step(copy_of(s), scratch)
    torch.cuda.current_stream().wait_stream(side)
    graphs, got = [], []
    for s in sets:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            got.append(step(s, scratch))
    for i in range(6):
        s = sets[i % 2]
        s["logits"].copy_(torch.randn(s["logits"].shape, device=DEV, generator=g))
        s["scores"].copy_(torch.rand(s["scores"].shape, device=DEV, generator=g))
        want = step(copy_of(s), None)
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got[i % 2], want))


# ---- move_rows in place: positions in any order ----


@pytest.mark.parametrize("batch,heads,capacity,keep,width", [(1, 2, 6000, 5000, 64), (1, 3, 90, 80, 33), (40, 8, 300, 200, 40), (2, 2, 700, 650, 5000)])
def test_moves_of_positions_in_any_order(batch, heads, capacity, keep, width):
    """At or past their slots, in no order, one for several slots; those before their slots stay where they are."""
    g = cache.gen(keep)
    rows = torch.randint(-2 ** 15, 2 ** 15, (batch, heads, capacity, width), device=DEV, generator=g).short()
    slots = torch.arange(keep, device=DEV)
    kept = slots + (torch.rand(batch, heads, keep, device=DEV, generator=g) * (capacity - slots)).long()
    kept = torch.where(torch.rand(kept.shape, device=DEV, generator=g) < 0.2, capacity - 1, kept)
    before = torch.rand(kept.shape, device=DEV, generator=g) < 0.1
    at = kept.clone()
    kept = torch.where(before, (torch.rand(kept.shape, device=DEV, generator=g) * slots).long(), kept)
    want = rows.clone()
    at = torch.where(before, slots, at)
    want[:, :, :keep] = rows.gather(2, at[..., None].expand(-1, -1, -1, width))
    for _ in range(3):
        assert torch.equal(ssc.move_rows(rows.clone(), kept.int()), want)


# ---- calls with nothing to do ----


def test_calls_of_no_sequences_and_no_positions():
    w, s = torch.rand(2, 4, 3, 0, device=DEV), torch.rand(2, 2, 9, device=DEV)
    keep = s.clone()
    assert torch.equal(ssc.accumulate_weights(s, w, fresh=2, decay=0.0), keep)
    assert torch.equal(ssc.accumulate_weights(s, torch.rand(2, 2, 200, 9, device=DEV), lengths=torch.zeros(2, dtype=torch.int32, device=DEV)), keep)
    assert ssc.accumulate_weights(s[:0], torch.rand(0, 4, 300, 9, device=DEV)).shape == (0, 2, 9)
    kept = torch.zeros(0, 2, 5, dtype=torch.int32, device=DEV)
    rows = torch.rand(0, 2, 9, 4, device=DEV)
    assert ssc.move_rows(rows, kept) is rows and ssc.move_rows(rows, kept, out=torch.rand(0, 2, 7, 4, device=DEV)).shape == (0, 2, 5, 4)
    kept, counts = ssc.evict_rows(s, 4, lengths=torch.zeros(2, dtype=torch.int32, device=DEV), recent=2)
    assert bool((kept == -1).all()) and bool((counts == 0).all())
