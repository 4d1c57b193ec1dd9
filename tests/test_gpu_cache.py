"""A cache cut to its heaviest rows, on the GPU: positions and moved rows are
equal to the definition's; accumulated weights are sums of R values of 0 or more
in fp32, R - 1 additions and one for the earlier score, its product and nothing
else, so within R + 2 half steps (2^-24 each) of the sum of the magnitudes."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import scan_stream_compaction_amd as ssc

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = [torch.float32, torch.bfloat16, torch.float16]


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


# ---- accumulate_weights ----


def check_accumulate(scores, weights, lengths=None, fresh=0, decay=1.0):
    before = scores.double().cpu()
    got = ssc.accumulate_weights(scores, weights, lengths=lengths, fresh=fresh, decay=decay)
    torch.cuda.synchronize()
    assert got is scores
    batch, heads, capacity = scores.shape
    length = weights.shape[3]
    w = torch.nan_to_num(weights.double().cpu(), nan=0.0, posinf=float("inf"), neginf=-float("inf"))
    group = weights.shape[1] // heads
    added = w.reshape(batch, heads, -1, length).sum(2)
    size = w.abs().reshape(batch, heads, -1, length).sum(2)
    rows = group * weights.shape[2]
    f = float(np.float32(decay))
    for b in range(batch):
        n = length if lengths is None else min(max(int(lengths[b]), 0), length)
        old = before[b, :, :n] * f
        old[:, max(0, n - fresh):] = 0
        want = old + added[b, :, :n]
        tol = (rows + 2) * 2.0 ** -24 * (old.abs() + size[b, :, :n])
        assert bool(((got[b, :, :n].double().cpu() - want).abs() <= tol).all())
        assert torch.equal(got[b, :, n:].double().cpu(), before[b, :, n:])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("batch,heads,group,queries,length,capacity", [
    (1, 1, 1, 1, 1, 1), (2, 3, 1, 1, 7, 9), (3, 2, 4, 1, 511, 512), (2, 2, 3, 5, 513, 600), (1, 2, 8, 2, 1000, 1000),
    (2, 1, 4, 16, 1025, 1025), (1, 2, 4, 17, 300, 301), (1, 1, 8, 64, 77, 100), (1, 1, 1, 200, 2049, 4000), (2, 1, 1, 0, 5, 5),
    (2, 1, 8, 57, 1390, 1390), (1, 2, 3, 700, 513, 600), (1, 1, 2, 3000, 33, 40), (1, 1, 1, 65_600, 9, 9)])
def test_accumulate_sizes(batch, heads, group, queries, length, capacity, dtype):
    g = gen(length + queries)
    w = torch.rand(batch, heads * group, queries, length, device=DEV, generator=g).to(dtype)
    s = torch.rand(batch, heads, capacity, device=DEV, generator=g)
    check_accumulate(s.clone(), w)
    check_accumulate(s.clone(), w, fresh=1, decay=0.9)
    lengths = torch.randint(-1, length + 2, (batch,), device=DEV, generator=g).int()
    check_accumulate(s.clone(), w, lengths, fresh=3)
    check_accumulate(s.clone(), w, lengths, fresh=2 ** 40)


@pytest.mark.parametrize("dtype", TYPES)
def test_accumulate_masked_places_and_fresh_scores(dtype):
    """NaN in queries that saw nothing adds nothing; what is behind a sequence is
    not read; a fresh position's old score may be anything."""
    g = gen(1)
    nan = float("nan")
    w = torch.rand(3, 4, 2, 100, device=DEV, generator=g).to(dtype)
    w[0, 1, 0] = nan
    w[1, :, :, 60:] = nan
    w[2] = nan
    s = torch.rand(3, 2, 130, device=DEV, generator=g)
    s[1, :, 57:] = nan
    lengths = torch.tensor([100, 60, 5], dtype=torch.int32, device=DEV)
    tail = s[1, :, 60:].clone()
    s[0] = 0.5
    got = s.clone()
    ssc.accumulate_weights(got, w, lengths=lengths, fresh=3)
    assert bool(torch.isfinite(got[1, :, :60]).all()) and bool(torch.isnan(got[1, :, 60:]).all()) and tail.shape[1] == 70
    assert torch.equal(got[2, :, :2], s[2, :, :2]) and bool((got[2, :, 2:5] == 0).all()) and torch.equal(got[2, :, 5:], s[2, :, 5:])
    got2 = s.clone()
    got2[1, :, 57:60] = 0
    check_accumulate(got2[:1], w[:1], lengths[:1], fresh=0)


@pytest.mark.parametrize("dtype", TYPES)
def test_accumulate_rows_that_start_anywhere(dtype):
    """Each start within 16 bytes and lengths around a wavefront's columns; guard
    values that no sum may take lie on both sides of every row."""
    g = gen(5)
    per = 16 // torch.empty(0, dtype=dtype).element_size()
    for start in range(per + 1):
        for length in (1, per - 1, per, per + 1, 63 * per - 1, 63 * per, 63 * per + 1, 64 * per, 2 * 63 * per + 3):
            for apart in (0, 1):
                full = torch.full((1, 6, 3, length + start + 5 + apart), 1e4, device=DEV).to(dtype)
                w = full[:, :, :, start:start + length]
                w.copy_(torch.rand(w.shape, device=DEV, generator=g))
                s = torch.rand(1, 2, length, device=DEV, generator=g)
                check_accumulate(s.clone(), w)
                check_accumulate(s.clone(), w.transpose(1, 2).contiguous().transpose(1, 2))


def test_accumulate_strides():
    """Weights of (batch, queries, heads, length), scores as every second head of a buffer."""
    g = gen(2)
    w = torch.rand(2, 3, 8, 333, device=DEV, generator=g).to(torch.bfloat16).transpose(1, 2)[:, :, :, 1:332]
    buf = torch.rand(2, 8, 400, device=DEV, generator=g)
    keep = buf.clone()
    view = buf[:, ::2, 5:336]
    assert not view.is_contiguous()
    check_accumulate(view, w)
    assert torch.equal(buf[:, 1::2], keep[:, 1::2]) and torch.equal(buf[:, :, :5], keep[:, :, :5])
    assert torch.equal(buf[:, :, 336:], keep[:, :, 336:])
    # a broadcast input: the same weights for every sequence
    one = torch.rand(1, 4, 2, 331, device=DEV, generator=g).expand(2, 4, 2, 331)
    check_accumulate(buf[:, ::2, 5:336], one)


# ---- evict_rows ----


def evict_reference(scores, keep, first, recent, lengths):
    s = scores.cpu().numpy()
    batch, heads, capacity = s.shape
    kept = np.full((batch, heads, keep), -1, np.int64)
    counts = np.zeros((batch, heads), np.int64)
    for b in range(batch):
        n = capacity if lengths is None else min(max(int(lengths[b]), 0), capacity)
        for h in range(heads):
            if n <= keep:
                at = np.arange(n)
            else:
                x = s[b, h, first:n - recent].astype(np.float64)
                x = np.where(np.isnan(x), -np.inf, x)
                # NaN below -infinity
                low = np.isnan(s[b, h, first:n - recent])
                order = np.lexsort((np.arange(len(x)), low, -x))[: keep - first - recent]
                at = np.concatenate([np.arange(first), first + np.sort(order), np.arange(n - recent, n)])
            kept[b, h, :len(at)] = at
            counts[b, h] = len(at)
    return kept, counts


def check_evict(scores, keep, first=0, recent=0, lengths=None):
    kept, counts = ssc.evict_rows(scores, keep, first=first, recent=recent, lengths=lengths)
    torch.cuda.synchronize()
    rk, rc = evict_reference(scores, keep, first, recent, lengths)
    assert np.array_equal(counts.cpu().numpy(), rc)
    assert np.array_equal(kept.cpu().numpy(), rk), np.argwhere(kept.cpu().numpy() != rk)[:5]
    return kept, counts


@pytest.mark.parametrize("capacity", [1, 2, 63, 64, 65, 1000, 4095, 4096, 4097, 8192, 8193, 20_000, 32_768, 32_769, 50_001, 131_072])
def test_evict_sizes(capacity):
    g = gen(capacity)
    s = torch.exp(2.5 * torch.randn(3, 2, capacity, device=DEV, generator=g))
    s = torch.where(torch.rand(s.shape, device=DEV, generator=g) < 0.1, 0.0, s)
    for keep in sorted({1, 2, capacity // 8, capacity // 2, capacity - 1, capacity}):
        if not 1 <= keep <= capacity:
            continue
        check_evict(s, keep)
        first, recent = min(4, keep // 3), keep // 4
        lengths = torch.tensor([capacity, keep + (capacity - keep) // 2, keep // 2], dtype=torch.int32, device=DEV)
        check_evict(s, keep, first, recent, lengths)
        check_evict(s, keep, keep // 2, keep - keep // 2)  # nothing left to choose
        check_evict(s, keep, 0, keep, lengths)


@pytest.mark.parametrize("capacity", [300, 5000, 40_000, 200_000])
def test_evict_equal_and_special_scores(capacity):
    """Few values, so that the border falls among equal scores; all equal; NaN,
    infinities, both zeros; neighbours of the last bits."""
    g = gen(capacity + 1)
    few = torch.randint(0, 4, (2, 3, capacity), device=DEV, generator=g).float()
    few[1, 0] = 0.25
    few[1, 1] = torch.where(few[1, 1] > 1, -0.0, 0.0)
    few[1, 2, ::3] = float("nan")
    few[0, 2, ::5] = float("inf")
    few[0, 2, 1::5] = -float("inf")
    few[0, 1] = 1.0 + torch.randint(0, 8, (capacity,), device=DEV, generator=g) * 2.0 ** -23
    for keep in (1, 17, capacity // 3, capacity // 2, capacity - 2):
        check_evict(few, keep)
        check_evict(few, keep, min(3, keep), (keep - min(3, keep)) // 2)
    nan = torch.full((1, 2, capacity), float("nan"), device=DEV)
    nan[0, 1, ::2] = -float("inf")
    check_evict(nan, capacity // 2 + 3)
    check_evict(-torch.rand(1, 1, capacity, device=DEV, generator=g), capacity // 4, 2, 5)


@pytest.mark.parametrize("capacity", [17_000, 66_000])
def test_evict_borders_in_every_digit(capacity):
    """Scores that share their first 11, 22 or 31 bits with the border's, spread over all splits."""
    g = gen(capacity + 7)
    one = torch.full((1,), 1.0, device=DEV).view(torch.int32)
    for spread in (2, 2 ** 9, 2 ** 12, 2 ** 20, 2 ** 22):
        s = (one + torch.randint(0, spread, (1, 2, capacity), device=DEV, generator=g)).int().view(torch.float32)
        s = torch.where(torch.rand(s.shape, device=DEV, generator=g) < 0.3, 0.5 * s, s)
        for keep in (5, capacity // 3, capacity // 2, capacity - 3):
            check_evict(s, keep, 1, 3)


def test_evict_lengths_strides_and_outputs():
    g = gen(8)
    buf = torch.rand(5, 6, 700, device=DEV, generator=g)
    view = buf.transpose(0, 1)[:, :, 3:603]
    lengths = torch.tensor([-5, 0, 1, 600, 2 ** 31 - 1, 77], dtype=torch.int32, device=DEV)
    want = check_evict(view, 100, 2, 10, lengths)
    out = torch.full((6 * 5 * 100 + 9,), -7, dtype=torch.int32, device=DEV)
    cnt = torch.full((40,), -7, dtype=torch.int32, device=DEV)
    for _ in range(3):
        kept, counts = ssc.evict_rows(view, 100, first=2, recent=10, lengths=lengths, kept=out[4:], counts=cnt)
        assert torch.equal(kept, want[0]) and torch.equal(counts, want[1])
    assert bool((out[:4] == -7).all()) and bool((out[3004:] == -7).all()) and bool((cnt[30:] == -7).all())
    kept, counts = ssc.evict_rows(view[:0], 10)
    assert kept.shape == (0, 5, 10) and counts.shape == (0, 5)


# ---- move_rows ----


def move_reference(cache, kept, out):
    c, k = cache.cpu(), kept.cpu().long()
    o = out.cpu().clone()
    for b in range(k.shape[0]):
        for h in range(k.shape[1]):
            ok = (k[b, h] >= 0) & (k[b, h] < c.shape[2])
            o[b, h, :k.shape[2]][ok] = c[b, h, k[b, h][ok]]
    return o


def positions(g, batch, heads, capacity, keep):
    return torch.rand(batch, heads, capacity, device=DEV, generator=g).argsort(2)[:, :, :keep].sort(2)[0].int().contiguous()


def bits(t):
    return t.contiguous().view(torch.uint8)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32, torch.float16, torch.uint8, torch.int64, torch.float8_e4m3fn])
@pytest.mark.parametrize("width", [1, 2, 3, 7, 8, 9, 16, 17, 63, 64, 65, 128, 576, 2049, 5000])
def test_move_widths(width, dtype):
    g = gen(width)
    batch, heads, capacity, keep = 2, 3, 150, 70
    es = torch.empty(0, dtype=dtype).element_size()
    raw = torch.randint(0, 256, (batch, heads, capacity, width * es), device=DEV, generator=g).to(torch.uint8)
    cache = raw.view(dtype)
    kept = positions(g, batch, heads, capacity, keep)
    fill = torch.full((batch, heads, keep + 5, width * es), 99, dtype=torch.uint8, device=DEV).view(dtype)
    want = move_reference(bits(cache).view(batch, heads, capacity, -1), kept, bits(fill).view(batch, heads, keep + 5, -1))
    out = fill.clone()
    got = ssc.move_rows(cache, kept, out=out)
    assert got.shape == (batch, heads, keep, width) and got.data_ptr() == out.data_ptr()
    assert torch.equal(bits(out).view(want.shape).cpu(), want)
    assert torch.equal(bits(cache), raw.view(-1).view(bits(cache).shape))
    want = move_reference(bits(cache).view(batch, heads, capacity, -1), kept, bits(cache).view(batch, heads, capacity, -1))
    assert ssc.move_rows(cache, kept) is cache
    assert torch.equal(bits(cache).view(want.shape).cpu(), want)


@pytest.mark.parametrize("batch,heads,capacity,keep,width", [(1, 1, 1, 1, 64), (1, 1, 5000, 4999, 128), (1, 8, 3001, 1000, 128),
                                                            (4, 8, 2000, 1999, 64), (1, 2, 20_000, 3, 96), (40, 8, 300, 200, 40)])
def test_move_in_place_of_each_shape(batch, heads, capacity, keep, width):
    g = gen(capacity + keep)
    cache = torch.randint(-2 ** 15, 2 ** 15, (batch, heads, capacity, width), device=DEV, generator=g).short()
    kept = positions(g, batch, heads, capacity, keep)
    for change in (None, "stay", "ends", "holes"):
        k = kept.clone()
        if change == "stay":
            k[:] = torch.arange(keep, device=DEV)
        if change == "ends":  # the first rows stay, the last ones move
            k[:, :, :keep // 2] = torch.arange(keep // 2, device=DEV)
            k[:, :, keep // 2:] = torch.arange(capacity - (keep - keep // 2), capacity, device=DEV)
        if change == "holes":
            k[:, :, ::3] = -1
            k[:, :, 1::7] = capacity
        c = cache.clone()
        ssc.move_rows(c, k)
        assert torch.equal(c.cpu(), move_reference(cache, k, cache))
        out = torch.full((batch, heads, keep, width), 7, dtype=torch.short, device=DEV)
        want = move_reference(cache, k, out)
        assert torch.equal(ssc.move_rows(cache, k, out=out).cpu(), want)


@pytest.mark.parametrize("batch,heads,keep,width", [(1, 3, 40, 64), (2, 4, 700, 128), (64, 8, 8, 9008), (64, 8, 8, 2051)])
def test_move_each_row_one_place(batch, heads, keep, width):
    """Each slot is stored where the slot before it is read from, rows of several
    column passes of a workgroup among them: no store may pass a load."""
    g = gen(width)
    cache = torch.randint(-2 ** 15, 2 ** 15, (batch, heads, keep + 1, width), device=DEV, generator=g).short()
    kept = torch.arange(1, keep + 1, dtype=torch.int32, device=DEV).expand(batch, heads, keep).contiguous()
    want = cache.clone()
    want[:, :, :keep] = cache[:, :, 1:]
    for _ in range(3):
        c = cache.clone()
        ssc.move_rows(c, kept)
        assert torch.equal(c, want)


def test_move_strides():
    """Caches of (batch, capacity, heads, width), keys and values in one buffer; the front of the same cache."""
    g = gen(3)
    both = torch.randn(2, 500, 2, 4, 64, device=DEV, generator=g).to(torch.bfloat16)
    k, v = both[:, :, 0].transpose(1, 2), both[:, :, 1].transpose(1, 2)
    assert k.shape == (2, 4, 500, 64) and not k.is_contiguous()
    keep = both.clone()
    kept = positions(g, 2, 4, 500, 200)
    want = move_reference(k, kept, k)
    ssc.move_rows(k, kept)
    assert torch.equal(k.cpu(), want) and torch.equal(v, keep[:, :, 1].transpose(1, 2))
    want = move_reference(v, kept, v)
    front = v[:, :, :200]
    got = ssc.move_rows(v, kept, out=front)
    assert torch.equal(v.cpu(), want) and torch.equal(got.cpu(), want[:, :, :200])
    smaller = torch.zeros(4, 2, 210, 64, device=DEV, dtype=torch.bfloat16).transpose(0, 1)
    want = move_reference(k, kept, smaller)
    ssc.move_rows(k, kept, out=smaller)
    assert torch.equal(smaller.cpu(), want)


def test_move_past_32_bits():
    """Rows whose offsets in bytes and elements pass 2^32."""
    capacity, width = 70_000, 65_536
    cache = torch.zeros(1, 1, capacity, width, dtype=torch.uint8, device=DEV)
    mark = torch.arange(capacity, device=DEV)
    cache[0, 0, :, 5] = (mark % 251).to(torch.uint8)
    cache[0, 0, :, -1] = (mark % 241).to(torch.uint8)
    kept = torch.arange(1, capacity, 2, device=DEV).int()[None, None].contiguous()
    ssc.move_rows(cache, kept)
    assert torch.equal(cache[0, 0, :capacity // 2, 5], (mark[1::2] % 251).to(torch.uint8))
    assert torch.equal(cache[0, 0, :capacity // 2, -1], (mark[1::2] % 241).to(torch.uint8))
    assert torch.equal(cache[0, 0, capacity // 2:, 5], (mark[capacity // 2:] % 251).to(torch.uint8))


# ---- together ----


def test_a_decoding_loop():
    """Drafts sampled, verified, their cache rows scored, and the cache cut
    whenever it is full, against the same steps on the host."""
    g = gen(20)
    batch, heads, group, capacity, keep, width, vocab, drafts = 3, 2, 2, 96, 40, 16, 50, 3
    cache = torch.zeros(batch, heads, capacity, width, device=DEV)
    scores = torch.full((batch, heads, capacity), float("nan"), device=DEV)
    lengths = torch.zeros(batch, dtype=torch.int32, device=DEV)
    host_cache, host_scores = cache.cpu(), scores.cpu()
    cuts = 0
    for step in range(120):
        logits = torch.randn(batch, drafts + 1, vocab, device=DEV, generator=g)
        q = torch.softmax(logits[:, :drafts], 2)
        u = torch.rand(batch, drafts, device=DEV, generator=g)
        drafted = ssc.sample_rows(logits[:, :drafts].reshape(-1, vocab), u.reshape(-1).contiguous())[0].view(batch, drafts)
        p = torch.softmax(logits + 0.3 * torch.randn(logits.shape, device=DEV, generator=g), 2)
        tokens, accepted = ssc.verify_rows(p, drafted, torch.rand(batch, drafts + 1, device=DEV, generator=g), q)
        assert bool((tokens.gather(1, accepted.long()[:, None]) >= 0).all())
        # the accepted drafts' rows and the drawn token's are appended
        rows = torch.randn(batch, heads, drafts + 1, width, device=DEV, generator=g)
        grown = lengths + accepted + 1
        for b in range(batch):
            a, z = int(lengths[b]), int(grown[b])
            cache[b, :, a:z] = rows[b, :, : z - a]
            host_cache[b, :, a:z] = rows[b, :, : z - a].cpu()
        for b in range(batch):  # sequences add different numbers of rows
            n, new = grown[b:b + 1].contiguous(), int(grown[b] - lengths[b])
            w = torch.rand(1, heads * group, 1, capacity, device=DEV, generator=g)
            ssc.accumulate_weights(scores[b:b + 1], w, lengths=n, fresh=new)
            z = int(n)
            old = host_scores[b, :, :z].clone()
            old[:, z - new:] = 0
            host_scores[b, :, :z] = old + w.cpu().view(heads, group, capacity).sum(1)[:, :z]
        lengths = grown
        if int(lengths.max()) + drafts + 1 > capacity:
            kept, counts = ssc.evict_rows(scores, keep, first=2, recent=8, lengths=lengths)
            rk, rc = evict_reference(scores, keep, 2, 8, lengths)
            assert np.array_equal(kept.cpu().numpy(), rk)
            host_cache = move_reference(host_cache, kept, host_cache)
            host_scores = move_reference(host_scores.unsqueeze(3), kept, host_scores.unsqueeze(3)).squeeze(3)
            ssc.move_rows(cache, kept)
            ssc.move_rows(scores.unsqueeze(3), kept)
            lengths = counts[:, 0].contiguous()
            cuts += 1
        for b in range(batch):
            z = int(lengths[b])
            assert torch.equal(cache[b, :, :z].cpu(), host_cache[b, :, :z])
            near = (scores[b, :, :z].cpu() - host_scores[b, :, :z]).abs() <= 1e-5 * host_scores[b, :, :z]
            assert bool(near.all())
    assert cuts >= 1


def test_graph_replays_and_streams():
    g = gen(30)
    w = torch.rand(4, 8, 1, 3000, device=DEV, generator=g).to(torch.bfloat16)
    s = torch.rand(4, 2, 3000, device=DEV, generator=g)
    cache = torch.randn(4, 2, 3000, 64, device=DEV, generator=g).to(torch.bfloat16)
    out = torch.empty(4, 2, 1000, 64, device=DEV, dtype=torch.bfloat16)

    def step(s):
        ssc.accumulate_weights(s, w, fresh=1)
        kept, counts = ssc.evict_rows(s, 1000, first=4, recent=100)
        return kept, counts, ssc.move_rows(cache, kept, out=out)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(s.clone())
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(s)
    for _ in range(4):
        w.copy_(torch.rand(w.shape, device=DEV, generator=g))
        cache.copy_(torch.randn(cache.shape, device=DEV, generator=g))
        other = s.clone()
        graph.replay()
        torch.cuda.synchronize()
        now = [x.clone() for x in got]
        want = step(other)
        assert torch.equal(s, other) and all(torch.equal(a, b) for a, b in zip(now, want))


def test_refusals_of_arguments():
    cache, kept = torch.zeros(1, 2, 8, 4, device=DEV), torch.zeros(1, 2, 3, dtype=torch.int32, device=DEV)
    for out in ([1.0], 3):
        with pytest.raises(TypeError, match="out must be a torch tensor"):
            ssc.move_rows(cache, kept, out=out)
    with pytest.raises(ValueError, match="at least keep"):
        ssc.move_rows(cache, kept, out=torch.zeros(1, 2, 2, 4, device=DEV))
    with pytest.raises(ssc.SSCError):  # another layout of the same memory
        ssc.move_rows(cache, kept, out=cache.as_strided((1, 2, 8, 4), (64, 4, 8, 1)))
    # a scratch is checked also where none is needed
    scores, weights = torch.zeros(1, 2, 8, device=DEV), torch.zeros(1, 2, 1, 8, device=DEV)
    wrong = torch.zeros(64, device=DEV)
    for call in (lambda: ssc.accumulate_weights(scores, weights, scratch=wrong),
                 lambda: ssc.move_rows(cache, kept, scratch=wrong),
                 lambda: ssc.move_rows(cache, kept, out=cache.clone(), scratch=wrong),
                 lambda: ssc.evict_rows(scores, 2, scratch=wrong)):
        with pytest.raises(TypeError, match="scratch"):
            call()
    none = torch.zeros(0, dtype=torch.uint8, device=DEV)
    ssc.move_rows(cache, kept, out=cache.clone(), scratch=none)
    ssc.accumulate_weights(scores, weights, scratch=none)


def _long_step(s, w, cache):
    """The forms that go by way of scratch: rows in parts, heads in splits, moves in place."""
    ssc.accumulate_weights(s, w, fresh=3)
    kept, counts = ssc.evict_rows(s, 9000, first=4, recent=100)
    ssc.move_rows(cache, kept)
    return kept, counts


def _long_inputs(g):
    return (torch.rand(1, 2, 20_000, device=DEV, generator=g), torch.rand(1, 4, 100, 20_000, device=DEV, generator=g).half(),
            torch.randn(1, 2, 20_000, 64, device=DEV, generator=g).to(torch.bfloat16))


def test_the_forms_with_scratch_in_a_graph():
    g = gen(31)
    s, w, cache = _long_inputs(g)
    assert ssc.accumulate_scratch_bytes(1, 2, 2, 100, 20_000, torch.float16) > 0
    assert ssc.evict_scratch_bytes(1, 2, 20_000) > 0 and ssc.move_scratch_bytes(2, 1, 2, 9000, 64) > 0
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _long_step(s.clone(), w, cache.clone())
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = _long_step(s, w, cache)
    for _ in range(4):
        w.copy_(torch.rand(w.shape, device=DEV, generator=g))
        cache.copy_(torch.randn(cache.shape, device=DEV, generator=g))
        other, moved = s.clone(), cache.clone()
        graph.replay()
        torch.cuda.synchronize()
        now = [x.clone() for x in got]
        want = _long_step(other, w, moved)
        assert torch.equal(s, other) and torch.equal(cache, moved)
        assert all(torch.equal(a, b) for a, b in zip(now, want))


def test_two_calls_at_once():
    g = gen(32)
    sets = [_long_inputs(g) for _ in range(2)]
    want = []
    for s, w, cache in sets:
        s, cache = s.clone(), cache.clone()
        want.append((*_long_step(s, w, cache), s, cache))
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(3):
        got = []
        copies = [(s.clone(), w, cache.clone()) for s, w, cache in sets]
        torch.cuda.synchronize()
        for stream, (s, w, cache) in zip(streams, copies):
            with torch.cuda.stream(stream):
                got.append((*_long_step(s, w, cache), s, cache))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
