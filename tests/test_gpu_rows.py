"""Rows moved by a key (group_by_key, embed_rows, dispatch_rows, combine_rows
and their gradients) on the GPU against plain definitions in 64 bits.

Tolerances. A product or sum of fp32 values rounds by at most u = 2^-24 of
itself, so a sum of m products is off by at most (m + 1) u times the sum of
their magnitudes (to first order; 1.01 covers the rest), and rounding to the
output's type adds half a step, eps / 2 of the value, or half the smallest
subnormal."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import scan_stream_compaction_amd as ssc

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = [torch.float32, torch.bfloat16, torch.float16]
U = 2.0 ** -24


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, device=DEV, generator=g).to(dtype)


def _close(got, want, magnitude, terms, dtype):
    """|got - want| within the rounding of `terms` fp32 operations on values
    whose magnitudes sum to `magnitude`, and of the output's type."""
    fi = torch.finfo(dtype)
    tol = 1.01 * (terms + 1) * U * magnitude
    tol = tol + fi.eps / 2 * (want.abs() + tol) + fi.smallest_normal * fi.eps / 2
    bad = (got.double() - want).abs() > tol
    assert not bool(bad.any()), f"{int(bad.sum())} of {bad.numel()} off, largest {float((got.double() - want).abs().max())}"


def _guarded(shape, dtype, fill):
    """A tensor inside a larger buffer, and a check that the words around it
    still hold `fill`."""
    n = int(np.prod(shape))
    buf = torch.full((n + 128,), fill, dtype=dtype, device=DEV)
    view = buf[64:64 + n].view(shape)
    return view, lambda: bool((buf[:64] == fill).all()) and bool((buf[64 + n:] == fill).all())


def _group_want(keys, groups):
    flat = keys.reshape(-1).astype(np.int64)
    inside = (flat >= 0) & (flat < groups)
    key = np.where(inside, flat, groups)
    order = np.argsort(key, kind="stable")
    kept = int(inside.sum())
    ranks = np.full(flat.size, -1, np.int32)
    ranks[order[:kept]] = np.arange(kept)
    offsets = np.zeros(groups + 1, np.int64)
    np.add.at(offsets, flat[inside] + 1, 1)
    return order[:kept].astype(np.int32), ranks.reshape(keys.shape), np.cumsum(offsets).astype(np.int32)


def _check_group(keys, groups, **kw):
    n = keys.size
    kd = torch.from_numpy(keys).to(DEV)
    order, order_ok = _guarded((n,), torch.int32, -77)
    ranks, ranks_ok = _guarded((n,), torch.int32, -78)
    offsets, offsets_ok = _guarded((groups + 1,), torch.int32, -79)
    ssc.group_by_key(kd, groups, order=order, ranks=ranks, offsets=offsets, **kw)
    torch.cuda.synchronize()
    worder, wranks, woffsets = _group_want(keys, groups)
    kept = worder.size
    assert np.array_equal(offsets.cpu().numpy(), woffsets)
    assert np.array_equal(order[:kept].cpu().numpy(), worder)
    assert bool((order[kept:] == -77).all())
    assert np.array_equal(ranks.cpu().numpy(), wranks.reshape(-1))
    assert order_ok() and ranks_ok() and offsets_ok()


GROUP_SIZES = [1, 2, 63, 64, 65, 1023, 1024, 1025, 4095, 4097, 8191, 8192, 8193, 17408, 40961, 300_001]


@pytest.mark.parametrize("groups", [1, 2, 8, 511, 512, 1000, 4096, 4097, 131_072])
@pytest.mark.parametrize("n", GROUP_SIZES)
def test_group_by_key(n, groups):
    r = np.random.RandomState(n * 7 + groups)
    keys = (r.randint(-1, groups + 1, n) if groups < 4 else
            np.minimum(np.exp(r.rand(n) * np.log(groups + 2)).astype(np.int64) - 2, groups))
    keys = keys.astype(np.int64 if n % 2 else np.int32)
    _check_group(keys, groups)


@pytest.mark.parametrize("groups", [37, 5000])
@pytest.mark.parametrize("n", [1500, 2048, 2049, 2900, 3500, 4999, 5121, 6144, 6145, 7168, 7169])
def test_group_one_workgroup(n, groups):
    """Each number of sets of 64 keys that a wavefront of the one workgroup holds."""
    r = np.random.RandomState(n + groups)
    _check_group(r.randint(-1, groups + 1, n).astype(np.int64), groups)


@pytest.mark.parametrize("n", [70, 1500, 9000, 50_000])
@pytest.mark.parametrize("groups", [3, 600, 300_000, 5_000_000, 2 ** 27 + 5])
def test_group_many_passes_and_odd_keys(n, groups):
    """Two to four passes; one key everywhere, no key inside, keys far outside."""
    if groups > 10_000_000 and n > 2000:
        pytest.skip("the offsets alone are half a gigabyte: two sizes are enough")
    r = np.random.RandomState(n + groups % 1000)
    for keys in (np.full(n, groups - 1, np.int64), np.full(n, -1, np.int64), np.full(n, 0, np.int64),
                 r.randint(0, groups, n), np.where(r.rand(n) < 0.5, r.randint(0, groups, n), 2 ** 40 + 1),
                 np.where(r.rand(n) < 0.5, r.randint(0, groups, n), -2 ** 63)):
        _check_group(keys.astype(np.int64), groups)
        if groups > 10_000_000:
            break


def test_group_large():
    """The largest spans: 256 workgroups with several steps each."""
    r = np.random.RandomState(5)
    n = 5_000_003
    _check_group(r.randint(-1, 64, n).astype(np.int32), 64)
    _check_group(r.randint(-1, 100_000, n).astype(np.int32), 100_000)


def test_group_int32_extremes_and_none():
    keys = np.array([0, -2 ** 31, 2 ** 31 - 1, 5, 5, 0, 6], np.int32)
    _check_group(keys, 6)
    order, ranks, offsets = ssc.group_by_key(torch.empty(0, dtype=torch.int64, device=DEV), 1000)
    assert order.numel() == 0 and ranks.numel() == 0 and bool((offsets == 0).all()) and offsets.numel() == 1001


def test_group_optional_outputs_and_shape():
    keys = torch.randint(0, 9, (100, 8), device=DEV, generator=_gen(1))
    order, ranks, offsets = ssc.group_by_key(keys, 9)
    assert ranks.shape == keys.shape
    none, r2, o2 = ssc.group_by_key(keys, 9, order=False)
    assert none is None and torch.equal(r2, ranks) and torch.equal(o2, offsets)
    o3, none, _ = ssc.group_by_key(keys, 9, ranks=False)
    assert none is None and torch.equal(o3, order)


WIDTHS = [1, 3, 4, 7, 8, 9, 64, 257, 1000, 2048, 4100]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("width", WIDTHS)
def test_embed(dtype, width):
    g = _gen(width)
    vocab = 301
    table = _randn(g, vocab, width, dtype=dtype)
    for n, idt in ((1, torch.int64), (777, torch.int32)):
        ids = torch.randint(-3, vocab + 3, (n,), device=DEV, generator=g).to(idt)
        for scale in (1.0, 0.3, float(np.sqrt(width))):
            out, ok = _guarded((n, width), dtype, -5.0)
            ssc.embed_rows(table, ids, scale, out=out)
            s = float(np.float32(scale))
            inside = (ids >= 0) & (ids < vocab)
            want = table.double()[ids.long().clamp(0, vocab - 1)] * s * inside[:, None]
            _close(out, want, want.abs(), 1, dtype)
            assert ok()


def test_embed_unaligned_rows_and_nonfinite():
    """A table that starts inside a buffer at an odd element, and rows of inf and NaN."""
    g = _gen(3)
    buf = _randn(g, 50 * 33 + 1, dtype=torch.bfloat16)
    table = buf[1:].view(50, 33)
    table[4] = float("inf")
    table[5] = float("nan")
    ids = torch.tensor([4, 5, 6, 4, -1], device=DEV)
    out = ssc.embed_rows(table, ids, 2.0)
    assert bool(out[0].isinf().all()) and bool(out[1].isnan().all()) and bool((out[4] == 0).all())
    assert torch.equal(out[2], table[6] * 2)
    assert ssc.embed_rows(table, ids.view(5, 1)).shape == (5, 1, 33)
    assert ssc.embed_rows(table, ids[:0]).shape == (0, 33)
    assert bool((ssc.embed_rows(table[:0], ids) == 0).all())


def test_many_wide_rows():
    """More workgroups than one dimension of a launch holds, and elements past
    2^32: 17,000,003 rows of 1030 bf16 (35 GB)."""
    if torch.cuda.mem_get_info()[0] < 80 << 30:
        pytest.skip("needs 80 GB of device memory")
    n, width, vocab = 17_000_003, 1030, 1000
    table = _randn(_gen(31), vocab, width, dtype=torch.bfloat16)
    ids = (torch.arange(n, device=DEV) * 7919) % vocab
    out = ssc.embed_rows(table, ids, 1.0)
    for first in range(0, n, 1_000_000):
        assert torch.equal(out[first:first + 1_000_000:997], table[ids[first:first + 1_000_000:997]])
    assert torch.equal(out[-5000:], table[ids[-5000:]])
    # back as one row a token, from the same buffer: ranks in reverse
    ranks = torch.arange(n - 1, -1, -1, device=DEV, dtype=torch.int32)
    back = ssc.combine_rows(out, ranks)
    del out
    for first in range(0, n, 1_000_000):
        assert torch.equal(back[first:first + 1_000_000:991], table[ids[ranks[first:first + 1_000_000:991].long()]])
    assert torch.equal(back[-5000:], table[ids[ranks[-5000:].long()]])


def _grad_case(ids, vocab, width, dtype, scale, gdtype, seed):
    g = _gen(seed)
    n = ids.numel()
    dout = _randn(g, n, width, dtype=dtype)
    order, _, offsets = ssc.group_by_key(ids, vocab, ranks=False)
    out, ok = _guarded((vocab, width), gdtype, 3.0)
    ssc.embed_rows_grad(dout, ids, order, offsets, scale, out=out)
    s = float(np.float32(scale))
    inside = (ids >= 0) & (ids < vocab)
    at = ids[inside].long()
    d = dout.double()[inside]
    want = torch.zeros(vocab, width, dtype=torch.float64, device=DEV).index_add_(0, at, d)
    mag = torch.zeros_like(want).index_add_(0, at, d.abs())
    terms = torch.bincount(at, minlength=vocab)[:, None].double()
    _close(out, want * s, mag * abs(s), terms + 1, gdtype)
    assert ok()
    # added to what is there; rows without tokens stay as they are
    base = _randn(g, vocab, width, dtype=gdtype)
    acc = base.clone()
    ssc.embed_rows_grad(dout, ids, order, offsets, scale, out=acc, accumulate=True)
    empty = terms[:, 0] == 0
    assert torch.equal(acc[empty], base[empty])
    _close(acc, base.double() + want * s, mag * abs(s) + base.double().abs(), terms + 2, gdtype)
    return dout, out


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("width", [1, 5, 8, 9, 64, 257, 1032])
def test_embed_grad(dtype, width):
    g = _gen(width + 17)
    vocab, n = 301, 2500
    ids = (torch.rand(n, device=DEV, generator=g) ** 4 * (vocab + 1)).long() - 1
    _grad_case(ids, vocab, width, dtype, 0.125, dtype, 1)
    _grad_case(ids.int(), vocab, width, dtype, -1.7, torch.float32, 2)


@pytest.mark.parametrize("n,vocab", [(1, 1), (1, 5000), (255, 3), (256, 1), (4096, 1), (4111, 2), (70_001, 3), (70_001, 70_001), (300_007, 2)])
def test_embed_grad_block_sums(n, vocab):
    """One id over whole blocks of 16, 256 and 4096 sorted tokens, ranges that
    begin and end inside blocks, and ids that occur once."""
    g = _gen(n)
    ids = torch.randint(0, vocab, (n,), device=DEV, generator=g)
    for i in (ids, torch.where(torch.rand(n, device=DEV, generator=g) < 0.9, 0, ids)):
        _grad_case(i, vocab, 24, torch.bfloat16, 1.0, torch.float32, n)


def test_embed_grad_none_and_differences():
    """No tokens; and the lookup's change along a direction d of the table is
    <grad, d>: exact for a linear map, up to the rounding of its outputs."""
    empty = torch.empty(0, dtype=torch.int64, device=DEV)
    order, _, offsets = ssc.group_by_key(empty, 7)
    out = ssc.embed_rows_grad(torch.empty(0, 12, device=DEV), empty, order, offsets, 1.0)
    assert out.shape == (7, 12) and bool((out == 0).all())
    g = _gen(8)
    table, d = _randn(g, 97, 40), _randn(g, 97, 40)
    ids = torch.randint(0, 97, (600,), device=DEV, generator=g)
    dout, grad = _grad_case(ids, 97, 40, torch.float32, 0.7, torch.float32, 9)
    moved = ssc.embed_rows(table + d, ids, 0.7).double() - ssc.embed_rows(table, ids, 0.7).double()
    lhs, rhs = float((moved * dout.double()).sum()), float((grad.double() * d.double()).sum())
    # each of the 600 x 40 differences and the table + d sums are off by a few u of values below 10
    assert abs(lhs - rhs) <= 600 * 40 * 6 * U * 10 * float(dout.abs().mean())


def _route(g, tokens, per, experts, drop, dtype=torch.int64):
    score = torch.rand(tokens, experts, device=DEV, generator=g)
    ids = torch.topk(score, per, dim=1).indices
    ids[torch.rand(tokens, per, device=DEV, generator=g) < drop] = -1
    ids = ids.to(dtype)
    _, ranks, offsets = ssc.group_by_key(ids, experts, order=False)
    return ids, ranks, int(offsets[-1])


ROUTED = [(1, 1, 1, 8, 0.0), (1, 8, 64, 2048, 0.0), (33, 2, 4, 1, 0.2), (33, 3, 7, 5, 0.2), (300, 8, 64, 257, 0.3),
          (300, 9, 16, 4100, 0.1), (1000, 4, 8, 64, 1.0), (2100, 6, 60, 200, 0.05), (17, 16, 20, 1000, 0.5)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tokens,per,experts,width,drop", ROUTED)
def test_dispatch_combine_and_gradients(dtype, tokens, per, experts, width, drop):
    g = _gen(tokens + width)
    ids, ranks, kept = _route(g, tokens, per, experts, drop)
    x = _randn(g, tokens, width, dtype=dtype)
    out, ok = _guarded((tokens * per, width), dtype, -3.0)
    ssc.dispatch_rows(x, ranks, out=out)
    t, k = torch.nonzero(ranks >= 0, as_tuple=True)
    slot = ranks[t, k].long()
    assert torch.equal(out[slot], x[t]) and bool((out[kept:] == -3.0).all()) and ok()
    # back, weighted: slots past the kept ones hold NaN, which must not spread
    y = _randn(g, tokens * per, width, dtype=dtype)
    y[kept:] = float("nan")
    w = torch.rand(tokens, per, device=DEV, generator=g)
    w[ranks < 0] = float("nan")
    got, ok = _guarded((tokens, width), dtype, -4.0)
    ssc.combine_rows(y, ranks, w, out=got)
    terms = w[t, k].double()[:, None] * y.double()[slot]
    want = torch.zeros(tokens, width, dtype=torch.float64, device=DEV).index_add_(0, t, terms)
    mag = torch.zeros_like(want).index_add_(0, t, terms.abs())
    _close(got, want, mag, per, dtype)
    assert ok()
    # the gradient of dispatch: ones for weights
    got = ssc.dispatch_rows_grad(y, ranks)
    want = torch.zeros_like(want).index_add_(0, t, y.double()[slot])
    mag = torch.zeros_like(want).index_add_(0, t, y.double()[slot].abs())
    _close(got, want, mag, per, dtype)
    # the gradients of combine
    dout = _randn(g, tokens, width, dtype=dtype)
    dy, dy_ok = _guarded((tokens * per, width), dtype, -6.0)
    dw, dw_ok = _guarded((tokens, per), torch.float32, -7.0)
    ssc.combine_rows_grad(dout, y, ranks, w, dy=dy, dweights=dw)
    want = w[t, k].double()[:, None] * dout.double()[t]
    _close(dy[slot], want, want.abs(), 1, dtype)
    assert bool((dy[kept:] == -6.0).all())
    prod = dout.double()[t] * y.double()[slot]
    want = torch.zeros(tokens, per, dtype=torch.float64, device=DEV)
    mag = torch.zeros_like(want)
    want[t, k], mag[t, k] = prod.sum(1), prod.abs().sum(1)
    _close(dw, want, mag, width, torch.float32)
    assert bool((dw[ranks < 0] == 0).all()) and dy_ok() and dw_ok()


def test_routed_rows_that_the_buffers_do_not_hold():
    """Ranks at or past the rows of the buffer move and add nothing."""
    g = _gen(4)
    _, ranks, kept = _route(g, 100, 4, 8, 0.1)
    x = _randn(g, 100, 32)
    short = torch.zeros(150, 32, device=DEV)
    ssc.dispatch_rows(x, ranks, out=short)
    full = ssc.dispatch_rows(x, ranks)
    assert kept > 150 and torch.equal(short, full[:150])
    got = ssc.combine_rows(short, ranks)
    want = ((ranks >= 0) & (ranks < 150)).sum(1)[:, None] * x.double()
    _close(got, want, want.abs(), 4, torch.float32)
    none = ssc.combine_rows(short[:0], ranks)
    assert bool((none == 0).all())
    w = torch.ones(100, 4, device=DEV)
    dy, dw = ssc.combine_rows_grad(x, short[:0], ranks, w)
    assert dy.shape == (0, 32) and bool((dw == 0).all())
    assert ssc.dispatch_rows(x[:0], ranks[:0]).shape == (0, 32)
    assert ssc.combine_rows(short, ranks[:0]).shape == (0, 32)


def test_gradients_by_differences():
    """combine is linear in y and in the weights: its change along a direction
    is the gradient's inner product with it, up to rounding."""
    g = _gen(6)
    _, ranks, kept = _route(g, 64, 4, 8, 0.0)
    y, d = _randn(g, 256, 96), _randn(g, 256, 96)
    w, e = torch.rand(64, 4, device=DEV, generator=g), torch.rand(64, 4, device=DEV, generator=g)
    dout = _randn(g, 64, 96)
    dy, dw = ssc.combine_rows_grad(dout, y, ranks, w)
    at = ssc.combine_rows(y, ranks, w).double()
    # sums of 64 x 96 terms, each off by a few u of values below 20
    tol = 64 * 96 * 8 * U * 20
    by = float(((ssc.combine_rows(y + d, ranks, w).double() - at) * dout.double()).sum())
    assert abs(by - float((dy.double() * d.double()).sum())) <= tol
    by = float(((ssc.combine_rows(y, ranks, w + e).double() - at) * dout.double()).sum())
    assert abs(by - float((dw.double() * e.double()).sum())) <= tol


def _token_path(table, ids, expert_ids, weights, dout, experts, head):
    """One training step's rows: lookup, to the experts and back, and all gradients."""
    vocab = table.shape[0]
    x = ssc.embed_rows(table, ids, 2.0)
    _, ranks, offsets = ssc.group_by_key(expert_ids, experts, order=False)
    rows = ssc.dispatch_rows(x, ranks)
    y = rows * head
    out = ssc.combine_rows(y, ranks, weights)
    dy, dw = ssc.combine_rows_grad(dout, y, ranks, weights)
    dx = ssc.dispatch_rows_grad(dy * head, ranks)
    order, _, voff = ssc.group_by_key(ids, vocab, ranks=False)
    return out, dw, ssc.embed_rows_grad(dx, ids, order, voff, 2.0), offsets


def _path_inputs(seed, tokens=200, per=4, experts=16, vocab=500, width=48):
    g = _gen(seed)
    ids = torch.randint(0, vocab, (tokens,), device=DEV, generator=g)
    expert_ids = torch.topk(torch.rand(tokens, experts, device=DEV, generator=g), per, dim=1).indices
    weights = torch.rand(tokens, per, device=DEV, generator=g)
    return (_randn(g, vocab, width), ids, expert_ids, weights, _randn(g, tokens, width), experts,
            _randn(g, 1, width))


def test_the_token_path_together():
    """The operators in a row against autograd of the plain form in 64 bits."""
    table, ids, eids, w, dout, experts, head = _path_inputs(21)
    out, dw, dtable, offsets = _token_path(table, ids, eids, w, dout, experts, head)
    t64, w64 = table.double().requires_grad_(), w.double().requires_grad_()
    x = t64[ids] * 2
    want = ((x * head.double())[:, None] * w64[:, :, None]).sum(1)
    want.backward(dout.double())
    # values of order 10 through at most 20 roundings, 48-term dots, 20 tokens an id
    assert torch.allclose(out.double(), want.detach(), rtol=0, atol=20 * U * 100)
    assert torch.allclose(dw.double(), w64.grad, rtol=0, atol=(48 + 20) * U * 1000)
    assert torch.allclose(dtable.double(), t64.grad, rtol=0, atol=(20 + 20) * U * 1000)
    assert np.array_equal(offsets.cpu().numpy(), _group_want(eids.cpu().numpy(), experts)[2])


def test_the_token_path_in_a_graph_and_on_a_side_stream():
    args = _path_inputs(22)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        eager = _token_path(*args)
        _token_path(*args)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = _token_path(*args)
    for round_ in range(4):
        for a, seed in ((args[1], 30 + round_), (args[2], 40 + round_)):
            a.copy_(a[torch.randperm(a.shape[0], device=DEV, generator=_gen(seed))])
        args[0].add_(0.25)
        graph.replay()
        torch.cuda.synchronize()
        eager = _token_path(*args)
        for a, b in zip(captured, eager):
            assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("chunks,extra", [(65, 0), (80, 1), (81, 3), (128, 0), (129, 0), (160, 1), (200, 0), (256, 0), (257, 1)])
def test_rows_by_half_the_threads(dtype, chunks, extra):
    """Widths around those at which a row's threads take two chunks each, with
    a last chunk that starts early; a table large enough for it too."""
    each = 16 // torch.empty(0, dtype=dtype).element_size()
    width = chunks * each - extra
    g = _gen(width)
    vocab, n = 16_400, 900
    ids = (torch.rand(n, device=DEV, generator=g) ** 6 * (vocab + 1)).long() - 1
    _grad_case(ids, vocab, width, dtype, 0.5, dtype, width)
    table = _randn(g, 301, width, dtype=dtype)
    few = ids % 300 - (ids < 0).long()
    inside = few >= 0
    want = torch.where(inside[:, None], table[few.clamp(min=0)], torch.zeros((), dtype=dtype, device=DEV))
    assert torch.equal(ssc.embed_rows(table, few), want)
    test_dispatch_combine_and_gradients(dtype, 130, 3, 5, width, 0.2)


def test_scale_of_other_number_types():
    table = torch.randn(9, 16, device=DEV)
    ids = torch.tensor([3, 8, -1, 0], device=DEV)
    want = ssc.embed_rows(table, ids, 0.5)
    order, _, offsets = ssc.group_by_key(ids, 9)
    dtable = ssc.embed_rows_grad(want, ids, order, offsets, 0.5)
    for scale in (np.float32(0.5), torch.tensor(0.5), torch.tensor(0.5, device=DEV)):
        assert torch.equal(ssc.embed_rows(table, ids, scale), want)
        assert torch.equal(ssc.embed_rows_grad(want, ids, order, offsets, scale), dtable)


def test_two_groupings_at_once():
    """Calls in flight on two streams, each with a scratch of its own."""
    r = np.random.RandomState(9)
    keys = [r.randint(-1, 1000, 100_003).astype(np.int64) for _ in range(2)]
    dev = [torch.from_numpy(k).to(DEV) for k in keys]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(ssc.group_by_key(dev[i], 1000))
    torch.cuda.synchronize()
    for i in range(2):
        order, ranks, offsets = _group_want(keys[i], 1000)
        for o, k, f in got[i]:
            assert np.array_equal(f.cpu().numpy(), offsets) and np.array_equal(k.cpu().numpy(), ranks)
            assert np.array_equal(o[:order.size].cpu().numpy(), order)


def test_results_repeat_bit_for_bit():
    g = _gen(12)
    n, vocab, width = 30_000, 200, 72
    ids = (torch.rand(n, device=DEV, generator=g) ** 5 * vocab).long()
    dout = _randn(g, n, width, dtype=torch.bfloat16)
    order, _, offsets = ssc.group_by_key(ids, vocab)
    first = ssc.embed_rows_grad(dout, ids, order, offsets, 1.0, dtype=torch.float32)
    for _ in range(5):
        assert torch.equal(first, ssc.embed_rows_grad(dout, ids, order, offsets, 1.0, dtype=torch.float32))


def test_refusals_on_the_gpu():
    x = torch.zeros(10, 8, device=DEV)
    ids = torch.zeros(10, dtype=torch.int64, device=DEV)
    ranks = torch.zeros(10, 2, dtype=torch.int32, device=DEV)
    w = torch.zeros(10, 2, device=DEV)
    with pytest.raises(TypeError):
        ssc.group_by_key(x, 4)
    for groups in (0, -1, 2 ** 31):
        with pytest.raises((ValueError, ssc.SSCError)):
            ssc.group_by_key(ids, groups)
    with pytest.raises(TypeError):
        ssc.group_by_key(ids, 4, order=torch.zeros(10, dtype=torch.int64, device=DEV))
    with pytest.raises(ValueError):
        ssc.group_by_key(ids, 4, offsets=torch.zeros(4, dtype=torch.int32, device=DEV))
    with pytest.raises(TypeError):
        ssc.embed_rows(x.double(), ids)
    with pytest.raises(ValueError):
        ssc.embed_rows(x[:, ::2], ids)
    with pytest.raises(TypeError):
        ssc.embed_rows(x, ids.float())
    with pytest.raises(ssc.SSCError):
        ssc.embed_rows(x, ids, out=x[:10])  # the output over the table
    with pytest.raises(ValueError):
        ssc.dispatch_rows(x[:9], ranks)
    with pytest.raises(TypeError):
        ssc.dispatch_rows(x, ranks.long())
    with pytest.raises(ValueError):
        ssc.combine_rows(x, ranks, w[:, :1].contiguous())
    with pytest.raises(TypeError):
        ssc.combine_rows(x, ranks, w.half())
    with pytest.raises(TypeError):
        ssc.combine_rows_grad(x, x.half(), ranks, w)
    with pytest.raises(ssc.SSCError):
        ssc.combine_rows_grad(x, x, ranks, w, dy=x)
    order, _, offsets = ssc.group_by_key(ids, 4)
    with pytest.raises(ValueError):
        ssc.embed_rows_grad(x, ids, order, offsets, accumulate=True)
    with pytest.raises(TypeError):
        ssc.embed_rows_grad(x, ids, order, offsets, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        ssc.embed_rows_grad(x[:5], ids, order, offsets)
    many = torch.zeros(300, dtype=torch.int64, device=DEV)
    order, _, offsets = ssc.group_by_key(many, 4)
    with pytest.raises(ValueError):
        ssc.embed_rows_grad(torch.zeros(300, 8, device=DEV), many, order, offsets,
                            scratch=torch.zeros(8, dtype=torch.uint8, device=DEV))
