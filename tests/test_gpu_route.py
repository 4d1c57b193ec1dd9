"""ssc_route_rows and its gradient on the GPU against the definition in 64 bits.

Ids and counts are equal. Steps below are half steps of fp32, 2^-24 of a value.
An exponential is 2 to the power of a difference d of two fp32 logits times log2(e):
the difference, the product and the constant are off by 2.3 |d| of them, |d| being
110 at most where anything is left, and it is itself within 4. A row's sum is added up
in at most 24 + 6 steps, and products and quotients round 4 times: under 60 + 2 |d| in
all, for 0.3 |d| is at most 22 of what 60 leaves. A mean adds up to 64 rows a
lane, 3 lane steps and 9 of the wavefronts in fp32, and the rest in fp64: with
the 38 + 2.3 |d| of a softmax below the 135 + 2 |d| allowed."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import scan_stream_compaction_amd as ssc

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = [torch.float32, torch.bfloat16, torch.float16]
STEP = 2.0 ** -24


def reference(logits, per, normalize, live=None):
    """(ids, weights, p, d): in 64 bits, on the host; d the row's distances from its largest logit."""
    x = logits.detach().double().cpu().numpy()
    n, experts = x.shape
    x = np.where(np.isnan(x), -np.inf, x)
    if live is not None:
        x = np.where(live.cpu().numpy().astype(bool)[:, None], x, -np.inf)
    top = x.max(1, keepdims=True)
    lifted = np.where(top == np.inf, np.where(x == np.inf, 0.0, -np.inf), x)
    top = np.where(np.isfinite(top), top, 0.0)
    d = np.where(lifted > -np.inf, lifted - top, -np.inf)
    e = np.exp(d)
    s = e.sum(1, keepdims=True)
    p = np.where(s > 0, e / np.where(s > 0, s, 1.0), 0.0)
    ids = np.argsort(-lifted, axis=1, kind="stable")[:, :per]
    expert = np.take_along_axis(lifted, ids, 1) > -np.inf
    w = np.where(expert, np.take_along_axis(p, ids, 1), 0.0)
    if normalize:
        s = w.sum(1, keepdims=True)
        w = np.where(s > 0, w / np.where(s > 0, s, 1.0), 0.0)
    return np.where(expert, ids, -1), w, p, np.where(np.isfinite(d), -d, 0.0)


def steps(d):
    return 60 + 2 * float(min(d.max(initial=0.0), 110.0))


def check_forward(logits, per, normalize=True, live=None):
    ids, weights, counts, share, loss = ssc.route_rows(logits, per, normalize=normalize, live=live, balance=True)
    alone = ssc.route_rows(logits, per, normalize=normalize, live=live)
    torch.cuda.synchronize()
    rid, rw, p, d = reference(logits, per, normalize, live)
    n, experts = p.shape
    assert np.array_equal(ids.cpu().numpy(), rid), np.argwhere(ids.cpu().numpy() != rid)[:5]
    assert torch.equal(alone[0], ids) and torch.equal(alone[1], weights)
    tol = steps(d) * STEP
    w = weights.double().cpu().numpy()
    assert np.all(np.abs(w - rw) <= rw * tol + 2.0 ** -126)
    alive = int((p.sum(1) > 0).sum())
    rc = np.bincount(rid[rid >= 0], minlength=experts)
    assert np.array_equal(counts.cpu().numpy(), np.append(rc, alive))
    rs = p.sum(0) / max(alive, 1)
    tol += 75 * STEP
    assert np.all(np.abs(share.double().cpu().numpy() - rs) <= rs * tol + 2.0 ** -126)
    rl = experts * (rc / (per * max(alive, 1)) * rs).sum()
    assert abs(float(loss) - rl) <= rl * tol + 2.0 ** -126
    return ids, weights, counts, share, loss


def inputs(seed, n, experts, dtype, spread=1.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    x = torch.randn(n, experts, device=DEV, generator=g) * spread + 0.5 * torch.randn(experts, device=DEV, generator=g)
    return x.to(dtype), g


SIZES = [(1, 1, 1), (2, 2, 2), (7, 3, 1), (33, 8, 8), (31, 9, 2), (64, 16, 5), (65, 17, 17), (100, 32, 4), (257, 33, 6),
         (63, 64, 64), (130, 65, 8), (1000, 128, 8), (999, 129, 64), (300, 160, 6), (50, 192, 9), (50, 193, 3), (70, 256, 33),
         (129, 257, 8), (40, 511, 64), (41, 512, 1), (17, 513, 16), (19, 1024, 64), (5, 1000, 8)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,experts,per", SIZES)
def test_forward_sizes(n, experts, per, dtype):
    x, g = inputs(n + experts, n, experts, dtype)
    check_forward(x, per)
    live = torch.rand(n, device=DEV, generator=g) < 0.7
    check_forward(x, per, normalize=False, live=live)
    # few values: equal logits, the lowest expert first
    check_forward((x.float() * 2).round().to(dtype), per)


@pytest.mark.parametrize("experts", [24, 150, 250, 500, 1000])
def test_tokens_of_one_workgroup_and_more(experts):
    alone = 4 * 16_384 // (8 * (1 if experts <= 128 else 2 if experts <= 256 else 4 if experts <= 512 else 8) * 16)
    for n in (alone, alone + 1):
        x, g = inputs(n, n, experts, torch.float32)
        check_forward(x, 5, live=torch.rand(n, device=DEV, generator=g) < 0.8)


@pytest.mark.parametrize("n", [16_383, 40_000, 300_001])
def test_many_tokens(n):
    x, g = inputs(n, n, 24, torch.bfloat16, 2.0)
    check_forward(x, 4, live=(torch.rand(n, device=DEV, generator=g) < 0.9).to(torch.uint8))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("experts", [5, 40, 128, 200, 700])
def test_masked_and_special_logits(dtype, experts):
    inf = float("inf")
    x, _ = inputs(3, 14, experts, dtype)
    x[0] = -inf
    x[1] = float("nan")
    x[2, 1:] = -inf
    x[3, :-1] = -inf
    x[4, ::2] = float("nan")
    x[5, 3] = inf
    x[6, [0, 2, experts - 1]] = inf
    x[7] = torch.finfo(dtype).min
    x[8, 2:] = torch.finfo(dtype).min
    x[9] = inf
    x[10] = torch.finfo(dtype).max
    x[11] = torch.where(torch.arange(experts, device=DEV) % 2 == 0, 0.0, -0.0).to(dtype)
    x[12, 1] = -inf
    for per in (1, 4, min(experts, 64)):
        for normalize in (True, False):
            check_forward(x, per, normalize)
    check_forward(x, 2, live=torch.zeros(14, dtype=torch.bool, device=DEV))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("experts", [7, 30, 100, 150, 300])
def test_logits_of_the_last_bits(dtype, experts):
    """Subnormal logits of both signs beside zeros, and neighbours of one step."""
    g = torch.Generator(device=DEV)
    g.manual_seed(experts)
    small = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
    x = (torch.randint(-3, 4, (40, experts), device=DEV, generator=g).double() * small).to(dtype)
    for per in (1, 4, 7):
        check_forward(x, per)
    near = (1.0 + torch.randint(0, 5, (40, experts), device=DEV, generator=g).double() * torch.finfo(dtype).eps).to(dtype)
    for sign in (1, -1):
        check_forward(near * sign, 5)


def gradient(logits, ids, dweights, normalize, live, counts, dloss):
    """(gradient, bound): the formula in 64 bits, and what |g| bounds its roundings by."""
    per = ids.shape[1]
    _, _, p, d = reference(logits, 1, False, live)
    n, experts = p.shape
    i = ids.cpu().numpy()
    ok = (i >= 0) & (i < experts)
    at = np.where(ok, i, 0)
    rows = np.arange(n)[:, None]
    dw = np.zeros_like(p[:, :1].repeat(per, 1)) if dweights is None else np.where(ok, dweights.double().cpu().numpy(), 0.0)
    g = np.zeros_like(p)
    out, size = np.zeros_like(p), np.zeros_like(p)
    if normalize:
        w = np.where(ok, p[rows, at], 0.0)
        s = w.sum(1, keepdims=True)
        w = np.where(s > 0, w / np.where(s > 0, s, 1.0), 0.0)
        np.add.at(out, (rows, at), w * (dw - (w * dw).sum(1, keepdims=True)))
        np.add.at(size, (rows, at), w * (np.abs(dw) + (w * np.abs(dw)).sum(1, keepdims=True)))
    else:
        np.add.at(g, (rows, at), dw)
    even = np.zeros(experts)
    if counts is not None and int(counts[-1]) > 0:
        c = counts.double().cpu().numpy()
        even = float(dloss) * experts * c[:-1] / (c[-1] * per) / c[-1]
    a = np.abs(g) + np.abs(even)
    g = g + even
    out += p * (g - (p * g).sum(1, keepdims=True))
    size += p * (a + (p * a).sum(1, keepdims=True))
    return out, size, d


def check_gradient(logits, ids, dweights, normalize=True, live=None, counts=None, dloss=None):
    got = ssc.route_rows_grad(logits, ids, dweights, normalize=normalize, live=live, counts=counts, dloss=dloss)
    torch.cuda.synchronize()
    want, size, d = gradient(logits, ids, dweights, normalize, live, counts, dloss)
    half = torch.finfo(logits.dtype).eps / 2
    tol = size * 2 * steps(d) * STEP + np.abs(want) * half + torch.finfo(logits.dtype).smallest_normal * half + 2.0 ** -126
    if logits.dtype == torch.float16:
        tol += 2.0 ** -25  # half a step of its smallest values
    assert got.shape == logits.shape and got.dtype == logits.dtype
    err = np.abs(got.double().cpu().numpy() - want)
    assert np.all(err <= tol), (np.argwhere(err > tol)[:5], (err / tol).max())
    return got


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,experts,per", SIZES)
def test_gradient_sizes(n, experts, per, dtype):
    x, g = inputs(n * 7 + experts, n, experts, dtype)
    live = torch.rand(n, device=DEV, generator=g) < 0.8
    dw = torch.randn(n, per, device=DEV, generator=g)
    dloss = torch.full((1,), 0.5 * n, device=DEV)
    for normalize in (True, False):
        ids, _, counts, _, _ = ssc.route_rows(x, per, normalize=normalize, live=live, balance=True)
        check_gradient(x, ids, dw, normalize, live, counts, dloss)
        check_gradient(x, ids, dw, normalize, live)
    check_gradient(x, ids, None, True, live, counts, dloss)


@pytest.mark.parametrize("dtype", TYPES)
def test_gradient_of_masked_rows(dtype):
    inf = float("inf")
    x, g = inputs(5, 12, 40, dtype)
    x[0] = -inf
    x[1] = float("nan")
    x[2, 1:] = -inf
    x[3, 3:] = -inf
    x[4, ::2] = float("nan")
    x[5, 3] = inf
    x[6, [0, 2, 39]] = inf
    x[7] = torch.finfo(dtype).min
    x[8, 5:] = torch.finfo(dtype).min
    dw = torch.randn(12, 6, device=DEV, generator=g)
    dloss = torch.ones(1, device=DEV)
    for normalize in (True, False):
        ids, _, counts, _, _ = ssc.route_rows(x, 6, normalize=normalize, balance=True)
        got = check_gradient(x, ids, dw, normalize, None, counts, dloss)
        assert bool((got[:2] == 0).all()) and bool(torch.isfinite(got).all())


def test_ids_of_any_kind():
    """Ids outside add nothing; one that is named twice counts twice."""
    x, g = inputs(6, 200, 24, torch.float32)
    ids = torch.randint(-2, 26, (200, 9), device=DEV, generator=g).int()
    ids[0] = 7
    ids[1] = -1
    ids[2] = 2 ** 31 - 1
    ids[3] = -2 ** 31
    dw = torch.randn(200, 9, device=DEV, generator=g)
    for normalize in (True, False):
        check_gradient(x, ids, dw, normalize)


def test_gradient_by_differences():
    """Along random directions, against central differences of the definition in 64 bits (their error is of second order: 1e-8)."""
    x, g = inputs(8, 40, 20, torch.float32)
    for normalize in (True, False):
        ids, _, counts, _, _ = ssc.route_rows(x, 3, normalize=normalize, balance=True)
        dw = torch.randn(40, 3, device=DEV, generator=g)
        dloss = torch.full((1,), 3.0, device=DEV)
        got = ssc.route_rows_grad(x, ids, dw, normalize=normalize, counts=counts, dloss=dloss).double()
        c = counts.double()

        def value(z):
            p = torch.softmax(z, 1)
            w = p.gather(1, ids.long())
            if normalize:
                w = w / w.sum(1, keepdim=True)
            return (w * dw.double()).sum() + 3.0 * 20 * (c[:-1] / (3 * c[-1]) * p.mean(0)).sum()

        for _ in range(5):
            v = torch.randn(40, 20, device=DEV, generator=g).double()
            h = 1e-4
            slope = (value(x.double() + h * v) - value(x.double() - h * v)) / (2 * h)
            size = float((got.abs() * v.abs()).sum())
            assert abs(float((got * v).sum() - slope)) <= 1e-5 * size + 1e-6


def test_counts_of_several_calls():
    """A batch in two parts, their counts added up: the gradient of the whole batch's loss."""
    x, _ = inputs(9, 300, 48, torch.float32)
    ids, _, counts, _, _ = ssc.route_rows(x, 4, balance=True)
    dloss = torch.full((1,), 100.0, device=DEV)
    whole = ssc.route_rows_grad(x, ids, None, counts=counts, dloss=dloss)
    parts = [ssc.route_rows(y, 4, balance=True) for y in (x[:100], x[100:])]
    total = parts[0][2] + parts[1][2]
    assert torch.equal(total, counts)
    got = torch.cat([ssc.route_rows_grad(y, p[0], None, counts=total, dloss=dloss) for y, p in zip((x[:100], x[100:]), parts)])
    assert torch.equal(got, whole)


def test_strided_rows_given_outputs_and_repeats():
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    full = torch.randn(60, 3, 101, device=DEV, generator=g).to(torch.bfloat16)
    x = full[:, 1, 1:98]
    assert not x.is_contiguous()
    want = check_forward(x, 5)
    buf = torch.full((5, 400), -9, dtype=torch.int32, device=DEV)
    outs = dict(ids=buf[0, 3:303], weights=buf[1, 3:303].view(torch.float32), counts=buf[2, 3:101],
                share=buf[3, 3:100].view(torch.float32), loss=buf[4, 3:4].view(torch.float32))
    scratch = torch.full((ssc.route_scratch_bytes(60, 97),), 255, dtype=torch.uint8, device=DEV)
    for _ in range(3):
        got = ssc.route_rows(x, 5, balance=True, scratch=scratch, **outs)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert got[0].shape == (60, 5)
    for i, n in enumerate((300, 300, 98, 97, 1)):
        assert bool((buf[i, :3] == -9).all()) and bool((buf[i, 3 + n:] == -9).all())
    dw = torch.randn(60, 5, device=DEV, generator=g)
    grad = torch.full((60 * 97 + 7,), 5.0, device=DEV, dtype=torch.bfloat16)
    first = ssc.route_rows_grad(x, want[0], dw, out=grad)
    assert first.shape == (60, 97) and bool((grad[60 * 97:] == 5).all())
    assert torch.equal(first, check_gradient(x, want[0], dw))


def test_no_tokens():
    x = torch.empty(0, 12, device=DEV)
    ids, weights, counts, share, loss = ssc.route_rows(x, 3, balance=True)
    assert ids.shape == (0, 3) and bool((counts == 0).all()) and bool((share == 0).all()) and float(loss) == 0
    assert ssc.route_rows_grad(x, ids, weights, counts=counts, dloss=loss).shape == (0, 12)


def test_the_layer_with_its_gradients():
    """Router, grouping, rows to the experts and back, and all gradients, against
    autograd of the dense formula in 64 bits: the library's fp32 sums of up to 32
    products of a few units lie within 1e-4 of the gradients' size."""
    g = torch.Generator(device=DEV)
    g.manual_seed(12)
    n, width, experts, per = 200, 32, 12, 3
    x = torch.randn(n, width, device=DEV, generator=g)
    router = torch.randn(width, experts, device=DEV, generator=g) * 0.3
    mats = torch.randn(experts, width, width, device=DEV, generator=g) * 0.2
    dout = torch.randn(n, width, device=DEV, generator=g)
    coef = 0.7
    logits = x @ router
    ids, weights, counts, _, loss = ssc.route_rows(logits, per, balance=True)
    _, ranks, offsets = ssc.group_by_key(ids, experts, order=False)
    rows = ssc.dispatch_rows(x, ranks)
    bounds = offsets.tolist()
    assert torch.equal(offsets.diff(), counts[:-1])
    y = torch.cat([rows[a:b] @ mats[e] for e, (a, b) in enumerate(zip(bounds, bounds[1:]))])
    out = ssc.combine_rows(y, ranks, weights)
    dy, dweights = ssc.combine_rows_grad(dout, y, ranks, weights)
    drows = torch.cat([dy[a:b] @ mats[e].T for e, (a, b) in enumerate(zip(bounds, bounds[1:]))])
    dlogits = ssc.route_rows_grad(logits, ids, dweights, counts=counts, dloss=torch.full((1,), coef, device=DEV))
    dx = ssc.dispatch_rows_grad(drows, ranks) + dlogits @ router.T

    xd, rd = x.double().cpu().requires_grad_(), router.double().cpu().requires_grad_()
    p = torch.softmax(xd @ rd, 1)
    w = p.gather(1, ids.long().cpu())
    w = w / w.sum(1, keepdim=True)
    full = torch.stack([xd @ m for m in mats.double().cpu()], 1)
    want = (w[..., None] * full.gather(1, ids.long().cpu()[..., None].expand(-1, -1, width))).sum(1)
    c = counts.double().cpu()
    balance = experts * (c[:-1] / (per * n) * p.mean(0)).sum()
    ((want * dout.double().cpu()).sum() + coef * balance).backward()
    near = lambda a, b: float((a.double().cpu() - b).abs().max() / b.abs().max()) < 1e-4  # noqa: E731
    assert near(out, want.detach()) and abs(float(loss) - float(balance.detach())) < 1e-5
    assert near(dx, xd.grad) and near(x.T @ dlogits, rd.grad)


def test_graph_replays_and_streams():
    """Captured on a side stream, replayed over changed inputs with other work between."""
    x, g = inputs(21, 500, 64, torch.float32)
    live = torch.rand(500, device=DEV, generator=g) < 0.9
    dloss = torch.ones(1, device=DEV)

    def both():
        ids, weights, counts, share, loss = ssc.route_rows(x, 4, live=live, balance=True)
        return ids, weights, counts, share, loss, ssc.route_rows_grad(x, ids, weights, live=live, counts=counts, dloss=dloss)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both()
    for i in range(4):
        x.copy_(torch.randn(500, 64, device=DEV, generator=g))
        live.copy_(torch.rand(500, device=DEV, generator=g) < 0.5)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, both()))


def test_two_calls_at_once():
    xs = [inputs(30 + i, 3000, 160, torch.bfloat16)[0] for i in range(2)]
    want = [ssc.route_rows(x, 8, balance=True) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = []
    for _ in range(5):
        for x, s in zip(xs, streams):
            with torch.cuda.stream(s):
                got.append(ssc.route_rows(x, 8, balance=True))
    torch.cuda.synchronize()
    for i, r in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(r, want[i % 2]))
