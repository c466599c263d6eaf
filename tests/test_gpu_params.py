"""Embedding, its gradient, and clipping of gradients against the oracle (64 bits),
on the GPU.

Tolerances, with u = 2^-24 the half step of 32 bits and w that of the result's type:

* lookup: one product in 32 bits and one rounding, (u + w) |value|;
* the table's gradient: sums of n terms in 32 bits and a product, (n + 1) u scale
  sum |terms|, with accumulate one addition more, and w |value|;
* the norm: the squares of up to 8 elements added in 32 bits (each addition rounds a sum
  of positive terms below the last: 8 u of it, 4 u of its root), those sums in 64 (2 n
  2^-53), rounded to 32 (u);
* a clipped gradient: the factor rounded to 32 bits and a product, 2 u and the norm's u
  in the factor, and w; fp16 by half its smallest step besides.
"""

import math

import numpy as np
import pytest

import oracle as O
from gpu_util import say

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {"bf16": (2.0 ** -8, 2.0 ** -126), "fp16": (2.0 ** -11, 2.0 ** -25), "fp32": (U, 2.0 ** -126)}


@pytest.fixture(scope="module")
def torch():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return torch


@pytest.fixture(scope="module")
def thd(torch):
    import context_packed_sequence_amd as thd
    return thd


def _dtype(torch, name):
    return {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[name]


def _name(torch, dtype):
    return {torch.bfloat16: "bf16", torch.float16: "fp16", torch.float32: "fp32"}[dtype]


def _host(t):
    return t.detach().double().cpu().numpy()


def _normal(torch, rng, shape, dtype, size=1.0):
    return torch.from_numpy(rng.normal(0, size, shape).astype(np.float32)).to(_dtype(torch, dtype)).cuda()


def _within(got, want, bound, what):
    got = _host(got)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    with np.errstate(invalid="ignore"):
        bad = ~(np.abs(got - want) <= bound) & ~(got == want) & ~(np.isnan(got) & np.isnan(want))
    if bad.any():
        i = tuple(int(x) for x in np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} off, first at {i}: {got[i]!r} for {want[i]!r}, "
                             f"bound {np.broadcast_to(bound, got.shape)[i]!r}")


def _tokens(rng, rows, vocab, kind):
    if kind == "one":
        return np.full(rows, vocab // 2)
    if kind == "all":
        return np.arange(rows) % vocab
    return np.minimum(vocab - 1, np.exp(rng.random(rows) * math.log(vocab)).astype(np.int64) - 1).clip(0)


# ---- embedding ------------------------------------------------------------------

ROWS = [(1, 1, 1), (24, 32000, 8), (33, 7, 1001), (64, 512, 64), (5, 100003, 3), (1000, 511, 260)]


@pytest.mark.parametrize("rows,vocab,width", ROWS + [(9001, 300, 17)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_lookup(torch, thd, rows, vocab, width, dtype):
    say("embedding", rows, vocab, width, dtype)
    rng = np.random.default_rng([1, rows, vocab, width])
    table = _normal(torch, rng, (vocab, width), dtype)
    ids, mask = _tokens(rng, rows, vocab, "text"), (rng.random(rows) < 0.8).astype(np.uint8)
    ids[mask == 0] = -5     # not looked at
    got, status = thd.embedding(torch.from_numpy(ids).cuda(), table, mask=torch.from_numpy(mask).cuda(), scale=0.37)
    want = O.embedding(ids, _host(table), mask, np.float32(0.37).astype(np.float64))
    half, tiny = HALF[dtype]
    assert int(status) == 0
    _within(got, want, (U + half) * np.abs(want) + tiny, "rows")


@pytest.mark.parametrize("rows", [40, 9000])
def test_lookup_of_no_row(torch, thd, rows):
    say("embedding ids outside the table", rows)
    rng = np.random.default_rng(2)
    table = _normal(torch, rng, (50, 24), "bf16")
    ids = rng.integers(0, 50, rows)
    ids[[3, 17, 39]] = [-1, 50, 2 ** 40]
    got, status = thd.embedding(torch.from_numpy(ids).cuda(), table)
    want = O.embedding(ids, _host(table))
    assert int(status) == thd.THD_ERR_TOKEN and np.isnan(want[17]).all()
    _within(got, want, 0.0, "rows")
    ids[:] = 3
    assert int(thd.embedding(torch.from_numpy(ids).cuda(), table)[1]) == 0


def test_lookup_layouts(torch, thd):
    say("embedding layouts")
    rng = np.random.default_rng(3)
    room = _normal(torch, rng, (60, 40), "bf16")
    table = room[:, 3:24]                                   # rows of 21 at a stride of 40, not 16-byte aligned
    ids = torch.from_numpy(rng.integers(0, 60, (4, 9))).cuda()
    got, _ = thd.embedding(ids, table)
    assert got.shape == (4, 9, 21) and torch.equal(got, table[ids])
    to = torch.full((36, 30), 5.0, device="cuda", dtype=torch.bfloat16)
    back, _ = thd.embedding(ids, table, out=to[:, 1:22])
    assert torch.equal(to[:, 1:22], got.view(36, 21)) and bool((to[:, 0] == 5).all() and (to[:, 22:] == 5).all())
    empty, status = thd.embedding(ids[:0], table)
    assert empty.shape == (0, 9, 21) and int(status) == 0


@pytest.mark.parametrize("rows,vocab,width", ROWS + [(31, 5, 8), (32, 5, 8), (65, 2, 8), (8192, 700, 12),
                                                     (8193, 700, 12), (20000, 262143, 5), (70000, 40, 9)])
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("bf16", "fp32"), ("fp16", "fp16"), ("fp32", "fp32")])
def test_table_gradient(torch, thd, rows, vocab, width, dtype, out):
    rng = np.random.default_rng([4, rows, vocab, width])
    half, tiny = HALF[out]
    for kind in ("text", "one", "all"):
        say("embedding gradient", rows, vocab, width, dtype, out, kind)
        drows = _normal(torch, rng, (rows, width), dtype)
        ids, mask = _tokens(rng, rows, vocab, kind), (rng.random(rows) < 0.9).astype(np.uint8)
        ids[mask == 0] = vocab + 3
        args = torch.from_numpy(ids).cuda(), vocab
        more = dict(mask=torch.from_numpy(mask).cuda(), scale=0.37)
        to = None if out == dtype else torch.full((vocab, width), 9.0, device="cuda")
        drows[torch.from_numpy(mask == 0).cuda()] = math.nan
        got, status = thd.embedding_backward(drows, *args, out=to, **more)
        assert int(status) == 0
        scale = np.float32(0.37).astype(np.float64)
        x = np.nan_to_num(_host(drows))
        want = O.embedding_backward(x, ids, vocab, mask, scale)
        n = np.bincount(ids[mask != 0], minlength=vocab)[:, None]
        total = O.embedding_backward(np.abs(x), ids, vocab, mask, scale)
        bound = (n + 1) * U * total + half * np.abs(want) + tiny * (n > 0)
        _within(got, want, bound, f"gradient {kind}")
        again, _ = thd.embedding_backward(drows, *args, out=None if to is None else torch.empty_like(to), **more)
        assert torch.equal(got, again)


@pytest.mark.parametrize("rows", [50, 9000])
def test_table_gradient_added(torch, thd, rows):
    say("embedding gradient added", rows)
    rng = np.random.default_rng(5)
    ids = rng.integers(0, 30, rows) * 2                    # odd tokens do not occur
    drows = _normal(torch, rng, (rows, 33), "bf16")
    old = _normal(torch, rng, (60, 33), "fp32")
    old[1::2] = math.nan                                   # not touched
    to = old.clone()
    got, status = thd.embedding_backward(drows, torch.from_numpy(ids).cuda(), 60, out=to, accumulate=True)
    assert got is to and int(status) == 0
    want = O.embedding_backward(_host(drows), ids, 60)
    total = O.embedding_backward(np.abs(_host(drows)), ids, 60)
    n = np.bincount(ids, minlength=60)[:, None]
    want[0::2] += _host(old)[0::2]
    want[1::2] = np.nan
    _within(to, want, (n + 1) * U * (total + np.abs(np.nan_to_num(_host(old)))) + U * np.abs(want), "sums")


@pytest.mark.parametrize("at", [0, 8191, 8192, 10000])
def test_status_of_long_rows(torch, thd, at):
    # many ids, looked through beside the copy of rows of 4096 bytes
    say("embedding status of long rows", at)
    table = torch.ones((50, 2048), device="cuda", dtype=torch.bfloat16)
    ids = torch.arange(10001, device="cuda") % 50
    mask = torch.ones(10001, device="cuda", dtype=torch.uint8)
    assert int(thd.embedding(ids, table, mask=mask)[1]) == 0
    ids[at] = 50
    got, status = thd.embedding(ids, table, mask=mask)
    assert int(status) == thd.THD_ERR_TOKEN and bool(got[at].isnan().all()) and int(got.isnan().sum()) == 2048
    mask[at] = 0
    got, status = thd.embedding(ids, table, mask=mask)
    assert int(status) == 0 and not got[at].any()


@pytest.mark.parametrize("rows", [64, 10000])
def test_table_gradient_of_no_row(torch, thd, rows):
    say("embedding gradient ids outside the table", rows)
    rng = np.random.default_rng(6)
    ids = rng.integers(0, 9, rows)
    ids[[0, 5, 60]] = [-1, 9, 2 ** 35]
    drows = torch.ones((rows, 4), device="cuda")
    got, status = thd.embedding_backward(drows, torch.from_numpy(ids).cuda(), 9)
    assert int(status) == thd.THD_ERR_TOKEN
    _within(got, O.embedding_backward(np.ones((rows, 4)), ids, 9), 0.0, "whole numbers")


def test_table_gradient_of_no_tokens(torch, thd):
    say("embedding gradient of no tokens")
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    got, status = thd.embedding_backward(torch.empty((0, 5), device="cuda"), none, 7)
    assert int(status) == 0 and got.shape == (7, 5) and not got.any()
    masked = torch.zeros(20, dtype=torch.uint8, device="cuda")
    ids = torch.zeros(20, dtype=torch.int64, device="cuda")
    got, _ = thd.embedding_backward(torch.full((20, 5), math.nan, device="cuda"), ids, 7, mask=masked)
    assert not got.any()


def test_table_gradient_layouts(torch, thd):
    say("embedding gradient layouts")
    rng = np.random.default_rng(7)
    ids = torch.from_numpy(rng.integers(0, 40, 300)).cuda()
    room = _normal(torch, rng, (300, 50), "bf16")
    want, _ = thd.embedding_backward(room[:, 5:38].contiguous(), ids, 40)
    to = torch.full((40, 64), 3.0, device="cuda", dtype=torch.bfloat16)
    thd.embedding_backward(room[:, 5:38], ids.view(3, 100), 40, out=to[:, 1:34])
    assert torch.equal(to[:, 1:34], want) and bool((to[:, 0] == 3).all() and (to[:, 34:] == 3).all())


# ---- gradients --------------------------------------------------------------------

SIZES = [[1], [0, 5, 0], [16383, 16384, 16385, 8192, 8193, 7], [3] * 95, [3] * 96, [5] * 97, [11] * 200,
         [100000, 1, 70001], []]


@pytest.mark.parametrize("sizes", SIZES)
@pytest.mark.parametrize("dtypes", [["bf16"], ["fp16"], ["fp32"], ["bf16", "fp32", "fp16"]])
def test_clipping(torch, thd, sizes, dtypes):
    say("clipping", sizes[:6], len(sizes), dtypes)
    rng = np.random.default_rng([8, len(sizes)])
    grads = [_normal(torch, rng, (n,), dtypes[i % len(dtypes)]) for i, n in enumerate(sizes)]
    host = [_host(g) for g in grads]
    scale = 0.75
    true = O.gradient_norm(host, scale)
    rel = 5 * U + 2 * sum(sizes) * 2.0 ** -53
    norm, status = thd.gradient_norm(grads, scale)
    assert int(status) == 0
    _within(norm, np.array([true]), rel * true, "norm")
    for max_norm in (0.4 * true + 1e-9, 2 * true + 1.0, math.inf):
        _, want = O.clip_gradients(host, max_norm, scale)
        inplace = [g.clone() for g in grads]
        same = [torch.empty_like(g) for g in grads]
        wide = [torch.empty(g.shape, device="cuda") for g in grads]
        for outs, kind in ((None, inplace), (same, same), (wide, wide)):
            got, status = thd.clip_gradients(inplace if outs is None else grads, max_norm, scale=scale, outs=outs)
            assert int(status) == 0
            _within(got, np.array([true]), rel * true, "norm")
            for i, (x, y) in enumerate(zip(kind, want)):
                half, tiny = HALF[_name(torch, x.dtype)]
                _within(x, y, (4 * U + rel + half) * np.abs(y) + tiny, f"gradient {i}")


def test_shapes_and_unaligned_views(torch, thd):
    say("clipping views")
    rng = np.random.default_rng(9)
    flat = _normal(torch, rng, (50000,), "bf16")
    cuts = [0, 1, 3, 17000, 17007, 40001, 50000]
    grads = [flat[a:b] for a, b in zip(cuts, cuts[1:])]
    host = [_host(g) for g in grads]
    out = torch.empty(50001, device="cuda", dtype=torch.bfloat16)
    outs = [out[a + 1:b + 1] for a, b in zip(cuts, cuts[1:])]
    out[0] = 9
    thd.clip_gradients(grads, 1.0, outs=outs)
    _, want = O.clip_gradients(host, 1.0)
    _within(out[1:], np.concatenate(want), (8 * U + 2.0 ** -8) * np.abs(np.concatenate(want)), "views")
    assert float(out[0]) == 9
    two = flat[:40000].view(200, 200)
    thd.clip_gradients([two], 2.0)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_not_finite(torch, thd, bad):
    say("clipping", bad)
    grads = [torch.ones(5000, device="cuda", dtype=torch.bfloat16), torch.ones(70000, device="cuda")]
    grads[1][69999] = bad
    outs = [torch.full_like(g, 3.0) for g in grads]
    norm, status = thd.clip_gradients(grads, 1.0, outs=outs)
    assert int(status) == thd.THD_ERR_NORM and not math.isfinite(float(norm))
    assert not any(o.any() for o in outs)
    assert int(thd.gradient_norm(grads)[1]) == thd.THD_ERR_NORM
    thd.clip_gradients(grads, math.inf)
    assert not any(g.any() for g in grads)


def test_squares_past_32_bits(torch, thd):
    say("clipping of squares past 32 bits")
    for size in (1e25, 1e-30):
        g = torch.full((1000,), size, device="cuda")
        value = float(g[0])
        norm, status = thd.clip_gradients([g], 1e-3 if size > 1 else 1.0)
        assert int(status) == 0 and abs(float(norm) / (value * math.sqrt(1000)) - 1) < 2 * U
        if size > 1:
            assert abs(float(g[0]) / (1e-3 / math.sqrt(1000)) - 1) < 8 * U
        else:
            assert float(g[0]) == value


def test_norm_given(torch, thd):
    # two ranks' parts: the joined norm scales both
    say("clipping with a norm given")
    rng = np.random.default_rng(10)
    grads = [_normal(torch, rng, (n,), "fp32") for n in (1000, 333)]
    parts = torch.cat([thd.gradient_norm([g])[0] for g in grads])
    joined = parts.square().sum().sqrt().view(1)
    whole, _ = thd.gradient_norm(grads)
    assert abs(float(joined) / float(whole) - 1) < 1e-6
    want = [g.clone() for g in grads]
    thd.clip_gradients(want, 2.0)
    for g, w in zip(grads, want):
        norm, status = thd.clip_gradients([g], 2.0, norm=joined)
        assert int(status) == 0 and torch.equal(norm, joined)
        assert float((g - w).abs().max()) <= 1e-6 * float(w.abs().max())


def test_streams_and_graphs(torch, thd):
    say("embedding and clipping in a graph and on a stream")
    rng = np.random.default_rng(11)
    for rows in (100, 9000):
        ids = torch.from_numpy(_tokens(rng, rows, 500, "text")).cuda()
        table = _normal(torch, rng, (500, 48), "bf16")
        grads = [_normal(torch, rng, (n,), "bf16") for n in (40000, 9)]

        def step(stream=None):
            x, s1 = thd.embedding(ids, table, scale=2.0, stream=stream)
            d, s2 = thd.embedding_backward(x, ids, 500, stream=stream)
            outs = [torch.empty_like(g) for g in grads]
            norm, s3 = thd.clip_gradients(grads, 1.0, outs=outs, stream=stream)
            return x, d, *outs, norm, s1, s2, s3
        want = step()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        got = step(side)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = step()
        for i in range(4):
            table.normal_()
            ids.random_(0, 500 + 40 * (i == 2))             # the third holds ids outside the table
            grads[0].normal_()
            graph.replay()
            want = step()
            torch.cuda.synchronize()
            assert int(got[-2]) == int(got[-3]) == (thd.THD_ERR_TOKEN if i == 2 else 0)
            for a, b in zip(want, got):
                assert torch.equal(torch.nan_to_num(a.float()), torch.nan_to_num(b.float()))


def test_table_past_32_bits(torch, thd):
    say("embedding table past 4 GiB")
    vocab, width = 600_000, 4096
    table = torch.empty((vocab, width), device="cuda", dtype=torch.bfloat16)
    assert table.numel() * 2 > 1 << 32
    table[-2:] = torch.randn((2, width), device="cuda").to(torch.bfloat16)
    table[0] = 1.0
    ids = torch.tensor([vocab - 1, 0, vocab - 2, vocab - 1], device="cuda")
    got, status = thd.embedding(ids, table)
    assert int(status) == 0 and torch.equal(got, table[ids])
    grad, status = thd.embedding_backward(got, ids, vocab, out=table)
    assert int(status) == 0
    assert torch.equal(grad[0], got[1]) and torch.equal(grad[-2], got[2]) and not grad[1:-2].any()
    assert torch.equal(grad[-1], (got[0].float() + got[3].float()).to(torch.bfloat16))
