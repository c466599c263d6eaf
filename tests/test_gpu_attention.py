"""Attention inside documents and its gradient against the oracle (64 bits), on
the GPU; the tolerances are those of attention_bounds.py."""

import math

import numpy as np
import pytest

import attention_bounds
import oracle as O
import workloads as W
from gpu_util import dev_i32, say

pytestmark = pytest.mark.gpu

NAMES = ("out", "lse", "dq", "dk", "dv")


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
    return {"bf16": torch.bfloat16, "fp16": torch.float16}[name]


def _host(t):
    return t.detach().double().cpu().numpy()


class Batch:
    """Inputs on the device, and the same numbers on the host; pads hold NaN."""

    def __init__(self, torch, lens, real=None, heads=2, kv_heads=1, dim=64, dtype="bf16", seed=0, spread=1.0,
                 grad=1.0, fused=False, **how):
        real = lens if real is None else real
        self.torch, self.how, self.dtype = torch, how, dtype
        self.cp, self.rank = how.get("cp", 1), how.get("rank", 0)
        self.cu, self.cu_real = W.cumulative(lens), W.cumulative(real)
        t = int(self.cu[-1])
        rng = np.random.default_rng([seed, t, heads, dim])
        dt = _dtype(torch, dtype)

        def tensor(n, h, size):
            return torch.from_numpy(rng.normal(0, size, (n, h, dim)).astype(np.float32)).to(dt).cuda()
        rows = t // self.cp
        if fused:
            both = tensor(t, heads + 2 * kv_heads, spread)
            self.q, self.k, self.v = both[:, :heads], both[:, heads:heads + kv_heads], both[:, heads + kv_heads:]
        else:
            self.q, self.k, self.v = tensor(rows, heads, spread), tensor(t, kv_heads, spread), tensor(t, kv_heads, 1.0)
        self.dout = tensor(rows, heads, grad)
        self.rows, self.tokens = rows, t
        live = np.zeros(rows, dtype=bool)
        for row, _, _, _ in O.share_rows(self.cu, self.cu_real, self.cp, self.rank):
            live[row] = True
        self.live = live
        pads = np.ones(t, dtype=bool)
        for s, n in enumerate(real):
            pads[self.cu[s]:self.cu[s] + n] = False
        gone = torch.from_numpy(~live).cuda()
        for x in (self.q, self.dout):
            x[gone] = math.nan
        for x in (self.k, self.v):
            x[torch.from_numpy(pads).cuda()] = math.nan
        self.pads = pads
        self.cu_dev, self.cu_real_dev = dev_i32(self.cu), dev_i32(self.cu_real)

    def call(self, thd, **more):
        how = dict(self.how)
        return dict(cu_seqlens=self.cu_real_dev, cp_size=how.pop("cp", 1), **how, **more)

    def forward(self, thd, **more):
        return thd.packed_attention(self.q, self.k, self.v, self.cu_dev, **self.call(thd, **more))

    def backward(self, thd, out, lse, **more):
        return thd.packed_attention_backward(self.dout, self.q, self.k, self.v, out, lse, self.cu_dev,
                                             **self.call(thd, **more))

    def expected(self, grad=True):
        q, k, v, d = (_host(x) for x in (self.q, self.k, self.v, self.dout))
        return attention_bounds.attention(self.dtype, q, k, v, self.cu, self.cu_real, dout=d if grad else None,
                                          **self.how)


def _within(got, want, bound, what):
    got = _host(got)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    with np.errstate(invalid="ignore"):
        bad = ~(np.abs(got - want) <= bound) & ~(got == want)
    if bad.any():
        i = tuple(int(x) for x in np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} off, first at {i}: {got[i]!r} for {want[i]!r}, "
                             f"bound {bound[i]!r}")


def _check(thd, b, what):
    out, lse, status = b.forward(thd)
    dq, dk, dv, status2 = b.backward(thd, out, lse)
    assert int(status) == 0 and int(status2) == 0
    want = b.expected()
    for name, x in zip(NAMES, (out, lse, dq, dk, dv)):
        _within(x, *want[name], f"{what} {name}")
    # pads: exactly 0 (the oracle's value and bound there are 0 or tiny)
    gone = b.torch.from_numpy(~b.live).cuda()
    pads = b.torch.from_numpy(b.pads).cuda()
    assert not out[gone].any() and not dq[gone].any() and not dk[pads].any() and not dv[pads].any()
    assert bool((lse[:, gone] == -math.inf).all())
    return out, lse, dq, dk, dv


# one token; ends of 32-row waves, 64-key steps and 128-row tiles; pads, empty and pad-only slots; many documents
LENS = [([1], None), ([31, 1, 32, 33], None), ([64, 65, 63], None), ([127, 128, 129], None), ([300], None),
        ([16, 8, 0, 24, 40], [13, 8, 0, 1, 0]), ([0, 0, 257, 130], [0, 0, 250, 128]), ([513], [385]),
        ([3] * 70, [2] * 70)]


@pytest.mark.parametrize("lens,real", LENS)
@pytest.mark.parametrize("dim,dtype", [(64, "bf16"), (128, "fp16")])
def test_lengths(torch, thd, lens, real, dim, dtype):
    say("attention lengths", lens[:6], real and real[:6], dim, dtype)
    _check(thd, Batch(torch, lens, real, heads=2, kv_heads=1, dim=dim, dtype=dtype), "lengths")


@pytest.mark.parametrize("dim", [8, 16, 24, 40, 64, 72, 96, 120, 128])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_head_sizes(torch, thd, dim, dtype):
    say("attention head size", dim, dtype)
    _check(thd, Batch(torch, [130, 70], [130, 61], heads=3, kv_heads=3, dim=dim, dtype=dtype, seed=dim), "head size")


@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (4, 4), (8, 1), (6, 2), (16, 8), (12, 3)])
def test_heads(torch, thd, heads, kv_heads):
    say("attention heads", heads, kv_heads)
    _check(thd, Batch(torch, [97, 160], [97, 150], heads=heads, kv_heads=kv_heads, dim=64), "heads")


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("window", [0, 1, 5, 64, 100, 129, 10 ** 6])
@pytest.mark.parametrize("cap", [0.0, 2.0])
def test_masks(torch, thd, causal, window, cap):
    say("attention masks", causal, window, cap)
    b = Batch(torch, [260, 40, 200], [251, 40, 200], heads=2, kv_heads=1, dim=64, causal=causal, window=window, cap=cap)
    _check(thd, b, "masks")


@pytest.mark.parametrize("dim", [32, 80, 96, 128])
@pytest.mark.parametrize("how", [dict(window=40), dict(window=129, cap=1.5), dict(causal=False, cap=0.7),
                                 dict(causal=False, window=70)])
def test_masks_of_head_sizes(torch, thd, dim, how):
    say("attention masks of head sizes", dim, how)
    _check(thd, Batch(torch, [170, 33], [161, 33], heads=4, kv_heads=2, dim=dim, **how), "masks")
    _check(thd, Batch(torch, [260, 40], [251, 36], heads=2, kv_heads=2, dim=dim, dtype="fp16", cp=2, rank=1, **how),
           "masks")


# caps far above and far below the scores, and among them
@pytest.mark.parametrize("cap", [1e-3, 0.5, 8.0, 3e3, 1e6, 1e30])
@pytest.mark.parametrize("spread", [1.0, 8.0])
def test_caps(torch, thd, cap, spread):
    say("attention cap", cap, spread)
    _check(thd, Batch(torch, [140], heads=2, dim=64, cap=cap, spread=spread), "cap")


@pytest.mark.parametrize("cap", [3e3, 1e6, 1e30])
def test_far_cap_changes_nothing(torch, thd, cap):
    # z - cap tanh(z / cap) is below |z|^3 / (3 cap^2): with |z| up to 8, 2e-5 for a cap of 3000
    say("attention far cap", cap)
    b = Batch(torch, [140], heads=2, dim=64)
    want, bound = b.expected(grad=False)["lse"]
    b.how["cap"] = cap
    assert np.abs(want).max() < 8
    _within(b.forward(thd)[1], want, bound + 8 ** 3 / (3 * cap ** 2), "lse")


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("cap", [0.0, 3.0])
def test_documents_of_one_token(torch, thd, dtype, cap):
    # dz = p dp (1 - p) with p = exp(z - lse) off by r_p from 1, where the formula's is 0; a
    # delta from the rounded out would be off by w |dout| |v|, hundreds of times as much
    say("attention documents of one token", dtype, cap)
    b = Batch(torch, [1] * 40, heads=3, kv_heads=3, dim=128, dtype=dtype, cap=cap)
    out, lse, _ = b.forward(thd)
    dq, dk, _, _ = b.backward(thd, out, lse)
    q, k, v, d = (np.abs(_host(x)) for x in (b.q, b.k, b.v, b.dout))
    scale, u = 128 ** -0.5, 2.0 ** -24
    e_z = (128 + 4) * u * scale * (q * k).sum(-1, keepdims=True) + 8 * u * cap
    e_z = e_z + 4 * u * np.abs(_host(lse)).T[:, :, None]
    bound = 1.02 * (2 * e_z + 17 * u) * scale * (d * v).sum(-1, keepdims=True)
    # fp16: dz is held to 2^-38 of 2 max |dout| max |v|, and dq's and dk's smallest step is 2^-24
    top = 2 * np.linalg.norm(d, axis=-1).max() * np.linalg.norm(v, axis=-1).max()
    bound += 2.0 ** -38 * top if dtype == "fp16" else 0.0
    tiny = 2.0 ** -25 if dtype == "fp16" else 2.0 ** -126
    _within(dq, np.zeros(dq.shape), bound * k + tiny, "dq")
    _within(dk, np.zeros(dk.shape), bound * q + tiny, "dk")


@pytest.mark.parametrize("cp", [2, 4, 8])
@pytest.mark.parametrize("how", [dict(), dict(causal=False), dict(window=50, cap=5.0)])
def test_zigzag_shares(torch, thd, cp, how):
    align = 2 * cp
    lens = [W.pad_to_multiple([n], align)[0] for n in (300, 1, 41, 150)]
    for rank in sorted({0, 1, cp - 1}):
        say("attention zigzag share", cp, rank, how)
        _check(thd, Batch(torch, lens, [300, 1, 41, 140], heads=2, kv_heads=1, dim=64, cp=cp, rank=rank, **how), "share")


@pytest.mark.parametrize("spread,grad", [(6.0, 1e3), (0.05, 1e-4), (30.0, 1.0)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_sizes_of_values(torch, thd, spread, grad, dtype):
    # sharp and flat softmaxes, large and small gradients (in fp16 near both ends of its range)
    say("attention values", spread, grad, dtype)
    _check(thd, Batch(torch, [200, 65], dim=64, dtype=dtype, spread=spread, grad=grad), "values")


def test_growing_maximum(torch, thd):
    # each 64 keys' scores far above the ones before: the running maximum moves at every step
    say("attention growing maximum")
    b = Batch(torch, [400], dim=64, heads=1)
    ramp = torch.arange(400, device="cuda", dtype=torch.float32)[:, None, None] / 16
    b.k.copy_((torch.ones_like(b.k) * ramp).to(b.k.dtype))
    b.q.copy_(torch.ones_like(b.q))
    _check(thd, b, "growing maximum")


def test_fused_views(torch, thd):
    say("attention on views of one projection")
    b = Batch(torch, [120, 88], [111, 88], heads=4, kv_heads=2, dim=72, fused=True)
    out, lse, _ = b.forward(thd)
    room = torch.full((b.tokens, 8, 72), 7.0, device="cuda", dtype=b.q.dtype)
    grads = room[:, :4], room[:, 4:6], room[:, 6:]
    b.backward(thd, out, lse, grads=grads)
    want = b.expected()
    for name, x in zip(NAMES, (out, lse, *grads)):
        _within(x, *want[name], f"fused {name}")
    # heads outermost
    heads_first = [x.transpose(0, 1).contiguous().transpose(0, 1) for x in (b.q, b.k, b.v)]
    again, _, _ = thd.packed_attention(*heads_first, b.cu_dev, **b.call(thd))
    assert torch.equal(again, out)
    to = torch.empty((4, b.tokens, 72), device="cuda", dtype=b.q.dtype).transpose(0, 1)
    got, _, _ = b.forward(thd, out=to)
    assert got is to and torch.equal(to, out)


def test_without_real_boundaries(torch, thd):
    say("attention without real boundaries")
    b = Batch(torch, [90, 30])
    out, lse, _ = b.forward(thd)
    other, other_lse, _ = thd.packed_attention(b.q, b.k, b.v, b.cu_dev)
    assert torch.equal(out, other) and torch.equal(lse, other_lse)


def test_not_finite_stays_in_its_document(torch, thd):
    say("attention values that are not finite")
    b = Batch(torch, [70, 64, 70], heads=2, dim=64)
    clean, lse, _ = b.forward(thd)
    grads = b.backward(thd, clean, lse)[:3]
    for x in (b.q, b.k, b.v, b.dout):
        x[70:134] = math.inf
        x[80] = math.nan
    out, lse2, _ = b.forward(thd)
    got = b.backward(thd, out, lse2)[:3]
    for part in (slice(0, 70), slice(134, 204)):
        assert torch.equal(out[part], clean[part]) and torch.equal(lse2[:, part], lse[:, part])
        for x, y in zip(got, grads):
            assert torch.equal(x[part], y[part])


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_same_bits_every_time(torch, thd, dtype):
    say("attention twice", dtype)
    b = Batch(torch, [500, 140, 300], heads=8, kv_heads=2, dim=128, dtype=dtype)
    out, lse, _ = b.forward(thd)
    grads = b.backward(thd, out, lse)[:3]
    for _ in range(3):
        again, lse2, _ = b.forward(thd)
        assert torch.equal(again, out) and torch.equal(lse2, lse)
        for x, y in zip(b.backward(thd, out, lse)[:3], grads):
            assert torch.equal(x, y)


# few slots and many of a plan's tables; 4096 boundaries fit its shared memory
@pytest.mark.parametrize("slots", [4095, 4096, 4097, 9000])
def test_many_slots(torch, thd, slots):
    say("attention slots", slots)
    lens = np.zeros(slots, dtype=np.int64)
    lens[[0, 7, slots // 2, slots - 2]] = [40, 129, 70, 1]
    real = lens.copy()
    real[7] = 120
    _check(thd, Batch(torch, list(lens), list(real), heads=2, kv_heads=1), "slots")


# a group's heads in 1, 2, 3 and 8 parts
@pytest.mark.parametrize("heads,kv_heads,lens", [(128, 32, [300]), (96, 32, [300]), (8, 1, [300]), (8, 2, [20] * 12)])
def test_parts_of_a_group(torch, thd, heads, kv_heads, lens):
    say("attention parts", heads, kv_heads, lens)
    for cap in (0.0, 4.0):
        _check(thd, Batch(torch, lens, [n - 3 for n in lens], heads=heads, kv_heads=kv_heads, dim=32, cap=cap), "parts")


BAD = [([1, 4, 8], None, -10), ([0, 6, 4, 8], None, -11), ([0, 4, 7], None, -12), ([0, 4, 8], [0, 5, 8], -14),
       ([0, 4, 8], [0, 4, 3], -11), ([0, 4, 8], [1, 4, 8], -10)]


@pytest.mark.parametrize("cu,real,code", BAD)
def test_bad_boundaries_write_nothing(torch, thd, cu, real, code):
    say("attention bad boundaries", cu, real)
    q = torch.randn((8, 2, 64), device="cuda", dtype=torch.bfloat16)
    out = torch.full_like(q, 3.0)
    more = dict(cu_seqlens=None if real is None else dev_i32(real))
    _, lse, status = thd.packed_attention(q, q, q, dev_i32(cu), out=out, **more)
    assert int(status) == code and bool((out == 3.0).all())
    grads = [torch.full_like(q, 5.0) for _ in range(3)]
    *_, status = thd.packed_attention_backward(q, q, q, q, q, lse, dev_i32(cu), grads=grads, **more)
    assert int(status) == code and all(bool((g == 5.0).all()) for g in grads)


def test_bad_chunks(torch, thd):
    say("attention chunks that do not divide")
    q = torch.randn((4, 2, 64), device="cuda", dtype=torch.bfloat16)
    k = torch.randn((8, 2, 64), device="cuda", dtype=torch.bfloat16)
    _, _, status = thd.packed_attention(q, k, k, dev_i32([0, 4, 6, 8]), cp_size=2, rank=1)
    assert int(status) == thd.THD_ERR_CU_DIVISIBLE


def test_nothing_to_do(torch, thd):
    say("attention of no tokens")
    e = torch.empty((0, 2, 64), device="cuda", dtype=torch.bfloat16)
    out, lse, status = thd.packed_attention(e, e, e, dev_i32([0]))
    assert out.shape == (0, 2, 64) and lse.shape == (2, 0) and int(status) == 0
    *_, status = thd.packed_attention_backward(e, e, e, e, e, lse, dev_i32([0, 0]))
    assert int(status) == 0


def test_offsets_past_32_bits(torch, thd):
    # the last document of a stream whose keys, and whose queries, take over 4 GiB
    say("attention past 4 GiB")
    tokens, tail, heads, dim = 2_200_000, 300, 8, 128
    q = torch.zeros((tokens, heads, dim), device="cuda", dtype=torch.bfloat16)
    assert q.numel() * 2 > 1 << 32
    small = Batch(torch, [tail], heads=heads, kv_heads=heads, dim=dim)
    k, v, d = torch.zeros_like(q), torch.zeros_like(q), torch.zeros_like(q)
    for big, x in zip((q, k, v, d), (small.q, small.k, small.v, small.dout)):
        big[-tail:] = x
    cu, real = dev_i32([0, tokens - tail, tokens]), dev_i32([0, 0, tail])
    out, lse, status = thd.packed_attention(q, k, v, cu, cu_seqlens=real)
    dq, dk, dv, _ = thd.packed_attention_backward(d, q, k, v, out, lse, cu, cu_seqlens=real)
    assert int(status) == 0
    want_out, want_lse, _ = small.forward(thd)
    want = small.backward(thd, want_out, want_lse)[:3]
    assert torch.equal(out[-tail:], want_out) and torch.equal(lse[:, -tail:], want_lse)
    for x, y in zip((dq, dk, dv), want):
        assert torch.equal(x[-tail:], y) and not x[:-tail].any()


def test_on_another_stream(torch, thd):
    say("attention on another stream")
    b = Batch(torch, [300, 90], heads=4, kv_heads=2)
    out, lse, _ = b.forward(thd)
    grads = b.backward(thd, out, lse)[:3]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out2, lse2, _ = b.forward(thd, stream=side)
    grads2 = b.backward(thd, out2, lse2, stream=side)[:3]
    side.synchronize()
    assert torch.equal(out, out2) and all(torch.equal(x, y) for x, y in zip(grads, grads2))


def test_in_a_graph(torch, thd):
    # replays with eager work between, new inputs and new boundaries in place
    say("attention in a graph")
    b = Batch(torch, [300, 84], heads=4, kv_heads=2)
    out, lse, _ = b.forward(thd)
    b.backward(thd, out, lse)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse, status = b.forward(thd)
        dq, dk, dv, _ = b.backward(thd, out, lse)
    for i in range(4):
        b.q.normal_()
        b.v.normal_()
        cut = [300, 84 + i, 384][i % 3] // 2 * 2
        b.cu_dev.copy_(dev_i32([0, cut, 384]))
        b.cu_real_dev.copy_(dev_i32([0, cut, 384]))
        graph.replay()
        want, want_lse, _ = b.forward(thd)
        want_grads = b.backward(thd, want, want_lse)[:3]
        torch.cuda.synchronize()
        assert int(status) == 0 and torch.equal(out, want) and torch.equal(lse, want_lse)
        assert all(torch.equal(x, y) for x, y in zip((dq, dk, dv), want_grads))


def test_with_the_layout_transform(torch, thd):
    # pack -> route -> each rank's share -> attention -> back to token order: the whole stream's result
    say("attention with the layout transform")
    cp = 2
    rows = torch.from_numpy(W.token_rows(9, 3, 150, eod_rate=0.03, pad_tail_max=30)).cuda()
    max_docs, capacity = 40, 640
    ids, cu, cu_pad, status = thd.pack(rows, 0, 1, 2 * cp, capacity, max_docs)
    assert int(status) == 0
    route = thd.Route(max_docs + 1, cp, capacity)
    route.build(cu_pad, cp, capacity)
    g = torch.Generator(device="cuda").manual_seed(3)
    x = [torch.randn((capacity, h, 64), generator=g, device="cuda", dtype=torch.bfloat16) for h in (4, 2, 2, 4)]
    q, k, v, dout = x
    whole, lse, _ = thd.packed_attention(q, k, v, cu_pad, cu_seqlens=cu)
    dq, dk, dv, _ = thd.packed_attention_backward(dout, q, k, v, whole, lse, cu_pad, cu_seqlens=cu)
    zq, zd = route.swap(q, thd.C2Z), route.swap(dout, thd.C2Z)
    n = capacity // cp
    outs, dqs, dks, dvs = [], [], 0, 0
    for rank in range(cp):
        mine = slice(rank * n, (rank + 1) * n)
        how = dict(cu_seqlens=cu, cp_size=cp, rank=rank)
        o, l, _ = thd.packed_attention(zq[mine], k, v, cu_pad, **how)
        a, b, c, _ = thd.packed_attention_backward(zd[mine], zq[mine], k, v, o, l, cu_pad, **how)
        outs.append(o)
        dqs.append(a)
        dks, dvs = dks + b.float(), dvs + c.float()
    back = route.swap(torch.cat(outs), thd.Z2C)
    # the same sums in another tiling: a few roundings of the type apart
    for got, want in ((back, whole), (route.swap(torch.cat(dqs), thd.Z2C), dq), (dks, dk), (dvs, dv)):
        assert float((got.float() - want.float()).abs().max()) <= 2.0 ** -6 * float(want.float().abs().max())
    route.close()
