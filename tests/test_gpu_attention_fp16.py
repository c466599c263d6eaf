"""Attention where fp16 has few exponents to spare: rows with one key far above the
others, and long documents, against closed forms and the oracle (64 bits)."""

import math

import numpy as np
import pytest

from gpu_util import dev_i32, say
from test_gpu_attention import Batch, _host, _within, thd, torch  # noqa: F401  (fixtures)

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}
# half the smallest step of a probability, of the row's largest: fp16's 2^-25 over the 2^9 it is held with
FLOOR = {"bf16": 2.0 ** -126, "fp16": 2.0 ** -34}
TINY = {"bf16": 2.0 ** -133, "fp16": 2.0 ** -25}


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("gap", [10, 12, 14, 15, 16, 17, 18, 20])
@pytest.mark.parametrize("n", [40, 4000, 20000])
@pytest.mark.parametrize("place", ["first", "last"])
def test_one_strong_key(torch, thd, n, gap, dtype, place):
    # z is `gap` for one key of value 0, and 0 for n - 1 keys of value 1:
    # out = (n - 1) / (n - 1 + e^gap)
    say("attention one strong key", n, gap, dtype, place)
    dt = {"bf16": torch.bfloat16, "fp16": torch.float16}[dtype]
    q = torch.zeros((n, 1, 64), device="cuda", dtype=dt)
    k, v = torch.zeros_like(q), torch.ones_like(q)
    at = 0 if place == "first" else n - 1
    q[:, :, 0], k[at, :, 0], v[at] = 8.0, float(gap), 0.0
    out, lse, status = thd.packed_attention(q, k, v, dev_i32([0, n]), causal=False)
    assert int(status) == 0
    total = n - 1 + math.exp(gap)
    want, true_lse = (n - 1) / total, math.log(total)
    # roundings as counted in attention_bounds.py; p of the largest key is at most 1
    e_z = (64 + 4) * U * gap + 4 * U * gap
    r_p = 2 * e_z + (n + 16) * U
    bound = (HALF[dtype] + r_p + n * U) * want + (n - 1) * FLOOR[dtype] + HALF[dtype] * want + TINY[dtype]
    _within(out, np.full(out.shape, want), np.full(out.shape, bound), "out")
    _within(lse, np.full(lse.shape, true_lse), np.full(lse.shape, e_z + (n + 16) * U + 4 * U * true_lse), "lse")


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("tokens,heads,dim,spread", [(4099, 2, 64, 1.0), (2500, 1, 128, 3.0)])
def test_long_document(torch, thd, tokens, heads, dim, spread, dtype):
    # hundreds of steps of the running softmax, and of both walks of the gradients
    say("attention of a long document", tokens, heads, dim, spread, dtype)
    b = Batch(torch, [tokens + 13], [tokens], heads=heads, kv_heads=1, dim=dim, dtype=dtype, spread=spread)
    out, lse, status = b.forward(thd)
    dq, dk, dv, status2 = b.backward(thd, out, lse)
    assert int(status) == 0 and int(status2) == 0
    want = b.expected()
    for name, x in zip(("lse", "dq", "dk", "dv"), (lse, dq, dk, dv)):
        _within(x, *want[name], f"long {name}")
    # fp16: attention_bounds allows each probability 2^-25 of the row's largest; 2^-34 is what is lost
    value, bound = want["out"]
    if dtype == "fp16":
        seen = np.cumsum(np.abs(np.nan_to_num(_host(b.v))), 0).repeat(heads, 1)
        bound = bound - np.where(b.live[:, None, None], (2.0 ** -25 - FLOOR[dtype]) * seen, 0.0)
    _within(out, value, bound, "long out")


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("gap", [12, 16, 18, 20])
def test_gradient_of_weak_values(torch, thd, gap, dtype):
    # the same keys, dout 1 in every row: dv of a weak key is n / (n - 1 + e^gap)
    n = 20000
    say("attention gradient of weak values", n, gap, dtype)
    dt = {"bf16": torch.bfloat16, "fp16": torch.float16}[dtype]
    q = torch.zeros((n, 1, 64), device="cuda", dtype=dt)
    k, v = torch.zeros_like(q), torch.ones_like(q)
    q[:, :, 0], k[0, :, 0], v[0] = 8.0, float(gap), 0.0
    cu = dev_i32([0, n])
    out, lse, _ = thd.packed_attention(q, k, v, cu, causal=False)
    *_, dv, status = thd.packed_attention_backward(torch.ones_like(q), q, k, v, out, lse, cu, causal=False)
    assert int(status) == 0
    want = n / (n - 1 + math.exp(gap))
    r_p = 2 * ((64 + 4) * U * gap + 4 * U * gap) + (n + 16) * U
    # p is held times 2^14: half of fp16's smallest step is 2^-39 of it
    floor = {"bf16": 2.0 ** -126, "fp16": 2.0 ** -39}[dtype]
    bound = (HALF[dtype] + r_p + n * U) * want + n * floor + HALF[dtype] * want + TINY[dtype]
    _within(dv[1:], np.full((n - 1, 1, 64), want), np.full((n - 1, 1, 64), bound), "dv")


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("cap", [0.0, 4.0])
@pytest.mark.parametrize("dim", [64, 128])
def test_not_finite_stays_in_its_document(torch, thd, dtype, cap, dim):
    # fp16 holds all documents' gradients of scores by one power of two, from the largest norms of
    # dout and v: they stand in a clean document, so that both runs take the same
    say("attention values that are not finite", dtype, cap, dim)
    b = Batch(torch, [70, 64, 70], heads=4, kv_heads=2, dim=dim, dtype=dtype, cap=cap)
    for x in (b.v, b.dout):
        x[3] = 8.0
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
    assert not out[70:134].isfinite().any()


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("spread", [300.0, 2000.0, 4000.0, 8000.0])
@pytest.mark.parametrize("cap", [0.0, 1e7])
def test_scores_past_their_precision(torch, thd, spread, dtype, cap):
    # scores up to 3e8 are known to some whole numbers only; out still is a mean of values,
    # and fp16's factors stay within the type, as no p passes 1
    say("attention scores past their precision", spread, dtype, cap)
    b = Batch(torch, [600], heads=4, kv_heads=4, dim=64, dtype=dtype, cap=cap)
    for x in (b.q, b.k):
        x.copy_((x.float() * spread).clamp(-6e4, 6e4))
    out, lse, _ = b.forward(thd)
    assert bool(lse.isfinite().all())
    most = b.v.double().abs().amax(0)
    assert bool((out.double().abs() <= most * (1 + 2 * HALF[dtype])).all())
    *_, dv, _ = b.backward(thd, out, lse)
    assert bool(dv.isfinite().all())
    if dtype == "fp16":
        assert bool((dv.double().abs() <= b.dout.double().abs().sum(0) * (1 + 4 * HALF[dtype])).all())
