"""The losses of few long rows, each cut into parts over several workgroups.

Rows take that form from 8193 16-byte words on for log-probabilities (up to 64
rows) and from 4097 on for the losses (up to 48 rows).  Oracle, cases and bounds
are those of test_gpu_losses.
"""

import numpy as np
import pytest

import oracle as O
from gpu_util import say
from test_gpu_losses import (  # noqa: F401  (the fixtures torch and thd)
    DTYPES, Case, _check_distill, _check_logp, _check_policy, _dtype, _host, _logp_error, _within, thd, torch)

pytestmark = pytest.mark.gpu


def _in_parts(thd, case, targets):
    kind = {"bf16": thd.THD_BF16, "fp16": thd.THD_FP16, "fp32": thd.THD_FP32}[case.dtype]
    return thd.thd_loss_workspace_bytes(case.rows, case.vocab, kind, targets) > 0


@pytest.mark.parametrize("rows", [3, 40])
@pytest.mark.parametrize("dtype,vocab,stride,offset", [
    ("fp32", 33003, 33003, 0), ("bf16", 50257, 50264, 0), ("fp16", 50257, 50257, 5), ("bf16", 131075, 131075, 0)])
def test_teacher_columns_at_both_ends(torch, thd, rows, dtype, vocab, stride, offset):
    # a gradient at another place than the logits: the elements before the first
    # and after the last whole word have one owner, targets or not
    say("ends of the row", rows, dtype, vocab)
    case = Case(torch, 31, 3, rows, vocab, dtype, stride=stride, offset=offset, k=20)
    assert _in_parts(thd, case, 20)
    case.mask[:] = 1
    case.ids[:, :8] = np.arange(8)
    case.ids[:, 8:16] = vocab - 1 - np.arange(8)
    case.ids[1, 16:] = vocab - 1                # the last column several times
    case.ids[2, 1:19] = -1                      # and hardly anything else
    case.ids[2, 19] = vocab - 1
    for _ in range(3):
        _check_distill(case, thd, out="elsewhere", tau=1.5, teacher_dtype=_dtype(torch, dtype))
    _check_distill(case, thd, out="in place", tau=1.5)


VOCAB = 70001       # in parts for every call and type


def _part_case(torch, thd, seed, n, rows, dtype, k, **kw):
    case = Case(torch, seed, n, rows, VOCAB, dtype, k=k, **kw)
    assert _in_parts(thd, case, 0) and _in_parts(thd, case, max(k, 1))
    return case


def _place_rows(case):
    """The host's rows ``case.z`` into the logits (again)."""
    torch = case.torch
    z = torch.from_numpy(case.z).to(case.logits.dtype).cuda()
    case.logits.copy_(z[torch.from_numpy(case.pick).cuda()])


@pytest.mark.parametrize("rows", [4, 48])
@pytest.mark.parametrize("dtype", DTYPES)
def test_masked_rows_are_not_looked_at(torch, thd, rows, dtype):
    say("masked, in parts", rows, dtype)
    case = _part_case(torch, thd, 60, 4, rows, dtype, 6)
    case.mask[:] = [1, 0, 1, 0]
    case.labels[1], case.labels[3] = -7, 1 << 40
    case.old[1], case.adv[3] = np.nan, np.inf
    case.ids[1], case.ids[3] = -9, 1 << 30
    case.logits[1::4], case.logits[3::4] = float("nan"), float("inf")
    labels, mask = case.dev(case.labels), case.dev(case.mask)
    logp, lse, st = thd.token_logprobs(case.logits, labels, mask=mask)
    assert int(st.item()) == 0 and not logp[1::2].any() and not lse[1::2].any()
    g = thd.token_logprobs_backward(case.dev(case.d), case.logits, labels, lse, mask=mask)
    _, _, p, st = thd.policy_loss(case.logits, labels, case.dev(case.old), case.dev(case.adv), mask=mask,
                                  ref_logp=case.dev(case.ref), kl_coef=0.1)
    assert int(st.item()) == 0
    loss, d, st = thd.distill_topk(case.logits, case.dev(case.teacher).contiguous(), case.dev(case.ids).contiguous(),
                                   mask=mask)
    assert int(st.item()) == 0 and not loss[1::2].any()
    for grad in (g, p, d):
        assert not grad[1::2].any() and bool(torch.isfinite(grad.float()).all()) and bool(grad[::2].any(1).all())


@pytest.mark.parametrize("dtype", DTYPES)
def test_excluded_columns_and_lowest_values(torch, thd, dtype):
    say("lowest, in parts", dtype)
    case = _part_case(torch, thd, 61, 4, 8, dtype, 8)
    lowest = torch.finfo(_dtype(torch, dtype)).min
    z = case.z
    z[0, 100:VOCAB - 100] = -np.inf          # whole parts taken out
    z[1, 7:] = lowest                        # or given the type's lowest value
    z[2, :] = lowest                         # a row of nothing else: uniform
    z[3, :VOCAB - 1] = -np.inf               # one column left
    case.labels[:] = [50, 3, 40000, VOCAB - 1]
    case.ids = np.tile(np.array([1, 2, 3, 4, 5, 6, 50, VOCAB - 1]), (4, 1))
    case.ids[3] = [VOCAB - 1, -1, -1, -1, -1, -1, -1, -1]
    case.ids[1] = [0, 1, 2, 3, 4, 5, 6, -1]
    case.mask[:] = 1
    _place_rows(case)
    logp, _ = O.token_logprobs(z, case.labels)
    case.old, case.ref = (logp + 0.1).astype(np.float32), (logp - 0.2).astype(np.float32)
    assert logp[2] == pytest.approx(-np.log(VOCAB)) and logp[3] == 0
    _check_policy(case, thd)
    _check_distill(case, thd)
    got, _, _ = thd.token_logprobs(case.logits, case.dev(case.labels))
    _within(_host(got), case.whole(logp), case.whole(_logp_error(z, case.labels)[0]), "logp")


@pytest.mark.parametrize("dtype", DTYPES)
def test_rows_without_a_softmax(torch, thd, dtype):
    say("nan rows, in parts", dtype)
    case = _part_case(torch, thd, 62, 6, 12, dtype, 4)
    z, labels = case.logits, case.dev(case.labels)
    z[1::6] = -float("inf")
    z[2::6, 12345] = float("inf")
    z[3::6, VOCAB - 1] = float("nan")
    logp, lse, st = thd.token_logprobs(z, labels)
    assert int(st.item()) == 0
    g = thd.token_logprobs_backward(case.dev(case.d), z, labels, lse)
    loss, logp_p, p, st = thd.policy_loss(z, labels, case.dev(case.old), case.dev(case.adv))
    assert int(st.item()) == 0
    loss_d, d, st = thd.distill_topk(z, case.dev(case.teacher).contiguous(), case.dev(case.ids).contiguous())
    assert int(st.item()) == 0
    for i in range(6):
        values = [x[i::6].float() for x in (logp, lse, loss, logp_p, loss_d, g, p, d)]
        if i in (1, 2, 3):
            assert all(bool(torch.isnan(x).all()) for x in values)
        else:
            assert all(bool(torch.isfinite(x).all()) for x in values)


@pytest.mark.parametrize("out", ["new", "in place"])
def test_logits_of_any_size(torch, thd, out):
    say("far from zero, in parts", out)
    for at in (4e8, -6.3e8, 1.5e9, -3e9, 2.5e38, -2.5e38):
        case = _part_case(torch, thd, 63, 5, 5, "fp32", 9)
        step = float(np.spacing(np.float32(abs(at))))
        z = at - step * np.random.default_rng(3).integers(0, 4, (5, VOCAB))
        case.z = z.astype(np.float32).astype(np.float64)
        _place_rows(case)
        logp, _ = O.token_logprobs(case.z, case.labels)
        case.old = (np.maximum(logp, -60) + 0.05).astype(np.float32)
        case.ref = (np.maximum(logp, -60) - 0.1).astype(np.float32)
        case.mask[:] = logp > -60
        _check_policy(case, thd, out=out, kl=0.1)
        _place_rows(case)
        case.mask[:] = 1
        _check_distill(case, thd, out=out, tau=1.5)


@pytest.mark.parametrize("out", ["in place", "elsewhere"])
@pytest.mark.parametrize("dtype,stride,offset", [
    ("bf16", 70008, 0), ("bf16", 70011, 3), ("fp16", 70004, 1), ("fp32", 70007, 3), ("fp32", 70001, 1)])
def test_strides_and_places(torch, thd, out, dtype, stride, offset):
    say("strides, in parts", out, dtype, stride, offset)
    for check, k in ((_check_logp, 0), (_check_policy, 0), (_check_distill, 7)):
        case = _part_case(torch, thd, 64, 4, 5, dtype, k, stride=stride, offset=offset)
        check(case, thd, out=out)
        if stride > VOCAB:     # nothing outside the rows is written
            pad = case.room.as_strided((4, stride - VOCAB), (stride, 1), offset + VOCAB)
            assert torch.isnan(pad).all() and torch.isnan(case.room[:offset]).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_targets_outside_the_vocabulary(torch, thd, dtype):
    say("bad targets, in parts", dtype)
    for bad in (-1, VOCAB, 1 << 33, -(1 << 40)):
        case = _part_case(torch, thd, 65, 5, 10, dtype, 3)
        case.labels[1] = bad
        _check_policy(case, thd, status=thd.THD_ERR_LABEL)
        labels = case.dev(case.labels)
        logp, lse, st = thd.token_logprobs(case.logits, labels, mask=case.dev(case.mask))
        assert int(st.item()) == thd.THD_ERR_LABEL
        assert bool(torch.isnan(logp[1::5]).all()) and bool(torch.isnan(lse[1::5]).all())
        assert bool(torch.isfinite(logp[0::5]).all())
        g = thd.token_logprobs_backward(case.dev(case.d), case.logits, labels, lse)
        assert bool(torch.isnan(g[1::5].float()).all()) and bool(torch.isfinite(g[0::5].float()).all())
        if bad != -1:
            case.ids[1, 2] = bad
            for out in ("new", "elsewhere"):
                _check_distill(case, thd, out=out, status=thd.THD_ERR_LABEL)


@pytest.mark.parametrize("k", [1, 3, 64, 65, 256])
def test_teacher_columns(torch, thd, k):
    say("teacher, in parts", k)
    case = _part_case(torch, thd, 66, 7, 14, "bf16", k)
    case.mask[:] = 1
    case.ids[1] = -1                                  # no column at all
    case.ids[2, k // 2:] = case.ids[2, 0]             # one column many times
    case.teacher[3] = -np.inf                         # no probability at all
    case.teacher[4, k // 2] = -np.inf
    case.ids[5, : k // 2] = -1
    case.ids[6] = np.arange(k) + VOCAB - k            # neighbours, up to the row's last element
    loss, grad = _check_distill(case, thd, tau=1.0)
    for i in (1, 3):
        assert not loss[i::7].any() and not grad[i::7].any()
    _check_distill(case, thd, tau=0.25, ids64=False, teacher_dtype=torch.float16)
    _check_distill(case, thd, tau=3.0, out="elsewhere")
    _check_distill(case, thd, tau=20.0, out="in place")


def test_same_bits_on_every_stream(torch, thd):
    say("streams, in parts")
    case = _part_case(torch, thd, 67, 6, 6, "bf16", 10)
    labels, old, adv = case.dev(case.labels), case.dev(case.old), case.dev(case.adv)
    t, ids = case.dev(case.teacher).contiguous(), case.dev(case.ids).contiguous()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    want = None
    for stream in (None, None, side, side.cuda_stream):
        got = [*thd.token_logprobs(case.logits, labels, stream=stream),
               *thd.policy_loss(case.logits, labels, old, adv, stream=stream),
               *thd.distill_topk(case.logits, t, ids, stream=stream)]
        torch.cuda.synchronize()
        want = want or got
        assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_in_a_graph(torch, thd):
    say("graph, in parts")
    case = _part_case(torch, thd, 68, 6, 6, "bf16", 10)
    labels, old, adv = case.dev(case.labels), case.dev(case.old), case.dev(case.adv)
    t, ids = case.dev(case.teacher).contiguous(), case.dev(case.ids).contiguous()

    def step():
        logp, lse, st = thd.token_logprobs(case.logits, labels)
        return (logp, lse, st, thd.token_logprobs_backward(adv, case.logits, labels, lse),
                *thd.policy_loss(case.logits, labels, old, adv), *thd.distill_topk(case.logits, t, ids))
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for i in range(4):
        case.logits.copy_(torch.randn((6, VOCAB), device="cuda"))
        want = step()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got)), i
