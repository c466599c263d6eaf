"""The losses on packed streams against the oracle (64 bits), on the GPU.

Tolerances, with u = 2^-24 the half step of 32 bits, before any run:

* a sum of exponentials: at most vocab/256 + 160 additions one after another,
  each term with its own rounding (exponential 2 u, its argument 3 u times its
  size, which weighted by the terms stays under 20): relative error
  (vocab/256 + 280) u;
* log-probability: that, plus 4 u of each summand;
* probability of column v: the sum's error plus (5 |z_v - max| / tau + 6) u;
* a gradient: |d| q times the probability's error, plus the error of d (the
  log-probability's, carried through the ratio and the KL term), plus half a
  step of its own type, plus what falls below the normal range of 32 bits or
  the smallest step of fp16.
"""

import numpy as np
import pytest

import oracle as O
import oracle.loss_oracle
from gpu_util import say

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DTYPES = ["bf16", "fp16", "fp32"]
# half a step relative to the value, and half the smallest step
HALF = {"bf16": (2.0 ** -8, 0.0), "fp16": (2.0 ** -11, 2.0 ** -25), "fp32": (U, 0.0)}


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


def _dev(torch, a, dtype=None):
    t = torch.as_tensor(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def _host(t):
    return t.detach().double().cpu().numpy()


# ---- bounds -------------------------------------------------------------------

def _sum_error(vocab):
    return (vocab / 256 + 280) * U


def _logp_error(z, labels):
    """Bound of each row's log-probability, and of its log-sum-exp."""
    vocab = z.shape[1]
    out = []
    for t, y in enumerate(labels):
        y = y if 0 <= y < vocab else 0
        top = z[t].max()
        ln_s = np.log(np.exp(z[t] - top).sum())
        logp = _sum_error(vocab) + 4 * U * (abs(z[t, y] - top) + ln_s)
        out.append((logp, logp + 4 * U * abs(top + ln_s)))
    return np.array(out).T


def _grad_error(z, d, d_error, grad, dtype, tau=1.0, base=None, sum_error=None):
    """Bound of a gradient matrix: rows z, factor d of the softmax, its error."""
    vocab = z.shape[1]
    top = z.max(1, keepdims=True) if base is None else base[:, None]
    q = np.abs(grad)
    x = z / tau
    soft = np.exp(x - x.max(1, keepdims=True))
    soft /= soft.sum(1, keepdims=True)
    rel = (_sum_error(vocab) if sum_error is None else sum_error) + (5 * np.abs(z - top) / tau + 6) * U
    rel = np.where(np.isfinite(rel), rel, 0.0)
    half, tiny = HALF[dtype]
    # the target's column: one more difference
    at_target = np.abs(grad - d[:, None] * soft) > 4 * U * np.abs(d)[:, None]
    err = np.abs(d)[:, None] * (soft * rel + 8 * U * at_target) + d_error[:, None] * (soft + 1)
    err = err + half * (q + err) + tiny + 2.0 ** -126 * (1 + np.abs(d)[:, None])
    return err


def _within(got, want, bound, what):
    got, want = np.asarray(got, dtype=np.float64), np.asarray(want, dtype=np.float64)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    both_nan = np.isnan(got) & np.isnan(want)
    with np.errstate(invalid="ignore"):
        bad = ~both_nan & ~(np.abs(got - want) <= bound) & ~(got == want)
    if bad.any():
        i = tuple(int(v) for v in np.argwhere(bad)[0])
        b = np.broadcast_to(bound, got.shape)[i]
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} off, first at {i}: {got[i]!r} for {want[i]!r}, "
                             f"bound {b!r}")


# ---- inputs ---------------------------------------------------------------------

class Case:
    """`n` distinct rows on the host; on the device they repeat over `rows`."""

    def __init__(self, torch, seed, n, rows, vocab, dtype, stride=None, offset=0, k=0, spread=3.0):
        rng = np.random.default_rng([seed, n, rows, vocab, k])
        self.torch, self.n, self.rows, self.vocab, self.dtype = torch, n, rows, vocab, dtype
        dt = _dtype(torch, dtype)
        z = rng.normal(0, spread, (n, vocab)).astype(np.float32)
        self.labels = rng.integers(0, vocab, n)
        z[np.arange(n), self.labels] += 4
        zt = torch.from_numpy(z).to(dt)
        self.z = zt.double().numpy()
        self.old = None
        self.adv = rng.normal(size=n).astype(np.float32)
        self.w = rng.uniform(0.1, 1, n).astype(np.float32)
        self.d = rng.normal(size=n).astype(np.float32)
        logp, _ = O.token_logprobs(self.z, self.labels)
        self.old = (logp + rng.choice([-0.5, -0.1, 0.05, 0.6], n)).astype(np.float32)
        self.ref = (logp + rng.normal(0, 0.4, n)).astype(np.float32)
        self.mask = np.ones(n, dtype=np.uint8)
        if n > 2:
            self.mask[n // 2] = 0
        if k:
            self.ids = np.stack([rng.choice(vocab, k, replace=False) for _ in range(n)])
            self.teacher = rng.normal(0, 2, (n, k)).astype(np.float32)
        self.pick = np.arange(rows) % n
        self.stride, self.offset = stride or vocab, offset
        room = torch.full((offset + rows * self.stride,), float("nan"), dtype=dt, device="cuda")
        self.logits = room.as_strided((rows, vocab), (self.stride, 1), offset)
        self.logits.copy_(zt.cuda()[torch.from_numpy(self.pick).cuda()])
        self.room = room

    def dev(self, a):
        return _dev(self.torch, np.asarray(a)[self.pick])

    def whole(self, a):
        return np.asarray(a)[self.pick]


def _out(case, kind):
    torch = case.torch
    if kind == "new":
        return None
    if kind == "in place":
        return case.logits
    # another place within 16 bytes than the logits
    room = torch.full((case.rows * (case.vocab + 3) + 5,), 7.0, dtype=case.logits.dtype, device="cuda")
    return room.as_strided((case.rows, case.vocab), (case.vocab + 3, 1), 1 + case.offset)


def _check_policy(case, thd, out="new", kl=0.3, status=0):
    loss, logp, grad, st = thd.policy_loss(
        case.logits, case.dev(case.labels), case.dev(case.old), case.dev(case.adv), mask=case.dev(case.mask),
        ref_logp=case.dev(case.ref), weights=case.dev(case.w), clip_low=0.2, clip_high=0.3, kl_coef=kl,
        out=_out(case, out))
    assert int(st.item()) == status
    want = O.policy_loss(case.z, case.labels, case.old, case.adv, case.mask, case.ref, case.w, 0.2, 0.3, kl)
    e_logp, _ = _logp_error(case.z, case.labels)
    r = np.exp(want[1] - case.old)
    u = case.ref - want[1]
    e_ratio = r * (e_logp + (np.abs(want[1] - case.old) * 4 + 6) * U)
    e_kl = kl * (np.abs(np.expm1(u)) * (e_logp + 4 * U) + np.exp(u) * (6 + 4 * np.abs(u)) * U)
    e_d = case.w * (np.abs(case.adv) * e_ratio + kl * np.exp(u) * (e_logp + (6 + 4 * np.abs(u)) * U))
    e_loss = case.w * (np.abs(case.adv) * (e_ratio + 4 * U * 1.3) + e_kl) + 6 * U * np.abs(want[0])
    live = case.mask != 0
    d = np.array([O.loss_oracle.policy_terms(want[1][t], case.old[t], case.adv[t], case.ref[t], case.w[t], 0.2, 0.3,
                                             kl)[1] if live[t] else 0.0 for t in range(case.n)])
    _within(_host(loss), case.whole(want[0]), case.whole(e_loss), "loss")
    _within(_host(logp), case.whole(want[1]), case.whole(e_logp), "logp")
    _check_matrix(case, grad, want[2], _grad_error(case.z, -d, e_d, want[2], case.dtype), "gradient")
    return loss, logp, grad


def _check_matrix(case, grad, want, bound, what):
    """Compared on the device: every row with its host row."""
    torch = case.torch
    assert grad.shape == (case.rows, case.vocab) and grad.dtype == case.logits.dtype
    w, b = torch.from_numpy(want).cuda(), torch.from_numpy(np.broadcast_to(bound, want.shape).copy()).cuda()
    for i in range(case.n):
        g = grad[i::case.n].double()
        ok = ((g - w[i]).abs() <= b[i]) | (torch.isnan(g) & torch.isnan(w[i])) | (g == w[i])
        if not bool(ok.all()):
            at = (~ok).nonzero()[0].tolist()
            raise AssertionError(f"{what}: host row {i}, copy {at[0]}, column {at[1]}: {g[at[0], at[1]].item()!r} for "
                                 f"{w[i, at[1]].item()!r}, bound {b[i, at[1]].item()!r}; {int((~ok).sum())} off")


def _check_logp(case, thd, out="new"):
    labels, mask = case.dev(case.labels), case.dev(case.mask)
    logp, lse, st = thd.token_logprobs(case.logits, labels, mask=mask)
    assert int(st.item()) == 0
    want = O.token_logprobs(case.z, case.labels, case.mask)
    e_logp, e_lse = _logp_error(case.z, case.labels)
    _within(_host(logp), case.whole(want[0]), case.whole(e_logp), "logp")
    _within(_host(lse), case.whole(want[1]), case.whole(e_lse), "lse")
    # the gradient from one given log-sum-exp per host row
    lse32 = want[1].astype(np.float32)
    grad = thd.token_logprobs_backward(case.dev(case.d), case.logits, labels, case.dev(lse32), mask=mask,
                                       out=_out(case, out))
    g = O.token_logprobs_backward(case.d, case.z, case.labels, lse32, case.mask)
    # d enters as given; the softmax is taken against the rounded log-sum-exp
    bound = _grad_error(case.z, -case.d.astype(np.float64) * case.mask, np.abs(case.d) * 2 * U, g, case.dtype,
                        base=lse32.astype(np.float64), sum_error=U * 2)
    bound = bound + np.abs(case.d)[:, None] * 2 * U * np.abs(g)
    _check_matrix(case, grad, g, bound, "gradient")


def _check_distill(case, thd, out="new", tau=2.0, ids64=True, teacher_dtype=None, status=0):
    torch = case.torch
    teacher = torch.from_numpy(case.teacher).to(teacher_dtype or torch.float32)
    ids = _dev(torch, case.ids[case.pick], None if ids64 else torch.int32)
    t_dev = teacher.cuda()[torch.from_numpy(case.pick).cuda()].contiguous()
    loss, grad, st = thd.distill_topk(case.logits, t_dev, ids, mask=case.dev(case.mask), weights=case.dev(case.w),
                                      temperature=tau, out=_out(case, out))
    assert int(st.item()) == status
    t_host = teacher.double().numpy()
    want = O.distill_topk(case.z, t_host, case.ids, case.mask, case.w, tau)
    k = case.ids.shape[1]
    e_loss = np.zeros(case.n)
    for t in range(case.n):
        part = [(i, x) for i, x in zip(case.ids[t], t_host[t]) if 0 <= i < case.vocab and x != -np.inf]
        if not part:
            continue
        x = np.array([v for _, v in part]) / tau
        lp = x - x.max() - np.log(np.exp(x - x.max()).sum())
        zt = case.z[t] / tau
        lq = zt - zt.max() - np.log(np.exp(zt - zt.max()).sum())
        term = np.abs(lp) + np.abs(lq[[i for i, _ in part]])
        gap = np.abs(lp - lq[[i for i, _ in part]])
        # ln p and ln q, p itself (k additions), the sum over k
        fine = np.isfinite(term)
        e_loss[t] = tau ** 2 * case.w[t] * (np.exp(lp) * np.where(
            fine, (8 * U * (term + np.log(case.vocab)) + _sum_error(case.vocab) + (k + 12) * U) +
            gap * (k + 20 + 6 * np.abs(x - x.max())) * U, 0)).sum()
    _within(_host(loss), case.whole(want[0]), case.whole(e_loss + 4 * U * np.abs(want[0])), "loss")
    c = tau * case.w * case.mask
    bound = _grad_error(case.z, c.astype(np.float64), c * 0.0, want[1], case.dtype, tau=tau)
    # a target: its probability's error, k additions and an argument of size |t - max|
    spread = np.nanmax(np.where(np.isfinite(t_host), t_host.max(1, keepdims=True) - t_host, 0), 1) if k else 0
    target = np.zeros_like(want[1])
    for t in range(case.n):
        for i in case.ids[t]:
            if 0 <= i < case.vocab:
                target[t, i] += c[t] * (k + 20 + 5 * spread[t] / tau) * U
    _check_matrix(case, grad, want[1], bound + target * (1 + HALF[case.dtype][0]), "gradient")
    return loss, grad


# ---- sizes, types, both forms (few rows in parts, many rows one workgroup each) --------------------

VOCABS = [1, 2, 7, 8, 9, 65, 1000, 2047, 2049, 4104, 8199, 16390, 32000, 33001, 65543, 131075, 163851]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab", VOCABS)
def test_few_rows(torch, thd, dtype, vocab):
    say("few rows", dtype, vocab)
    case = Case(torch, 1, 3, 3, vocab, dtype)
    _check_logp(case, thd)
    _check_policy(case, thd)
    case = Case(torch, 2, 3, 3, vocab, dtype, k=min(vocab, 13))
    _check_distill(case, thd)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab", VOCABS)
def test_many_rows(torch, thd, dtype, vocab):
    # odd vocabularies put the rows at every place within 16 bytes
    say("many rows", dtype, vocab)
    rows = 1100 if vocab <= 33001 else 530
    case = Case(torch, 3, 5, rows, vocab, dtype)
    _check_logp(case, thd)
    _check_policy(case, thd)
    case = Case(torch, 4, 5, rows, vocab, dtype, k=min(vocab, 40))
    _check_distill(case, thd, ids64=False, teacher_dtype=_dtype(torch, dtype))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("words", [256, 512, 1024, 2048, 4096, 8192, 12288, 16384, 26624])
def test_rows_that_just_fit(torch, thd, dtype, words):
    # rows on whole lines that fill a form's registers (and LDS), and a word more
    per = 8 if dtype == "bf16" else 4
    for vocab in (words * per, words * per + per):
        say("full registers", dtype, vocab)
        case = Case(torch, 18, 3, 70, vocab, dtype)
        _check_policy(case, thd)
        case = Case(torch, 18, 3, 70, vocab, dtype, k=33)
        _check_distill(case, thd)


@pytest.mark.parametrize("rows", [5, 1100])
@pytest.mark.parametrize("out", ["new", "in place"])
def test_logits_of_any_size(torch, thd, rows, out):
    # a row's logits may lie far from zero: only their distances count. 32-bit
    # steps at 2^k are 2^(k-23), so the distances are whole numbers of those.
    say("far from zero", rows, out)
    for at in (0.0, 4e8, -4e8, 6.2e8, -6.3e8, 1.5e9, -3e9, 1e20, 2.5e38, -2.5e38):
        case = Case(torch, 19, 5, rows, 3001, "fp32", k=9)
        step = float(np.spacing(np.float32(max(abs(at), 1.0))))
        case.z = at - step * np.random.default_rng(3).integers(0, 4, (5, 3001)) if at else case.z
        case.z = case.z.astype(np.float32).astype(np.float64)
        case.logits.copy_(torch.from_numpy(case.z).float().cuda()[torch.from_numpy(case.pick).cuda()])
        logp, _ = O.token_logprobs(case.z, case.labels)
        case.old = (np.maximum(logp, -60) + 0.05).astype(np.float32)
        case.ref = (np.maximum(logp, -60) - 0.1).astype(np.float32)
        live = logp > -60        # labels further off have a ratio of zero, and a KL term beyond 32 bits
        case.mask[:] = live
        _check_policy(case, thd, out=out, kl=0.1)
        case.logits.copy_(torch.from_numpy(case.z).float().cuda()[torch.from_numpy(case.pick).cuda()])
        case.mask[:] = 1
        _check_distill(case, thd, out=out, tau=1.5)


@pytest.mark.parametrize("rows", [5, 40, 1100])
@pytest.mark.parametrize("vocab", [2, 9, 1003, 70001])
def test_labels_near_certainty(torch, thd, rows, vocab):
    # ln q and 1 - q of a label far above the rest keep their relative precision:
    # the sum's, and 6 u of the gap from the exponentials' arguments
    say("near certainty", rows, vocab)
    case = Case(torch, 20, 5, rows, vocab, "fp32")
    case.mask[:] = 1
    case.labels[:] = [0, vocab - 1, vocab // 2, min(3, vocab - 1), vocab - 2]
    top = case.z.max(1)
    case.z[np.arange(5), case.labels] = np.float32(top + [5, 10, 15, 20, 25])
    case.logits.copy_(torch.from_numpy(case.z).float().cuda()[torch.from_numpy(case.pick).cuda()])
    gap = np.array([5, 10, 15, 20, 25]) + 30
    rel = _sum_error(vocab) + (6 * gap + 12) * U
    logp, lse, _ = thd.token_logprobs(case.logits, case.dev(case.labels))
    want, _ = O.token_logprobs(case.z, case.labels)
    _within(_host(logp), case.whole(want), case.whole(rel * np.abs(want) + 1e-15), "logp")
    # the policy that the batch was drawn with: the gradient is A (q - [y])
    old = want.astype(np.float32)
    loss, got, g, _ = thd.policy_loss(case.logits, case.dev(case.labels), case.dev(old),
                                      torch.ones(rows, device="cuda"), clip_high=0.5)
    _within(_host(got), case.whole(want), case.whole(rel * np.abs(want) + 1e-15), "logp of the policy loss")
    at = g[torch.arange(rows, device="cuda"), case.dev(case.labels)]
    not_q = -np.expm1(want)
    _within(_host(at), case.whole(-not_q), case.whole((rel + 4 * U) * not_q + 1e-15), "label's gradient")


@pytest.mark.parametrize("vocab", [200003, 300007])
def test_rows_longer_than_the_registers(torch, thd, vocab):
    say("long rows", vocab)
    case = Case(torch, 5, 3, 530, vocab, "bf16", k=100)
    _check_policy(case, thd, out="in place")
    case = Case(torch, 5, 3, 530, vocab, "bf16", k=100)
    _check_distill(case, thd, out="in place")


@pytest.mark.parametrize("rows", [1, 2, 17, 64, 255, 257, 511, 513, 1025])
def test_row_counts(torch, thd, rows):
    say("rows", rows)
    case = Case(torch, 6, min(rows, 4), rows, 12345, "bf16", k=5)
    _check_logp(case, thd)
    _check_policy(case, thd)
    _check_distill(case, thd)


@pytest.mark.parametrize("rows", [3, 1100])
@pytest.mark.parametrize("out", ["in place", "elsewhere"])
@pytest.mark.parametrize("dtype,vocab,stride,offset", [
    ("bf16", 5003, 5008, 0), ("bf16", 5003, 5011, 3), ("fp16", 4096, 4099, 1), ("fp32", 2001, 2007, 3),
    ("fp32", 2000, 2000, 1)])
def test_strides_and_places(torch, thd, rows, out, dtype, vocab, stride, offset):
    say("strides", rows, out, dtype, vocab, stride, offset)
    for check, k in ((_check_logp, 0), (_check_policy, 0), (_check_distill, 7)):
        case = Case(torch, 7, 4, rows, vocab, dtype, stride=stride, offset=offset, k=k)
        check(case, thd, out=out)
        if stride > vocab:     # nothing outside the rows is written
            pad = case.room.as_strided((rows - 1, stride - vocab), (stride, 1), offset + vocab)
            assert torch.isnan(pad).all() and torch.isnan(case.room[:offset]).all()


@pytest.mark.parametrize("rows", [4, 700])
def test_calls_of_the_c_names(torch, thd, rows):
    # caller-owned outputs and workspaces, teacher rows with a stride of their own
    say("c names", rows)
    case = Case(torch, 21, 4, rows, 70001, "bf16", k=6)
    v, z = case.vocab, case.logits
    labels, mask, old, adv = (case.dev(x) for x in (case.labels, case.mask, case.old, case.adv))
    f = lambda *n: torch.full(n, 7.0, device="cuda")
    st = torch.full((1,), 99, dtype=torch.int32, device="cuda")
    g = torch.empty_like(z)

    def room(targets):
        n = thd.thd_loss_workspace_bytes(rows, v, thd.THD_BF16, targets)
        assert (n > 0) == (rows == 4)
        return torch.full((max(n, 1),), 255, dtype=torch.uint8, device="cuda"), n
    ws, n = room(0)
    logp, lse = f(rows), f(rows)
    thd.thd_token_logprobs(z.data_ptr(), thd.THD_BF16, rows, v, v, labels, mask, logp, lse, st, ws, n)
    want = thd.token_logprobs(z, labels, mask=mask)
    assert torch.equal(logp, want[0]) and torch.equal(lse, want[1]) and int(st.item()) == 0
    thd.thd_token_logprobs_backward(adv, z.data_ptr(), thd.THD_BF16, rows, v, v, labels, lse, mask, g.data_ptr(), v)
    assert torch.equal(g, thd.token_logprobs_backward(adv, z, labels, lse, mask=mask))
    ws, n = room(1)
    loss = f(rows)
    thd.thd_policy_loss(z.data_ptr(), thd.THD_BF16, rows, v, v, labels, mask, old, None, adv, None, 0.2, 0.3, 0.0, loss,
                        logp, g.data_ptr(), v, st, ws, n)
    want = thd.policy_loss(z, labels, old, adv, mask=mask, clip_high=0.3)
    assert torch.equal(loss, want[0]) and torch.equal(logp, want[1]) and torch.equal(g, want[2])
    # no status word, no mask
    thd.thd_policy_loss(z.data_ptr(), thd.THD_BF16, rows, v, v, labels, None, old, None, adv, None, 0.2, 0.3, 0.0, loss,
                        logp, g.data_ptr(), v, None, ws, n)
    assert torch.equal(g, thd.policy_loss(z, labels, old, adv, clip_high=0.3)[2])
    ws, n = room(6)
    teacher, ids = case.dev(case.teacher).contiguous(), case.dev(case.ids).to(torch.int32).contiguous()
    wide_t = torch.full((rows, 11), float("nan"), device="cuda")
    wide_i = torch.full((rows, 11), -77, dtype=torch.int32, device="cuda")
    wide_t[:, :6], wide_i[:, :6] = teacher, ids
    thd.thd_distill_topk(z.data_ptr(), thd.THD_BF16, rows, v, v, wide_t.data_ptr(), thd.THD_FP32, wide_i.data_ptr(), 4,
                         6, 11, mask, None, 1.5, loss, g.data_ptr(), v, st, ws, n)
    want = thd.distill_topk(z, teacher, ids, mask=mask, temperature=1.5)
    assert torch.equal(loss, want[0]) and torch.equal(g, want[1]) and int(st.item()) == 0
    cu = torch.tensor([0, rows // 2, rows], dtype=torch.int32, device="cuda")
    pairs = torch.tensor([[1, 0]], dtype=torch.int32, device="cuda")
    n = thd.thd_preference_workspace_bytes(rows, 2)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    loss, rewards, d = f(1), f(1, 2), f(rows)
    thd.thd_preference_loss(logp, old, mask, cu, 2, rows, pairs, 1, 0.1, 0.0, 1.0, loss, rewards, d, st, ws, n)
    want = thd.preference_loss(logp, old, pairs, cu, mask=mask)
    assert torch.equal(loss, want[0]) and torch.equal(rewards, want[1]) and torch.equal(d, want[2])


def test_new_gradient_has_the_logits_shape(torch, thd):
    z = torch.randn((2, 3, 37), device="cuda", dtype=torch.bfloat16)
    y = torch.zeros((2, 3), dtype=torch.int64, device="cuda")
    f = torch.zeros((2, 3), device="cuda")
    loss, logp, grad, _ = thd.policy_loss(z, y, f, f + 1)
    assert grad.shape == z.shape and loss.shape == (6,)
    wide = torch.randn((6, 48), device="cuda", dtype=torch.bfloat16)
    view = wide[:, 5:42]
    view.copy_(z.view(6, 37))
    again = thd.policy_loss(view, y, f, f + 1)
    assert again[2].shape == view.shape
    # rows at another place sum in another order, so the bits may differ: each
    # is checked against the oracle elsewhere
    assert (again[2].data_ptr() - view.data_ptr()) % 16 == 0


# ---- masks, infinities, bad data ---------------------------------------------------------------------

@pytest.mark.parametrize("rows", [4, 1100])
@pytest.mark.parametrize("dtype", DTYPES)
def test_masked_rows_are_not_looked_at(torch, thd, rows, dtype):
    say("masked", rows, dtype)
    case = Case(torch, 8, 4, rows, 5001, dtype, k=6)
    case.mask[:] = [1, 0, 1, 0]
    case.labels[1], case.labels[3] = -7, 1 << 40
    case.old[1], case.adv[3] = np.nan, np.inf
    case.ids[1], case.ids[3] = -9, 1 << 30
    case.logits[1::4], case.logits[3::4] = float("nan"), float("inf")
    case.z[[1, 3]] = 0.0
    safe = case.labels.copy()
    logp, lse, st = thd.token_logprobs(case.logits, case.dev(safe), mask=case.dev(case.mask))
    assert int(st.item()) == 0
    assert not logp[1::2].any() and not lse[1::2].any() and bool((logp[::2] != 0).all())
    g = thd.token_logprobs_backward(case.dev(case.d), case.logits, case.dev(safe), lse, mask=case.dev(case.mask))
    assert not g[1::2].any() and bool(torch.isfinite(g.float()).all()) and bool(g[::2].any(1).all())
    loss, logp, g, st = thd.policy_loss(case.logits, case.dev(safe), case.dev(case.old), case.dev(case.adv),
                                        mask=case.dev(case.mask), ref_logp=case.dev(case.ref), kl_coef=0.1)
    assert int(st.item()) == 0
    assert not loss[1::2].any() and not logp[1::2].any() and not g[1::2].any()
    assert bool(torch.isfinite(g.float()).all())
    loss, g, st = thd.distill_topk(case.logits, case.dev(case.teacher).contiguous(), case.dev(case.ids).contiguous(),
                                   mask=case.dev(case.mask))
    assert int(st.item()) == 0 and not loss[1::2].any() and not g[1::2].any()
    assert bool(torch.isfinite(g.float()).all()) and bool((loss[::2] > 0).all())
    # nothing left at all
    none = torch.zeros(rows, dtype=torch.uint8, device="cuda")
    loss, logp, g, st = thd.policy_loss(case.logits, case.dev(safe), case.dev(case.old), case.dev(case.adv), mask=none)
    assert not loss.any() and not logp.any() and not g.any() and int(st.item()) == 0


@pytest.mark.parametrize("rows", [4, 1100])
@pytest.mark.parametrize("dtype", DTYPES)
def test_excluded_columns_and_lowest_values(torch, thd, rows, dtype):
    say("lowest", rows, dtype)
    case = Case(torch, 9, 4, rows, 4099, dtype, k=8)
    lowest = torch.finfo(_dtype(torch, dtype)).min
    z = case.z
    z[0, 100:4000] = -np.inf                 # columns taken out
    z[1, 7:] = lowest                        # or given the type's lowest value
    z[2, :] = lowest                         # a row of nothing else: uniform
    z[3, :4098] = -np.inf                    # one column left
    case.labels[:] = [50, 3, 4000, 4098]
    case.ids = np.tile(np.array([1, 2, 3, 4, 5, 6, 50, 4098]), (4, 1))
    case.ids[3] = [4098, -1, -1, -1, -1, -1, -1, -1]
    case.ids[1] = [0, 1, 2, 3, 4, 5, 6, -1]
    case.mask[:] = 1
    case.logits.copy_(torch.from_numpy(z).to(case.logits.dtype).cuda()[torch.from_numpy(case.pick).cuda()])
    logp, _ = O.token_logprobs(z, case.labels)
    case.old = (logp + 0.1).astype(np.float32)
    case.ref = (logp - 0.2).astype(np.float32)
    assert logp[2] == pytest.approx(-np.log(4099)) and logp[3] == 0
    _check_policy(case, thd)
    _check_distill(case, thd)
    got, lse, _ = thd.token_logprobs(case.logits, case.dev(case.labels))
    e, _ = _logp_error(z, case.labels)
    _within(_host(got), case.whole(logp), case.whole(e), "logp")


@pytest.mark.parametrize("rows", [6, 1100])
def test_rows_without_a_softmax(torch, thd, rows):
    say("nan rows", rows)
    case = Case(torch, 10, 6, rows, 3001, "bf16", k=4)
    case.mask[:] = 1
    keep = [0, 4, 5]
    z = case.logits
    z[1::6] = -float("inf")
    z[2::6, 1234] = float("inf")
    z[3::6, 17] = float("nan")
    labels = case.dev(case.labels)
    logp, lse, st = thd.token_logprobs(z, labels)
    assert int(st.item()) == 0
    for i in (1, 2, 3):
        assert bool(torch.isnan(logp[i::6]).all())
    loss, logp, g, st = thd.policy_loss(z, labels, case.dev(case.old), case.dev(case.adv))
    loss_d, g_d, _ = thd.distill_topk(z, case.dev(case.teacher).contiguous(), case.dev(case.ids).contiguous())
    for i in (1, 2, 3):
        assert bool(torch.isnan(loss[i::6]).all()) and bool(torch.isnan(logp[i::6]).all())
        assert bool(torch.isnan(g[i::6].float()).any(1).all())
        assert bool(torch.isnan(loss_d[i::6]).all())
    want = O.policy_loss(case.z[keep], case.labels[keep], case.old[keep], case.adv[keep])
    e, _ = _logp_error(case.z[keep], case.labels[keep])
    for j, i in enumerate(keep):
        assert bool(torch.isfinite(g[i::6].float()).all()) and bool(torch.isfinite(g_d[i::6].float()).all())
        assert float((logp[i::6].double() - want[1][j]).abs().max()) <= e[j]


@pytest.mark.parametrize("rows", [5, 1100])
@pytest.mark.parametrize("dtype", DTYPES)
def test_targets_outside_the_vocabulary(torch, thd, rows, dtype):
    say("bad targets", rows, dtype)
    for bad in (-1, 777, 1 << 33, -(1 << 40)):
        case = Case(torch, 11, 5, rows, 777, dtype, k=3)
        case.labels[1] = bad
        _check_policy(case, thd, status=thd.THD_ERR_LABEL)
        logp, lse, st = thd.token_logprobs(case.logits, case.dev(case.labels), mask=case.dev(case.mask))
        assert int(st.item()) == thd.THD_ERR_LABEL
        assert bool(torch.isnan(logp[1::5]).all()) and bool(torch.isfinite(logp[0::5]).all())
        g = thd.token_logprobs_backward(case.dev(case.d), case.logits, case.dev(case.labels), lse)
        assert bool(torch.isnan(g[1::5].float()).all()) and bool(torch.isfinite(g[0::5].float()).all())
        if bad != -1:
            case.ids[1, 2] = bad
            _check_distill(case, thd, status=thd.THD_ERR_LABEL)


# ---- distillation ----------------------------------------------------------------------------------------

@pytest.mark.parametrize("rows", [7, 1100])
@pytest.mark.parametrize("k", [1, 3, 64, 65, 256])
def test_teacher_columns(torch, thd, rows, k):
    say("teacher", rows, k)
    case = Case(torch, 12, 7, rows, 9001, "bf16", k=k)
    case.mask[:] = 1
    case.ids[1] = -1                                  # no column at all
    case.ids[2, k // 2:] = case.ids[2, 0]             # one column many times
    case.teacher[3] = -np.inf                         # no probability at all
    case.teacher[4, k // 2] = -np.inf
    case.ids[5, : k // 2] = -1
    case.ids[6] = np.arange(k) + 9001 - k             # neighbours, up to the row's last element
    loss, grad = _check_distill(case, thd, tau=1.0)
    for i in (1, 3):
        assert not loss[i::7].any() and not grad[i::7].any()
    _check_distill(case, thd, tau=0.25, ids64=False, teacher_dtype=torch.float16)
    _check_distill(case, thd, tau=20.0, out="in place")


def test_a_teacher_equal_to_the_student(torch, thd):
    # over the whole vocabulary: the loss is zero, up to the bound
    case = Case(torch, 13, 4, 900, 200, "fp32", k=200)
    case.ids[:] = np.arange(200)
    case.teacher = case.z.astype(np.float32)
    _check_distill(case, thd)


# ---- preference loss ---------------------------------------------------------------------------------------

def _preference(torch, thd, seed, lengths, pairs, masked=0.2, ref=True, **kw):
    rng = np.random.default_rng([seed, len(lengths)])
    cu = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
    total = int(cu[-1])
    logp = -np.exp(rng.normal(size=total)).astype(np.float32)
    r = (logp + rng.normal(0, 0.1, total)).astype(np.float32) if ref else None
    mask = (rng.random(total) >= masked).astype(np.uint8)
    if masked:
        logp[mask == 0] = np.nan
    pairs = np.asarray(pairs, dtype=np.int32).reshape(-1, 2)
    loss, rewards, d, st = thd.preference_loss(
        _dev(torch, logp), None if r is None else _dev(torch, r), _dev(torch, pairs), _dev(torch, cu),
        mask=_dev(torch, mask), **kw)
    want = O.preference_loss(np.where(mask, logp, 0), r, pairs, cu, mask, **kw)
    # sums and their functions are taken in 64 bits; results are rounded once
    # to 32. A sum's own error, 64-bit steps of up to `total` terms, is far
    # below that step except where a sum cancels.
    beta, scale = abs(kw.get("beta", 0.1)), abs(kw.get("scale", 1.0))
    lost = total * 2.0 ** -52 * np.abs(np.where(mask, logp, 0)).sum() * beta
    for got, w, f, what in ((loss, want[0], scale, "loss"), (rewards, want[1], 1.0, "rewards"),
                            (d, want[2], scale * beta, "dlogp")):
        _within(_host(got), w, 1.01 * U * np.abs(w) + 2 * lost * f + 2.0 ** -149, what)
    return loss, rewards, d, int(st.item())


@pytest.mark.parametrize("lengths,pairs", [
    ([5, 3], [(0, 1)]),
    ([1, 1, 1], [(2, 0)]),
    ([0, 512, 0, 512, 0], [(1, 3)]),
    ([511, 2, 1023, 1, 0, 600], [(0, 2), (5, 1), (3, 4)]),
    ([300] * 40, [(i, 39 - i) for i in range(20)]),
    ([17] * 700, [(i, i + 1) for i in range(0, 700, 2)]),
    ([1] * 3000, [(i, 2999 - i) for i in range(1500)]),
    ([100000, 5, 77777], [(0, 2), (2, 0), (0, 1), (0, 0), (-1, -1)]),
    ([64] * 6, [(0, j) for j in range(1, 6)]),
])
def test_preference(torch, thd, lengths, pairs):
    say("preference", len(lengths), len(pairs))
    assert _preference(torch, thd, 1, lengths, pairs)[3] == 0
    assert _preference(torch, thd, 2, lengths, pairs, ref=False, masked=0.0, beta=0.02, label_smoothing=0.3,
                       scale=1 / len(pairs))[3] == 0
    _, _, d, _ = _preference(torch, thd, 3, lengths, pairs, masked=1.0, label_smoothing=1.0)
    assert not d.any()


def test_preference_of_a_million_tokens(torch, thd):
    say("preference 1M")
    lengths = [262144 + 13, 300000, 100001, 262144 + 120000 - 100014 - 37856]
    assert _preference(torch, thd, 4, lengths, [(0, 1), (3, 2)], scale=0.5, beta=0.001)[3] == 0


def test_preference_without_tokens_or_pairs(torch, thd):
    assert _preference(torch, thd, 5, [0, 0], [(0, 1)], masked=0.0)[3] == 0
    loss, rewards, d, st = _preference(torch, thd, 6, [40, 7], [])
    assert st == 0 and loss.numel() == 0 and not d.any()


def test_preference_reports_bad_pairs_and_boundaries(torch, thd):
    say("preference errors")
    _, _, _, st = _preference(torch, thd, 7, [30, 40, 50], [(0, 1), (2, 3), (-1, 1), (1 << 30, 0), (-1, -1)])
    assert st == thd.THD_ERR_PAIR
    logp = torch.zeros(1000, device="cuda")
    pairs = torch.tensor([[0, 1]], dtype=torch.int32, device="cuda")
    for cu, code in (([1, 500, 1000], thd.THD_ERR_CU_START), ([0, 600, 500, 1000], thd.THD_ERR_CU_MONOTONE),
                     ([0, 500, 999], thd.THD_ERR_CU_TOTAL), ([0, 500, 1 << 30], thd.THD_ERR_CU_TOTAL),
                     ([0, -5, 1000], thd.THD_ERR_CU_MONOTONE), ([-(1 << 31), 2000, 1000], thd.THD_ERR_CU_START)):
        out = thd.preference_loss(logp, None, pairs, torch.tensor(cu, dtype=torch.int32, device="cuda"))
        assert int(out[3].item()) == code, cu


# ---- how the calls behave on a GPU ---------------------------------------------------------------------------

def test_offsets_beyond_32_bits(torch, thd):
    say("beyond 2^31 elements")
    rows, vocab = 8200, 262147
    z = torch.empty((rows, vocab), dtype=torch.bfloat16, device="cuda")
    assert z.numel() > 2 ** 31
    base = torch.randn((4, vocab), device="cuda").to(torch.bfloat16)
    for i in range(4):
        z[i::4] = base[i]
    labels = torch.arange(rows, device="cuda") % 4 * 60000
    old = torch.full((rows,), -12.0, device="cuda")
    adv = torch.ones(rows, device="cuda")
    _, _, g, st = thd.policy_loss(z, labels, old, adv, clip_high=3.0)
    assert int(st.item()) == 0
    host = base.double().cpu().numpy()
    want = O.policy_loss(host, [0, 60000, 120000, 180000], [-12.0] * 4, [1.0] * 4, clip_high=3.0)
    e, _ = _logp_error(host, [0, 60000, 120000, 180000])
    r = np.exp(want[1] + 12)
    bound = _grad_error(host, np.where(r <= 4, r, 0), np.where(r <= 4, r, 0) * (e + 30 * U), want[2], "bf16")
    for t in (0, 1, rows - 2, rows - 1):
        _within(_host(g[t]), want[2][t % 4], bound[t % 4], f"row {t}")
    del g
    logp, lse, _ = thd.token_logprobs(z, labels)
    assert float((logp[-4:].double().cpu() - torch.from_numpy(want[1])).abs().max()) <= e.max()
    out = thd.token_logprobs_backward(adv, z, labels, lse, out=z)
    assert out.data_ptr() == z.data_ptr()
    got = _host(z[rows - 1])
    one = np.zeros(vocab)
    one[labels[-1].item()] = 1
    soft = np.exp(host[(rows - 1) % 4] - float(lse[-1]))
    _within(got, one - soft, 2.0 ** -8 * np.abs(one - soft) + 200 * U * (soft + one), "last row")


def test_same_bits_every_time(torch, thd):
    say("same bits")
    for rows in (5, 700):
        case = Case(torch, 14, 5, rows, 33333, "bf16", k=50)
        first = None
        for _ in range(3):
            got = [*thd.policy_loss(case.logits, case.dev(case.labels), case.dev(case.old), case.dev(case.adv))[:3],
                   *thd.distill_topk(case.logits, case.dev(case.teacher).contiguous(),
                                     case.dev(case.ids).contiguous())[:2],
                   *thd.token_logprobs(case.logits, case.dev(case.labels))[:2]]
            first = first or got
            for a, b in zip(first, got):
                assert torch.equal(a, b)


@pytest.mark.parametrize("rows", [6, 700])
def test_on_another_stream(torch, thd, rows):
    say("stream", rows)
    case = Case(torch, 15, 6, rows, 20000, "bf16", k=10)
    args = (case.logits, case.dev(case.labels), case.dev(case.old), case.dev(case.adv))
    t, ids = case.dev(case.teacher).contiguous(), case.dev(case.ids).contiguous()
    want = thd.policy_loss(*args)
    want_d = thd.distill_topk(case.logits, t, ids)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (side, side.cuda_stream):
        got = thd.policy_loss(*args, stream=stream)
        got_d = thd.distill_topk(case.logits, t, ids, stream=stream)
        side.synchronize()
        for a, b in zip((*want, *want_d), (*got, *got_d)):
            assert torch.equal(a, b)
    del got, got_d


@pytest.mark.parametrize("rows", [6, 700])
def test_in_a_graph(torch, thd, rows):
    say("graph", rows)
    case = Case(torch, 16, 6, rows, 20000, "bf16", k=10)
    labels, old, adv = case.dev(case.labels), case.dev(case.old), case.dev(case.adv)
    t, ids = case.dev(case.teacher).contiguous(), case.dev(case.ids).contiguous()
    cu = torch.tensor([0, rows // 2, rows], dtype=torch.int32, device="cuda")
    pairs = torch.tensor([[0, 1]], dtype=torch.int32, device="cuda")

    def step():
        logp, lse, st = thd.token_logprobs(case.logits, labels)
        loss, _, d, _ = thd.preference_loss(logp, old, pairs, cu)
        g = thd.token_logprobs_backward(d, case.logits, labels, lse)
        return (logp, lse, st, loss, g, *thd.policy_loss(case.logits, labels, old, adv),
                *thd.distill_topk(case.logits, t, ids))
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for i in range(4):
        case.logits.copy_(torch.randn((rows, 20000), device="cuda"))
        want = step()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert torch.equal(a, b), i


def test_nothing_to_do(torch, thd):
    z = torch.zeros((0, 100), device="cuda")
    y = torch.zeros(0, dtype=torch.int64, device="cuda")
    f = torch.zeros(0, device="cuda")
    logp, lse, st = thd.token_logprobs(z, y)
    assert logp.numel() == 0 and int(st.item()) == 0
    assert thd.token_logprobs_backward(f, z, y, lse).shape == (0, 100)
    assert int(thd.policy_loss(z, y, f, f)[3].item()) == 0
    assert int(thd.distill_topk(z, torch.zeros((0, 4), device="cuda"),
                                torch.zeros((0, 4), dtype=torch.int64, device="cuda"))[2].item()) == 0


def test_gradients_against_differences(torch, thd):
    # fp32 logits: a step of 2^-7 in a logit, the loss's second derivative below
    # 1 and its own error E = bound of the log-probability, leave an error of at
    # most (2^-7)^2 + E / 2^-7
    say("differences")
    rows, vocab, step = 64, 40, 2.0 ** -7
    case = Case(torch, 17, 64, rows, vocab, "fp32", k=6, spread=1.0)
    e, _ = _logp_error(case.z, case.labels)
    bound = step ** 2 + (e.max() + 20 * U) * 4 / step
    old = (O.token_logprobs(case.z, case.labels)[0] + 0.05).astype(np.float32)   # inside the clip for every step
    args = (case.dev(case.labels), case.dev(old), case.dev(np.clip(case.adv, -1, 1)))
    t, ids = case.dev(case.teacher).contiguous(), case.dev(case.ids).contiguous()
    kw = dict(ref_logp=case.dev(case.ref), kl_coef=0.1, clip_low=0.5, clip_high=0.5)
    g = thd.policy_loss(case.logits, *args, **kw)[2]
    g_d = thd.distill_topk(case.logits, t, ids, temperature=1.0)[1]
    for v in (0, 1, 17, 39):
        up, down = case.logits.clone(), case.logits.clone()
        up[:, v] += step
        down[:, v] -= step
        width = (up[:, v] - down[:, v]).double()
        d = (thd.policy_loss(up, *args, **kw)[0].double() - thd.policy_loss(down, *args, **kw)[0].double()) / width
        assert float((d - g[:, v].double()).abs().max()) <= bound
        d = (thd.distill_topk(up, t, ids, temperature=1.0)[0].double()
             - thd.distill_topk(down, t, ids, temperature=1.0)[0].double()) / width
        assert float((d - g_d[:, v].double()).abs().max()) <= bound
