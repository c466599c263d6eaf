"""What the loss calls refuse, on the host, before any device work (CPU)."""

import os
import shutil
import subprocess
import sys

import pytest

import context_packed_sequence_amd as thd
from conftest import ROOT

# addresses far apart; nothing is read through them
Z, G, LAB, MASK, OLD, REF, ADV, W, LOSS, LOGP, STATUS, WS, T, ID = (i << 32 for i in range(1, 15))


@pytest.fixture(scope="module")
def lib():
    return thd.binding.library()


def _call(lib, name, order, good):
    def call(**kw):
        assert set(kw) <= set(good)
        return getattr(lib, name)(*[{**good, **kw}[k] for k in order])
    return call


LOGITS = dict(z=Z, dtype=thd.THD_BF16, rows=600, vocab=32000, stride=32000)
BAD_SIZES = [dict(rows=-1), dict(rows=2 ** 31), dict(vocab=0), dict(vocab=thd.THD_MAX_VOCAB + 1), dict(dtype=3),
             dict(dtype=-1), dict(stride=31999), dict(stride=2 ** 62), dict(z=None), dict(z=Z + 1)]


@pytest.fixture
def logp(lib):
    good = dict(LOGITS, labels=LAB, mask=MASK, logp=LOGP, lse=LOSS, status=STATUS, ws=None, ws_bytes=0, stream=None)
    return _call(lib, "thd_token_logprobs", list(good), good)


@pytest.fixture
def logp_backward(lib):
    good = dict(d=LOSS, **LOGITS, labels=LAB, lse=LOGP, mask=MASK, g=G, gstride=32000, stream=None)
    return _call(lib, "thd_token_logprobs_backward", list(good), good)


@pytest.fixture
def policy(lib):
    good = dict(LOGITS, labels=LAB, mask=MASK, old=OLD, ref=REF, adv=ADV, w=W, low=0.2, high=0.2, kl=0.1, loss=LOSS,
                logp=LOGP, g=G, gstride=32000, status=STATUS, ws=None, ws_bytes=0, stream=None)
    return _call(lib, "thd_policy_loss", list(good), good)


@pytest.fixture
def distill(lib):
    good = dict(LOGITS, t=T, tdtype=thd.THD_FP32, ids=ID, id_bytes=8, k=16, tstride=16, mask=MASK, w=W, tau=1.0,
                loss=LOSS, g=G, gstride=32000, status=STATUS, ws=None, ws_bytes=0, stream=None)
    return _call(lib, "thd_distill_topk", list(good), good)


@pytest.fixture
def preference(lib):
    need = lib.thd_preference_workspace_bytes(4096, 8)
    good = dict(logp=LOGP, ref=REF, mask=MASK, cu=T, n_slots=8, total=4096, pairs=ID, n_pairs=4, beta=0.1, e=0.0,
                scale=1.0, loss=LOSS, rewards=W, d=G, status=STATUS, ws=WS, ws_bytes=need, stream=None)
    return _call(lib, "thd_preference_loss", list(good), good)


@pytest.mark.parametrize("bad", BAD_SIZES)
def test_sizes(logp, logp_backward, policy, distill, bad):
    for call in (logp, logp_backward, policy, distill):
        assert call(**bad) == thd.THD_ERR_ARG


def test_missing_pointers(logp, logp_backward, policy, distill, preference):
    for call, names in ((logp, ["labels", "logp", "lse"]), (logp_backward, ["d", "labels", "lse", "g"]),
                        (policy, ["labels", "old", "ref", "adv", "loss", "logp", "g"]),
                        (distill, ["t", "ids", "loss", "g"]),
                        (preference, ["logp", "cu", "pairs", "loss", "rewards", "d", "ws"])):
        for n in names:
            assert call(**{n: None}) == thd.THD_ERR_ARG, n


def test_policy_parameters(policy):
    for bad in (dict(low=-0.1), dict(low=1.1), dict(high=-0.1), dict(high=float("inf")), dict(low=float("nan")),
                dict(kl=float("nan")), dict(kl=float("inf")), dict(gstride=31999), dict(g=G + 1)):
        assert policy(**bad) == thd.THD_ERR_ARG, bad


def test_distill_parameters(distill):
    for bad in (dict(k=0), dict(k=thd.THD_MAX_TOPK + 1), dict(id_bytes=2), dict(tdtype=5), dict(tstride=15),
                dict(tau=0.0), dict(tau=-1.0), dict(tau=float("inf")), dict(tau=float("nan")), dict(tau=1e-45),
                dict(ids=ID + 4), dict(t=T + 2)):
        assert distill(**bad) == thd.THD_ERR_ARG, bad


def test_preference_parameters(preference, lib):
    for bad in (dict(n_slots=-1), dict(total=-1), dict(total=2 ** 31), dict(n_pairs=-1),
                dict(n_pairs=thd.THD_MAX_PAIRS + 1), dict(e=-0.1), dict(e=1.1), dict(e=float("nan")),
                dict(beta=float("inf")), dict(scale=float("nan")), dict(ws=WS + 4), dict(ws_bytes=0)):
        assert preference(**bad) == thd.THD_ERR_ARG, bad
    assert lib.thd_preference_workspace_bytes(-1, 1) == -1
    assert lib.thd_preference_workspace_bytes(1, -1) == -1


def test_overlaps(logp, logp_backward, policy, distill, preference):
    n = 600 * 32000 * 2
    for call in (logp_backward, policy, distill):
        assert call(g=Z + 16) == thd.THD_ERR_ALIAS
        assert call(g=Z + n - 2) == thd.THD_ERR_ALIAS
        assert call(g=Z, gstride=32008) == thd.THD_ERR_ALIAS      # in place needs the same stride
        assert call(g=MASK) == thd.THD_ERR_ALIAS
    for call in (policy, distill):
        assert call(loss=Z) == thd.THD_ERR_ALIAS
        assert call(loss=G + 64) == thd.THD_ERR_ALIAS
        assert call(status=LOSS) == thd.THD_ERR_ALIAS
        assert call(g=Z, loss=Z + 64) == thd.THD_ERR_ALIAS
    assert policy(logp=OLD + 4) == thd.THD_ERR_ALIAS
    assert logp(lse=LOGP) == thd.THD_ERR_ALIAS
    assert preference(d=LOGP) == thd.THD_ERR_ALIAS
    assert preference(rewards=LOSS + 4) == thd.THD_ERR_ALIAS


def test_workspace(lib, logp, policy, distill):
    need = lib.thd_loss_workspace_bytes
    assert need(600, 32000, thd.THD_BF16, 0) >= 0
    for bad in ((-1, 8, 0, 0), (8, 0, 0, 0), (8, 8, 7, 0), (8, 8, 0, -1), (8, 8, 0, thd.THD_MAX_TOPK + 1)):
        assert need(*bad) == -1
    # two rows of a large vocabulary are cut into parts: without a workspace the calls refuse
    for call, targets in ((logp, 0), (policy, 1), (distill, 16)):
        n = need(2, 131072, thd.THD_BF16, targets)
        assert n > 0
        for bad in (dict(ws=None, ws_bytes=n), dict(ws=WS, ws_bytes=n - 1), dict(ws=WS + 4, ws_bytes=n)):
            assert call(rows=2, vocab=131072, stride=131072, **bad) == thd.THD_ERR_ARG


def test_wrappers_refuse_before_any_device_call():
    torch = pytest.importorskip("torch")
    z = torch.zeros((4, 10))
    y = torch.zeros(4, dtype=torch.int64)
    f = torch.zeros(4)
    cu = torch.tensor([0, 2, 4], dtype=torch.int32)
    pairs = torch.tensor([[0, 1]], dtype=torch.int32)
    for text, call in (
            ("must be bfloat16", lambda: thd.token_logprobs(z.double(), y)),
            ("last dimension", lambda: thd.token_logprobs(torch.zeros((10, 4)).t(), y)),
            ("must not overlap", lambda: thd.token_logprobs(torch.zeros((1, 10)).expand(4, 10), y)),
            ("flattened", lambda: thd.token_logprobs(torch.zeros((2, 2, 10)).transpose(0, 1), y)),
            ("at least one column", lambda: thd.token_logprobs(torch.zeros((4, 0)), y)),
            ("labels must be torch.int64", lambda: thd.token_logprobs(z, y.int())),
            ("labels must have 4", lambda: thd.token_logprobs(z, y[:3])),
            ("labels is required", lambda: thd.token_logprobs(z, None)),
            ("mask must be torch.uint8", lambda: thd.token_logprobs(z, y, y)),
            ("must live on the GPU", lambda: thd.token_logprobs(z, y)),
            ("dlogp must have 4", lambda: thd.token_logprobs_backward(f[:2], z, y, f)),
            ("must live on the GPU", lambda: thd.token_logprobs_backward(f, z, y, f)),
            ("needs ref_logp", lambda: thd.policy_loss(z, y, f, f, kl_coef=0.1)),
            ("advantages must be torch.float32", lambda: thd.policy_loss(z, y, f, f.double())),
            ("must be contiguous", lambda: thd.policy_loss(z, y, torch.zeros(8)[::2], f)),
            ("must live on the GPU", lambda: thd.policy_loss(z, y, f, f)),
            ("teacher_ids must be int32", lambda: thd.distill_topk(z, z[:, :2].contiguous(), f)),
            ("at most 256", lambda: thd.distill_topk(z, torch.zeros((4, 257)), torch.zeros((4, 257)).long())),
            ("must be \\[4, 2\\]", lambda: thd.distill_topk(z, torch.zeros((4, 2)), torch.zeros((4, 3)).long())),
            ("must live on the GPU", lambda: thd.distill_topk(z, torch.zeros((4, 2)), torch.zeros((4, 2)).long())),
            ("pairs must be \\[pairs, 2\\]", lambda: thd.preference_loss(f, f, pairs[0], cu)),
            ("pairs must be torch.int32", lambda: thd.preference_loss(f, f, pairs.long(), cu)),
            ("cu_seqlens_padded must be torch.int32", lambda: thd.preference_loss(f, f, pairs, cu.long())),
            ("must live on the GPU", lambda: thd.preference_loss(f, f, pairs, cu))):
        with pytest.raises(ValueError, match=text):
            call()


def test_header_is_plain_c(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    src = tmp_path / "uses_header.c"
    src.write_text('#include "thd_loss.h"\n'
                   "int main(void) { return thd_loss_workspace_bytes(2, 131072, THD_BF16, 1) > 0 ? 0 : 1; }\n")
    pkg = os.path.join(ROOT, "context_packed_sequence_amd")
    exe = str(tmp_path / "uses_header")
    res = subprocess.run([cc, "-std=c11", "-Wall", "-Wextra", "-Werror", f"-I{ROOT}/include", str(src), "-o", exe,
                          f"-L{pkg}", "-lthdcp", f"-Wl,-rpath,{pkg}"], capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
    assert subprocess.run([exe], timeout=60).returncode == 0


def test_one_hip_runtime_whatever_is_imported_first():
    # the library's HIP runtime and torch's are different files of one name:
    # with both in a process, each has devices of its own
    code = ("import context_packed_sequence_amd, torch\n"
            "print(len({l.split()[-1] for l in open('/proc/self/maps') if 'libamdhip64' in l}))\n")
    res = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=ROOT, timeout=300)
    assert res.returncode == 0, res.stderr
    assert res.stdout.split()[-1] == "1"
