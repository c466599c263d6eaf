"""A whole step of examples/packed_losses.py: its gradients against automatic
differentiation of the same model in 64 bits on the CPU."""

import importlib.util
import math
import os

import pytest

from conftest import ROOT
from gpu_util import say

pytestmark = pytest.mark.gpu


def _model(torch, e, first):
    """The example's loss from its parameters, with its documents one by one."""
    p = {n: x.double().cpu().requires_grad_() for n, x in first["parameters"].items()}
    ids, cu, cu_padded = (first[n].cpu() for n in ("ids", "cu", "cu_padded"))
    total, count = 0.0, 0
    for s in range(len(cu) - 1):
        n, at = int(cu[s + 1] - cu[s]), int(cu_padded[s])
        if n < 1:
            continue
        x = p["table"][ids[at:at + n]]
        qkv = (x @ p["qkv"].t()).view(n, -1, e.HEAD_DIM).transpose(0, 1)
        q, k, v = qkv[:e.HEADS], qkv[e.HEADS:e.HEADS + e.KV_HEADS], qkv[e.HEADS + e.KV_HEADS:]
        k, v = (y.repeat_interleave(e.HEADS // e.KV_HEADS, 0) for y in (k, v))
        z = q @ k.transpose(1, 2) / math.sqrt(e.HEAD_DIM)
        z = z.masked_fill(torch.ones(n, n).triu(1).bool(), -math.inf)
        h = x + (z.softmax(2) @ v).transpose(0, 1).reshape(n, -1) @ p["out"].t()
        logq = (h @ p["head"].t()).log_softmax(1)
        if n > 1:
            total = total - logq[:n - 1].gather(1, ids[at + 1:at + n, None]).sum()
            count += n - 1
    return total / count, p


def test_a_whole_step():
    say("example: a whole step")
    import torch
    spec = importlib.util.spec_from_file_location("packed_losses", os.path.join(ROOT, "examples", "packed_losses.py"))
    e = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(e)
    losses, first = e.train(steps=3)
    assert all(math.isfinite(v) for v in losses)
    loss, p = _model(torch, e, first)
    loss.backward()
    loss = loss.item()
    # activations and their gradients are rounded to bf16 some six times on the way, each up to 2^-8 of its size
    assert abs(losses[0] - loss) <= 6 * 2.0 ** -8 * loss
    for name, g in first["grads"].items():
        want = p[name].grad
        off = (g.double().cpu() - want).norm() / want.norm()
        assert off <= 6 * 2.0 ** -8, (name, float(off))
    norm = math.sqrt(sum(float(g.double().square().sum()) for g in first["grads"].values()))
    assert abs(float(first["norm"]) / norm - 1) <= 2.0 ** -22
