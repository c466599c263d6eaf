"""Training a linear head on a packed batch with the losses of this library.

    python examples/packed_losses.py

Token rows are packed on the device, the zigzag route of two context-parallel
ranks is built from the padded boundaries, and the hidden states are brought
into zigzag order, as a context-parallel model holds them.  Labels and masks
come from the label roll in the same order.  Then one head learns in turn from

* a clipped policy loss against its own earlier log-probabilities, with a KL term
  towards a reference head;
* a preference between document pairs: per-token log-probabilities go back to
  token order through the route, where documents are contiguous, and their
  gradient returns the same way;
* a teacher head's top logits.

Every loss hands back the gradient of the logits, from which ``backward`` starts.
"""

import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import context_packed_sequence_amd as thd  # noqa: E402

PAD, EOD = 0, 1
VOCAB, HIDDEN, RANKS = 1003, 64, 2


def batch(generator, rows=8, seq=96):
    """[rows, seq] token rows of several documents each, with pads at the end."""
    tokens = torch.randint(2, VOCAB, (rows, seq), generator=generator)
    for r in range(rows):
        tokens[r, torch.randint(8, 64, (2,), generator=generator)] = EOD
        tokens[r, seq - int(torch.randint(1, 9, (1,), generator=generator)):] = PAD
    return tokens.cuda()


def run(steps=8, seed=0):
    """Returns {name: [loss of each step]}."""
    generator = torch.Generator().manual_seed(seed)
    torch.manual_seed(seed)
    tokens = batch(generator)
    max_docs, align, capacity = 64, 2 * RANKS, 1024
    ids, cu, cu_padded, pack_status = thd.pack(tokens, PAD, EOD, align, capacity, max_docs)

    route = thd.Route(max_docs + 1, RANKS, capacity)
    route.build(cu_padded, RANKS, capacity)
    shifted, masks, roll_status = route.roll_labels_zigzag(ids, cu_padded, cu)
    labels, mask = shifted[0], masks[1]
    per_token = mask.float() / mask.sum()

    embedding = torch.randn((VOCAB, HIDDEN), device="cuda", dtype=torch.bfloat16)
    hidden = route.swap(embedding[ids], thd.C2Z)

    def head():
        return torch.nn.Linear(HIDDEN, VOCAB, bias=False, device="cuda", dtype=torch.bfloat16)
    model, reference, teacher = head(), head(), head()
    reference.load_state_dict(model.state_dict())
    optimizer = torch.optim.SGD(model.parameters(), lr=0.5)
    status = [pack_status, roll_status]
    history = {"policy": [], "preference": [], "distillation": []}

    def step(logits, dlogits):
        optimizer.zero_grad()
        logits.backward(dlogits)
        optimizer.step()

    with torch.no_grad():
        ref_logp, _, s = thd.token_logprobs(reference(hidden), labels, mask=mask)
        teacher_logits, teacher_ids = teacher(hidden).topk(32)
    status.append(s)

    # policy loss: several steps on the log-probabilities the batch was drawn with
    old_logp = ref_logp.clone()
    advantages = torch.randn(capacity, device="cuda")
    for _ in range(steps):
        logits = model(hidden)
        loss, _, dlogits, s = thd.policy_loss(logits.detach(), labels, old_logp, advantages, mask=mask,
                                              ref_logp=ref_logp, weights=per_token, kl_coef=0.05)
        step(logits, dlogits)
        history["policy"].append(loss.sum())
        status.append(s)

    # preference loss: document 2i preferred to document 2i + 1; an entry of -1 is unused
    pairs = torch.full((max_docs // 2, 2), -1, dtype=torch.int32, device="cuda")
    lengths = cu_padded[1:max_docs + 1] - cu_padded[:max_docs]
    slots = torch.arange(max_docs, dtype=torch.int32, device="cuda").view(-1, 2)
    real = cu[1:max_docs + 1] - cu[:max_docs] > 0
    pairs.copy_(torch.where(((lengths > 0) & real).view(-1, 2).all(1, keepdim=True), slots, pairs))
    ref_natural, mask_natural = route.swap_many([ref_logp, mask], thd.Z2C)
    for _ in range(steps):
        logits = model(hidden)
        logp, lse, s = thd.token_logprobs(logits.detach(), labels, mask=mask)
        loss, rewards, dlogp, s2 = thd.preference_loss(route.swap(logp, thd.Z2C), ref_natural, pairs, cu_padded,
                                                       mask=mask_natural, beta=0.1, scale=1.0 / pairs.shape[0])
        dlogits = thd.token_logprobs_backward(route.swap(dlogp, thd.C2Z), logits.detach(), labels, lse, mask=mask)
        step(logits, dlogits)
        history["preference"].append(loss.sum())
        status += [s, s2]

    # distillation from the teacher's 32 largest logits
    for _ in range(steps):
        logits = model(hidden)
        loss, dlogits, s = thd.distill_topk(logits.detach(), teacher_logits, teacher_ids, mask=mask,
                                            weights=per_token, temperature=2.0)
        step(logits, dlogits)
        history["distillation"].append(loss.sum())
        status.append(s)

    # the one place that waits for the GPU
    codes = torch.cat(status).tolist()
    assert not any(codes) and route.status() == 0, [thd.thd_strerror(c) for c in codes if c]
    route.close()
    return {name: [float(v) for v in values] for name, values in history.items()}


if __name__ == "__main__":
    for name, values in run().items():
        print(f"{name:13s}", " ".join(f"{v:.4f}" for v in values))
