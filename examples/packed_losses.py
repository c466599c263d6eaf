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

``train`` goes the whole way: embedding, attention inside the documents with the
queries of each rank's zigzag share, a head, the label's log-probability, the
gradients of all of it back to the embedding table, and clipping by their norm.
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
    rows, embed_status = thd.embedding(ids, embedding)
    hidden = route.swap(rows, thd.C2Z)

    def head():
        return torch.nn.Linear(HIDDEN, VOCAB, bias=False, device="cuda", dtype=torch.bfloat16)
    model, reference, teacher = head(), head(), head()
    reference.load_state_dict(model.state_dict())
    optimizer = torch.optim.SGD(model.parameters(), lr=0.5)
    status = [pack_status, roll_status, embed_status]
    history = {"policy": [], "preference": [], "distillation": []}

    def step(logits, dlogits):
        optimizer.zero_grad()
        logits.backward(dlogits)
        status.append(thd.clip_gradients([p.grad for p in model.parameters()], 100.0)[1])
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


HEADS, KV_HEADS, HEAD_DIM = 4, 2, 32


def train(steps=4, seed=0, lr=0.1, max_norm=1.0):
    """One attention layer between the embedding and the head.  Returns the losses of
    the steps, and of the first step the inputs, parameters and gradients."""
    generator = torch.Generator().manual_seed(seed)
    tokens = batch(generator)
    max_docs, capacity = 64, 1024
    ids, cu, cu_padded, pack_status = thd.pack(tokens, PAD, EOD, 2 * RANKS, capacity, max_docs)
    route = thd.Route(max_docs + 1, RANKS, capacity)
    route.build(cu_padded, RANKS, capacity)
    shifted, masks, roll_status = route.roll_labels_zigzag(ids, cu_padded, cu)
    labels, mask = shifted[0], masks[1]
    _, tokens_of, s = thd.roll_labels(ids, cu_padded, cu)
    valid = tokens_of[0]
    status = [pack_status, roll_status, s]

    def weight(rows, columns):
        return (torch.randn((rows, columns), generator=generator) / columns ** 0.5).cuda().to(torch.bfloat16)
    qkv_heads = HEADS + 2 * KV_HEADS
    table = (torch.randn((VOCAB, HIDDEN), generator=generator)).cuda().to(torch.bfloat16)
    w_qkv, w_out = weight(qkv_heads * HEAD_DIM, HIDDEN), weight(HIDDEN, HEADS * HEAD_DIM)
    w_head = weight(VOCAB, HIDDEN)
    parameters = {"table": table, "qkv": w_qkv, "out": w_out, "head": w_head}
    kept = {name: p.clone() for name, p in parameters.items()}
    share = capacity // RANKS
    scale = -1.0 / mask.sum()
    losses, first = [], None
    for _ in range(steps):
        x, s1 = thd.embedding(ids, table, mask=valid)
        qkv = (x @ w_qkv.t()).view(capacity, qkv_heads, HEAD_DIM)
        k, v = qkv[:, HEADS:HEADS + KV_HEADS], qkv[:, HEADS + KV_HEADS:]
        q = route.swap(qkv[:, :HEADS].contiguous(), thd.C2Z)
        outs, lses = [], []
        for rank in range(RANKS):
            o, lse, s2 = thd.packed_attention(q[rank * share:(rank + 1) * share], k, v, cu_padded, cu_seqlens=cu,
                                              cp_size=RANKS, rank=rank)
            outs.append(o)
            lses.append(lse)
            status.append(s2)
        mixed = torch.cat(outs)
        hidden = route.swap(x, thd.C2Z) + mixed.view(capacity, -1) @ w_out.t()
        logits = hidden @ w_head.t()
        logp, row_lse, s3 = thd.token_logprobs(logits, labels, mask=mask)
        losses.append(logp.sum() * scale)

        dlogits = thd.token_logprobs_backward(scale * mask, logits, labels, row_lse, mask=mask, out=logits)
        dhead = dlogits.t() @ hidden
        dhidden = dlogits @ w_head
        dout = dhidden.t() @ mixed.view(capacity, -1)
        dmixed = (dhidden @ w_out).view(capacity, HEADS, HEAD_DIM)
        dq, dk, dv = [], 0, 0
        for rank in range(RANKS):
            mine = slice(rank * share, (rank + 1) * share)
            a, b, c, s4 = thd.packed_attention_backward(dmixed[mine], q[mine], k, v, outs[rank], lses[rank], cu_padded,
                                                        cu_seqlens=cu, cp_size=RANKS, rank=rank)
            dq.append(a)
            dk, dv = dk + b.float(), dv + c.float()       # the sum over the ranks
            status.append(s4)
        dqkv = torch.cat([route.swap(torch.cat(dq), thd.Z2C), dk.to(k.dtype), dv.to(v.dtype)], 1).view(capacity, -1)
        dx = dqkv @ w_qkv + route.swap(dhidden, thd.Z2C)
        dtable, s5 = thd.embedding_backward(dx, ids, VOCAB, mask=valid)
        grads = {"table": dtable, "qkv": dqkv.t() @ x, "out": dout, "head": dhead}
        if first is None:
            first = {"ids": ids, "cu": cu, "cu_padded": cu_padded, "parameters": kept,
                     "grads": {name: g.clone() for name, g in grads.items()}}
        norm, s6 = thd.clip_gradients(list(grads.values()), max_norm)
        first.setdefault("norm", norm)
        for name, p in parameters.items():
            p.sub_(lr * grads[name])
        status += [s1, s3, s5, s6]

    codes = torch.cat(status).tolist()
    assert not any(codes) and route.status() == 0, [thd.thd_strerror(c) for c in codes if c]
    route.close()
    return [float(v) for v in losses], first


if __name__ == "__main__":
    for name, values in run().items():
        print(f"{name:13s}", " ".join(f"{v:.4f}" for v in values))
    print("one layer    ", " ".join(f"{v:.4f}" for v in train()[0]))
