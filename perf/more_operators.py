"""Measured cases of the operators of a training step on a packed stream, between the packing and the optimizer.

Documents lie end to end in a stream of `tokens` positions, as the packing writes them: padded boundaries say where each
one starts, real boundaries how long it is, the last slot may hold pads only, and slots may be empty.

Operators (`op` of a case):

* ``attn``        attention inside each document: queries of the whole stream, or of one context-parallel rank's zigzag
                  share, over the keys and values of the whole stream; causal or not, with a window, with scores capped
                  by a tanh
* ``attn_grad``   the same and its backward pass, as one training step runs them
* ``embed``       rows of the embedding table for the stream's token ids, scaled
* ``embed_grad``  the table's gradient from the rows' gradients
* ``clip``        norm of all gradients and the gradients scaled down to a largest norm
"""

import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}

MAX_PAIR_WORK = 2.0e11          # pairs x query heads x head size of one drawn case
MAX_ELEMENTS = 1 << 28          # of one drawn table, batch of rows, or set of gradients
CLIP_EPS = 1e-6


def _attn(name, op, tokens, low, high, align, heads, kv_heads, dim, dtype, causal=True, window=0, cap=0.0, cp=1, rank=0):
    case = dict(op=op, tokens=tokens, low=low, high=high, align=align, heads=heads, kv_heads=kv_heads, dim=dim,
                dtype=dtype, causal=causal, window=window, cap=cap, cp=cp, rank=rank)
    return dict(case, name=name) if name else case


def listed():
    return [
        # scoring the smallest packed batch: latency counts
        _attn("attn_few", "attn", 24, 4, 12, 4, 4, 2, 64, "bf16"),
        # scoring many short documents, as a fine-tuning batch holds them: tiles that documents fill badly
        _attn("attn_sft", "attn", 32768, 64, 1024, 16, 32, 8, 128, "bf16"),
        # every token sees its whole document (no causal mask), odd lengths and a head size that fills no tile
        _attn("attn_full_odd", "attn", 5003, 1, 4001, 1, 12, 12, 72, "fp16", causal=False),
        # a small training step with a window and capped scores, in half precision
        _attn("attn_grad_few", "attn_grad", 515, 30, 300, 1, 8, 2, 64, "fp16", window=64, cap=30.0),
        # a training step on many short documents
        _attn("attn_grad_sft", "attn_grad", 16384, 64, 1024, 16, 32, 8, 128, "bf16"),
        # one of 4 ranks trains on its zigzag share of long documents, capped scores
        _attn("attn_grad_share", "attn_grad", 32768, 8192, 32768, 8, 16, 4, 128, "bf16", cap=50.0, cp=4, rank=1),
        # a few positions in full precision, odd row size
        dict(name="embed_few", op="embed", rows=24, vocab=32000, width=1001, dtype="fp32", masked=0.1),
        # one rank's share of a 128K batch with this repository's vocabulary and row size
        dict(name="embed_share", op="embed", rows=32768, vocab=32000, width=4096, dtype="bf16", masked=0.05),
        # its gradient where the table is far larger than the batch, odd sizes
        dict(name="embed_grad_odd", op="embed_grad", rows=4099, vocab=100003, width=1001, dtype="fp32", masked=0.1),
        # its gradient for the share above
        dict(name="embed_grad_share", op="embed_grad", rows=32768, vocab=32000, width=4096, dtype="bf16", masked=0.05),
        # many small gradients of odd sizes
        dict(name="clip_many", op="clip", tensors=293, elements=1 << 20, dtype="fp32", clipped=False),
        # a model's gradients, clipped
        dict(name="clip_large", op="clip", tensors=147, elements=1 << 29, dtype="bf16", clipped=True),
    ]


def _log_uniform(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn_grad", "attn_grad", "embed", "embed_grad", "clip"])
    if op == "clip":
        elements = _log_uniform(rng, 1000, MAX_ELEMENTS)
        return dict(op=op, tensors=_log_uniform(rng, 1, min(600, elements // 10)), elements=elements,
                    dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]), clipped=rng.random() < 0.7)
    if op in ("embed", "embed_grad"):
        width = _log_uniform(rng, 8, 8192)
        return dict(op=op, rows=_log_uniform(rng, 1, min(131072, MAX_ELEMENTS // width)),
                    vocab=_log_uniform(rng, 100, min(262144, MAX_ELEMENTS // width)), width=width,
                    dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]), masked=rng.choice([0.0, 0.1, 0.4]))
    while True:
        cp = rng.choice([1, 1, 1, 2, 4, 8])
        align = 2 * cp * rng.choice([1, 1, 2, 8]) if cp > 1 else rng.choice([1, 1, 8, 16])
        tokens = max(1, _log_uniform(rng, 1, 32768) // align) * align
        high = _log_uniform(rng, 1, tokens)
        kv_heads = rng.choice([1, 2, 4, 8])
        case = _attn(None, op, tokens, max(1, high // rng.choice([1, 4, 16])), high, align,
                     kv_heads * rng.choice([1, 2, 4, 8]), kv_heads, rng.choice([64, 128, 128, 8 * rng.randint(1, 16)]),
                     rng.choice(["bf16", "bf16", "fp16"]), causal=rng.random() < 0.8,
                     window=rng.choice([0, 0, 0, _log_uniform(rng, 1, tokens)]), cap=rng.choice([0.0, 0.0, 30.0, 50.0]),
                     cp=cp, rank=rng.randrange(cp))
        pairs, rows = _pairs(case), sum(n for _, n, _, _, _ in _pieces(case))
        # a row that sees one key alone has no gradient but rounding's: rows see several on average
        enough = rows > 0 and (op == "attn" or pairs >= 6 * rows)
        if enough and pairs * case["heads"] * case["dim"] <= MAX_PAIR_WORK and len(_documents(case)) <= 300:
            return case


# ---- documents --------------------------------------------------------------


def _documents(case):
    """[(padded start, padded length, real length)]: lengths spread over [low, high] by their logarithm, padded to
    `align`; a pad-only slot takes what is left of the stream, and a few slots are empty."""
    rng = random.Random("%(tokens)d %(low)d %(high)d %(align)d" % case)
    docs, at, align = [], 0, case["align"]
    while at < case["tokens"]:
        real = _log_uniform(rng, case["low"], case["high"])
        padded = -(-real // align) * align
        if at + padded > case["tokens"]:
            real, padded = (0, case["tokens"] - at) if docs else (case["tokens"], case["tokens"])
        docs.append((at, padded, real))
        at += padded
        if rng.random() < 0.05:
            docs.append((at, 0, 0))
    return docs


def _pieces(case):
    """The share's queries as runs of one document: (first row, rows, first position, document's start, real length).
    A rank's zigzag share holds chunks rank and 2 cp - 1 - rank of each document."""
    cp, out = case["cp"], []
    for start, padded, real in _documents(case):
        chunk = padded // (2 * cp)
        cuts = [(start, padded, 0)] if cp == 1 else [
            (start // cp, chunk, case["rank"] * chunk), (start // cp + chunk, chunk, (2 * cp - 1 - case["rank"]) * chunk)]
        for row, n, pos in cuts:
            n = min(n, real - pos)
            if n > 0:
                out.append((row, n, pos, start, real))
    return out


def _seen(case, pos, real):
    """First and end position of the keys that position `pos` sees."""
    w = case["window"]
    end = pos + 1 if case["causal"] else min(real, pos + w) if w else real
    return (max(0, pos - w + 1) if w else 0), end


def _pairs(case):
    total = 0
    for _, n, pos, _, real in _pieces(case):
        if case["window"]:
            total += sum(e - b for b, e in (_seen(case, p, real) for p in range(pos, pos + n)))
        else:
            total += n * pos + n * (n + 1) // 2 if case["causal"] else n * real
    return total


def work(case):
    op = case["op"]
    b = BYTES[case["dtype"]]
    if op == "clip":
        n = case["elements"]
        return {"bytes": 2 * n * b, "flops": 3 * n}
    if op in ("embed", "embed_grad"):
        t, live, width = case["rows"], case["rows"] * (1.0 - case["masked"]), case["width"]
        if op == "embed":
            # no more rows of the table than there are
            return {"bytes": int(min(live, case["vocab"]) * width * b + t * width * b + t * 9), "flops": int(live * width)}
        return {"bytes": int(live * width * b + case["vocab"] * width * b + t * 9), "flops": int(live * width)}
    h, kv, d, tokens = case["heads"], case["kv_heads"], case["dim"], case["tokens"]
    rows, pairs = tokens // case["cp"], _pairs(case)
    q, k = rows * h * d * b, tokens * kv * d * b
    if op == "attn":
        return {"bytes": 2 * q + 2 * k + 4 * rows * h, "flops": 4 * d * h * pairs}
    # forward: two products; backward: five
    return {"bytes": 4 * q + 4 * k + 4 * rows * h, "flops": 14 * d * h * pairs}


# ---- inputs -----------------------------------------------------------------


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, dtype = case["op"], DTYPES[case["dtype"]]

    def normal(*shape, scale=1.0):
        x = torch.empty(shape, device="cuda", dtype=dtype)
        return x.normal_(0.0, scale, generator=g)

    s = {"op": op, "case": case}
    if op == "clip":
        gc = random.Random(seed)
        # sizes spread over a factor of a thousand, as weights, biases and norms of one model are
        shares = [math.exp(gc.uniform(0.0, math.log(1000.0))) for _ in range(case["tensors"])]
        rest = case["elements"] - case["tensors"]
        ends = [0]
        for share in shares:
            ends.append(ends[-1] + 1 + int(rest * share / sum(shares)))
        ends[-1] = case["elements"]
        scale = 1e-3
        s["grads"] = [normal(e - a, scale=scale) for a, e in zip(ends, ends[1:])]
        s["flat"] = torch.empty(case["elements"], device="cuda", dtype=dtype)
        s["outs"] = [s["flat"][a:e] for a, e in zip(ends, ends[1:])]
        norm = scale * math.sqrt(case["elements"])
        s["max_norm"] = 0.3 * norm if case["clipped"] else 3.0 * norm
        return s
    if op in ("embed", "embed_grad"):
        t, v, width = case["rows"], case["vocab"], case["width"]
        # token ranks as text has them: the n-th frequent one about 1 / n of the time, spread over the table
        rank = torch.exp(torch.rand(t, generator=g, device="cuda", dtype=torch.float64) * math.log(v)).long() - 1
        places = torch.randperm(v, generator=g, device="cuda")
        s["ids"] = places[rank.clamp(0, v - 1)]
        s["mask"] = (torch.rand(t, generator=g, device="cuda") >= case["masked"]).to(torch.uint8)
        s["mask"][0] = 1
        s["vocab"], s["scale"] = v, math.sqrt(width)
        s["table" if op == "embed" else "drows"] = normal(v if op == "embed" else t, width, scale=0.02)
        return s
    h, kv, d, tokens = case["heads"], case["kv_heads"], case["dim"], case["tokens"]
    # one projection's output: queries, keys and values side by side where a rank holds the whole stream
    if case["cp"] == 1:
        qkv = normal(tokens, h + 2 * kv, d)
        s["q"], s["k"], s["v"] = qkv[:, :h], qkv[:, h:h + kv], qkv[:, h + kv:]
    else:
        kvs = normal(tokens, 2 * kv, d)
        s["q"], s["k"], s["v"] = normal(tokens // case["cp"], h, d), kvs[:, :kv], kvs[:, kv:]
    s["q"].mul_(2.0)
    if op == "attn_grad":
        s["dout"] = normal(tokens // case["cp"], h, d)
    docs = _documents(case)
    ends = [0]
    for _, _, real in docs:
        ends.append(ends[-1] + real)
    s["cu_padded"] = torch.tensor([start for start, _, _ in docs] + [tokens], dtype=torch.int32, device="cuda")
    s["cu"] = torch.tensor(ends, dtype=torch.int32, device="cuda")
    s["pieces"] = _pieces(case)
    return s


# ---- one pass ---------------------------------------------------------------


def run(s):
    return _run_own(s) if own else _PLAIN[s["op"]](s)


def _run_own(s):
    import context_packed_sequence_amd as thd
    op, case = s["op"], s["case"]
    if op == "clip":
        norm, _ = thd.clip_gradients(s["grads"], s["max_norm"], outs=s["outs"])
        return norm, s["flat"]
    if op == "embed":
        return thd.embedding(s["ids"], s["table"], mask=s["mask"], scale=s["scale"])[0]
    if op == "embed_grad":
        return thd.embedding_backward(s["drows"], s["ids"], s["vocab"], mask=s["mask"], scale=s["scale"])[0]
    how = dict(cu_seqlens=s["cu"], causal=case["causal"], window=case["window"], cap=case["cap"], cp_size=case["cp"],
               rank=case["rank"])
    out, lse, _ = thd.packed_attention(s["q"], s["k"], s["v"], s["cu_padded"], **how)
    if op == "attn":
        return out, lse
    dq, dk, dv, _ = thd.packed_attention_backward(s["dout"], s["q"], s["k"], s["v"], out, lse, s["cu_padded"], **how)
    return out, lse, dq, dk, dv


def _plain_clip(s):
    # sums of up to 2^29 squares: 64 bits where a tensor's sum meets the others'
    total = torch.stack([(x.float() * x.float()).sum() for x in s["grads"]]).double().sum()
    norm = torch.sqrt(total).float()
    factor = (s["max_norm"] / (norm + CLIP_EPS)).clamp(max=1.0)
    for x, out in zip(s["grads"], s["outs"]):
        out.copy_(x.float() * factor)
    return norm.view(1), s["flat"]


def _plain_embed(s):
    rows = s["table"][s["ids"]].float() * s["scale"]
    return (rows * s["mask"][:, None]).to(s["table"].dtype)


def _plain_embed_grad(s):
    drows = s["drows"].float() * (s["mask"].float() * s["scale"])[:, None]
    grad = torch.zeros((s["vocab"], drows.shape[1]), device="cuda")
    return grad.index_add_(0, s["ids"], drows).to(s["drows"].dtype)


def _plain_attn(s):
    """Attention, and its gradient where there is one to start from; a few rows of a document at a time, so that
    their scores over all heads fit."""
    case, q, k, v, dout = s["case"], s["q"], s["k"], s["v"], s.get("dout")
    rows, h, d = q.shape
    kv = k.shape[1]
    scale, cap, w = 1.0 / math.sqrt(d), case["cap"], case["window"]
    out = torch.zeros((rows, h, d), device="cuda", dtype=q.dtype)
    lse = torch.full((h, rows), -math.inf, device="cuda")
    if dout is not None:
        dq = torch.zeros((rows, h, d), device="cuda", dtype=q.dtype)
        dk, dv = torch.zeros(k.shape, device="cuda"), torch.zeros(v.shape, device="cuda")

    def heads_first(x):      # [n, heads, d] -> [kv heads, heads of the group x n, d]
        return x.float().transpose(0, 1).reshape(kv, -1, d)

    for row0, total, pos0, start, real in s["pieces"]:
        step = max(16, (1 << 27) // (h * real))
        for a in range(0, total, step):
            n, pos, row = min(step, total - a), pos0 + a, row0 + a
            low = _seen(case, pos, real)[0]
            high = _seen(case, pos + n - 1, real)[1]
            x, ks, vs = heads_first(q[row:row + n]), heads_first(k[start + low:start + high]), heads_first(v[start + low:start + high])
            z = torch.matmul(x, ks.transpose(1, 2)).view(h, n, high - low) * scale
            if cap:
                t = torch.tanh(z / cap)
                z = t * cap
            if case["causal"] or w:
                gap = torch.arange(pos, pos + n, device="cuda")[:, None] - torch.arange(low, high, device="cuda")[None]
                hidden = gap < (0 if case["causal"] else 1 - w)
                if w:
                    hidden = hidden | (gap >= w)
                z.masked_fill_(hidden, -math.inf)
            top = z.amax(2, keepdim=True)
            p = torch.exp(z - top)
            total_p = p.sum(2, keepdim=True)
            lse[:, row:row + n] = (top + torch.log(total_p))[:, :, 0]
            p /= total_p
            o = torch.matmul(p.view(kv, -1, high - low), vs).view(h, n, d)
            out[row:row + n] = o.transpose(0, 1).to(q.dtype)
            if dout is None:
                continue
            g = heads_first(dout[row:row + n])
            dv[start + low:start + high] += torch.matmul(p.view(kv, -1, high - low).transpose(1, 2), g).transpose(0, 1)
            dz = torch.matmul(g, vs.transpose(1, 2)).view(h, n, high - low)
            dz = p * (dz - (g.view(h, n, d) * o).sum(2, keepdim=True))
            if cap:
                dz *= 1.0 - t * t
            dz = (dz * scale).view(kv, -1, high - low)
            dq[row:row + n] = torch.matmul(dz, ks).view(h, n, d).transpose(0, 1).to(q.dtype)
            dk[start + low:start + high] += torch.matmul(dz.transpose(1, 2), x).transpose(0, 1)
    return (out, lse) if dout is None else (out, lse, dq, dk.to(k.dtype), dv.to(v.dtype))


_PLAIN = {"attn": _plain_attn, "attn_grad": _plain_attn, "embed": _plain_embed, "embed_grad": _plain_embed_grad,
          "clip": _plain_clip}


# ---- the definitions in 64 bits -----------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "clip":
        norm = math.sqrt(math.fsum(float(torch.linalg.vector_norm(x.double())) ** 2 for x in s["grads"]))
        factor = min(1.0, s["max_norm"] / (norm + CLIP_EPS))
        flat = torch.cat([x.double() for x in s["grads"]]) * factor
        return torch.tensor([norm], dtype=torch.float64), flat
    if op == "embed":
        return torch.nn.functional.embedding(s["ids"], s["table"].double()) * (s["scale"] * s["mask"].double())[:, None]
    if op == "embed_grad":
        # sorted by token, ends of a running sum in 64 bits
        kept = s["mask"].bool().nonzero()[:, 0]
        ids, order = torch.sort(s["ids"][kept], stable=True)
        out = torch.zeros((case["vocab"], case["width"]), dtype=torch.float64, device="cuda")
        if ids.numel():
            names, counts = torch.unique_consecutive(ids, return_counts=True)
            ends = torch.cumsum(counts, 0)
            for a in range(0, case["width"], 1024):
                run_sum = torch.cumsum(s["drows"][kept[order], a:a + 1024].double(), 0)[ends - 1]
                run_sum[1:] -= run_sum[:-1].clone()
                out[names, a:a + 1024] = run_sum * s["scale"]
        return out
    return _exact_attn(case, s)


def _exact_attn(case, s):
    """Each key head of each document by itself, its gradient by differentiating the definition."""
    rows, h, d = s["q"].shape
    group, wide = h // case["kv_heads"], case["op"] == "attn_grad"
    out = torch.zeros((rows, h, d), dtype=torch.float64, device="cuda")
    lse = torch.full((h, rows), -math.inf, dtype=torch.float64, device="cuda")
    dq, dk, dv = torch.zeros_like(out), torch.zeros_like(s["k"], dtype=torch.float64), torch.zeros_like(s["v"], dtype=torch.float64)
    for row0, total, pos0, start, real in s["pieces"]:
        step = max(1, (1 << 26) // (real * group))
        for a in range(0, total, step):
            at = torch.arange(a, min(a + step, total), device="cuda")
            i, j = (pos0 + at)[:, None], torch.arange(real, device="cuda")[None]
            sees = torch.ones((1, 1), dtype=torch.bool, device="cuda").expand(at.numel(), real)
            if case["causal"]:
                sees = sees & (j <= i)
            if case["window"]:
                sees = sees & ((i - j).abs() < case["window"])
            r = row0 + at
            for b in range(case["kv_heads"]):
                mine = slice(b * group, (b + 1) * group)
                x = s["q"][r, mine].double().permute(1, 0, 2).contiguous().requires_grad_(wide)
                y = s["k"][start:start + real, b].double().contiguous().requires_grad_(wide)
                u = s["v"][start:start + real, b].double().contiguous().requires_grad_(wide)
                z = (x.reshape(-1, d) @ y.t()).view(group, -1, real) / math.sqrt(d)
                if case["cap"]:
                    z = case["cap"] * torch.tanh(z / case["cap"])
                z = torch.where(sees, z, -math.inf)
                o = (torch.softmax(z, 2).view(-1, real) @ u).view(group, -1, d)
                out[r, mine] = o.detach().permute(1, 0, 2)
                lse[mine, r[0]:r[-1] + 1] = torch.logsumexp(z.detach(), 2)
                if wide:
                    gx, gy, gu = torch.autograd.grad(o, (x, y, u), s["dout"][r, mine].double().permute(1, 0, 2))
                    dq[r, mine] = gx.permute(1, 0, 2)
                    dk[start:start + real, b] += gy
                    dv[start:start + real, b] += gu
    return (out, lse, dq, dk, dv) if wide else (out, lse)
