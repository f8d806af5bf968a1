"""Cases of the operators of one batched decode step: filling the paged cache, attention over it, and the next token.

``run`` computes an operator in elementary torch operations, or, where ``own`` is true, by the call that a program
makes of this package.  ``exact`` is the definition in float64."""

import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # one token of the 57.7M model's attention (8 heads of 64, rotary): the latency of a single-user decode step
        {"name": "append_one", "op": "append", "tokens": 1, "seqs": 1, "before": 1000, "heads": 8, "kv_heads": 8, "dim": 64,
         "page": 16, "rope": 64, "type": "bf16"},
        # one decode step of 256 sequences with shared key heads
        {"name": "append_step", "op": "append", "tokens": 256, "seqs": 256, "before": 1024, "heads": 32, "kv_heads": 8,
         "dim": 128, "page": 16, "rope": 128, "type": "bf16"},
        # a few prompts of the 162M model's heads in fp32, half of each head rotated
        {"name": "append_prompts_fp32", "op": "append", "tokens": 4095, "seqs": 5, "before": 3, "heads": 12, "kv_heads": 12,
         "dim": 64, "page": 32, "rope": 32, "type": "fp32"},
        # the largest: a full batch of prompts at once
        {"name": "append_prompts", "op": "append", "tokens": 32768, "seqs": 24, "before": 0, "heads": 32, "kv_heads": 8,
         "dim": 128, "page": 64, "rope": 128, "type": "bf16"},
        # one sequence of the 162M model at its full context, the serving partition's cache type
        {"name": "attend_one_fp32", "op": "attend", "seqs": 1, "shortest": 513, "longest": 513, "heads": 12, "kv_heads": 12,
         "dim": 64, "page": 16, "type": "fp32"},
        # the 350M model's heads, sequences of every length up to its context
        {"name": "attend_batch", "op": "attend", "seqs": 200, "shortest": 1, "longest": 1024, "heads": 16, "kv_heads": 16,
         "dim": 64, "page": 16, "type": "bf16"},
        # shared key heads, ragged lengths into the thousands
        {"name": "attend_shared", "op": "attend", "seqs": 64, "shortest": 17, "longest": 8192, "heads": 32, "kv_heads": 8,
         "dim": 128, "page": 16, "type": "bf16"},
        # one very long sequence: all of the GPU on one row of the batch
        {"name": "attend_long", "op": "attend", "seqs": 1, "shortest": 131071, "longest": 131071, "heads": 32, "kv_heads": 8,
         "dim": 128, "page": 64, "type": "bf16"},
        # one row of the 57.7M model's vocabulary
        {"name": "token_one", "op": "token", "rows": 1, "vocab": 12288, "history": 1000, "type": "bf16", "mask": False},
        # a batch of the 162M model's logits, grammar masks on
        {"name": "token_batch", "op": "token", "rows": 64, "vocab": 50304, "history": 1024, "type": "fp32", "mask": True},
        # a vocabulary of odd size: rows begin at any alignment
        {"name": "token_odd", "op": "token", "rows": 33, "vocab": 49999, "history": 3001, "type": "bf16", "mask": True},
        # the largest: many rows of a large vocabulary
        {"name": "token_large", "op": "token", "rows": 512, "vocab": 131072, "history": 2048, "type": "fp32", "mask": True},
    ]


def _log_int(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "token"])
    kind = rng.choice(["bf16", "bf16", "fp32"])
    if op == "token":
        vocab = _log_int(rng, 256, 131072)
        rows = _log_int(rng, 1, min(512, (1 << 25) // vocab))
        return {"op": op, "rows": rows, "vocab": vocab, "history": _log_int(rng, 1, 4096), "type": kind,
                "mask": rng.random() < 0.5}
    dim = rng.choice([32, 64, 64, 80, 96, 128, 128])
    kv_heads = rng.choice([1, 2, 4, 8, 12, 16])
    heads = kv_heads * rng.choice([1, 1, 2, 3, 4, 7, 8])
    page = rng.choice([8, 16, 24, 32, 64, 128])
    row = kv_heads * dim * (2 if kind == "bf16" else 4)  # bytes of a key of all heads
    if op == "append":
        tokens = _log_int(rng, 1, min(32768, (1 << 28) // (row + heads * dim * 2)))
        seqs = rng.choice([tokens, max(1, tokens // 100), 1]) if tokens <= 512 else _log_int(rng, 1, 32)
        return {"op": op, "tokens": tokens, "seqs": min(seqs, tokens), "before": _log_int(rng, 1, 1500), "heads": heads,
                "kv_heads": kv_heads, "dim": dim, "page": page, "rope": rng.choice([0, dim // 4, dim // 2, dim, dim]),
                "type": kind}
    seqs = _log_int(rng, 1, 256)
    most = max(2, min(131072, (1 << 28) // (row * seqs)))
    longest = _log_int(rng, 1, most)
    return {"op": op, "seqs": seqs, "shortest": min(longest, _log_int(rng, 1, longest)), "longest": longest, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "page": page, "type": kind}


def _spread(n, low, high):
    """n whole numbers from low to high, evenly spread (the same for every seed: the work of a case is fixed)."""
    if n == 1:
        return [high]
    return [low + (high - low) * i // (n - 1) for i in range(n)]


def _counts(case):
    """New tokens of each sequence, unevenly: together case["tokens"], one at least."""
    n, s = case["tokens"], case["seqs"]
    spare = n - s
    weight = [i + 1 for i in range(s)]
    got = [1 + spare * w // sum(weight) for w in weight]
    got[-1] += n - sum(got)
    return got


def _lens(case):
    return _spread(case["seqs"], case["shortest"], case["longest"])


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _cache(case, lens, g):
    """Key and value pages in a random order over a pool with some spare pages, and the table of each sequence's pages."""
    page, shape = case["page"], (case["kv_heads"], case["dim"])
    used = [(n + page - 1) // page for n in lens]
    n_pages = sum(used) + 3
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros(len(lens), max(used), dtype=torch.int32, device="cuda")
    at = 0
    for i, n in enumerate(used):
        table[i, :n] = order[at:at + n]
        at += n
    kind = TYPES[case["type"]]
    k, v = (torch.randn(n_pages, page, *shape, generator=g, device="cuda", dtype=kind) for _ in range(2))
    return k, v, table


def prepare(case, seed):
    g = _generator(seed)
    kind = TYPES[case["type"]]
    s = dict(case)
    if case["op"] == "append":
        counts = _counts(case)
        before = torch.randint(0, case["before"] + 1, (case["seqs"],), generator=g, device="cuda").tolist()
        s["k_cache"], s["v_cache"], s["table"] = _cache(case, [case["before"] + n for n in counts], g)
        # one projection's output, q | k | v side by side in a token's row
        width = (case["heads"] + 2 * case["kv_heads"]) * case["dim"]
        qkv = torch.randn(case["tokens"], width, generator=g, device="cuda", dtype=kind)
        q, k, v = qkv.split([case["heads"] * case["dim"]] + 2 * [case["kv_heads"] * case["dim"]], dim=1)
        s["q"], s["k"], s["v"] = (x.unflatten(1, (-1, case["dim"])) for x in (q, k, v))
        seq, pos = [], []
        for i, n in enumerate(counts):
            seq += [i] * n
            pos += range(before[i], before[i] + n)
        s["seq"] = torch.tensor(seq, dtype=torch.int32, device="cuda")
        s["positions"] = torch.tensor(pos, dtype=torch.int32, device="cuda")
    elif case["op"] == "attend":
        lens = _lens(case)
        order = torch.randperm(len(lens), generator=g, device="cuda").tolist()
        lens = [lens[i] for i in order]
        s["k_cache"], s["v_cache"], s["table"] = _cache(case, lens, g)
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s["q"] = torch.randn(case["seqs"], case["heads"], case["dim"], generator=g, device="cuda", dtype=kind)
    else:
        rows, vocab, most = case["rows"], case["vocab"], case["history"]
        s["logits"] = 3.0 * torch.randn(rows, vocab, generator=g, device="cuda").to(kind)
        # tokens repeat as in text: a few ids are frequent
        u = torch.rand(rows, most, generator=g, device="cuda")
        s["history_ids"] = (u.pow(4) * vocab).to(torch.int32).clamp_(max=vocab - 1)
        s["history_lens"] = torch.tensor(_spread(rows, max(1, most // 2), most), dtype=torch.int32, device="cuda")
        s["prompt_lens"] = (s["history_lens"] // 3).to(torch.int32)
        s["repetition"] = 1.0 + 0.5 * torch.rand(rows, generator=g, device="cuda")
        s["presence"] = torch.rand(rows, generator=g, device="cuda")
        s["frequency"] = 0.2 * torch.rand(rows, generator=g, device="cuda")
        n_bias = min(32, vocab)
        s["bias_ids"] = torch.rand(rows, vocab, generator=g, device="cuda").topk(n_bias, dim=1).indices.to(torch.int32)
        s["bias_values"] = 4.0 * torch.randn(rows, n_bias, generator=g, device="cuda")
        if case["mask"]:  # one bit for each token id
            s["allowed"] = torch.randint(-(1 << 31), 1 << 31, (rows, (vocab + 31) // 32), generator=g, device="cuda").to(torch.int32)
    return s


def _rotated(x, positions, rope):
    """Pairs (2i, 2i+1) of the first `rope` dims turned by position * 10000^(-2i/rope); angles in 64 bits, the rest in 32."""
    x = x.float()
    if rope == 0:
        return x
    i = torch.arange(0, rope, 2, device=x.device, dtype=torch.float64)
    angle = positions.double()[:, None] * torch.pow(10000.0, -i / rope)
    c, s = angle.cos().float()[:, None, :], angle.sin().float()[:, None, :]
    even, odd = x[..., 0:rope:2], x[..., 1:rope:2]
    turned = torch.stack([even * c - odd * s, even * s + odd * c], dim=-1).flatten(-2)
    return torch.cat([turned, x[..., rope:]], dim=-1)


def _append(s):
    pos = s["positions"].long()
    page = s["table"][s["seq"].long(), pos // s["page"]].long()
    kind = s["k_cache"].dtype
    s["k_cache"][page, pos % s["page"]] = _rotated(s["k"], pos, s["rope"]).to(kind)
    s["v_cache"][page, pos % s["page"]] = s["v"]
    return _rotated(s["q"], pos, s["rope"]).to(kind), s["k_cache"], s["v_cache"]


def _attend(s):
    n, heads, dim = s["q"].shape
    groups = heads // s["kv_heads"]
    k = s["k_cache"][s["table"].long()].flatten(1, 2).float()  # [sequence, key, head, dim]
    v = s["v_cache"][s["table"].long()].flatten(1, 2).float()
    q = s["q"].float().unflatten(1, (s["kv_heads"], groups))
    z = torch.matmul(q, k.permute(0, 2, 3, 1)) * (1.0 / math.sqrt(dim))  # [sequence, kv head, group, key]
    past = torch.arange(k.shape[1], device=k.device) >= s["lens"][:, None]
    z = z.masked_fill(past[:, None, None, :], -math.inf)
    m = z.amax(dim=-1, keepdim=True)
    p = torch.exp(z - m)
    total = p.sum(dim=-1, keepdim=True)
    o = torch.matmul(p, v.permute(0, 2, 1, 3)) / total
    return o.flatten(1, 2).to(s["q"].dtype), (m + torch.log(total)).flatten(1)


def _token(s):
    z = s["logits"].float()
    rows, vocab = z.shape
    ids = s["history_ids"].long()
    at = torch.arange(ids.shape[1], device=z.device)
    inside = at < s["history_lens"][:, None]
    made = inside & (at >= s["prompt_lens"][:, None])
    seen = torch.zeros_like(z).scatter_add_(1, ids, inside.float()) > 0
    count = torch.zeros_like(z).scatter_add_(1, ids, made.float())
    r = s["repetition"][:, None]
    z = torch.where(seen, torch.where(z > 0, z / r, z * r), z)
    z = z - s["frequency"][:, None] * count
    z = z - s["presence"][:, None] * (count > 0)
    z = z + torch.zeros_like(z).scatter_add_(1, s["bias_ids"].long(), s["bias_values"])
    if s["mask"]:
        bits = (s["allowed"][:, :, None] >> torch.arange(32, device=z.device)) & 1
        z = z.masked_fill(bits.flatten(1)[:, :vocab] == 0, -math.inf)
    m = z.amax(dim=1, keepdim=True)
    first = torch.where(z == m, torch.arange(vocab, device=z.device), vocab).amin(dim=1).to(torch.int32)
    return first, z, (m + torch.log(torch.exp(z - m).sum(dim=1, keepdim=True))).squeeze(1)


def run(s):
    if own:
        from persistent_gpt_step_gb300 import binding as B
        if s["op"] == "append":
            q = B.kv_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["positions"], seq=s["seq"], q=s["q"],
                            rope_dims=s["rope"])
            return q, s["k_cache"], s["v_cache"]
        if s["op"] == "attend":
            return B.decode_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"])
        return B.next_token(s["logits"], history=s["history_ids"], history_lens=s["history_lens"], prompt_lens=s["prompt_lens"],
                            repetition=s["repetition"], presence=s["presence"], frequency=s["frequency"],
                            bias_ids=s["bias_ids"], bias_values=s["bias_values"], allowed=s.get("allowed"))
    return {"append": _append, "attend": _attend, "token": _token}[s["op"]](s)


def work(case):
    size = 2 if case["type"] == "bf16" else 4
    if case["op"] == "append":
        row = case["dim"] * size
        turned = case["heads"] + case["kv_heads"]
        return {"bytes": case["tokens"] * ((2 * case["heads"] + 4 * case["kv_heads"]) * row + 12),
                "flops": case["tokens"] * turned * case["rope"] * 3}
    if case["op"] == "attend":
        keys = sum(_lens(case))
        pages = sum((n + case["page"] - 1) // case["page"] for n in _lens(case))
        return {"bytes": 2 * keys * case["kv_heads"] * case["dim"] * size + 2 * case["seqs"] * case["heads"] * case["dim"] * size
                + 4 * case["seqs"] * case["heads"] + 4 * (pages + case["seqs"]),
                "flops": 4 * keys * case["heads"] * case["dim"]}
    values = case["rows"] * case["vocab"]
    kept = sum(_spread(case["rows"], max(1, case["history"] // 2), case["history"]))
    return {"bytes": values * (size + 4) + (values // 8 if case["mask"] else 0) + 4 * kept + case["rows"] * (28 + 8 * min(32, case["vocab"])),
            "flops": 5 * values}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        pos, rope = s["positions"].long(), case["rope"]

        def turned(x):  # as complex numbers times e^(i angle)
            x = x.double()
            if rope == 0:
                return x
            rate = torch.tensor([10000.0 ** (-2.0 * i / rope) for i in range(rope // 2)], dtype=torch.float64, device="cuda")
            angle = pos[:, None].double() * rate[None, :]
            pairs = torch.view_as_complex(x[..., :rope].contiguous().unflatten(-1, (rope // 2, 2)))
            pairs = pairs * torch.polar(torch.ones_like(angle), angle)[:, None, :]
            return torch.cat([torch.view_as_real(pairs).reshape(*x.shape[:-1], rope), x[..., rope:]], dim=-1)

        flat = s["table"][s["seq"].long(), torch.div(pos, case["page"], rounding_mode="floor")].long() * case["page"] + pos % case["page"]
        k = s["k_cache"].double().flatten(0, 1).index_copy(0, flat, turned(s["k"]))
        v = s["v_cache"].double().flatten(0, 1).index_copy(0, flat, s["v"].double())
        return turned(s["q"]), k.view(s["k_cache"].shape), v.view(s["v_cache"].shape)
    if case["op"] == "attend":
        outs, lses = [], []
        groups = case["heads"] // case["kv_heads"]
        for b, n in enumerate(s["lens"].tolist()):
            at = torch.arange(n, device="cuda")
            page = s["table"][b, at // case["page"]].long()
            k = s["k_cache"][page, at % case["page"]].double().repeat_interleave(groups, dim=1)
            v = s["v_cache"][page, at % case["page"]].double().repeat_interleave(groups, dim=1)
            z = torch.einsum("hd,nhd->hn", s["q"][b].double(), k) / math.sqrt(case["dim"])
            lses.append(torch.logsumexp(z, dim=1))
            outs.append(torch.einsum("hn,nhd->hd", torch.softmax(z, dim=1), v))
        return torch.stack(outs), torch.stack(lses)
    z = s["logits"].double()
    for row in range(case["rows"]):
        n, first = int(s["history_lens"][row]), int(s["prompt_lens"][row])
        seen = torch.unique(s["history_ids"][row, :n].long())
        z[row, seen] = torch.where(z[row, seen] > 0, z[row, seen] / s["repetition"][row].double(),
                                   z[row, seen] * s["repetition"][row].double())
        made, count = torch.unique(s["history_ids"][row, first:n].long(), return_counts=True)
        z[row, made] -= s["frequency"][row].double() * count + s["presence"][row].double()
        z[row, s["bias_ids"][row].long()] += s["bias_values"][row].double()
        if case["mask"]:
            ids = torch.arange(case["vocab"], device="cuda")
            z[row, (s["allowed"][row, ids // 32].long() >> (ids % 32)) & 1 == 0] = -math.inf
    return None, z, torch.logsumexp(z, dim=1)
