"""Cases of the decode-step operators over a cache held in 8 bits, and of drawing a token: filling the scaled e4m3
cache, attention over it, and sampling with temperature, top-k, top-p and min-p from given random numbers.

``run`` computes an operator in elementary torch operations, or, where ``own`` is true, by the call that a program
makes of this package.  ``exact`` is the definition in float64."""

import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
E4M3 = torch.float8_e4m3fn


def listed():
    return [
        # one token of the 57.7M model's attention (8 heads of 64, rotary): the latency of a single-user decode step
        {"name": "append8_one", "op": "append", "tokens": 1, "seqs": 1, "before": 1000, "heads": 8, "kv_heads": 8, "dim": 64,
         "page": 16, "rope": 64, "type": "bf16"},
        # one decode step of 256 sequences with shared key heads
        {"name": "append8_step", "op": "append", "tokens": 256, "seqs": 256, "before": 1024, "heads": 32, "kv_heads": 8,
         "dim": 128, "page": 16, "rope": 128, "type": "bf16"},
        # a few prompts of the 162M model's heads in fp32, half of each head rotated, continued in pages begun before
        {"name": "append8_prompts_fp32", "op": "append", "tokens": 4095, "seqs": 5, "before": 45, "heads": 12, "kv_heads": 12,
         "dim": 64, "page": 32, "rope": 32, "type": "fp32"},
        # the largest: a full batch of prompts at once
        {"name": "append8_prompts", "op": "append", "tokens": 32768, "seqs": 24, "before": 0, "heads": 32, "kv_heads": 8,
         "dim": 128, "page": 64, "rope": 128, "type": "bf16"},
        # one sequence of the 162M model at its full context, queries of the serving partition's type
        {"name": "attend8_one_fp32", "op": "attend", "seqs": 1, "shortest": 513, "longest": 513, "heads": 12, "kv_heads": 12,
         "dim": 64, "page": 16, "type": "fp32"},
        # the 350M model's heads, sequences of every length up to its context
        {"name": "attend8_batch", "op": "attend", "seqs": 200, "shortest": 1, "longest": 1024, "heads": 16, "kv_heads": 16,
         "dim": 64, "page": 16, "type": "bf16"},
        # shared key heads, ragged lengths into the thousands
        {"name": "attend8_shared", "op": "attend", "seqs": 64, "shortest": 17, "longest": 8192, "heads": 32, "kv_heads": 8,
         "dim": 128, "page": 16, "type": "bf16"},
        # one very long sequence: all of the GPU on one row of the batch
        {"name": "attend8_long", "op": "attend", "seqs": 1, "shortest": 131071, "longest": 131071, "heads": 32, "kv_heads": 8,
         "dim": 128, "page": 64, "type": "bf16"},
        # one row of the 57.7M model's vocabulary, a chat program's usual settings
        {"name": "sample_one", "op": "sample", "rows": 1, "vocab": 12288, "filters": "all", "type": "bf16"},
        # a batch of the 162M model's logits, every request with settings of its own
        {"name": "sample_batch", "op": "sample", "rows": 64, "vocab": 50304, "filters": "mixed", "type": "fp32"},
        # a vocabulary of odd size (rows begin at any alignment), the nucleus alone
        {"name": "sample_odd", "op": "sample", "rows": 33, "vocab": 49999, "filters": "top_p", "type": "bf16"},
        # the largest: many rows of a large vocabulary from the whole distribution, as rollouts for training are drawn
        {"name": "sample_large", "op": "sample", "rows": 512, "vocab": 131072, "filters": "none", "type": "fp32"},
    ]


def _log_int(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "sample"])
    kind = rng.choice(["bf16", "bf16", "fp32"])
    if op == "sample":
        vocab = _log_int(rng, 256, 131072)
        rows = _log_int(rng, 1, min(512, (1 << 25) // vocab))
        return {"op": op, "rows": rows, "vocab": vocab, "filters": rng.choice(["none", "top_k", "top_p", "min_p", "all", "mixed"]),
                "type": kind}
    dim = rng.choice([32, 64, 64, 80, 96, 128, 128])
    kv_heads = rng.choice([1, 2, 4, 8, 12, 16])
    heads = kv_heads * rng.choice([1, 1, 2, 3, 4, 7, 8])
    page = rng.choice([8, 16, 24, 32, 64, 128])
    row = kv_heads * dim  # bytes of a key of all heads
    if op == "append":
        tokens = _log_int(rng, 1, min(32768, (1 << 28) // (4 * row + heads * dim * 2)))
        seqs = rng.choice([tokens, max(1, tokens // 100), 1]) if tokens <= 512 else _log_int(rng, 1, 32)
        return {"op": op, "tokens": tokens, "seqs": min(seqs, tokens), "before": _log_int(rng, 1, 1500), "heads": heads,
                "kv_heads": kv_heads, "dim": dim, "page": page, "rope": rng.choice([0, dim // 4, dim // 2, dim, dim]),
                "type": kind}
    seqs = _log_int(rng, 1, 256)
    most = max(2, min(131072, (1 << 28) // (2 * row * seqs)))
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


def _scale(top):
    """The scale of a block whose largest magnitude is `top`: the power of two that brings it to 128 up to 256."""
    exponent = torch.where(top > 0, torch.frexp(top).exponent - 1, torch.full_like(top, -119, dtype=torch.int32))
    return torch.ldexp(torch.ones_like(top), exponent.clamp(min=-119) - 7)


def _int32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _cache(case, lens, g):
    """Scaled key and value pages in a random order over a pool with some spare pages, and the table of each sequence's pages."""
    page, shape = case["page"], (case["kv_heads"], case["dim"])
    used = [(n + page - 1) // page for n in lens]
    n_pages = sum(used) + 3
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    seq = torch.repeat_interleave(torch.arange(len(lens), device="cuda"), torch.tensor(used, device="cuda"))
    at = torch.arange(sum(used), device="cuda") - (torch.tensor(used, device="cuda").cumsum(0) - torch.tensor(used, device="cuda"))[seq]
    table = torch.zeros(len(lens), max(used), dtype=torch.int32, device="cuda")
    table[seq, at] = order[:sum(used)]
    codes, scales = [], []
    for _ in range(2):
        x = torch.randn(n_pages, page, *shape, generator=g, device="cuda")
        s = _scale(x.abs().amax(dim=(1, 3)))
        codes.append((x / s[:, None, :, None]).to(E4M3))
        scales.append(s)
    return codes[0], codes[1], scales[0], scales[1], table


def prepare(case, seed):
    g = _generator(seed)
    kind = TYPES[case["type"]]
    s = dict(case)
    if case["op"] == "append":
        counts = _counts(case)
        before = torch.randint(0, case["before"] + 1, (case["seqs"],), generator=g, device="cuda").tolist()
        s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["table"] = _cache(case, [case["before"] + n for n in counts], g)
        # one projection's output, q | k | v side by side in a token's row
        width = (case["heads"] + 2 * case["kv_heads"]) * case["dim"]
        qkv = torch.randn(case["tokens"], width, generator=g, device="cuda", dtype=kind)
        q, k, v = qkv.split([case["heads"] * case["dim"]] + 2 * [case["kv_heads"] * case["dim"]], dim=1)
        s["q"], s["k"], s["v"] = (x.unflatten(1, (-1, case["dim"])) for x in (q, k, v))
        s["before_lens"] = _int32(before)
        s["starts"] = _int32([sum(counts[:i]) for i in range(len(counts) + 1)]) if case["tokens"] > case["seqs"] else None
    elif case["op"] == "attend":
        lens = _lens(case)
        order = torch.randperm(len(lens), generator=g, device="cuda").tolist()
        lens = [lens[i] for i in order]
        s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["table"] = _cache(case, lens, g)
        s["lens"] = _int32(lens)
        s["q"] = torch.randn(case["seqs"], case["heads"], case["dim"], generator=g, device="cuda", dtype=kind)
    else:
        rows, vocab = case["rows"], case["vocab"]
        # a few likely tokens and a long tail, weights falling off about as a power of the rank
        tail = torch.rand(rows, vocab, generator=g, device="cuda").clamp_(min=1e-9).log_()
        s["logits"] = (2.5 * torch.randn(rows, vocab, generator=g, device="cuda") - 1.5 * tail).to(kind)
        s["uniform"] = torch.rand(rows, generator=g, device="cuda")
        s["temperature"] = 0.5 + 0.8 * torch.rand(rows, generator=g, device="cuda")
        top_k = torch.randint(1, max(2, min(200, vocab)), (rows,), generator=g, device="cuda").to(torch.int32)
        top_p = 0.7 + 0.29 * torch.rand(rows, generator=g, device="cuda")
        min_p = 0.01 + 0.1 * torch.rand(rows, generator=g, device="cuda")
        on = {"none": (), "all": ("top_k", "top_p", "min_p"), "mixed": ("top_k", "top_p", "min_p")}.get(case["filters"], (case["filters"],))
        if case["filters"] == "mixed":  # each setting off (0, 1, 0) for half of the rows, in every combination
            row = torch.arange(rows, device="cuda")
            top_k = torch.where(row % 2 == 0, top_k, 0)
            top_p = torch.where(row // 2 % 2 == 0, top_p, 1.0)
            min_p = torch.where(row // 4 % 2 == 0, min_p, 0.0)
        s["top_k"], s["top_p"], s["min_p"] = (x if name in on else None for name, x in (("top_k", top_k), ("top_p", top_p), ("min_p", min_p)))
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


def _append_one_side(cache, scale, x, turned, s, first_page, first_slot, page, slot):
    """x's rows, `turned` already, into the pages: a page begun in this call has the scale of its new rows, one begun
    before the larger of that and its own, and the codes before the new rows are brought to it."""
    codes = cache.view(torch.uint8)
    top = torch.zeros_like(scale).scatter_reduce_(0, page[:, None].expand(-1, scale.shape[1]), x.abs().amax(dim=2).float(), "amax")
    begun = torch.zeros(scale.shape[0], dtype=torch.bool, device=x.device)
    begun[first_page] = first_slot > 0
    old = scale[first_page]
    new = torch.where(begun[:, None], torch.maximum(scale, _scale(top)), _scale(top))
    scale[page] = new[page]
    kept = codes[first_page]  # [sequence, slot, head, dim]
    brought = (kept.view(E4M3).float() * (old / scale[first_page])[:, None, :, None]).to(E4M3).view(torch.uint8)
    before = torch.arange(kept.shape[1], device=x.device) < first_slot[:, None]
    codes[first_page] = torch.where(before[:, :, None, None], brought, kept)
    codes[page, slot] = (turned / scale[page][:, :, None]).to(E4M3).view(torch.uint8)


def _append(s):
    before = s["before_lens"].long()
    row = torch.arange(s["tokens"], device=before.device)
    seq = row if s["starts"] is None else torch.searchsorted(s["starts"][1:].long(), row, right=True)
    pos = before[seq] + (0 if s["starts"] is None else row - s["starts"][seq].long())
    size = s["page"]
    page = s["table"][seq, pos // size].long()
    first_page = s["table"][torch.arange(s["seqs"], device=before.device), before // size].long()
    _append_one_side(s["k_cache"], s["k_scale"], s["k"], _rotated(s["k"], pos, s["rope"]), s, first_page, before % size, page, pos % size)
    _append_one_side(s["v_cache"], s["v_scale"], s["v"], s["v"].float(), s, first_page, before % size, page, pos % size)
    return _rotated(s["q"], pos, s["rope"]).to(s["q"].dtype), s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]


def _attend(s):
    n, heads, dim = s["q"].shape
    groups = heads // s["kv_heads"]
    pages = s["table"].long()

    def values(cache, scale):  # [sequence, key, head, dim]
        x = cache.view(torch.uint8)[pages].view(E4M3).float() * scale[pages][:, :, None, :, None]
        return x.flatten(1, 2)

    k, v = values(s["k_cache"], s["k_scale"]), values(s["v_cache"], s["v_scale"])
    q = s["q"].float().unflatten(1, (s["kv_heads"], groups))
    z = torch.matmul(q, k.permute(0, 2, 3, 1)) * (1.0 / math.sqrt(dim))  # [sequence, kv head, group, key]
    past = torch.arange(k.shape[1], device=k.device) >= s["lens"][:, None]
    z = z.masked_fill(past[:, None, None, :], -math.inf)
    m = z.amax(dim=-1, keepdim=True)
    p = torch.exp(z - m)
    total = p.sum(dim=-1, keepdim=True)
    o = torch.matmul(p, v.permute(0, 2, 1, 3)) / total
    return o.flatten(1, 2).to(s["q"].dtype), (m + torch.log(total)).flatten(1)


def _sample(s):
    z = s["logits"].float()
    rows, vocab = z.shape
    z, order = z.sort(dim=1, descending=True, stable=True)  # equal logits: the lowest id first
    w = torch.exp((z.double() - z[:, :1].double()) / s["temperature"].double()[:, None])
    rank = torch.arange(vocab, device=z.device)
    keep = torch.ones_like(z, dtype=torch.bool)
    if s["top_k"] is not None:
        keep &= (rank < s["top_k"][:, None]) | (s["top_k"][:, None] < 1)
    if s["top_p"] is not None:  # a token stays while those before it do not hold top_p of what top-k left
        sums = (w * keep).cumsum(dim=1)
        keep &= (sums - w * keep < s["top_p"].double()[:, None] * sums[:, -1:]) | (s["top_p"][:, None] >= 1)
    if s["min_p"] is not None:
        keep &= w >= s["min_p"].double()[:, None]
    keep[:, 0] = True
    w = torch.zeros_like(w).scatter_(1, order, w * keep)  # by id again
    sums = w.cumsum(dim=1)
    token = (sums > s["uniform"].double()[:, None] * sums[:, -1:]).to(torch.int8).argmax(dim=1, keepdim=True)
    logprob = torch.log(w.gather(1, token) / sums[:, -1:])
    return token.squeeze(1).to(torch.int32), logprob.squeeze(1).float(), keep.sum(dim=1).to(torch.int32)


def run(s):
    if own:
        from persistent_gpt_step_gb300 import binding as B
        if s["op"] == "append":
            q = B.kv_append_fp8(s["k"], s["v"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["table"], s["before_lens"],
                                starts=s["starts"], q=s["q"], rope_dims=s["rope"])
            return q, s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]
        if s["op"] == "attend":
            return B.decode_attention_fp8(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["table"], s["lens"])
        return B.sample_token(s["logits"], s["uniform"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
                              min_p=s["min_p"])
    return {"append": _append, "attend": _attend, "sample": _sample}[s["op"]](s)


def work(case):
    size = 2 if case["type"] == "bf16" else 4
    if case["op"] == "append":
        # q read and written, k and v read and written as codes; the positions, the pages' ids and scales
        pages = sum((n + case["page"] - 1) // case["page"] for n in _counts(case))
        values = case["tokens"] * case["dim"]
        return {"bytes": values * (2 * size * case["heads"] + 2 * (size + 1) * case["kv_heads"]) + 8 * case["seqs"]
                + pages * (4 + 8 * case["kv_heads"]),
                "flops": values * (2 * case["kv_heads"] + (case["heads"] + case["kv_heads"]) * 3 * case["rope"] / case["dim"])}
    if case["op"] == "attend":
        keys = sum(_lens(case))
        pages = sum((n + case["page"] - 1) // case["page"] for n in _lens(case))
        return {"bytes": 2 * keys * case["kv_heads"] * case["dim"] + 2 * case["seqs"] * case["heads"] * case["dim"] * size
                + 4 * case["seqs"] * case["heads"] + pages * (4 + 8 * case["kv_heads"]) + 4 * case["seqs"],
                "flops": 4 * keys * case["heads"] * case["dim"]}
    values = case["rows"] * case["vocab"]
    return {"bytes": values * size + case["rows"] * 32, "flops": 5 * values}


def _nearest_e4m3(x):
    """x (float64, below 448) to the nearest value of 4 significant bits, steps of 2^-9 at least, ties to even."""
    exponent = torch.frexp(x).exponent.clamp(min=-5)
    step = torch.ldexp(torch.ones_like(x), exponent - 4)
    return torch.round(x / step) * step


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        counts, before, size, rope = _counts(case), s["before_lens"].tolist(), case["page"], case["rope"]
        pos = torch.cat([torch.arange(b, b + n, device="cuda") for b, n in zip(before, counts)])

        def turned(x):  # as complex numbers times e^(i angle)
            x = x.double()
            if rope == 0:
                return x
            rate = torch.tensor([10000.0 ** (-2.0 * i / rope) for i in range(rope // 2)], dtype=torch.float64, device="cuda")
            angle = pos[:, None].double() * rate[None, :]
            pairs = torch.view_as_complex(x[..., :rope].contiguous().unflatten(-1, (rope // 2, 2)))
            pairs = pairs * torch.polar(torch.ones_like(angle), angle)[:, None, :]
            return torch.cat([torch.view_as_real(pairs).reshape(*x.shape[:-1], rope), x[..., rope:]], dim=-1)

        if sum((n + size - 1) // size + 1 for n in counts) > 4000:
            return None
        table = s["table"].tolist()
        sides = []
        for raw, values, codes, scales in ((s["k"], turned(s["k"]), s["k_cache"], s["k_scale"]), (s["v"], s["v"].double(), s["v_cache"], s["v_scale"])):
            codes, scales, row = codes.double(), scales.double(), 0
            for i, (b, n) in enumerate(zip(before, counts)):
                end = b + n
                while b < end:
                    page, slot = table[i][b // size], b % size
                    many = min(size - slot, end - b)
                    top = raw[row:row + many].double().abs().amax(dim=(0, 2))
                    scale = torch.exp2(torch.floor(torch.log2(top)) - 7)
                    if slot > 0:
                        scale = torch.maximum(scale, scales[page])
                        codes[page, :slot] = _nearest_e4m3(codes[page, :slot] * (scales[page] / scale)[:, None])
                    codes[page, slot:slot + many] = _nearest_e4m3(values[row:row + many] / scale[:, None])
                    scales[page] = scale
                    row, b = row + many, b + many
            sides.append((codes, scales))
        return turned(s["q"]), sides[0][0], sides[1][0], sides[0][1], sides[1][1]
    if case["op"] == "attend":
        outs, lses = [], []
        groups = case["heads"] // case["kv_heads"]
        for b, n in enumerate(s["lens"].tolist()):
            pages = s["table"][b, :(n + case["page"] - 1) // case["page"]].long()

            def values(cache, scale):
                x = torch.cat([cache[p][None] for p in pages.tolist()]) if len(pages) < 64 else cache.view(torch.uint8)[pages].view(E4M3)
                return (x.double() * scale[pages].double()[:, None, :, None]).flatten(0, 1)[:n].repeat_interleave(groups, dim=1)

            z = torch.einsum("hd,nhd->hn", s["q"][b].double(), values(s["k_cache"], s["k_scale"])) / math.sqrt(case["dim"])
            lses.append(torch.logsumexp(z, dim=1))
            outs.append(torch.einsum("hn,nhd->hd", torch.softmax(z, dim=1), values(s["v_cache"], s["v_scale"])))
        return torch.stack(outs), torch.stack(lses)
    logprobs = []
    for row in range(case["rows"]):
        z = s["logits"][row].double() / s["temperature"][row].double()
        value, ids = torch.sort(z, descending=True, stable=True)
        p = torch.softmax(value, dim=0)
        n = case["vocab"]
        if s["top_k"] is not None and int(s["top_k"][row]) > 0:
            n = min(n, int(s["top_k"][row]))
        if s["min_p"] is not None:
            n = min(n, max(1, int((p >= s["min_p"][row].double() * p[0]).sum())))
        if s["top_p"] is not None and float(s["top_p"][row]) < 1:
            most = case["vocab"] if s["top_k"] is None or int(s["top_k"][row]) < 1 else int(s["top_k"][row])
            sums = p[:most].cumsum(0)
            n = min(n, 1 + int((sums < s["top_p"][row].double() * sums[-1]).sum()))
        kept = ids[:n].sort().values
        share = torch.softmax(z[kept], dim=0)
        at = min(int((share.cumsum(0) <= s["uniform"][row].double()).sum()), n - 1)
        logprobs.append(torch.log(share[at]))
    return None, torch.stack(logprobs), None
