"""The paged cache's operators: what is timed, and their plain forms.

A pool holds, for each layer, pages of `page` tokens; sequences own lists of
pages and share them after a fork. The arrays of a pool (L layers, N pages, H
key/value heads, S sequences of at most W pages, C = W * page):

    K, V    [L, N, H, page, d]   bf16, or E4M3 codes with scales [L, N, H, page]
    pos     [L, N, H, page]      position of the token that a slot holds
    score   [L, S, H, C]         accumulated attention of a sequence's slots
    table   [L, S, W]            pages of a sequence, -1 behind the last
    meta    [L, S, 2]            length, next position
    ref     [L, N]               sequences that hold a page

Four operators: writing tokens into sequences, forking (and freeing) sequences,
compacting them to their heavy hitters and recent tokens, and single-token
attention of a batch over a shared prefix and each sequence's own tokens.
"""
import math

import torch

own = False

BF16 = torch.bfloat16
E4M3 = torch.float8_e4m3fn


# ---------------------------------------------------------------------- cases
def listed():
    return [
        # the first tokens of one small sequence: latency alone
        dict(name="attend_tiny", op="attend", kv="bf16", batch=1, q_heads=4, heads=4, d=64, page=16,
             prefix=0, shortest=33, longest=33),
        # an OPT-6.7B-shaped layer: a system prompt once for all, own tokens up to the 20 % budget
        dict(name="attend_opt-6.7b", op="attend", kv="bf16", batch=8, q_heads=32, heads=32, d=128, page=64,
             prefix=2048, shortest=1, longest=460),
        # a LLaMA-7B-shaped layer over a document of 32768 tokens that 16 questions share
        dict(name="attend_llama-7b-32k", op="attend", kv="bf16", batch=16, q_heads=32, heads=32, d=128, page=128,
             prefix=32768, shortest=64, longest=1024),
        # a large batch: nearly all the bytes are the sequences' own
        dict(name="attend_batch-256", op="attend", kv="bf16", batch=256, q_heads=32, heads=32, d=128, page=32,
             prefix=1024, shortest=300, longest=410),
        # grouped heads and an E4M3 cache, 256 query rows a head over a ragged prefix
        dict(name="attend_grouped_fp8", op="attend", kv="fp8", batch=64, q_heads=32, heads=8, d=128, page=32,
             prefix=8197, shortest=0, longest=1000),
        # one short prompt down to 16 + 16 tokens
        dict(name="compact_tiny", op="compact", kv="bf16", n=1, heads=4, d=64, page=16, shortest=128, longest=128,
             h=16, r=16),
        # four prompts of 32768 tokens down to 2048 + 2048
        dict(name="compact_llama-7b-32k", op="compact", kv="bf16", n=4, heads=32, d=128, page=64, shortest=32768,
             longest=32768, h=2048, r=2048),
        # ragged prompts, some already inside the budget, of an E4M3 cache
        dict(name="compact_opt-6.7b_fp8", op="compact", kv="fp8", n=8, heads=32, d=128, page=32, shortest=301,
             longest=2048, h=230, r=230),
        # a step of a beam search in one layer: half the beams go, the others are forked
        dict(name="fork_beams", op="fork", kv="bf16", layers=1, src=4, dst=4, heads=32, d=128, page=64, shortest=201,
             longest=300),
        # eight prompts forked to 56 samples in all layers of an OPT-30B-shaped stack
        dict(name="fork_opt-30b-stack", op="fork", kv="bf16", layers=48, src=8, dst=56, heads=56, d=128, page=16,
             shortest=198, longest=206),
        # the first few tokens of many sequences, E4M3
        dict(name="write_few_fp8", op="write", kv="fp8", n=64, heads=8, d=128, page=16, shortest=0, longest=5),
        # eight prompts of 2048 tokens with their scores
        dict(name="write_opt-6.7b", op="write", kv="bf16", n=8, heads=32, d=128, page=64, shortest=1500,
             longest=2048),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "compact", "fork", "write"])
    kv = rng.choice(["bf16", "bf16", "fp8"])
    d = rng.choice([64, 128, 128])
    page = rng.choice([16, 32, 64, 128])
    if op == "attend":
        group = rng.choice([1, 1, 2, 3, 4, 5, 8])
        heads = rng.choice([1, 2, 4, 7, 8, 16, 32])
        batch = _log(rng, 1, 256)
        prefix = rng.choice([0, 1, 1]) * _log(rng, 1, 32768)
        longest = _log(rng, 1, 2048)
        # no more bytes, rows or plain-form work than the largest listed cases
        while heads * (prefix + batch * longest) > 3_000_000 or batch * group * heads * prefix > 16_000_000:
            prefix, longest, batch = prefix * 2 // 3, max(1, longest * 2 // 3), max(1, batch * 3 // 4)
        shortest = rng.choice([0, 1, longest // 2, longest])
        if not prefix:
            shortest = max(1, shortest)
        return dict(op=op, kv=kv, batch=batch, q_heads=heads * group, heads=heads, d=d, page=page, prefix=prefix,
                    shortest=min(shortest, longest), longest=longest)
    heads = _log(rng, 1, 32)
    if op == "compact":
        n = _log(rng, 1, 16)
        h, r = _log(rng, 1, 2048) - 1, _log(rng, 1, 2048)
        longest = min(32768, h + r + _log(rng, 1, 30000))
        while n * heads * longest > 4_000_000:
            n, heads = max(1, n // 2), max(1, heads * 3 // 4)
        return dict(op=op, kv=kv, n=n, heads=heads, d=d, page=page, shortest=max(1, longest // rng.choice([1, 1, 2, 5])),
                    longest=longest, h=h, r=r)
    if op == "fork":
        layers, src = _log(rng, 1, 48), _log(rng, 1, 8)
        longest = _log(rng, 1, 2000)
        while layers * heads * (src + 1) * longest > 4_000_000:
            layers, longest = max(1, layers * 2 // 3), max(1, longest * 2 // 3)
        return dict(op=op, kv=kv, layers=layers, src=src, dst=_log(rng, 1, 56), heads=heads, d=d, page=page,
                    shortest=max(1, longest // 2), longest=longest)
    n, longest = _log(rng, 1, 64), _log(rng, 1, 2048)
    while n * heads * longest > 500_000:
        n, longest = max(1, n * 2 // 3), max(1, longest * 2 // 3)
    return dict(op=op, kv=kv, n=n, heads=heads, d=d, page=page, shortest=rng.choice([0, longest // 2, longest]),
                longest=longest)


def _lengths(case, n):
    """n lengths spread over [shortest, longest], the longest among them; the case alone decides them."""
    lo, hi = case["shortest"], case["longest"]
    return [hi if i == 0 else lo + (i * 2654435761 >> 7) % (hi - lo + 1) for i in range(n)]


def _pages(tokens, page):
    return -(-tokens // page)


# ------------------------------------------------------------------ the inputs
def _quantise(x):
    """E4M3 codes (as float8) and one scale a vector: scale = amax / 448, code = E4M3(x * (448 / amax))."""
    x = x.float()
    amax = x.abs().amax(-1, keepdim=True)
    top = torch.full_like(amax, 448.0)  # tensors on both sides: a scalar's reciprocal would round once more
    inv = torch.where(amax > 0, top / amax, 0.0)
    return (x * inv).clamp(-448, 448).to(E4M3), (amax / top).squeeze(-1)


def _pool(case, gen, layers, lengths, room, spare, width):
    """The arrays of a pool whose first sequences have `lengths`, with `room` more empty sequences and `spare` free pages.

    A few tokens of every page attract most of the attention, along a direction that the queries share; the scores
    follow a power law. The pages of a sequence lie anywhere in the pool."""
    dev, heads, d, page = "cuda", case["heads"], case["d"], case["page"]
    used = [_pages(t, page) for t in lengths]
    n, s = sum(used) + spare, len(lengths) + room
    shape = (layers, n, heads, page)
    direction = torch.randn(heads, 1, d, generator=gen, device=dev)
    direction = direction / direction.norm(dim=-1, keepdim=True)
    arrays = {}
    for name in "KV":
        x = torch.empty(*shape, d, dtype=BF16, device=dev)
        for layer in range(layers):  # a layer at a time, to bound the memory of the random numbers
            x[layer] = torch.randn(*shape[1:], d, generator=gen, device=dev, dtype=BF16)
            if name == "K":
                rank = torch.rand(*shape[1:], 1, generator=gen, device=dev) * 4096 + 1
                x[layer] += (8 * rank.pow(-0.8) * direction).to(BF16)
        if case["kv"] == "fp8":
            both = [_quantise(x[layer]) for layer in range(layers)]
            arrays[name] = torch.stack([b[0].view(torch.uint8) for b in both])
            arrays[name.lower() + "scale"] = torch.stack([b[1] for b in both])
        else:
            arrays[name] = x
    table = torch.full((layers, s, width), -1, dtype=torch.int32)
    meta = torch.zeros(layers, s, 2, dtype=torch.int32)
    order = torch.randperm(n, generator=torch.Generator().manual_seed(int(gen.initial_seed()) + 1)).int()
    at = 0
    for i, t in enumerate(lengths):
        table[:, i, :used[i]] = order[at:at + used[i]]
        meta[:, i] = torch.tensor([t, t + 3 * i], dtype=torch.int32)  # some tokens were dropped before
        at += used[i]
    ref = torch.zeros(layers, n, dtype=torch.int32)
    ref[:, order[:at].long()] = 1
    arrays["pos"] = torch.randint(0, 1 << 20, shape, generator=gen, device=dev, dtype=torch.int32)
    u = torch.rand(layers, s, heads, width * page, generator=gen, device=dev)
    arrays["score"] = 0.02 / (u + 1e-3)
    # many tokens of equal score: a few values only, in a quarter of the slots
    arrays["score"] = torch.where(u < 0.25, (arrays["score"] * 2).round() / 2, arrays["score"])
    arrays["table"], arrays["meta"], arrays["ref"] = table.to(dev), meta.to(dev), ref.to(dev)
    return arrays, direction


def _ints(values):
    return torch.tensor(list(values), dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    op, heads, d, page = case["op"], case["heads"], case["d"], case["page"]
    state = {"case": case, "page": page}
    layers = case.get("layers", 1)
    if op == "attend":
        lengths = _lengths(case, case["batch"])
        prefix = [case["prefix"]] if case["prefix"] else []
        width = max(_pages(t, page) for t in lengths + prefix)
        arrays, direction = _pool(case, gen, 1, lengths + prefix, 0, 2, width)
        q = torch.randn(case["batch"], case["q_heads"], d, generator=gen, device="cuda")
        q += 2 * direction.repeat_interleave(case["q_heads"] // heads, 0).squeeze(1)
        state |= {"q": q.to(BF16), "seqs": _ints(range(case["batch"])), "prefix": len(lengths) if prefix else -1,
                  "reach": max(_pages(t, page) for t in lengths)}
    elif op == "compact":
        # the sequences are kept as they are; forks of them are compacted
        lengths = _lengths(case, case["n"])
        width = max(_pages(t, page) for t in lengths)
        k = case["h"] + case["r"]
        spare = sum(1 + _pages(min(t, k), page) for t in lengths)
        arrays, _ = _pool(case, gen, 1, lengths, case["n"], spare, width)
        state |= {"src": _ints(range(case["n"])), "dst": _ints(range(case["n"], 2 * case["n"]))}
    elif op == "fork":
        # the sequences that are dropped have a page of their own each
        lengths = _lengths(case, case["src"]) + [min(page, case["longest"])] * case["dst"]
        width = max(_pages(t, page) for t in lengths) + 1
        arrays, _ = _pool(case, gen, layers, lengths, 0, 2, width)
        state |= {"src": _ints((i * 5) % case["src"] for i in range(case["dst"])),
                  "dst": _ints(range(case["src"], case["src"] + case["dst"]))}
    else:
        lengths = _lengths(case, case["n"])
        width = max(1, max(_pages(t, page) for t in lengths))
        arrays, direction = _pool(case, gen, 1, [1], case["n"], sum(_pages(t, page) for t in lengths) + 2, width)
        tokens = torch.randn(2, case["n"], heads, case["longest"], d, generator=gen, device="cuda").to(BF16)
        state |= {"new_K": tokens[0].contiguous(), "new_V": tokens[1].contiguous(),
                  "new_score": torch.rand(case["n"], heads, case["longest"], generator=gen, device="cuda"),
                  "lens": _ints(lengths), "seqs": _ints(range(1, case["n"] + 1))}
    state["pool"] = arrays
    if own:
        import h2o_heavy_hitter_gb300 as h2o

        state["handle"] = h2o.h2o_pool_create(layers, arrays["ref"].shape[1], page, heads, d, arrays["meta"].shape[1],
                                              arrays["table"].shape[2], kv=case["kv"])
        view = h2o.h2o_pool_view(state["handle"])
        for name in arrays:
            view[name].copy_(arrays[name])
        state["pool"] = view
    return state


# --------------------------------------------------------------- the operators
def run(state):
    op, pool = state["case"]["op"], state["pool"]
    if own:
        import h2o_heavy_hitter_gb300 as h2o

        handle = state["handle"]
    if op == "attend":
        if own:
            out, lse = h2o.h2o_pool_attend(handle, 0, state["seqs"], state["q"], prefix=state["prefix"])
        else:
            out, lse = _attend(state)
        return {"out": out, "lse": lse, "score": pool["score"]}
    if op == "compact":
        if own:
            h2o.h2o_pool_free(handle, 0, state["dst"])
            h2o.h2o_pool_fork(handle, 0, state["src"], state["dst"])
            h2o.h2o_pool_compact(handle, 0, state["dst"], state["case"]["h"], state["case"]["r"])
        else:
            _free(pool, state["dst"])
            _fork(pool, state["src"], state["dst"], state["page"])
            _compact(pool, state["dst"], state["case"]["h"], state["case"]["r"], state["page"])
    elif op == "fork":
        if own:
            h2o.h2o_pool_free(handle, -1, state["dst"])
            h2o.h2o_pool_fork(handle, -1, state["src"], state["dst"])
        else:
            _free(pool, state["dst"])
            _fork(pool, state["src"], state["dst"], state["page"])
    else:
        if own:
            h2o.h2o_pool_free(handle, 0, state["seqs"])
            h2o.h2o_pool_write(handle, 0, state["seqs"], state["new_K"], state["new_V"], lens=state["lens"],
                               score=state["new_score"])
        else:
            _free(pool, state["seqs"])
            _write(state)
    return _values(pool)


def _values(pool):
    """A pool's arrays, codes as the values that they stand for before their scale."""
    return {k: v.view(E4M3) if v.dtype == torch.uint8 else v for k, v in pool.items()}


def _stored(pool, name, layer, pages):
    """The tokens of `pages` [..., n] in 32 bits, as [..., n, heads, page, d]."""
    x = pool[name][layer][pages]
    if x.dtype == torch.uint8:
        return x.view(E4M3).float() * pool[name.lower() + "scale"][layer][pages].unsqueeze(-1)
    return x.float()


def _attend(state):
    pool, page, q = state["pool"], state["page"], state["q"].float()
    batch, q_heads, d = q.shape
    seqs, prefix, reach = state["seqs"].long(), state["prefix"], state["reach"]
    heads = pool["score"].shape[2]
    q = q.view(batch, heads, q_heads // heads, d) / math.sqrt(d)
    # each sequence's own tokens
    pages = pool["table"][0][seqs, :reach].long().clamp(min=0)
    own_len = pool["meta"][0][seqs, 0]
    keep = torch.arange(reach * page, device=q.device) < own_len[:, None]
    both = [_stored(pool, n, 0, pages).transpose(1, 2).reshape(batch, heads, reach * page, d) for n in "KV"]
    k, v = both[0], torch.where(keep[:, None, :, None], both[1], 0)
    s = torch.where(keep[:, None, None], q @ k.transpose(2, 3), -math.inf)
    if prefix >= 0:
        at = pool["table"][0][prefix].long().clamp(min=0)
        stays = torch.arange(at.numel() * page, device=q.device) < pool["meta"][0][prefix, 0]
        pk, pv = (_stored(pool, n, 0, at).transpose(0, 1).reshape(heads, -1, d) for n in "KV")
        rows = q.transpose(0, 1).reshape(heads, -1, d)
        ps = torch.where(stays, rows @ pk.transpose(1, 2), -math.inf)
        pv = torch.where(stays[:, None], pv, 0)
        ps = ps.view(heads, batch, -1, ps.shape[2]).transpose(0, 1)
        top = torch.maximum(s.amax(-1, keepdim=True), ps.amax(-1, keepdim=True))
        e, pe = (s - top).exp(), (ps - top).exp()
        total = e.sum(-1, keepdim=True) + pe.sum(-1, keepdim=True)
        p, pp = e / total, pe / total
        flat = pp.transpose(0, 1).reshape(heads, -1, pp.shape[3])
        more = (flat @ pv).view(heads, batch, -1, d).transpose(0, 1)
        out = p @ v + more
        pool["score"][0][prefix] += flat.sum(1)
    else:
        top = s.amax(-1, keepdim=True)
        e = (s - top).exp()
        total = e.sum(-1, keepdim=True)
        p = e / total
        out = p @ v
    pool["score"][0][:, :, :reach * page].index_add_(0, seqs, p.sum(2))
    lse = (top + total.log()).view(batch, q_heads)
    return out.reshape(batch, q_heads, d).to(BF16), lse


def _free(pool, seqs):
    seqs = seqs.long()
    held = pool["table"][:, seqs].flatten(1).long()
    pool["ref"].scatter_add_(1, held.clamp(min=0), -(held >= 0).int())
    pool["table"][:, seqs] = -1
    pool["meta"][:, seqs] = 0


def _fresh(pool, need):
    """Free pages, the lowest first, for each entry of `need` [L, n] in its turn: [L, n, W]; what is behind an entry's need is not its own."""
    free = torch.argsort((pool["ref"] != 0).int(), dim=1, stable=True)
    width = pool["table"].shape[2]
    rank = (need.cumsum(1) - need).unsqueeze(-1) + torch.arange(width, device=need.device)
    return free.gather(1, rank.clamp(max=free.shape[1] - 1).flatten(1)).view(rank.shape)


def _fork(pool, src, dst, page):
    src, dst = src.long(), dst.long()
    layers, _, width = pool["table"].shape
    held, length = pool["table"][:, src].long(), pool["meta"][:, src, 0].long()
    whole, rest = (length // page).unsqueeze(-1), length % page
    j = torch.arange(width, device=src.device)
    fresh = _fresh(pool, (rest > 0).long())[:, :, :1]
    table = torch.where(j < whole, held, torch.where((j == whole) & (rest > 0).unsqueeze(-1), fresh, -1))
    shared = (j < whole).flatten(1)
    pool["ref"].scatter_add_(1, held.clamp(min=0).flatten(1), shared.int())
    layer, i = torch.nonzero(rest > 0, as_tuple=True)
    to = fresh[layer, i, 0]
    pool["ref"][layer, to] = 1
    at = held[layer, i, length[layer, i] // page]
    live = torch.arange(page, device=src.device) < rest[layer, i].unsqueeze(-1)
    for name in ("K", "V", "kscale", "vscale", "pos"):
        if name in pool:
            x = pool[name]
            mask = live.view(live.shape[0], 1, page, *[1] * (x.dim() - 4))
            x[layer, to] = torch.where(mask, x[layer, at], x[layer, to])
    behind = torch.arange(width * page, device=src.device) >= length[:, :, None, None]
    pool["score"][:, dst] = torch.where(behind, pool["score"][:, dst], pool["score"][:, src])
    pool["table"][:, dst] = table.int()
    pool["meta"][:, dst] = pool["meta"][:, src]


def _compact(pool, seqs, h, r, page):
    k, width = h + r, pool["table"].shape[2]
    seqs = seqs.long()
    seqs = seqs[pool["meta"][0][seqs, 0] > k]
    length = pool["meta"][0][seqs, 0].long()
    c = torch.arange(width * page, device=seqs.device)
    key = torch.where(c < length[:, None, None], pool["score"][0][seqs], -1.0)
    key = torch.where((c >= (length - r)[:, None, None]) & (c < length[:, None, None]), math.inf, key)
    # descending, the later of equal ones first
    order = torch.argsort(key.flip(-1), dim=-1, descending=True, stable=True)[..., :k]
    kept = (c.numel() - 1 - order).sort(-1).values
    held = pool["table"][0][seqs].long()
    heads = torch.arange(kept.shape[1], device=seqs.device)[None, :, None]
    at = held.unsqueeze(1).expand(-1, kept.shape[1], -1).gather(2, kept // page)
    need = torch.full_like(length, -(-k // page))
    fresh = _fresh(pool, need[None])[0]
    mine = torch.arange(width, device=seqs.device) < need[:, None]
    j = torch.arange(k, device=seqs.device)
    to = fresh[:, None, :].expand(-1, kept.shape[1], -1)[..., j // page]
    for name in ("K", "V", "kscale", "vscale", "pos"):
        if name in pool:
            x = pool[name][0]
            x[to, heads, j % page] = x[at, heads, kept % page]
    pool["score"][0][seqs, :, :k] = pool["score"][0][seqs].gather(2, kept)
    pool["ref"][0].scatter_add_(0, held.clamp(min=0).flatten(), -(held >= 0).int().flatten())
    pool["ref"][0][fresh[mine]] = 1
    pool["table"][0][seqs] = torch.where(mine, fresh, -1).int()
    pool["meta"][0][seqs, 0] = k


def _write(state):
    pool, page = state["pool"], state["page"]
    seqs, lens = state["seqs"].long(), state["lens"].long()
    begin, first = pool["meta"][0][seqs].long().unbind(1)
    width, longest = pool["table"].shape[2], state["new_K"].shape[2]
    p0, p1 = -(-begin // page), -(-(begin + lens) // page)
    j = torch.arange(width, device=seqs.device)
    fresh = _fresh(pool, (p1 - p0)[None])[0]
    fresh = fresh.gather(1, (j - p0[:, None]).clamp(min=0))
    new = (j >= p0[:, None]) & (j < p1[:, None])
    pool["table"][0][seqs] = torch.where(new, fresh, pool["table"][0][seqs].long()).int()
    pool["ref"][0][fresh[new]] = 1
    i, t = torch.nonzero(torch.arange(longest, device=seqs.device) < lens[:, None], as_tuple=True)
    slot = begin[i] + t
    at = pool["table"][0][seqs[i], slot // page].long()
    for name in "KV":
        x = state["new_" + name][i, :, t]
        if pool[name].dtype == torch.uint8:
            x, scale = _quantise(x)
            x = x.view(torch.uint8)
            pool[name.lower() + "scale"][0][at, :, slot % page] = scale
        pool[name][0][at, :, slot % page] = x
    pool["pos"][0][at, :, slot % page] = (first[i] + t).int()[:, None]
    pool["score"][0][seqs[i], :, slot] = state["new_score"][i, :, t]
    pool["meta"][0][seqs] = torch.stack([begin + lens, first + lens], 1).int()


# -------------------------------------------------------------------- its work
def work(case):
    """Bytes and operations that a pass cannot do without."""
    page, heads, d = case["page"], case["heads"], case["d"]
    vector = 2 * d if case["kv"] == "bf16" else d + 4
    slot = heads * (2 * vector + 8)  # a token's keys and values, position and score
    if case["op"] == "attend":
        lengths = _lengths(case, case["batch"])
        rows = case["batch"] * case["q_heads"]
        tokens = sum(lengths) + case["prefix"]
        pairs = case["q_heads"] * (sum(lengths) + case["batch"] * case["prefix"])
        return {"bytes": tokens * heads * (2 * vector + 8) + rows * (4 * d + 4), "flops": 4 * d * pairs}
    if case["op"] == "compact":
        k = case["h"] + case["r"]
        lengths = _lengths(case, case["n"])
        kept = sum(k if t > k else 0 for t in lengths)
        copied = sum(t % page for t in lengths)  # by the fork, and its scores
        return {"bytes": 2 * kept * slot + 4 * heads * sum(2 * t + (t if t > k else 0) for t in lengths)
                + 2 * copied * (slot - 8 * heads), "flops": 0}
    if case["op"] == "fork":
        lengths = _lengths(case, case["src"])
        to = [lengths[(i * 5) % case["src"]] for i in range(case["dst"])]
        return {"bytes": 2 * case["layers"] * sum((t % page) * (slot - 4 * heads) + 4 * heads * t + 4 * (t // page)
                                                  for t in to), "flops": 0}
    tokens = sum(_lengths(case, case["n"]))
    return {"bytes": tokens * (heads * (4 * d + 4) + slot), "flops": 0}


# -------------------------------------------------- the definition, in 64 bits
def _e4m3_steps(x):
    """The nearest E4M3 value, ties to even, of float64 values within +-448."""
    mant, exp = torch.frexp(x)
    step = torch.ldexp(torch.ones_like(x), exp.clamp(min=-5) - 4)
    return torch.round(x / step) * step


def exact(case, seed):
    state = prepare(case, seed)
    pool = state["pool"]
    wide = {n: (pool[n].view(E4M3) if pool[n].dtype == torch.uint8 else pool[n]).double()
            for n in ("K", "V", "kscale", "vscale", "score") if n in pool}
    table, meta, ref = pool["table"].cpu(), pool["meta"].cpu(), pool["ref"].cpu()
    page, op = case["page"], case["op"]

    def take(layer, n):
        free = torch.nonzero(ref[layer] == 0).flatten()[:n].tolist()
        ref[layer, free] = 1
        return free

    def tokens(name, layer, seq):
        """All stored tokens of a sequence, [heads, length, d]."""
        pages, length = table[layer, seq].tolist(), int(meta[layer, seq, 0])
        got = [wide[name][layer, p] for p in pages if p >= 0]
        if name.lower() + "scale" in wide:
            got = [g * wide[name.lower() + "scale"][layer, p].unsqueeze(-1) for g, p in zip(got, pages)]
        return torch.cat(got, 1)[:, :length] if got else wide[name].new_zeros(case["heads"], 0, case["d"])

    def drop(layer, seq):
        for p in table[layer, seq].tolist():
            if p >= 0:
                ref[layer, p] -= 1
        table[layer, seq], meta[layer, seq] = -1, 0

    def fork(layer, a, b):
        length = int(meta[layer, a, 0])
        table[layer, b], meta[layer, b] = table[layer, a], meta[layer, a]
        for p in table[layer, a, :length // page].tolist():
            ref[layer, p] += 1
        if length % page:
            old, (p,) = int(table[layer, a, length // page]), take(layer, 1)
            table[layer, b, length // page] = p
            for n in ("K", "V", "kscale", "vscale"):
                if n in wide:
                    wide[n][layer, p, :, :length % page] = wide[n][layer, old, :, :length % page]
        wide["score"][layer, b, :, :length] = wide["score"][layer, a, :, :length]

    if op == "attend":
        q, seqs = state["q"].double(), state["seqs"].tolist()
        group = case["q_heads"] // case["heads"]
        prefix = state["prefix"]
        shared = [tokens(n, 0, prefix) for n in "KV"] if prefix >= 0 else None
        out, lse = torch.empty_like(q), q.new_empty(q.shape[:2])
        for i, seq in enumerate(seqs):
            k, v = (tokens(n, 0, seq) for n in "KV")
            own_len = k.shape[1]
            if shared:
                k, v = torch.cat([k, shared[0]], 1), torch.cat([v, shared[1]], 1)
            s = q[i].view(case["heads"], group, -1) @ k.mT * case["d"] ** -0.5
            p = torch.softmax(s, -1)
            out[i] = (p @ v).flatten(0, 1)
            lse[i] = torch.logsumexp(s, -1).flatten()
            mass = p.sum(1)
            wide["score"][0, seq, :, :own_len] += mass[:, :own_len]
            if shared:
                wide["score"][0, prefix, :, :mass.shape[1] - own_len] += mass[:, own_len:]
        return {"out": out, "lse": lse, "score": wide["score"]}
    if op == "write":
        for i, seq in enumerate(state["seqs"].tolist()):
            drop(0, seq)
        for i, seq in enumerate(state["seqs"].tolist()):
            t = int(state["lens"][i])
            pages = take(0, _pages(t, page))
            for n in "KV":
                x = state["new_" + n][i, :, :t].double()
                if case["kv"] == "fp8":
                    amax = x.abs().amax(-1, keepdim=True)
                    inv = torch.where(amax > 0, (448 / amax).float().double(), 0)  # each operation is rounded to 32 bits
                    x = _e4m3_steps((x * inv).float().double().clamp(-448, 448))
                    scale = (amax / 448).float().double().squeeze(-1)
                    for at, p in enumerate(pages):
                        part = scale[:, at * page:(at + 1) * page]
                        wide[n.lower() + "scale"][0, p, :, :part.shape[1]] = part
                for at, p in enumerate(pages):
                    part = x[:, at * page:(at + 1) * page]
                    wide[n][0, p, :, :part.shape[1]] = part
            wide["score"][0, seq, :, :t] = state["new_score"][i, :, :t].double()
        return {n: wide.get(n) for n in pool}
    src, dst = state["src"].tolist(), state["dst"].tolist()
    for layer in range(ref.shape[0]):
        for b in dst:
            drop(layer, b)
        for a, b in zip(src, dst):
            fork(layer, a, b)
    if op == "compact":
        k = case["h"] + case["r"]
        moves = []
        for b in dst:
            length = int(meta[0, b, 0])
            if length <= k:
                continue
            score, pages = wide["score"][0, b, :, :length], table[0, b].tolist()
            order = torch.arange(length, device="cuda")
            # by (score, slot) in two stable sorts; the window counts as above every score
            ranked = torch.where(order >= length - case["r"], math.inf, score)
            kept = ranked.sort(stable=True, dim=-1).indices[:, length - k:].sort(-1).values
            moves.append((b, kept, pages, take(0, _pages(k, page)), score.gather(1, kept)))
        heads = torch.arange(case["heads"], device="cuda")[:, None]
        j = torch.arange(k, device="cuda")
        for b, kept, pages, fresh, score in moves:
            old, new = torch.tensor(pages, device="cuda"), torch.tensor(fresh, device="cuda")
            for n in ("K", "V", "kscale", "vscale"):
                if n in wide:
                    wide[n][0][new[j // page].expand(case["heads"], -1), heads, j % page] = \
                        wide[n][0][old[kept // page], heads, kept % page]
            wide["score"][0, b, :, :k] = score
    return {n: wide.get(n) for n in pool}
