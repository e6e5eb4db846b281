"""Rotary positions and drafted tokens over the paged cache: what is timed, and the plain forms.

A pool's arrays (one layer, N pages of `page` tokens, H key/value heads, S sequences of at most W
pages, C = W * page):

    K, V    [N, H, page, d]   bf16, or E4M3 codes with scales [N, H, page]
    pos     [N, H, page]      position of the token that a slot holds
    score   [S, H, C]         accumulated attention of a sequence's slots
    table   [S, W]            pages of a sequence, -1 behind the last
    meta    [S, 2]            length, next position
    ref     [N]               sequences that hold a page

Four operators: norms of queries and keys with the rotation of their positions, from a projection's
token-major output to head-major prompts (rotate); the same into the pages of sequences (append);
attention of a tree of drafted tokens over a sequence and a shared prefix (tree); and keeping the
drafts that were accepted, with the probabilities of their rows added to the scores (accept).
"""
import math

import torch

own = False

BF16 = torch.bfloat16
E4M3 = torch.float8_e4m3fn
EPS = 1e-6


# ---------------------------------------------------------------------- cases
def listed():
    return [
        # one token of one small sequence: latency alone
        dict(name="rotate_tiny", op="rotate", batch=1, T=1, q_heads=4, heads=4, d=64, dim=64, layout="half",
             scaling="none", base=10000.0, norm=False, first=129),
        # a prompt of a LLaMA-7B-shaped layer
        dict(name="rotate_llama-7b-32k", op="rotate", batch=1, T=32768, q_heads=32, heads=32, d=128, dim=128,
             layout="half", scaling="none", base=10000.0, norm=False, first=0),
        # prompts of odd length behind long ones, grouped heads with norms, half of each head rotated
        dict(name="rotate_grouped", op="rotate", batch=8, T=1021, q_heads=32, heads=8, d=128, dim=64,
             layout="interleaved", scaling="parts", base=500000.0, norm=True, first=100000),
        # a step of many sequences with grouped heads into an E4M3 cache
        dict(name="append_step_fp8", op="append", kv="fp8", n=64, T=1, shortest=1, longest=300, q_heads=32, heads=8,
             d=128, page=32, dim=128, layout="half", scaling="parts", base=500000.0, norm=True, draft=True),
        # the drafts of a LLaMA-7B-shaped layer for 16 sequences
        dict(name="append_tree", op="append", kv="bf16", n=16, T=24, shortest=64, longest=1024, q_heads=32, heads=32,
             d=128, page=64, dim=128, layout="half", scaling="linear", base=10000.0, norm=False, draft=True),
        # eight prompts of up to 2048 tokens
        dict(name="append_prompts", op="append", kv="bf16", n=8, T=2048, shortest=0, longest=0, q_heads=32, heads=32,
             d=128, page=64, dim=128, layout="half", scaling="none", base=10000.0, norm=False, draft=False),
        # five drafts of one small sequence: latency alone
        dict(name="tree_tiny", op="tree", kv="bf16", n=1, nodes=5, q_heads=4, heads=4, d=64, page=16, prefix=0,
             shortest=33, longest=33),
        # 16 drafts each over four documents of 32768 tokens, LLaMA-7B-shaped
        dict(name="tree_llama-7b-32k", op="tree", kv="bf16", n=4, nodes=16, q_heads=32, heads=32, d=128, page=128,
             prefix=0, shortest=32000, longest=32768),
        # a batch of sequences with up to 32 drafts each, grouped heads and an E4M3 cache
        dict(name="tree_grouped_fp8", op="tree", kv="fp8", n=64, nodes=32, q_heads=32, heads=8, d=128, page=32,
             prefix=0, shortest=300, longest=2000),
        # a long system prompt once for all and wide trees: 256 query rows a head
        dict(name="tree_prefix", op="tree", kv="bf16", n=16, nodes=64, q_heads=32, heads=8, d=128, page=64,
             prefix=8197, shortest=1, longest=1000),
        # what the grouped batch above keeps of its drafts
        dict(name="accept_grouped_fp8", op="accept", kv="fp8", n=64, nodes=32, q_heads=32, heads=8, d=128, page=32,
             prefix=0, shortest=300, longest=2000),
        # what the documents' trees keep
        dict(name="accept_llama-7b-32k", op="accept", kv="bf16", n=4, nodes=16, q_heads=32, heads=32, d=128, page=128,
             prefix=0, shortest=32000, longest=32768),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotate", "append", "tree", "tree", "accept"])
    kv = rng.choice(["bf16", "bf16", "fp8"])
    d = rng.choice([64, 128, 128])
    page = rng.choice([16, 32, 64, 128])
    heads, group = rng.choice([1, 2, 4, 7, 8, 16, 32]), rng.choice([1, 1, 2, 3, 4, 5, 8])
    rotary = dict(dim=rng.choice([16, 48, d // 2, d, d]), layout=rng.choice(["half", "interleaved"]),
                  scaling=rng.choice(["none", "linear", "ntk", "parts"]), base=rng.choice([10000.0, 500000.0, 1e6]),
                  norm=rng.random() < 0.5)
    if op == "rotate":
        batch, T = _log(rng, 1, 64), _log(rng, 1, 32768)
        while batch * T * heads * (group + 2) > 32768 * 96:
            batch, T = max(1, batch * 2 // 3), max(1, T * 2 // 3)
        return dict(op=op, batch=batch, T=T, q_heads=heads * group, heads=heads, d=d,
                    first=rng.choice([0, 1]) * _log(rng, 1, (1 << 20) - T), **rotary)
    if op == "append":
        draft = rng.random() < 0.6
        n, T, longest = _log(rng, 1, 256), _log(rng, 1, 64 if draft else 2048), _log(rng, 1, 4096) if draft else 0
        while n * T * heads * (group + 2) > 8 * 2048 * 96 or n * heads * (T + longest) > 2_000_000:
            n, longest = max(1, n * 2 // 3), longest * 2 // 3
            T = T if draft else max(1, T * 2 // 3)
        return dict(op=op, kv=kv, n=n, T=T, shortest=longest // rng.choice([1, 2, 50]), longest=longest,
                    q_heads=heads * group, heads=heads, d=d, page=page, draft=draft, **rotary)
    n, nodes = _log(rng, 1, 128), _log(rng, 1, 64)
    prefix = rng.choice([0, 0, 1]) * _log(rng, 1, 16384)
    longest = _log(rng, 1, 32768)
    while heads * (prefix + n * (longest + nodes)) > 4_000_000 or heads * group * n * nodes * (prefix + longest) > 210_000_000:
        n, longest, prefix = max(1, n * 3 // 4), max(1, longest * 3 // 4), prefix * 3 // 4
    return dict(op=op, kv=kv, n=n, nodes=nodes, q_heads=heads * group, heads=heads, d=d, page=page, prefix=prefix,
                shortest=rng.choice([0, longest // 2, longest]), longest=longest)


def _spread(lo, hi, n):
    """n whole numbers spread over [lo, hi], hi among them; nothing but the numbers decides them."""
    return [hi if i == 0 else lo + (i * 2654435761 >> 7) % (hi - lo + 1) for i in range(n)]


def _pages(tokens, page):
    return -(-tokens // page)


def _sizes(case):
    """(tokens before the new ones, new tokens) of each sequence."""
    if case["op"] == "append":
        new = _spread(case["T"] if case["draft"] else case["T"] * 3 // 4, case["T"], case["n"])
    else:
        new = _spread(max(1, case["nodes"] // 2), case["nodes"], case["n"])
    return _spread(case["shortest"], case["longest"], case["n"]), new


# ------------------------------------------------------------------ the inputs
SCALINGS = {"none": {}, "linear": dict(factor=4.0), "ntk": dict(factor=4.0),
            "parts": dict(factor=8.0, original=8192, low=1.0, high=32.0, attention=0.1 * math.log(8.0) + 1.0)}


def _quantise(x):
    """E4M3 codes (as float8) and one scale a vector: scale = amax / 448, code = E4M3(x * (448 / amax))."""
    x = x.float()
    amax = x.abs().amax(-1, keepdim=True)
    top = torch.full_like(amax, 448.0)  # tensors on both sides: a scalar's reciprocal would round once more
    inv = torch.where(amax > 0, top / amax, 0.0)
    return (x * inv).clamp(-448, 448).to(E4M3), (amax / top).squeeze(-1)


def _ints(values):
    return torch.tensor(list(values), dtype=torch.int32, device="cuda")


def _pool(case, gen, lengths, room, spare, width):
    """The arrays of a pool whose first sequences have `lengths`, with `room` more empty sequences and `spare` free pages.

    A few tokens of every page attract most of the attention, along a direction that the queries share; the scores
    follow a power law. The pages of a sequence lie anywhere in the pool."""
    dev, heads, d, page = "cuda", case["heads"], case["d"], case["page"]
    length = torch.tensor(lengths)
    used = -(-length // page)
    n, s = int(used.sum()) + spare, len(lengths) + room
    shape = (n, heads, page)
    direction = torch.randn(heads, 1, d, generator=gen, device=dev)
    direction = direction / direction.norm(dim=-1, keepdim=True)
    k = torch.randn(*shape, d, generator=gen, device=dev, dtype=BF16)
    rank = torch.rand(*shape, 1, generator=gen, device=dev) * 4096 + 1
    k += (8 * rank.pow(-0.8) * direction).to(BF16)
    v = torch.randn(*shape, d, generator=gen, device=dev, dtype=BF16)
    arrays = {"K": k, "V": v}
    if case["kv"] == "fp8":
        (k, ks), (v, vs) = _quantise(k), _quantise(v)
        arrays = {"K": k.view(torch.uint8), "V": v.view(torch.uint8), "kscale": ks, "vscale": vs}
    table = torch.full((s, width), -1, dtype=torch.int32)
    order = torch.randperm(n, generator=torch.Generator().manual_seed(int(gen.initial_seed()) + 1)).int()
    table[:len(lengths)][torch.arange(width) < used[:, None]] = order[:int(used.sum())]
    meta = torch.zeros(s, 2, dtype=torch.int32)
    meta[:len(lengths), 0] = length
    meta[:len(lengths), 1] = length + 5003 * torch.arange(len(lengths))  # some tokens were dropped before
    ref = torch.zeros(n, dtype=torch.int32)
    ref[order[:int(used.sum())].long()] = 1
    arrays["pos"] = torch.randint(0, 1 << 20, shape, generator=gen, device=dev, dtype=torch.int32)
    arrays["score"] = 0.02 / (torch.rand(s, heads, width * page, generator=gen, device=dev) + 1e-3)
    arrays["table"], arrays["meta"], arrays["ref"] = table.to(dev), meta.to(dev), ref.to(dev)
    return arrays, direction


def _parents(gen, n, nodes):
    """Random trees: node t hangs below one of the 60 % before it that came last, or begins a branch of its own."""
    t = torch.arange(nodes, device="cuda")
    r = 0.4 + 0.6 * torch.rand(n, nodes, generator=gen, device="cuda")
    return ((t + 1) * r).floor().clamp(max=t).int() - 1


def _frequencies(case):
    """Radians a position of each pair, in 64 bits, and the factor of cosines and sines."""
    dim, kind = case["dim"], SCALINGS[case["scaling"]]
    base = case["base"]
    if case["scaling"] == "ntk":
        base = base * kind["factor"] ** (dim / (dim - 2))
    f = torch.pow(base, -torch.arange(0, dim, 2, dtype=torch.float64, device="cuda") / dim)
    if case["scaling"] == "linear":
        f = f / kind["factor"]
    if case["scaling"] == "parts":
        turns = kind["original"] * f / (2 * math.pi)
        g = ((turns - kind["low"]) / (kind["high"] - kind["low"])).clamp(0, 1)
        f = g * f + (1 - g) * f / kind["factor"]
    return f, kind.get("attention", 1.0)


def _projection(case, gen, n, T):
    """q, k, v [n, T, heads, d]: views of one projection's output, and the norms' weights."""
    qh, h, d = case["q_heads"], case["heads"], case["d"]
    x = torch.randn(n, T, (qh + 2 * h) * d, generator=gen, device="cuda", dtype=BF16)
    x = x.view(n, T, qh + 2 * h, d)
    weights = [1 + 0.2 * torch.randn(d, generator=gen, device="cuda") if case["norm"] else None for _ in range(2)]
    state = {"q": x[:, :, :qh], "k": x[:, :, qh:qh + h], "v": x[:, :, qh + h:], "q_norm": weights[0], "k_norm": weights[1]}
    if own:
        import h2o_heavy_hitter_gb300 as h2o

        state["rotary"] = h2o.h2o_rotary(case["dim"], case["base"], layout=case["layout"], scaling=case["scaling"],
                                         **SCALINGS[case["scaling"]])
    else:
        state["freq"], state["factor"] = _frequencies(case)
    return state


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    op = case["op"]
    state = {"case": case}
    if op == "rotate":
        state |= _projection(case, gen, case["batch"], case["T"])
        first = torch.randint(case["first"] // 2, case["first"] + 1, (case["batch"], 1), generator=gen, device="cuda")
        state["positions"] = (first + torch.arange(case["T"], device="cuda")).int()
        return state
    before, new = _sizes(case)
    n, page, heads, d = case["n"], case["page"], case["heads"], case["d"]
    T = max(new)
    state |= {"lens": _ints(new), "seqs": _ints(range(n))}
    if op == "append":
        width = max(_pages(a + b, page) for a, b in zip(before, new))
        spare = sum(_pages(a + b, page) - _pages(a, page) for a, b in zip(before, new)) + 2
        arrays, _ = _pool(case, gen, before, 0, spare, width)
        state |= _projection(case, gen, n, T)
        state["parent"] = _parents(gen, n, T) if case["draft"] else None
        state["out"] = torch.zeros(n, T, case["q_heads"], d, dtype=BF16, device="cuda")
    else:
        shared = [case["prefix"]] if case["prefix"] else []
        state |= {"parent": _parents(gen, n, T), "prefix": -1}
        q_shape = (n, T, case["q_heads"], d)
        if op == "tree":
            lengths = [a + b for a, b in zip(before, new)] + shared
            arrays, direction = _pool(case, gen, lengths, 0, 2, max(_pages(t, page) for t in lengths))
            state |= {"out": torch.zeros(q_shape, dtype=BF16, device="cuda"), "lse": torch.zeros(q_shape[:3], device="cuda")}
        else:
            # the sequences are kept as they are; forks of them get the drafts
            lengths = before + shared
            width = max(_pages(t, page) for t in [a + b for a, b in zip(before, new)] + shared)
            spare = sum(_pages(a + b, page) - a // page for a, b in zip(before, new)) + 2
            arrays, direction = _pool(case, gen, lengths, n, spare, width)
            state["dst"] = _ints(range(len(lengths), len(lengths) + n))
        if shared:
            state["prefix"] = n
        q = torch.randn(q_shape, generator=gen, device="cuda")
        q += 2 * direction.repeat_interleave(case["q_heads"] // heads, 0).squeeze(1)
        state["q"] = q.to(BF16)
    if op == "accept":
        drafts = torch.randn(2, n, heads, T, d, generator=gen, device="cuda").to(BF16)
        state |= {"new_K": drafts[0].contiguous(), "new_V": drafts[1].contiguous()}
        # the first up to eight nodes of a branch; one sequence in eight keeps nothing
        leaf = (torch.rand(n, generator=gen, device="cuda") * state["lens"]).long()
        branch = _reach(state["parent"])[torch.arange(n, device="cuda"), leaf]
        node = torch.arange(T, device="cuda")
        path = torch.where(branch, node, T).sort(-1).values[:, :8]
        none = torch.rand(n, 1, generator=gen, device="cuda") < 0.125
        state["path"] = torch.where((path == T) | none, -1, path).int()
    state["pool"] = arrays
    if op == "accept":
        _stage(state)
        state["lse"] = torch.where(node < state["lens"][:, None], 0, math.nan)[:, :, None] + _log_sums(state)
        _free(arrays, state["dst"])
    if own:
        import h2o_heavy_hitter_gb300 as h2o

        state["handle"] = h2o.h2o_pool_create(1, arrays["ref"].shape[0], page, heads, d, arrays["meta"].shape[0],
                                              arrays["table"].shape[1], kv=case["kv"])
        view = h2o.h2o_pool_view(state["handle"], 0)
        torch._foreach_copy_([view[name] for name in arrays], list(arrays.values()))
        state["pool"] = view
    return state


# --------------------------------------------------------------- the operators
def run(state):
    op = state["case"]["op"]
    if own:
        return _run_own(state)
    if op == "rotate":
        angle = _angles(state, state["positions"])
        q = _rotated(state, state["q"], state["q_norm"], angle)
        k = _rotated(state, state["k"], state["k_norm"], angle)
        return [x.transpose(1, 2).to(BF16).contiguous() for x in (q, k, state["v"])]
    pool = state["pool"]
    if op == "append":
        if not state["case"]["draft"]:
            _free(pool, state["seqs"])
        _append(state)
        if state["case"]["draft"]:
            _accept(pool, state["seqs"], state["lens"], torch.full_like(state["parent"][:, :1], -1))
        return {"q": state["out"]} | _values(pool)
    if op == "tree":
        _attend(state)
        return {"out": state["out"], "lse": state["lse"]}
    _free(pool, state["dst"])
    _stage(state)
    _accept(pool, state["dst"], state["lens"], state["path"])
    _add_scores(state)
    return _values(pool)


def _run_own(state):
    import h2o_heavy_hitter_gb300 as h2o

    op = state["case"]["op"]
    if op == "rotate":
        return list(h2o.h2o_rotate_qkv(state["rotary"], state["q"], state["k"], state["v"], positions=state["positions"],
                                       q_norm=state["q_norm"], k_norm=state["k_norm"], eps=EPS))
    handle, pool, seqs = state["handle"], state["pool"], state["seqs"]
    if op == "append":
        if not state["case"]["draft"]:
            h2o.h2o_pool_free(handle, 0, seqs)
        out = h2o.h2o_pool_append(handle, 0, seqs, state["q"], state["k"], state["v"], rotary=state["rotary"],
                                  lens=state["lens"], parent=state["parent"], q_norm=state["q_norm"],
                                  k_norm=state["k_norm"], eps=EPS, out=state["out"])
        if state["case"]["draft"]:
            h2o.h2o_pool_accept(handle, 0, seqs, state["q"].shape[1], lens=state["lens"])
        return {"q": out} | _values(pool)
    if op == "tree":
        out, lse = h2o.h2o_pool_attend_tree(handle, 0, seqs, state["q"], prefix=state["prefix"], lens=state["lens"],
                                            parent=state["parent"], out=state["out"], lse=state["lse"])
        return {"out": out, "lse": lse}
    dst = state["dst"]
    h2o.h2o_pool_free(handle, 0, dst)
    h2o.h2o_pool_fork(handle, 0, seqs, dst)
    h2o.h2o_pool_write(handle, 0, dst, state["new_K"], state["new_V"], lens=state["lens"])
    h2o.h2o_pool_accept(handle, 0, dst, state["q"].shape[1], path=state["path"], lens=state["lens"], q=state["q"],
                        lse=state["lse"], prefix=state["prefix"])
    return _values(pool)


def _values(pool):
    """A pool's arrays, codes as the values that they stand for before their scale."""
    return {k: v.view(E4M3) if v.dtype == torch.uint8 else v for k, v in pool.items()}


def _angles(state, positions):
    """Cosines and sines [..., 1, dim / 2] in 32 bits, of angles in 64."""
    a = positions.double()[..., None, None] * state["freq"]
    return a.cos().float() * state["factor"], a.sin().float() * state["factor"]


def _rotated(state, x, weight, angle):
    """x [..., heads, d] in 32 bits, normed and rotated."""
    dim, (c, s) = state["case"]["dim"], angle
    x = x.float()
    if weight is not None:
        x = x * (x.square().mean(-1, keepdim=True) + EPS).rsqrt() * weight
    rest = x[..., dim:]
    if state["case"]["layout"] == "half":
        a, b = x[..., :dim // 2], x[..., dim // 2:dim]
        return torch.cat([a * c - b * s, a * s + b * c, rest], -1)
    a, b = x[..., :dim:2], x[..., 1:dim:2]
    return torch.cat([torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2), rest], -1)


def _reach(parent):
    """[n, T, T]: whether node t's branch (itself and those that it hangs below) holds node j."""
    n, T = parent.shape
    up = torch.nn.functional.one_hot(parent.long() + 1, T + 1)[..., 1:].float()
    m = up + torch.eye(T, device=parent.device)
    for _ in range(6):  # branches of 2, 4, ... 64 nodes
        m = ((m @ m) > 0).float()
    return m > 0


def _free(pool, seqs):
    seqs = seqs.long()
    held = pool["table"][seqs].flatten().long()
    pool["ref"].scatter_add_(0, held.clamp(min=0), -(held >= 0).int())
    pool["table"][seqs] = -1
    pool["meta"][seqs] = 0


def _fresh(pool, need):
    """Free pages, the lowest first, for each entry of `need` [n] in its turn: [n, W]; what is behind an entry's need is not its own."""
    free = torch.argsort((pool["ref"] != 0).int(), stable=True)
    rank = (need.cumsum(0) - need).unsqueeze(-1) + torch.arange(pool["table"].shape[1], device=need.device)
    return free[rank.clamp(max=free.shape[0] - 1)]


def _fork(pool, src, dst, page):
    src, dst = src.long(), dst.long()
    held, length = pool["table"][src].long(), pool["meta"][src, 0].long()
    whole, rest = (length // page).unsqueeze(-1), length % page
    j = torch.arange(held.shape[1], device=src.device)
    fresh = _fresh(pool, (rest > 0).long())[:, :1]
    pool["table"][dst] = torch.where(j < whole, held, torch.where((j == whole) & (rest > 0).unsqueeze(-1), fresh, -1)).int()
    pool["ref"].scatter_add_(0, held.clamp(min=0).flatten(), (j < whole).flatten().int())
    i = torch.nonzero(rest > 0).squeeze(1)
    to, at = fresh[i, 0], held[i, length[i] // page]
    pool["ref"][to] = 1
    live = torch.arange(page, device=src.device) < rest[i].unsqueeze(-1)
    for name in ("K", "V", "kscale", "vscale", "pos"):
        if name in pool:
            x = pool[name]
            x[to] = torch.where(live.view(live.shape[0], 1, page, *[1] * (x.dim() - 3)), x[at], x[to])
    behind = torch.arange(pool["score"].shape[2], device=src.device) >= length[:, None, None]
    pool["score"][dst] = torch.where(behind, pool["score"][dst], pool["score"][src])
    pool["meta"][dst] = pool["meta"][src]


def _place(pool, seqs, lens, T, page):
    """Pages for lens[i] more tokens of each sequence; (entry, token, page, offset, slot) of each, and the next positions before."""
    begin, first = pool["meta"][seqs].long().unbind(1)
    p0, p1 = -(-begin // page), -(-(begin + lens) // page)
    j = torch.arange(pool["table"].shape[1], device=seqs.device)
    fresh = _fresh(pool, p1 - p0).gather(1, (j - p0[:, None]).clamp(min=0))
    new = (j >= p0[:, None]) & (j < p1[:, None])
    pool["table"][seqs] = torch.where(new, fresh, pool["table"][seqs].long()).int()
    pool["ref"][fresh[new]] = 1
    i, t = torch.nonzero(torch.arange(T, device=seqs.device) < lens[:, None], as_tuple=True)
    slot = begin[i] + t
    pool["meta"][seqs, 0] = (begin + lens).int()
    return i, t, pool["table"][seqs[i], slot // page].long(), slot % page, slot, first


def _put(pool, at, off, k, v):
    """Keys and values [tokens, heads, d] into their slots."""
    for name, x in (("K", k), ("V", v)):
        if pool[name].dtype == torch.uint8:
            x, scale = _quantise(x)
            x = x.view(torch.uint8)
            pool[name.lower() + "scale"][at, :, off] = scale
        pool[name][at, :, off] = x.to(pool[name].dtype)


def _append(state):
    pool, page = state["pool"], state["case"]["page"]
    seqs, lens = state["seqs"].long(), state["lens"].long()
    i, t, at, off, slot, first = _place(pool, seqs, lens, state["k"].shape[1], page)
    ahead = t if state["parent"] is None else _reach(state["parent"]).sum(-1)[i, t] - 1
    position = first[i] + ahead
    angle = _angles(state, position)
    state["out"][i, t] = _rotated(state, state["q"][i, t], state["q_norm"], angle).to(BF16)
    _put(pool, at, off, _rotated(state, state["k"][i, t], state["k_norm"], angle), state["v"][i, t])
    pool["pos"][at, :, off] = position.int()[:, None]
    pool["score"][seqs[i], :, slot] = 0
    if state["parent"] is None:
        pool["meta"][seqs, 1] = (first + lens).int()


def _stage(state):
    """The drafts in forks of the sequences."""
    pool, page = state["pool"], state["case"]["page"]
    _fork(pool, state["seqs"], state["dst"], page)
    seqs, lens = state["dst"].long(), state["lens"].long()
    i, t, at, off, slot, first = _place(pool, seqs, lens, state["new_K"].shape[2], page)
    _put(pool, at, off, state["new_K"][i, :, t], state["new_V"][i, :, t])
    pool["pos"][at, :, off] = (first[i] + t).int()[:, None]
    pool["score"][seqs[i], :, slot] = 0
    pool["meta"][seqs, 1] = (first + lens).int()


def _stored(pool, name, pages):
    """The tokens of `pages` [..., n] in 32 bits, as [..., heads, n * page, d]."""
    x = pool[name][pages]
    x = x.view(E4M3).float() * pool[name.lower() + "scale"][pages].unsqueeze(-1) if x.dtype == torch.uint8 else x.float()
    return x.transpose(-4, -3).flatten(-3, -2)


def _rows(state):
    """The queries as rows of their key heads, [n, heads, nodes * group, d], in 32 bits and scaled."""
    n, T, q_heads, d = state["q"].shape
    heads = state["case"]["heads"]
    q = state["q"].float() / math.sqrt(d)
    return q.view(n, T, heads, q_heads // heads, d).transpose(1, 2).reshape(n, heads, -1, d)


def _own_logits(state, seqs, q):
    """Logits of the rows against their sequence's tokens, -inf where a row does not attend, and the tokens' pages."""
    pool, page = state["pool"], state["case"]["page"]
    seqs, lens, T = seqs.long(), state["lens"].long(), state["q"].shape[1]
    pages = pool["table"][seqs].long().clamp(min=0)
    begin = (pool["meta"][seqs, 0].long() - lens)[:, None, None]
    slot = torch.arange(pages.shape[1] * page, device=q.device)
    node = (slot - begin).clamp(0, T - 1).expand(-1, T, -1)
    keep = (slot < begin) | (_reach(state["parent"]).gather(2, node) & (slot >= begin) & (slot < begin + lens[:, None, None]))
    keep = keep.repeat_interleave(q.shape[2] // T, 1)[:, None]
    return torch.where(keep, q @ _stored(pool, "K", pages).transpose(2, 3), -math.inf), pages, slot < begin[:, 0] + lens[:, None]


def _prefix_logits(state, q):
    """The same against the prefix's, [heads, n * rows, tokens]."""
    pool, page, prefix = state["pool"], state["case"]["page"], state["prefix"]
    pages = pool["table"][prefix].long().clamp(min=0)
    stays = torch.arange(pages.numel() * page, device=q.device) < pool["meta"][prefix, 0]
    rows = q.transpose(0, 1).reshape(q.shape[1], -1, q.shape[3])
    return torch.where(stays, rows @ _stored(pool, "K", pages).transpose(1, 2), -math.inf), pages, stays


def _by_token(state, x):
    """[n, heads, nodes * group, ...] as [n, nodes, q_heads, ...]."""
    n, T, q_heads, _ = state["q"].shape
    heads = state["case"]["heads"]
    x = x.view(n, heads, T, q_heads // heads, *x.shape[3:])
    return x.transpose(1, 2).reshape(n, T, q_heads, *x.shape[4:])


def _attend(state):
    pool, q = state["pool"], _rows(state)
    s, pages, live = _own_logits(state, state["seqs"], q)
    top = s.amax(-1, keepdim=True)
    if state["prefix"] >= 0:
        ps, at, stays = _prefix_logits(state, q)
        ps = ps.view(s.shape[1], s.shape[0], -1, ps.shape[2]).transpose(0, 1)
        top = torch.maximum(top, ps.amax(-1, keepdim=True))
    e = (s - top).exp()
    total = e.sum(-1, keepdim=True)
    out = e @ torch.where(live[:, None, :, None], _stored(pool, "V", pages), 0)
    if state["prefix"] >= 0:
        pe = (ps - top).exp()
        total = total + pe.sum(-1, keepdim=True)
        flat = pe.transpose(0, 1).reshape(s.shape[1], -1, pe.shape[3])
        more = flat @ torch.where(stays[:, None], _stored(pool, "V", at), 0)
        out = out + more.view(s.shape[1], s.shape[0], -1, more.shape[2]).transpose(0, 1)
    n, T = state["q"].shape[:2]
    valid = torch.arange(T, device=q.device) < state["lens"][:, None]
    state["out"].copy_(torch.where(valid[..., None, None], _by_token(state, out / total).to(BF16), state["out"]))
    state["lse"].copy_(torch.where(valid[..., None], _by_token(state, (top + total.log()).squeeze(-1)), state["lse"]))


def _log_sums(state):
    """The natural log of every row's normaliser over its sequence's drafts' fork and the prefix, [n, nodes, q_heads]."""
    q = _rows(state)
    s = _own_logits(state, state["dst"], q)[0]
    lse = torch.logsumexp(s, -1)
    if state["prefix"] >= 0:
        ps = torch.logsumexp(_prefix_logits(state, q)[0], -1).view(s.shape[1], s.shape[0], -1).transpose(0, 1)
        lse = torch.logaddexp(lse, ps)
    return _by_token(state, lse)


def _accept(pool, seqs, lens, path):
    """Keeps the nodes path[i] (ascending, -1 behind the last) of the last lens[i] tokens of each sequence."""
    page, width = pool["pos"].shape[2], pool["table"].shape[1]
    seqs, begin, count = seqs.long(), pool["meta"][seqs.long(), 0].long() - lens.long(), (path >= 0).sum(1)
    held = pool["table"][seqs].long()
    first = pool["pos"][held[torch.arange(len(seqs), device=seqs.device), begin // page], 0, begin % page]
    i, j = torch.nonzero(path >= 0, as_tuple=True)
    old, new = begin[i] + path[i, j].long(), begin[i] + j
    for name in ("K", "V", "kscale", "vscale", "pos"):
        if name in pool:
            pool[name][held[i, new // page], :, new % page] = pool[name][held[i, old // page], :, old % page]
    gone = (torch.arange(width, device=seqs.device) >= (-(-(begin + count) // page))[:, None]) & (held >= 0)
    pool["ref"].scatter_add_(0, held[gone], torch.full_like(held[gone], -1).int())
    pool["table"][seqs] = torch.where(gone, -1, held).int()
    pool["meta"][seqs] = torch.stack([begin + count, first + count], 1).int()


def _add_scores(state):
    pool, page, path = state["pool"], state["case"]["page"], state["path"].long()
    dst, count = state["dst"].long(), (state["path"] >= 0).sum(1)
    n, P = path.shape
    heads, group = state["case"]["heads"], state["q"].shape[2] // state["case"]["heads"]
    row = torch.arange(n, device=path.device)[:, None]
    q = state["q"].float()[row, path.clamp(min=0)] / math.sqrt(state["case"]["d"])
    lse = torch.where((path >= 0)[..., None], state["lse"][row, path.clamp(min=0)], math.inf)
    q = q.view(n, P, heads, group, -1).transpose(1, 2).flatten(2, 3)
    lse = lse.view(n, P, heads, group).transpose(1, 2).flatten(2, 3).unsqueeze(-1)
    pages = pool["table"][dst].long().clamp(min=0)
    slot = torch.arange(pages.shape[1] * page, device=q.device)
    begin = (pool["meta"][dst, 0].long() - count)[:, None, None]
    keep = slot <= begin + torch.arange(P, device=q.device).repeat_interleave(group)[:, None]
    p = torch.where(keep[:, None], (q @ _stored(pool, "K", pages).transpose(2, 3) - lse).exp(), 0)
    more = torch.where((slot < begin + count[:, None, None])[:, 0][:, None], p.sum(2), 0)
    pool["score"].index_add_(0, dst, more)
    if state["prefix"] >= 0:
        ps, _, stays = _prefix_logits(state, q)
        p = (ps - lse.transpose(0, 1).reshape(heads, -1, 1)).exp().sum(1)
        pool["score"][state["prefix"]] += torch.where(stays, p, 0)


# -------------------------------------------------------------------- its work
def work(case):
    """Bytes and operations that a pass cannot do without."""
    heads, q_heads, d = case["heads"], case["q_heads"], case["d"]
    if case["op"] == "rotate":
        tokens = case["batch"] * case["T"]
        return {"bytes": tokens * ((q_heads + 2 * heads) * 4 * d + 4), "flops": tokens * (q_heads + heads) * 3 * case["dim"]}
    before, new = _sizes(case)
    vector = 2 * d if case["kv"] == "bf16" else d + 4
    tokens = sum(new)
    if case["op"] == "append":
        return {"bytes": tokens * ((q_heads + 2 * heads) * 2 * d + q_heads * 2 * d + heads * (2 * vector + 8)),
                "flops": tokens * (q_heads + heads) * 3 * case["dim"]}
    seen = sum(before) + case["prefix"]
    if case["op"] == "tree":
        pairs = q_heads * sum(b * (a + case["prefix"]) for a, b in zip(before, new))
        return {"bytes": (seen + tokens) * heads * 2 * vector + tokens * q_heads * (4 * d + 4), "flops": 4 * d * pairs}
    # four accepted drafts a sequence; the staging's own bytes are not counted
    pairs = q_heads * 4 * (sum(before) + case["n"] * case["prefix"])
    return {"bytes": seen * heads * (vector + 8) + case["n"] * 4 * (q_heads * (2 * d + 4) + heads * 4 * vector),
            "flops": 2 * d * pairs}


# -------------------------------------------------- the definition, in 64 bits
def _e4m3_steps(x):
    """The nearest E4M3 value, ties to even, of float64 values within +-448."""
    _, exp = torch.frexp(x)
    step = torch.ldexp(torch.ones_like(x), exp.clamp(min=-5) - 4)
    return torch.round(x / step) * step


def _codes(x):
    """E4M3 values and scales of float64 vectors that are rounded to 32 bits first."""
    amax = x.float().double().abs().amax(-1, keepdim=True)
    inv = torch.where(amax > 0, (448 / amax).float().double(), 0)
    return _e4m3_steps((x.float().double() * inv).float().double().clamp(-448, 448)), (amax / 448).float().double().squeeze(-1)


def _turned(case, x, weight, positions):
    """x [..., heads, d] in 64 bits at positions [...], as products of complex numbers."""
    dim, kind = case["dim"], SCALINGS[case["scaling"]]
    x = x.double()
    if weight is not None:
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / case["d"] + EPS) * weight.double()
    stretch = kind["factor"] ** (dim / (dim - 2)) if case["scaling"] == "ntk" else 1.0
    angles = []
    for i in range(dim // 2):
        f = (case["base"] * stretch) ** (-2.0 * i / dim)
        if case["scaling"] == "linear":
            f /= kind["factor"]
        if case["scaling"] == "parts":
            share = (kind["original"] * f / (2 * math.pi) - kind["low"]) / (kind["high"] - kind["low"])
            share = min(1.0, max(0.0, share))
            f = share * f + (1 - share) * f / kind["factor"]
        angles.append(positions.double() * f)
    size = torch.full((), kind.get("attention", 1.0), dtype=torch.float64, device=x.device)
    turn = torch.polar(size, torch.stack(angles, -1)).unsqueeze(-2)
    out = x.clone()
    first = torch.arange(dim // 2) * (1 if case["layout"] == "half" else 2)
    second = first + (dim // 2 if case["layout"] == "half" else 1)
    z = torch.complex(x[..., first], x[..., second]) * turn
    out[..., first], out[..., second] = z.real, z.imag
    return out


def exact(case, seed):
    state = prepare(case, seed)
    op = case["op"]
    if op == "rotate":
        q = _turned(case, state["q"], state["q_norm"], state["positions"]).transpose(1, 2)
        k = _turned(case, state["k"], state["k_norm"], state["positions"]).transpose(1, 2)
        return [q, k, state["v"].double().transpose(1, 2)]
    pool, page = state["pool"], case["page"]
    wide = {n: (pool[n].view(E4M3) if pool[n].dtype == torch.uint8 else pool[n]).double()
            for n in ("K", "V", "kscale", "vscale", "score") if n in pool}
    table, meta, ref = pool["table"].cpu(), pool["meta"].cpu(), pool["ref"].cpu()
    parent = None if state["parent"] is None else state["parent"].tolist()
    lens = state["lens"].tolist()

    def branch(i, t):
        """Node t of entry i and those that it hangs below, the first first."""
        got = []
        while t >= 0:
            got.append(t)
            t = parent[i][t]
        return got[::-1]

    def take(count):
        free = torch.nonzero(ref == 0).flatten()[:count].tolist()
        ref[free] = 1
        return free

    def tokens(name, seq):
        """All stored tokens of a sequence, [heads, length, d]."""
        pages, length = [p for p in table[seq].tolist() if p >= 0], int(meta[seq, 0])
        if not pages:
            return wide[name].new_zeros(case["heads"], 0, case["d"])
        x = wide[name][pages]
        if name.lower() + "scale" in wide:
            x = x * wide[name.lower() + "scale"][pages].unsqueeze(-1)
        return x.transpose(0, 1).reshape(case["heads"], -1, case["d"])[:, :length]

    def put(seq, k, v):
        """Appends [heads, tokens, d]; the first slot."""
        begin, T = int(meta[seq, 0]), k.shape[1]
        have, need = _pages(begin, page), _pages(begin + T, page)
        table[seq, have:need] = torch.tensor(take(need - have), dtype=torch.int32)
        meta[seq, 0] += T
        slot = torch.arange(begin, begin + T)
        at, off = table[seq][slot // page].long().cuda(), (slot % page).cuda()
        for name, x in (("K", k), ("V", v)):
            x = x.transpose(0, 1)
            if case["kv"] == "fp8":
                x, scale = _codes(x)
                wide[name.lower() + "scale"][at, :, off] = scale
            wide[name][at, :, off] = x
        wide["score"][seq, :, begin:begin + T] = 0
        return begin

    def drop(seq, length):
        for j in range(_pages(length, page), _pages(int(meta[seq, 0]), page)):
            ref[table[seq, j]] -= 1
            table[seq, j] = -1
        meta[seq, 0] = length

    if op == "append":
        out = state["out"].double()
        for i, seq in enumerate(state["seqs"].tolist()):
            if not case["draft"]:
                drop(seq, 0)
                meta[seq, 1] = 0
        for i, seq in enumerate(state["seqs"].tolist()):
            T, next_ = lens[i], int(meta[seq, 1])
            ahead = range(T) if parent is None else [len(branch(i, t)) - 1 for t in range(T)]
            positions = torch.tensor([next_ + a for a in ahead], device="cuda")
            out[i, :T] = _turned(case, state["q"][i, :T], state["q_norm"], positions)
            k = _turned(case, state["k"][i, :T], state["k_norm"], positions)
            put(seq, k.transpose(0, 1), state["v"][i, :T].double().transpose(0, 1))
        return {"q": out} | {n: wide.get(n) for n in pool}

    q = state["q"].double()
    n, T, q_heads, d = q.shape
    group = q_heads // case["heads"]
    prefix = state["prefix"]
    shared = {m: tokens(m, prefix) for m in "KV"} if prefix >= 0 else None
    if op == "tree":
        out, lse = state["out"].double(), state["lse"].double()
        for i, seq in enumerate(state["seqs"].tolist()):
            k, v = tokens("K", seq), tokens("V", seq)
            begin = k.shape[1] - lens[i]
            for t in range(lens[i]):
                at = torch.cat([torch.arange(begin), begin + torch.tensor(branch(i, t))]).cuda() if t else None
                kt, vt = (k[:, :begin + 1], v[:, :begin + 1]) if t == 0 else (k, v)
                s = q[i, t].view(case["heads"], group, d) @ kt.mT / math.sqrt(d)
                if t:
                    gone = torch.ones(k.shape[1], dtype=torch.bool, device="cuda")
                    gone[at] = False
                    s = s.masked_fill(gone, -math.inf)
                if shared:
                    s = torch.cat([s, q[i, t].view(case["heads"], group, d) @ shared["K"].mT / math.sqrt(d)], -1)
                p = torch.softmax(s, -1)
                y = p[..., :kt.shape[1]] @ vt
                if shared:
                    y = y + p[..., kt.shape[1]:] @ shared["V"]
                out[i, t], lse[i, t] = y.flatten(0, 1), torch.logsumexp(s, -1).flatten()
        return {"out": out, "lse": lse}
    dst, given = state["dst"].tolist(), state["lse"].double()
    for seq, to in zip(state["seqs"].tolist(), dst):  # the forks
        length = int(meta[seq, 0])
        table[to], meta[to] = table[seq], meta[seq]
        ref[table[seq, :length // page].long()] += 1
        if length % page:
            old, (new,) = int(table[seq, length // page]), take(1)
            table[to, length // page] = new
            for m in ("K", "V", "kscale", "vscale"):
                if m in wide:
                    wide[m][new, :, :length % page] = wide[m][old, :, :length % page]
        wide["score"][to, :, :length] = wide["score"][seq, :, :length]
    begins = [put(to, state["new_K"][i, :, :lens[i]].double(), state["new_V"][i, :, :lens[i]].double())
              for i, to in enumerate(dst)]
    for i, to in enumerate(dst):
        kept = [t for t in state["path"][i].tolist() if t >= 0]
        begin = begins[i]
        where = lambda slots: (table[to][slots // page].long().cuda(), (slots % page).cuda())  # noqa: E731
        old, new = where(begin + torch.tensor(kept, dtype=torch.long)), where(begin + torch.arange(len(kept)))
        for m in ("K", "V", "kscale", "vscale"):
            if m in wide and kept:
                wide[m][new[0], :, new[1]] = wide[m][old[0], :, old[1]]
        drop(to, begin + len(kept))
        k = tokens("K", to)
        for j, t in enumerate(kept):
            rows, less = q[i, t].view(case["heads"], group, d), given[i, t].view(case["heads"], group, 1)
            p = torch.exp(rows @ k[:, :begin + j + 1].mT / math.sqrt(d) - less)
            wide["score"][to, :, :begin + j + 1] += p.sum(1)
            if shared:
                wide["score"][prefix, :, :shared["K"].shape[1]] += torch.exp(rows @ shared["K"].mT / math.sqrt(d) - less).sum(1)
    return {m: wide.get(m) for m in pool}
