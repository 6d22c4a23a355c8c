"""Workloads of the paged KV cache operators: the calls a user makes of them, and their plain form in torch.

The cache is the framework's INT8 KV cache (one float32 scale per head_dim group) cut into pages of
[kv_heads, page_tokens, head_dim]. Five operators work on it: ``shn_kv_plan`` (block tables and slot maps from
request lengths), ``shn_kv_store`` (norm and rotation of queries and keys, keys and values quantised into their
slots), ``shn_kv_load`` (rows of the cache as bf16), ``shn_kv_attn_prompt`` (causal attention of packed prompts)
and ``shn_kv_attn_shared`` (attention of single tokens that share a prefix).
"""
import math
import random

import torch

own = False

DEV = "cuda"
# Angles of the rotation: base 10000, positions up to the longest sequence of a case.
ROPE_BASE = 10000.0
EPS = 1e-6


def listed():
    return [
        # one decoding step of a serving batch: every request gets one token, few need a new page
        dict(name="plan_step_256", op="plan", reqs=256, new=256, ctx=4096, page=16),
        # admission of a large batch of prompts on top of what the requests hold already
        dict(name="plan_prompts_1000", op="plan", reqs=1000, new=131072, ctx=300, page=32),
        # the cache write of one decoding step, 32 query and 8 key heads of 128 (the framework's KV cache shape)
        dict(name="store_step_64", op="store", tokens=64, heads=32, kv_heads=8, dim=128, page=16, norm=True, rot=128, pairs=False),
        # a chunk of prompts of the same model, an odd number of tokens
        dict(name="store_prompt_8191", op="store", tokens=8191, heads=32, kv_heads=8, dim=128, page=32, norm=True, rot=128, pairs=False),
        # the rows of one short request, to look at or to move
        dict(name="load_rows_129", op="load", tokens=129, kv_heads=8, dim=128, page=16),
        # a reloaded layer as bf16 for a consumer that has no INT8 path
        dict(name="load_rows_65536", op="load", tokens=65536, kv_heads=8, dim=128, page=64),
        # three short prompts, one of them a single token
        dict(name="prompt_short", op="prompt", reqs=3, new=300, ctx=0, heads=32, kv_heads=8, dim=128, page=16, lens=1),
        # chunks of ragged prompts that hold cached context already, heads of 64, one key head per query head
        dict(name="prompt_chunks_d64", op="prompt", reqs=9, new=5001, ctx=5000, heads=16, kv_heads=16, dim=64, page=32, lens=2),
        # one whole long prompt
        dict(name="prompt_8192", op="prompt", reqs=1, new=8192, ctx=0, heads=32, kv_heads=8, dim=128, page=64, lens=3),
        # a few users on a common system prompt: latency
        dict(name="shared_4", op="shared", reqs=4, prefix=1000, own_tokens=200, heads=32, kv_heads=8, dim=128, page=16, lens=4),
        # many users on one long document, with long tails of their own
        dict(name="shared_128", op="shared", reqs=128, prefix=16384, own_tokens=128000, heads=32, kv_heads=8, dim=128, page=64, lens=5),
        # heads of 64, six query heads to a key head, a prefix that ends inside a page
        dict(name="shared_33_d64", op="shared", reqs=33, prefix=7001, own_tokens=9000, heads=24, kv_heads=4, dim=64, page=32, lens=6),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "store", "load", "prompt", "shared"])
    page = rng.choice([16, 32, 64, 128])
    dim = rng.choice([64, 128, 128])
    kv_heads = rng.choice([1, 2, 4, 8])
    heads = kv_heads * rng.choice([1, 2, 3, 4, 5, 8])
    if op == "plan":
        reqs = _log(rng, 1, 1500)
        return dict(op=op, reqs=reqs, new=_log(rng, reqs, 131072), ctx=_log(rng, 1, 5000), page=page)
    if op == "store":
        rot = rng.choice([0, dim // 2, dim])
        return dict(op=op, tokens=_log(rng, 1, 8000), heads=heads, kv_heads=kv_heads, dim=dim, page=page, norm=rng.random() < 0.6, rot=rot, pairs=rng.random() < 0.4)
    if op == "load":
        return dict(op=op, tokens=_log(rng, 1, 60000), kv_heads=kv_heads, dim=dim, page=page)
    lens = rng.randrange(1 << 20)
    if op == "prompt":
        reqs = _log(rng, 1, 24)
        new = _log(rng, reqs, 2900)
        return dict(op=op, reqs=reqs, new=new, ctx=rng.choice([0, _log(rng, 1, 2900)]), heads=heads, kv_heads=kv_heads, dim=dim, page=page, lens=lens)
    reqs = _log(rng, 1, 128)
    return dict(op=op, reqs=reqs, prefix=_log(rng, 1, 16384), own_tokens=_log(rng, reqs, 500 * reqs + 1), heads=heads, kv_heads=kv_heads, dim=dim, page=page, lens=lens)


def _split(total, parts, least, rng):
    """`total` in `parts` ragged lengths of `least` at the least (parts * least <= total)."""
    cuts = sorted(rng.randint(0, total - parts * least) for _ in range(parts - 1))
    return [b - a + least for a, b in zip([0] + cuts, cuts + [total - parts * least])]


def _lengths(case):
    """(new, context) tokens of each request of an attention case."""
    rng = random.Random(case["lens"])
    if case["op"] == "prompt":
        new = _split(case["new"], case["reqs"], 1, rng)
        ctx = [rng.randint(0, 2 * (case["ctx"] // case["reqs"])) for _ in new]
        return new, ctx
    return [1] * case["reqs"], _split(case["own_tokens"], case["reqs"], 1, rng)


def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _cache(pages, kv_heads, page, dim, g):
    """Pages as the framework's KV caches are made: normal values times a scale per channel, absmax INT8 per head_dim group."""
    def half():
        x = torch.randn(pages, kv_heads, page, dim, generator=g, device=DEV)
        x *= torch.exp(0.5 * torch.randn(kv_heads, 1, dim, generator=g, device=DEV))
        s = x.abs().amax(-1, keepdim=True).clamp_min(1e-30) / 127.0
        return torch.round(x / s).clamp_(-127, 127).to(torch.int8), s.squeeze(-1).contiguous()

    k, ks = half()
    v, vs = half()
    return dict(k=k, v=v, k_scale=ks, v_scale=vs)


def _angles(positions, rot):
    """cos and sin of the rotation, [positions, rot]: the cosines first, then the sines; from 64-bit angles."""
    inv = ROPE_BASE ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)
    a = torch.arange(positions, dtype=torch.float64, device=DEV)[:, None] * inv
    return torch.cat([a.cos(), a.sin()], 1).float()


def _bf16(*shape, g):
    return torch.randn(*shape, generator=g, device=DEV).to(torch.bfloat16)


def _tables(counts, spare, g, shared=0, wide=0):
    """Block tables [len(counts), widest]: `shared` pages in front that all have, then counts[r] pages of its own, in random
    order of a pool with `spare` more; -1 behind them. And the pool's size."""
    own_pages, widest = sum(counts), max(max(counts), wide)
    pool = own_pages + shared + spare
    order = torch.randperm(pool, generator=g, device=DEV).to(torch.int32)
    n = _ints(counts).long()
    j = torch.arange(widest, device=DEV)
    at = (n.cumsum(0) - n)[:, None] + j
    mine = torch.where(j < n[:, None], order[shared:][at.clamp_max(own_pages + spare - 1)], -1)
    return torch.cat([order[:shared].expand(len(counts), shared), mine], 1).contiguous(), pool, order


def prepare(case, seed):
    g = _generator(seed)
    op, page = case["op"], case["page"]
    st = dict(op=op, page=page)
    if op == "plan":
        rng = random.Random(int(seed))
        mean, more = divmod(case["new"], case["reqs"])
        off = [rng.randint(-mean, mean) if mean > 1 else 0 for _ in range(case["reqs"] // 2)]  # two by two around the mean: the total is the case's
        off = [o for pair in off for o in (pair, -pair)] + [0] * (case["reqs"] % 2)
        new = [mean + o + (i < more) for i, o in enumerate(off)]
        ctx = [rng.randint(0, 2 * case["ctx"]) for _ in new]
        held = [-(-c // page) for c in ctx]
        total = [-(-(c + n) // page) for c, n in zip(ctx, new)]
        table, pool, order = _tables(held, sum(total) - sum(held) + 64, g, wide=(2 * (case["ctx"] + mean) + 1) // page + 2)
        free = order[sum(held):].contiguous()
        n, tokens = case["reqs"], case["new"] + 64  # the buffers of a captured step are a little larger than the step
        st.update(ctx=_ints(ctx), new=_ints(new), table=table, free=free, head=_ints([3]), next=_ints([0]), cu=_ints([0] * (n + 1)), kv_len=_ints([0] * n),
                  positions=torch.zeros(tokens, dtype=torch.int32, device=DEV), slots=torch.zeros(tokens, dtype=torch.int32, device=DEV))
    elif op in ("store", "load"):
        tokens, hk, d = case["tokens"], case["kv_heads"], case["dim"]
        pages = -(-tokens // page) + 4
        st.update(slots=torch.randperm(pages * page, generator=g, device=DEV)[:tokens].to(torch.int32))
        if op == "load":
            st.update(_cache(pages, hk, page, d, g), k_out=torch.empty(tokens, hk, d, dtype=torch.bfloat16, device=DEV), v_out=torch.empty(tokens, hk, d, dtype=torch.bfloat16, device=DEV))
        else:
            h, longest = case["heads"], 16384
            qkv = _bf16(tokens, (h + 2 * hk) * d, g=g)  # one projection's output: the three are strided views of it
            q, k, v = (t.unflatten(1, (-1, d)) for t in qkv.split([h * d, hk * d, hk * d], 1))
            st.update(q=q, k=k, v=v, eps=EPS, pairs=case["pairs"], positions=torch.randint(0, longest, (tokens,), generator=g, device=DEV).to(torch.int32),
                      wq=(1 + 0.2 * torch.randn(d, generator=g, device=DEV)).to(torch.bfloat16) if case["norm"] else None,
                      wk=(1 + 0.2 * torch.randn(d, generator=g, device=DEV)).to(torch.bfloat16) if case["norm"] else None,
                      cos_sin=_angles(longest, case["rot"]) if case["rot"] else None,
                      cache_shape=(pages, hk, page, d), q_out=torch.empty(tokens, h, d, dtype=torch.bfloat16, device=DEV),
                      k_out=torch.empty(tokens, hk, d, dtype=torch.bfloat16, device=DEV), v_out=torch.empty(tokens, hk, d, dtype=torch.bfloat16, device=DEV))
    else:
        new, ctx = _lengths(case)
        h, hk, d = case["heads"], case["kv_heads"], case["dim"]
        prefix = case.get("prefix", 0)
        shared = prefix // page  # whole pages of the prefix are everyone's; the rest of it each request has again in a page of its own
        kv = [prefix + c for c in ctx] if op == "shared" else [n + c for n, c in zip(new, ctx)]
        table, pool, order = _tables([-(-x // page) - shared for x in kv], 8, g, shared)
        st.update(_cache(pool, hk, page, d, g), table=table, kv_len=_ints(kv), scale=1.0 / math.sqrt(d), q=_bf16(sum(new), h, d, g=g), out=torch.empty(sum(new), h, d, dtype=torch.bfloat16, device=DEV))
        if op == "shared":
            st.update(prefix_pages=order[:shared].contiguous() if shared else _ints([0]), prefix=shared * page, prefix_len=_ints([shared * page]))
        else:
            cu = [sum(new[:i]) for i in range(len(new) + 1)]
            st.update(cu=_ints(cu), longest=max(new))
    if own:
        from entropy_coded_lossless_b200 import kv as shn_kv

        if op == "store":
            st["cache"] = shn_kv.Cache.empty(*st["cache_shape"], device=DEV)
        elif op != "plan":
            st["cache"] = shn_kv.Cache(st["k"], st["v"], st["k_scale"], st["v_scale"])
        nbytes = shn_kv.attn_shared_workspace_bytes(st["cache"], len(st["kv_len"]), st["q"].shape[1]) if op == "shared" else shn_kv.WORKSPACE_BYTES
        st["work"] = shn_kv.workspace(nbytes, DEV)
    return st


def _run_own(st):
    from entropy_coded_lossless_b200 import kv as shn_kv

    op = st["op"]
    if op == "plan":
        shn_kv.shn_kv_plan(st["ctx"], st["new"], st["page"], st["table"], st["free"], st["head"], st["next"], st["cu"], st["kv_len"], st["positions"], st["slots"], st["work"])
        return st["table"], st["next"], st["cu"], st["kv_len"], st["positions"], st["slots"]
    if op == "store":
        shn_kv.shn_kv_store(st["q"], st["k"], st["v"], st["positions"], st["slots"], st["cache"], st["q_out"], st["work"], q_weight=st["wq"], k_weight=st["wk"], eps=st["eps"],
                            cos_sin=st["cos_sin"], pairs=st["pairs"])
        shn_kv.shn_kv_load(st["cache"], st["slots"], st["k_out"], st["v_out"], st["work"])
        return st["q_out"], st["k_out"], st["v_out"]
    if op == "load":
        shn_kv.shn_kv_load(st["cache"], st["slots"], st["k_out"], st["v_out"], st["work"])
        return st["k_out"], st["v_out"]
    if op == "prompt":
        shn_kv.shn_kv_attn_prompt(st["q"], st["cache"], st["table"], st["cu"], st["kv_len"], st["scale"], st["out"], st["work"])
    else:
        shn_kv.shn_kv_attn_shared(st["q"], st["cache"], st["prefix_pages"], st["prefix_len"], st["table"], st["kv_len"], st["scale"], st["out"], st["work"])
    return st["out"]


def _plan(st):
    ctx, new, page, table = st["ctx"].long(), st["new"].long(), st["page"], st["table"]
    kv_len, held = ctx + new, (ctx + page - 1) // page
    need = (kv_len + page - 1) // page - held
    first = st["head"].long() + need.cumsum(0) - need
    j = torch.arange(table.shape[1], device=DEV)[None] - held[:, None]
    at = (first[:, None] + j).clamp(0, st["free"].numel() - 1)
    table = torch.where((j >= 0) & (j < need[:, None]), st["free"][at], table)
    ends = new.cumsum(0)
    cu = torch.cat([ends.new_zeros(1), ends])
    i = torch.arange(st["slots"].numel(), device=DEV)
    r = torch.searchsorted(ends, i, right=True).clamp_max(ends.numel() - 1)
    real = i < ends[-1]
    position = torch.where(real, ctx[r] + i - cu[r], 0)
    slot = torch.where(real, table[r, position // page].long() * page + position % page, -1)
    return table, (st["head"] + need.sum()).int(), cu.int(), kv_len.int(), position.int(), slot.int()


def _rotated(x, cos_sin, positions, pairs):
    """x [tokens, heads, dim] with its first dimensions rotated: (i, i + rot/2), or with `pairs` (2i, 2i + 1)."""
    rot = cos_sin.shape[1]
    c, s = cos_sin[positions.long()][:, None].split(rot // 2, -1)
    a, b = (x[..., :rot:2], x[..., 1:rot:2]) if pairs else (x[..., :rot // 2], x[..., rot // 2:rot])
    u, w = a * c - b * s, b * c + a * s
    return torch.cat([torch.stack([u, w], -1).flatten(-2) if pairs else torch.cat([u, w], -1), x[..., rot:]], -1)


def _normed(x, w, eps):
    return x if w is None else x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * w.float()


def _quantised(x):
    """The values that absmax INT8 of each row stands for."""
    s = x.abs().amax(-1, keepdim=True).clamp_min(1e-30) / 127.0
    return torch.round(x / s).clamp(-127, 127) * s


def _store(st):
    q, k = _normed(st["q"].float(), st["wq"], st["eps"]), _normed(st["k"].float(), st["wk"], st["eps"])
    if st["cos_sin"] is not None:
        q, k = (_rotated(x, st["cos_sin"], st["positions"], st["pairs"]) for x in (q, k))
    return q, _quantised(k), _quantised(st["v"].float())


def _load(st):
    s = st["slots"].long()
    p, t = s // st["page"], s % st["page"]
    return tuple((st[n][p, :, t].float() * st[n + "_scale"][p, :, t][..., None]).bfloat16() for n in ("k", "v"))


def _pages(st, name, pages):
    """Pages [..., n] of the cache as values [..., kv_heads, n * page_tokens, dim] in 32 bits (page -1: any page, masked later)."""
    at = pages.clamp_min(0).long()
    x = st[name][at].float() * st[name + "_scale"][at][..., None]
    return x.transpose(-4, -3).flatten(-3, -2)


def _weights(s, seen):
    """Softmax over the last axis of the scores that are seen, in place; a row that sees nothing has weights of zero."""
    s.masked_fill_(~seen, -math.inf)
    s.sub_(s.amax(-1, keepdim=True).clamp_min(-3e38)).exp_()
    return s.div_(s.sum(-1, keepdim=True).clamp_min(1e-30))


def _prompt(st):
    cu, kv_len, q = st["cu"].long(), st["kv_len"].long(), st["q"]
    n, h, d = q.shape
    new = cu[1:] - cu[:-1]
    i = torch.arange(st["longest"], device=DEV)
    at = (cu[:-1, None] + i).clamp_max(n - 1)
    k, v = (_pages(st, x, st["table"]) for x in ("k", "v"))
    b, hk, t, _ = k.shape
    x = q[at].float().reshape(b, -1, hk, h // hk, d).permute(0, 2, 3, 1, 4).flatten(2, 3)
    s = (x * st["scale"]) @ k.transpose(-1, -2)
    seen = torch.arange(t, device=DEV) <= (kv_len - new)[:, None, None] + i[:, None]
    o = _weights(s.view(b, hk, h // hk, -1, t), seen[:, None, None]).view(b, hk, -1, t) @ v
    o = o.view(b, hk, h // hk, -1, d).permute(0, 3, 1, 2, 4).reshape(b, -1, h, d)
    r = torch.searchsorted(cu[1:], torch.arange(n, device=DEV), right=True)
    return o[r, torch.arange(n, device=DEV) - cu[r]].bfloat16()


def _shared(st):
    q, kv_len, prefix = st["q"], st["kv_len"].long(), st["prefix"]
    b, h, d = q.shape
    first = prefix // st["page"]
    kp, vp = (_pages(st, x, st["prefix_pages"])[:, :prefix] for x in ("k", "v"))
    k, v = (_pages(st, x, st["table"][:, first:]) for x in ("k", "v"))
    hk, t = k.shape[1:3]
    x = q.float().view(b, hk, h // hk, d) * st["scale"]
    s = torch.cat([(x.transpose(0, 1).flatten(1, 2) @ kp.transpose(-1, -2)).view(hk, b, h // hk, prefix).transpose(0, 1), x @ k.transpose(-1, -2)], -1)
    seen = torch.arange(prefix + t, device=DEV) < kv_len[:, None, None, None]
    w = _weights(s, seen)
    o = (w[..., :prefix].transpose(0, 1).flatten(1, 2) @ vp).view(hk, b, h // hk, d).transpose(0, 1) + w[..., prefix:] @ v
    return o.reshape(b, h, d).bfloat16()


def run(st):
    if own:
        return _run_own(st)
    op = st["op"]
    if op == "plan":
        return _plan(st)
    if op == "store":
        return tuple(x.bfloat16() for x in _store(st))
    if op == "load":
        return _load(st)
    return _prompt(st) if op == "prompt" else _shared(st)


def work(case):
    op = case["op"]
    if op == "plan":
        pages = case["new"] / case["page"] + (case["reqs"] / 2 if case["new"] > case["reqs"] else 0)
        return dict(bytes=8 * case["reqs"] + 8 * pages + 8 * (case["new"] + 64) + 4 * (2 * case["reqs"] + 1), flops=0)
    hk, d = case["kv_heads"], case["dim"]
    row = 2 * hk * (d + 4)  # a token's keys and values in the cache with their scales
    if op == "load":
        return dict(bytes=case["tokens"] * (row + 4 * hk * d + 4), flops=case["tokens"] * 2 * hk * d)
    h = case["heads"]
    if op == "store":
        return dict(bytes=case["tokens"] * (4 * h * d + 8 * hk * d + row + 8 + 4 * case["rot"]), flops=case["tokens"] * 10 * (h + 2 * hk) * d)
    new, ctx = _lengths(case)
    if op == "prompt":
        seen = sum(n * c + n * (n + 1) // 2 for n, c in zip(new, ctx))
        cached = sum(new) + sum(ctx)
    else:
        shared = case["prefix"] // case["page"] * case["page"]
        seen = sum(case["prefix"] + c for c in ctx)
        cached = shared + sum(case["prefix"] - shared + c for c in ctx)
    return dict(bytes=cached * row + 4 * sum(new) * h * d + 4 * cached / case["page"], flops=4 * h * d * seen)


def exact(case, seed):
    """The operators from their definitions in 64 bits, one request and one head after another."""
    st = prepare(case, seed)
    op, page = st["op"], st["page"]
    if op == "plan":
        return None
    if op == "load":
        at = st["slots"].long()
        return tuple(st[n].transpose(1, 2).flatten(0, 1)[at].double() * st[n + "_scale"].transpose(1, 2).flatten(0, 1)[at].double()[..., None] for n in ("k", "v"))
    if op == "store":
        turn = None
        if case["rot"]:
            half = case["rot"] // 2
            table = st["cos_sin"].double()[st["positions"].long()]
            turn = torch.complex(table[:, :half], table[:, half:])[:, None]  # the rotation as a product of complex numbers
        found = []
        for x, w in ((st["q"], st["wq"]), (st["k"], st["wk"])):
            x = x.double()
            if w is not None:
                x = x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * w.double()
            if turn is not None:
                z = x[..., :2 * half].unflatten(-1, (half, 2) if case["pairs"] else (2, half))
                z = torch.view_as_real(torch.complex(*z.unbind(-1 if case["pairs"] else -2)) * turn)
                x = torch.cat([(z if case["pairs"] else z.transpose(-1, -2)).flatten(-2), x[..., 2 * half:]], -1)
            found.append(x)
        found.append(st["v"].double())
        for i in (1, 2):
            step = torch.linalg.vector_norm(found[i], math.inf, -1, keepdim=True).clamp_min(1e-30) / 127
            found[i] = (found[i] / step).round() * step
        return tuple(found)
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device=DEV)
    group = case["heads"] // case["kv_heads"]
    new, ctx = _lengths(case)
    at = 0
    for r, n in enumerate(new):
        length = int(st["kv_len"][r])
        pages = st["table"][r, : -(-length // page)].long()
        for h in range(case["kv_heads"]):
            k, v = ((st[x][pages, h].double() * st[x + "_scale"][pages, h].double()[..., None]).reshape(-1, case["dim"])[:length] for x in ("k", "v"))
            for j in range(h * group, (h + 1) * group):
                s = st["q"][at:at + n, j].double() @ k.T * st["scale"]
                if n > 1:
                    s += torch.full_like(s, -math.inf).triu(length - n + 1)
                out[at:at + n, j] = torch.softmax(s, -1) @ v
        at += n
    return out
