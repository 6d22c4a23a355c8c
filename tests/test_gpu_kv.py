"""The paged KV cache operators (include/shn_kv.h) against their definitions in 64 bits (kv_spec)."""
import math
import random

import pytest
import torch

from entropy_coded_lossless_b200 import build as shn_build

shn_build.build()  # the binding is an extension module: it is there before it is imported
from entropy_coded_lossless_b200 import kv, shn  # noqa: E402
from tests import kv_spec as spec  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16_HALF = 2.0**-8  # torch.finfo(torch.bfloat16).eps / 2


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    shn.lib()


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def work(n=kv.WORKSPACE_BYTES):
    w = shn.empty_aligned(n, DEV)
    w.fill_(0x5A)  # a workspace needs no preparation
    return w


def status(w):
    return shn.shn_get_device_status(w)


def filled_cache(pages, hk, pt, d, seed=0, scales=None):
    g = gen(seed)
    k, v = (torch.randint(-127, 128, (pages, hk, pt, d), generator=g, device=DEV).to(torch.int8) for _ in range(2))
    ks, vs = (torch.exp(0.5 * torch.randn(pages, hk, pt, generator=g, device=DEV)) / 90 for _ in range(2))
    if scales is not None:
        vs *= scales
    return kv.Cache(k, v, ks, vs)


def bf16(*shape, seed=0):
    return torch.randn(*shape, generator=gen(seed), device=DEV).to(torch.bfloat16)


# ---- plan ------------------------------------------------------------------------------------------


def plan_buffers(n, max_tokens):
    z = lambda m: torch.full((m,), -7, dtype=torch.int32, device=DEV)  # noqa: E731
    return z(1), z(n + 1), z(n), z(max_tokens), z(max_tokens)


@pytest.mark.parametrize("n,pt,mean,most,pad", [(1, 16, 1, 1, 0), (1, 32, 0, 5000, 3), (7, 16, 40, 50, 100), (300, 64, 200, 9, 1), (1023, 16, 10, 2, 5),
                                                (1025, 32, 33, 40, 64), (2500, 16, 3, 3, 0), (40, 1024, 3000, 3000, 11)])
def test_plan(n, pt, mean, most, pad):
    rng = random.Random(n * pt)
    ctx = [rng.choice([0, rng.randint(0, 2 * mean), pt, pt - 1, pt + 1]) for _ in range(n)]
    new = [rng.choice([0, 1, rng.randint(0, most)]) for _ in range(n)]
    width = max(-(-(c + m) // pt) for c, m in zip(ctx, new)) + 1
    held = [-(-c // pt) for c in ctx]
    need = sum(-(-(c + m) // pt) for c, m in zip(ctx, new)) - sum(held)
    pool = list(range(sum(held) + need + 5))
    rng.shuffle(pool)
    table, at = [], 0
    for h in held:
        table.append(pool[at:at + h] + [-1] * (width - h))
        at += h
    free, head = [999_999, 999_998] + pool[at:], 2  # the first two are taken already
    tokens = sum(new) + pad
    expect = spec.plan(ctx, new, pt, table, free, head, tokens)
    t, w = ints(table), work()
    nxt, cu, kv_len, pos, slots = plan_buffers(n, tokens)
    kv.shn_kv_plan(ints(ctx), ints(new), pt, t, ints(free), ints([head]), nxt, cu, kv_len, pos, slots, w)
    assert status(w) == (0, 0)
    assert (t.tolist(), nxt.item(), cu.tolist(), kv_len.tolist(), pos.tolist(), slots.tolist()) == expect


def test_plan_head_in_place_over_steps():
    """The head updated in place, step after step: every token keeps a slot of its own."""
    n, pt = 5, 16
    table, free, head, ctx = ints([[-1] * 8] * n), ints(list(range(40))[::-1]), ints([0]), ints([0] * n)
    seen, w = set(), work()
    for step in range(12):
        new = ints([step % 3, 1, 7 * (step % 2), 0, 2])
        _, cu, kv_len, pos, slots = plan_buffers(n, 24)
        kv.shn_kv_plan(ctx, new, pt, table, free, head, head, cu, kv_len, pos, slots, w)
        assert status(w) == (0, 0)
        total = int(cu[-1])
        mine = slots[:total].tolist()
        assert not seen & set(mine) and len(set(mine)) == total and min(mine, default=0) >= 0
        assert slots[total:].tolist() == [-1] * (24 - total)
        seen |= set(mine)
        ctx = kv_len
    assert head.item() == sum(-(-c // pt) for c in ctx.tolist())


@pytest.mark.parametrize("what,code", [("tokens", shn.SHN_ERR_CAPACITY), ("blocks", shn.SHN_ERR_CAPACITY), ("pages", shn.SHN_ERR_CAPACITY),
                                       ("negative", shn.SHN_ERR_INVALID_ARG), ("head", shn.SHN_ERR_INVALID_ARG), ("huge", shn.SHN_ERR_INVALID_ARG)])
def test_plan_refuses_and_takes_nothing(what, code):
    ctx, new = [5, 0, 40], [3, 20, 30]
    if what == "negative":
        new[1] = -1
    if what == "huge":
        ctx[1], new[1] = 2**31 - 1, 2**31 - 1
    table = [[9, -1, -1, -1, -1], [-1] * 5, [8, 7, 6, -1, -1]]
    if what == "blocks":
        table = [r[:4] for r in table]
    t, w = ints(table), work()
    free = ints([0, 1] if what == "pages" else [0, 1, 2, 3, 4, 5])
    head = ints([7 if what == "head" else 0])
    nxt, cu, kv_len, pos, slots = plan_buffers(3, 40 if what == "tokens" else 64)
    kv.shn_kv_plan(ints(ctx), ints(new), 16, t, free, head, nxt, cu, kv_len, pos, slots, w)
    st, detail = status(w)
    assert st == code
    if what in ("negative", "huge", "blocks"):
        assert detail == (2 if what == "blocks" else 1)
    assert t.tolist() == table and nxt.item() == head.item()
    assert set(cu.tolist()) == {0} and set(kv_len.tolist()) == {0} and set(pos.tolist()) == {0} and set(slots.tolist()) == {-1}


def test_plan_reports_a_bad_page():
    w = work()
    nxt, cu, kv_len, pos, slots = plan_buffers(2, 8)
    t = ints([[-5, -1], [3, -1]])
    kv.shn_kv_plan(ints([4, 14]), ints([2, 4]), 16, t, ints([2**31 - 1]), ints([0]), nxt, cu, kv_len, pos, slots, w)
    assert status(w)[0] == shn.SHN_ERR_INVALID_ARG
    assert slots.tolist() == [-1, -1, 3 * 16 + 14, 3 * 16 + 15, -1, -1, -1, -1]


@pytest.mark.parametrize("n,new", [(40, 100), (1500, 3)])
def test_plan_of_many_tokens_reports_the_first_bad_page(n, new):
    """Pages that are begun and pages from the list, those of a request that takes no token aside; the head in place or not."""
    pt = 16
    ctx = [5 if r % 3 else 0 for r in range(n)]
    fresh = [new if r % 5 else 0 for r in range(n)]
    pages = [-(-(c + m) // pt) - -(-c // pt) for c, m in zip(ctx, fresh)]
    begun = [r for r in range(n) if ctx[r] and fresh[r]]
    takes = [r for r in range(n) if pages[r]]
    far = (2**31 - 1) // pt
    width = max(pages) + 1
    for bad_begun, bad_new in ((begun[3], None), (None, takes[1]), (None, takes[-1]), (begun[-1], takes[2]), (begun[1], takes[-2]), (None, None)):
        for in_place in (False, True):
            table = [[r] + [-1] * (width - 1) if c else [-1] * width for r, c in enumerate(ctx)]
            table[5][0] = -3  # (request 5 takes no token)
            if bad_begun is not None:
                table[bad_begun][0] = -2
            free = [n + i for i in range(sum(pages) + 2)]
            if bad_new is not None:
                free[1 + sum(pages[:bad_new])] = far
            nxt, cu, kv_len, pos, slots = plan_buffers(n, sum(fresh) + 9)
            head, w = ints([1]), work()
            kv.shn_kv_plan(ints(ctx), ints(fresh), pt, ints(table), ints(free), head, head if in_place else nxt, cu, kv_len, pos, slots, w)
            bad = [r for r in (bad_begun, bad_new) if r is not None]
            assert status(w) == ((shn.SHN_ERR_INVALID_ARG, min(bad)) if bad else (0, 0))
            assert (head if in_place else nxt).item() == 1 + sum(pages)
            none = sum(min(fresh[r], pt - ctx[r]) for r in bad[:1] if r == bad_begun) + sum(
                min(pt, fresh[r] - (pt - ctx[r]) % pt) for r in bad if r == bad_new)
            assert (slots[:sum(fresh)] < 0).sum().item() == none


def test_plan_of_nothing():
    w = work()
    e = ints([])
    nxt, cu, kv_len, pos, slots = plan_buffers(0, 3)
    kv.shn_kv_plan(e, e, 16, e.view(0, 4), e, ints([0]), nxt, cu, kv_len, pos, slots, w)
    assert status(w) == (0, 0) and cu.tolist() == [0] and slots.tolist() == [-1] * 3 and nxt.item() == 0


# ---- store and load --------------------------------------------------------------------------------


def angles(n, rot, seed):
    a = torch.rand(n, rot // 2, generator=gen(seed), device=DEV) * 6.3
    return torch.cat([a.cos(), a.sin()], 1)


@pytest.mark.parametrize("tokens,h,hk,d,pt,norm,rot,pairs", [
    (1, 32, 8, 128, 16, True, 128, False), (37, 8, 8, 128, 32, False, 128, True), (130, 6, 2, 64, 64, True, 32, False), (5, 5, 1, 64, 16, True, 64, True),
    (64, 16, 4, 128, 1024, True, 0, False), (300, 3, 3, 128, 128, False, 16, False), (9, 0, 7, 64, 16, True, 48, True), (2, 64, 1, 128, 16, False, 0, False),
])
def test_store_and_load(tokens, h, hk, d, pt, norm, rot, pairs):
    pages = -(-tokens // pt) + 3
    cache = filled_cache(pages, hk, pt, d, seed=1)
    before = [t.clone() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)]
    qkv = bf16(tokens, (h + 2 * hk) * d + 24, seed=2) * 3  # rows with a tail that belongs to something else
    q, k, v = (qkv[:, a * d:b * d].unflatten(1, (b - a, d)) for a, b in ((0, h), (h, h + hk), (h + hk, h + 2 * hk)))
    slots = torch.randperm(pages * pt, generator=gen(3), device=DEV)[:tokens].to(torch.int32)
    if tokens > 4:
        slots[tokens // 2] = -1
    positions = torch.randint(0, 500, (tokens,), generator=gen(4), device=DEV).to(torch.int32)
    wq, wk = ((1 + 0.3 * torch.randn(d, generator=gen(s), device=DEV)).to(torch.bfloat16) if norm else None for s in (5, 6))
    cs = angles(500, rot, 7) if rot else None
    out, w = torch.full((tokens, h + 1, d), 7.0, dtype=torch.bfloat16, device=DEV), work()
    kv.shn_kv_store(q if h else None, k, v, positions if rot else None, slots, cache, out[:, :h] if h else None, w, q_weight=wq, k_weight=wk, eps=1e-5, cos_sin=cs,
                    pairs=pairs)
    assert status(w) == (0, 0)
    assert (out[:, h] == 7.0).all()

    def near(x, weight, y):
        """float32 error of y: the norm's sum over d and a handful of roundings, of the row's size."""
        return (d + 16) * 2.0**-24 * 2 * y.abs().amax(-1, keepdim=True)

    if h:
        y = spec.normed_rotated(q, wq, 1e-5, cs, positions, pairs)
        assert ((out[:, :h].double() - y).abs() <= BF16_HALF * y.abs() + near(q, wq, y)).all()
    real = slots >= 0
    for name, src, y in (("k", k, spec.normed_rotated(k, wk, 1e-5, cs, positions, pairs)), ("v", v, v.double())):
        y = y[real]
        p, t = slots[real].long() // pt, slots[real].long() % pt
        got, s = getattr(cache, name)[p, :, t].double(), getattr(cache, name + "_scale")[p, :, t].double()
        want = y.abs().amax(-1) / 127
        e = near(src, wk, y) if name == "k" else 0 * near(src, wk, y)
        assert ((s - want).abs() <= want * 2.0**-23 + e[..., 0] / 127).all()
        # the integer is the nearest to y / s: off by half a step, by the error of y and by the division's rounding
        assert ((got * s[..., None] - y).abs() <= 0.5 * s[..., None] * (1 + 2.0**-14) + e).all()
        assert got.abs().max() == 127
    # everything else in the cache is as it was
    mask = torch.ones(pages, pt, dtype=torch.bool, device=DEV)
    mask[slots[real].long() // pt, slots[real].long() % pt] = False
    for now, was in zip((cache.k, cache.v, cache.k_scale, cache.v_scale), before):
        assert torch.equal(now.transpose(1, 2)[mask], was.transpose(1, 2)[mask])
    # load: bit for bit the product rounded once
    ko, vo = (torch.full((tokens, hk, d), 5.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    kv.shn_kv_load(cache, slots, ko, vo, w)
    assert status(w) == (0, 0)
    for name, o in (("k", ko), ("v", vo)):
        p, t = slots[real].long() // pt, slots[real].long() % pt
        ref = (getattr(cache, name)[p, :, t].float() * getattr(cache, name + "_scale")[p, :, t][..., None]).to(torch.bfloat16)
        assert torch.equal(o[real].view(torch.int16), ref.view(torch.int16))
        assert (o[~real] == 5.0).all()


def test_store_query_in_place_and_odd_rows():
    """A zero row, a row with an infinity, one with a NaN, one of the smallest values; the query in place."""
    hk, d, pt = 2, 128, 16
    cache = filled_cache(2, hk, pt, d)
    k = bf16(4, hk, d, seed=1)
    k[0], k[1, 0, 5], k[2, 1, 9], k[3] = 0, math.inf, math.nan, 2.0**-120
    q = bf16(4, 4, d, seed=2)
    was = q.clone()
    w = work()
    kv.shn_kv_store(q, k, k, None, ints([3, 4, 5, 6]), cache, q, w)
    assert status(w) == (0, 0)
    assert torch.equal(q, was)  # neither norm nor rotation: the same values
    for name in ("k", "v"):
        x, s = getattr(cache, name)[0, :, 3:7], getattr(cache, name + "_scale")[0, :, 3:7]
        assert (x[:, 0] == 0).all() and (s[:, 0] == torch.tensor(1e-30, device=DEV) / 127).all()
        assert s[0, 1] == math.inf and torch.isfinite(s[1, 1]) and torch.isnan(s[1, 2]) and torch.isfinite(s[0, 2])
        assert torch.isnan(x[1, 2].float() * s[1, 2]).all()  # a poisoned row reads as NaN
        assert not torch.isfinite(x[0, 1].float() * s[0, 1]).any()
        assert (s[:, 3] == torch.tensor(1e-30, device=DEV) / 127).all() and (x[:, 3] == 0).all()  # 2^-120 < 1e-30 / 254


def test_load_repeats_and_one_side():
    cache = filled_cache(3, 2, 16, 64)
    slots = ints([5, 5, 47, 0, 5])
    ko, w = torch.zeros(5, 2, 64, dtype=torch.bfloat16, device=DEV), work()
    kv.shn_kv_load(cache, slots, ko, None, w)
    assert status(w) == (0, 0)
    ref = spec.rows_of(cache, slots, "k").float().to(torch.bfloat16)
    assert torch.equal(ko, ref)
    vo = torch.zeros(5, 3, 64, dtype=torch.bfloat16, device=DEV)[:, :2]
    kv.shn_kv_load(cache, slots, None, vo, w)
    assert torch.equal(vo, spec.rows_of(cache, slots, "v").float().to(torch.bfloat16))


def test_store_and_load_report_bad_slots_and_positions():
    cache = filled_cache(2, 2, 16, 64)
    was = [t.clone() for t in (cache.k, cache.k_scale)]
    q, k, w = bf16(3, 4, 64, seed=1), bf16(3, 2, 64, seed=2), work()
    out = torch.full((3, 4, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    kv.shn_kv_store(q, k, k, None, ints([-1, 32, -1]), cache, out, w)
    assert status(w) == (shn.SHN_ERR_INVALID_ARG, 1)
    assert (out[1] == 7.0).all() and torch.equal(out[0], q[0]) and torch.equal(out[2], q[2])
    cs = angles(10, 64, 1)
    for bad in (-1, 10):
        kv.shn_kv_store(q, k, k, ints([0, 0, bad]), ints([-1, -1, 4]), cache, out, w, cos_sin=cs)
        assert status(w) == (shn.SHN_ERR_INVALID_ARG, 2)
    assert torch.equal(cache.k, was[0]) and torch.equal(cache.k_scale, was[1])
    ko = torch.full((2, 2, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    kv.shn_kv_load(cache, ints([2**31 - 1, 1]), ko, None, w)
    assert status(w) == (shn.SHN_ERR_INVALID_ARG, 0)
    assert (ko[0] == 7.0).all() and torch.equal(ko[1], spec.rows_of(cache, ints([1]), "k").float().to(torch.bfloat16)[0])
    kv.shn_kv_load(cache, ints([1]), ko[:1], None, w)
    assert status(w) == (0, 0)  # every call clears the word


@pytest.mark.parametrize("n", [1, 2, 3, 5, 255, 1030, 8191, 8192, 8197, 40000])
def test_a_bad_index_anywhere_is_reported(n):
    """Slots and positions that start at any place within 16 bytes, bad ones at both ends and between. Of several bad ones a
    call of up to 8192 tokens reports the first."""
    cache = filled_cache(2, 1, 16, 64)
    k, w, cs = bf16(n, 1, 64, seed=n), work(), angles(6, 64, 1)
    out, none = torch.zeros_like(k), torch.full((n,), -1, dtype=torch.int32, device=DEV)
    was = cache.k.clone()
    for lead in range(4):
        slots, positions = (torch.zeros(lead + n, dtype=torch.int32, device=DEV)[lead:] for _ in range(2))
        slots -= 1
        for at in sorted({0, n // 2, n - 1}):
            last = n - 1 if n <= 8192 else at  # the later one is bad as well
            slots[at], slots[last] = 32, 33
            kv.shn_kv_load(cache, slots, out, None, w)
            assert status(w) == (shn.SHN_ERR_INVALID_ARG, at)
            kv.shn_kv_store(None, k, k, positions, slots, cache, None, w, cos_sin=cs)
            assert status(w) == (shn.SHN_ERR_INVALID_ARG, at)
            slots[at] = slots[last] = -1
            positions[at], positions[last] = -1, 6
            kv.shn_kv_store(None, k, k, positions, none, cache, None, w, cos_sin=cs)
            assert status(w) == (shn.SHN_ERR_INVALID_ARG, at)
            positions[at] = positions[last] = 0
        kv.shn_kv_store(None, k, k, positions, slots, cache, None, w, cos_sin=cs)
        assert status(w) == (0, 0)
    assert torch.equal(cache.k, was) and not out.any()


# ---- attention -------------------------------------------------------------------------------------


def tables(kv_lens, pt, seed, extra=0):
    """A random block table for these lengths; -1 behind a row's pages."""
    counts = [-(-n // pt) for n in kv_lens]
    order = torch.randperm(sum(counts) + 2, generator=gen(seed), device=DEV).to(torch.int32)
    table = torch.full((len(kv_lens), max(counts + [1]) + extra), -1, dtype=torch.int32, device=DEV)
    at = 0
    for r, c in enumerate(counts):
        table[r, :c] = order[at:at + c]
        at += c
    return table, sum(counts) + 2


def run_prompt(cache, table, new, kv_lens, h, d, seed, scale=None, padding=0, strided=False):
    cu = [sum(new[:i]) for i in range(len(new) + 1)]
    n = cu[-1] + padding
    if strided:
        q = bf16(n, h + 3, d, seed=seed)[:, 2:2 + h]
        out = torch.full((n, h + 1, d), 7.0, dtype=torch.bfloat16, device=DEV)[:, :h]
    else:
        q, out = bf16(n, h, d, seed=seed), torch.full((n, h, d), 7.0, dtype=torch.bfloat16, device=DEV)
    w = work()
    scale = 1 / math.sqrt(d) if scale is None else scale
    kv.shn_kv_attn_prompt(q, cache, table, ints(cu), ints(kv_lens), scale, out, w)
    assert status(w) == (0, 0)
    assert (out[cu[-1]:] == 7.0).all()
    ref, tol = spec.cache_attention(q[:cu[-1]], cache, lambda r: table[r], [max(0, x) for x in kv_lens], cu, scale)
    bad = ~((out[:cu[-1]].double() - ref).abs() <= tol)
    assert not bad.any(), (bad.sum().item(), bad.nonzero()[:4].tolist(), out[:cu[-1]][bad][:4], ref[bad][:4], tol[bad][:4])
    return out


@pytest.mark.parametrize("h,hk,d,pt,new,ctx", [
    (8, 2, 128, 16, [1], [0]),
    (4, 4, 128, 32, [1, 127, 128, 129, 0, 3], [0, 0, 0, 0, 9, 0]),
    (32, 8, 128, 16, [300, 77, 1], [0, 5, 130]),
    (6, 2, 64, 64, [65, 64, 63, 257], [1, 1000, 64, 0]),
    (5, 1, 64, 16, [200, 31], [17, 0]),
    (16, 1, 128, 128, [33, 2, 2, 50], [0, 700, 1, 127]),
    (64, 1, 64, 1024, [9, 30], [1500, 0]),
    (7, 7, 128, 16, [513], [511]),
    (2, 1, 64, 16, [1000, 1], [0, 2000]),
])
def test_prompt(h, hk, d, pt, new, ctx):
    kv_lens = [n + c for n, c in zip(new, ctx)]
    table, pages = tables(kv_lens, pt, 3, extra=1)
    cache = filled_cache(pages, hk, pt, d, seed=4)
    run_prompt(cache, table, new, kv_lens, h, d, seed=5, padding=2)
    run_prompt(cache, table, new, kv_lens, h, d, seed=6, scale=0.5, strided=True)  # a sharper softmax


@pytest.mark.parametrize("n", [32, 33, 900, 1800])
def test_prompt_of_many_requests(n):
    """As many requests as a warp has lanes, one more, more than a block has threads and two for each of them."""
    rng = random.Random(n)
    new = [rng.choice([0, 1, 2, 5]) for _ in range(n)]
    kv_lens = [m + rng.choice([0, 0, 3, 40]) for m in new]
    table, pages = tables(kv_lens, 16, 1)
    cache = filled_cache(pages, 1, 16, 64, seed=2)
    run_prompt(cache, table, new, kv_lens, 2, 64, seed=3, padding=1)


def test_prompt_rows_that_see_nothing():
    """More queries than tokens: the first ones see nothing and are zero; a request without tokens; padding requests."""
    new, kv_lens = [40, 5, 0, 0, 150], [10, 0, 0, 7, 149]
    table, pages = tables(kv_lens, 16, 1)
    cache = filled_cache(pages, 2, 16, 128, seed=2)
    out = run_prompt(cache, table, new, kv_lens, 4, 128, seed=3)
    assert (out[:30] == 0).all() and (out[30] != 0).any() and (out[40:45] == 0).all() and (out[45] == 0).all() and (out[46] != 0).any()


@pytest.mark.parametrize("d", [64, 128])
def test_attention_masked_places_hold_anything(d):
    """Tokens behind a sequence's end, in its last page and in pages that are nobody's, hold NaN and infinite scales, and
    a later token of the sequence an infinite value: no query that does not see them is touched."""
    new, kv_lens, pt, hk, h = [200, 21], [200, 150], 32, 2, 4
    table, pages = tables(kv_lens, pt, 8, extra=2)
    table[0, 7:] = 2**31 - 1  # behind the pages a row needs anything may stand
    cache = filled_cache(pages, hk, pt, d, seed=9)
    clean = run_prompt(cache, table, new, kv_lens, h, d, seed=5)
    used = torch.zeros(pages * pt, dtype=torch.bool, device=DEV)
    for r, n in enumerate(kv_lens):
        used[spec.token_slots(table[r], pt, n)] = True
    for s, x in ((cache.k_scale, math.nan), (cache.v_scale, math.inf)):
        s.transpose(1, 2).reshape(-1, hk)  # a view check only
        flat = s.permute(0, 2, 1).reshape(-1, hk).clone()
        flat[~used] = x
        s.copy_(flat.view(pages, pt, hk).permute(0, 2, 1))
    last = spec.token_slots(table[0], pt, 200)[199].item()
    cache.v_scale[last // pt, :, last % pt] = math.inf
    cache.k_scale[last // pt, :, last % pt] = math.nan
    q, out, w = bf16(221, h, d, seed=5), torch.zeros(221, h, d, dtype=torch.bfloat16, device=DEV), work()
    kv.shn_kv_attn_prompt(q, cache, table, ints([0, 200, 221]), ints(kv_lens), 1 / math.sqrt(d), out, w)
    assert status(w) == (0, 0)
    assert torch.equal(out[:199], clean[:199]) and torch.equal(out[200:], clean[200:])
    assert torch.isnan(out[199]).all()
    one, w = torch.zeros(2, h, d, dtype=torch.bfloat16, device=DEV), work(kv.attn_shared_workspace_bytes(cache, 2, h))
    kv.shn_kv_attn_shared(q[:2], cache, None, ints([0]), table, ints([199, 150]), 1 / math.sqrt(d), one, w)
    assert status(w) == (0, 0) and torch.isfinite(one).all()


@pytest.mark.parametrize("d", [64, 128])
def test_attention_extreme_scores(d):
    """Scores far apart (one key takes all), very large and very negative ones, and maxima that rise along the sequence."""
    pt, hk, h, n = 16, 1, 2, 700
    table, pages = tables([n], pt, 1)
    cache = filled_cache(pages, hk, pt, d, seed=2)
    flat = torch.linspace(0.001, 6.0, pages * pt, device=DEV)
    order = spec.token_slots(table[0], pt, n)
    ks = torch.ones(pages * pt, device=DEV)
    ks[order] = flat[:n]
    cache.k_scale.copy_(ks.view(pages, hk, pt))
    run_prompt(cache, table, [n], [n], h, d, seed=3)
    ks[order] = flat[:n].flip(0)
    cache.k_scale.copy_(ks.view(pages, hk, pt))
    run_prompt(cache, table, [60], [n], h, d, seed=4)
    run_shared(cache, table, [n], 0, h, d, seed=4)


@pytest.mark.parametrize("h,hk,d,pt,new,ctx", [
    (2, 1, 64, 16, [1], [511]),  # a few tiles: two parts
    (2, 1, 128, 16, [1], [640]),
    (8, 1, 128, 64, [1], [2900]),  # 8 parts of 2 or 3 tiles
    (5, 1, 64, 128, [3, 1, 0], [3000, 0, 700]),  # short requests beside a long one: parts without tiles
    (4, 4, 128, 1024, [9], [2040]),  # parts that begin inside a page
    (12, 3, 64, 32, [70, 130], [1500, 900]),  # rows of several blocks, the last one odd
    (32, 8, 128, 16, [7], [1283]),
    (16, 2, 64, 64, [400], [1000]),  # the causal end lies in several parts
    (1, 1, 128, 32, [300], [500]),
    (64, 1, 64, 16, [5], [1200]),
])
def test_prompt_of_few_rows(h, hk, d, pt, new, ctx):
    """Few rows and many tokens: the tokens are shared by several blocks."""
    kv_lens = [n + c for n, c in zip(new, ctx)]
    table, pages = tables(kv_lens, pt, 3, extra=1)
    cache = filled_cache(pages, hk, pt, d, seed=4)
    run_prompt(cache, table, new, kv_lens, h, d, seed=5, padding=2)
    run_prompt(cache, table, new, kv_lens, h, d, seed=6, scale=0.5, strided=True)
    # value scales that grow and fall along the sequence: the parts hold their sums in different ranges
    grow = torch.logspace(-9, 9, cache.v_scale.numel(), device=DEV).view_as(cache.v_scale)
    cache.v_scale *= grow
    run_prompt(cache, table, new, kv_lens, h, d, seed=7)
    cache.v_scale /= grow * grow
    run_prompt(cache, table, new, kv_lens, h, d, seed=8)


@pytest.mark.parametrize("d", [64, 128])
def test_prompt_of_few_rows_masked_and_empty(d):
    """Rows that see no token, or none of the later parts, and what masked places of those hold; wide tables of short
    requests; a bad page in a later part; all of it captured and replayed."""
    new, kv_lens, pt, hk, h = [20, 1], [1024, 9], 32, 1, 4
    table, pages = tables(kv_lens, pt, 8, extra=2)
    cache = filled_cache(pages, hk, pt, d, seed=9)
    clean, scale = run_prompt(cache, table, new, kv_lens, h, d, seed=5), 1 / math.sqrt(d)
    last = spec.token_slots(table[0], pt, 1024)[1010:].tolist()
    for x in last:
        cache.v_scale[x // pt, :, x % pt] = math.inf
        cache.k_scale[x // pt, :, x % pt] = math.nan
    q, out, w = bf16(21, h, d, seed=5), torch.zeros(21, h, d, dtype=torch.bfloat16, device=DEV), work()
    args = (q, cache, table, ints([0, 20, 21]), ints(kv_lens), scale, out, w)
    kv.shn_kv_attn_prompt(*args)
    assert status(w) == (0, 0)
    # Weights enter fp16 times a power of two that the value scales of 32 tokens give, masked ones among them: below fp16's
    # normal numbers a weight's rounding depends on it, by no more than the tolerance's part for lost weights.
    ref, tol = spec.cache_attention(q, filled_cache(pages, hk, pt, d, seed=9), lambda r: table[r], kv_lens, [0, 20, 21], scale)
    assert ((out[:6].double() - ref[:6]).abs() <= tol[:6]).all() and torch.isnan(out[6:20]).all() and torch.equal(out[20], clean[20])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kv.shn_kv_attn_prompt(*args)
    first = out.clone()
    out.zero_()
    graph.replay()
    assert torch.equal(out.view(torch.int16), first.view(torch.int16))
    run_prompt(filled_cache(pages, hk, pt, d, seed=9), table, [1100, 1], [1024, 9], 1, d, seed=2)  # 76 rows see nothing
    table[0, 30] = pages
    kv.shn_kv_attn_prompt(*args)
    assert status(w) == (shn.SHN_ERR_INVALID_ARG, 0) and torch.equal(out[20], clean[20])


def test_prompt_far_slots():
    """A cache whose bytes pass 2^32: pages at its end are read where they are."""
    hk, pt, d = 8, 64, 128
    pages = (1 << 32) // (hk * pt * d) + 300
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB")
    k, v = (torch.zeros(pages, hk, pt, d, dtype=torch.int8, device=DEV) for _ in range(2))
    ks, vs = (torch.ones(pages, hk, pt, device=DEV) / 100 for _ in range(2))
    cache = kv.Cache(k, v, ks, vs)
    tail = torch.arange(pages - 6, pages, dtype=torch.int32, device=DEV)
    for x in (k, v):
        x[-6:] = torch.randint(-127, 128, (6, hk, pt, d), generator=gen(1), device=DEV).to(torch.int8)
    table = tail.flip(0).view(1, 6).contiguous()
    run_prompt(cache, table, [130], [380], 16, d, seed=2)
    run_shared(cache, table, [380], 200, 16, d, seed=2)
    slots = (tail[-1:] * pt + pt - 1).to(torch.int32)
    ko, vo, w = *(torch.zeros(1, hk, d, dtype=torch.bfloat16, device=DEV) for _ in range(2)), work()
    kv.shn_kv_store(None, bf16(1, hk, d, seed=3), bf16(1, hk, d, seed=4), None, slots, cache, None, w)
    kv.shn_kv_load(cache, slots, ko, vo, w)
    assert status(w) == (0, 0)
    assert torch.equal(ko, spec.rows_of(cache, slots, "k").float().to(torch.bfloat16)) and ko.abs().max() > 0


def run_shared(cache, table, kv_lens, prefix, h, d, seed, scale=None, strided=False, n_prefix=None):
    b = len(kv_lens)
    pt = cache.page_tokens
    blocks = -(-prefix // pt) if n_prefix is None else n_prefix
    longest = max(range(b), key=lambda r: kv_lens[r])
    pages = table[longest, :blocks].contiguous()  # its first pages are the prefix's
    if strided:
        q, out = bf16(b, h + 3, d, seed=seed)[:, 2:2 + h], torch.full((b, h + 1, d), 7.0, dtype=torch.bfloat16, device=DEV)[:, :h]
    else:
        q, out = bf16(b, h, d, seed=seed), torch.full((b, h, d), 7.0, dtype=torch.bfloat16, device=DEV)
    scale = 1 / math.sqrt(d) if scale is None else scale
    w = work(kv.attn_shared_workspace_bytes(cache, b, h))
    kv.shn_kv_attn_shared(q, cache, pages if blocks else None, ints([prefix]), table, ints(kv_lens), scale, out, w)
    assert status(w) == (0, 0)

    ref, tol = spec.cache_attention(q, cache, lambda r: table[r], kv_lens, list(range(b + 1)), scale, (pages, prefix))
    bad = ~((out.double() - ref).abs() <= tol)
    assert not bad.any(), (bad.sum().item(), bad.nonzero()[:4].tolist(), out[bad][:4], ref[bad][:4], tol[bad][:4])
    return out


def shared_tables(own, prefix, pt, seed):
    """Block tables of requests that share `prefix` tokens (whole pages) and hold own[r] more."""
    front = prefix // pt
    table, pages = tables([n + 1 for n in own] or [1], pt, seed)
    shared = torch.randperm(front, generator=gen(seed + 1), device=DEV).to(torch.int32) + pages
    return torch.cat([shared.expand(len(own), front), table], 1).contiguous(), pages + front


@pytest.mark.parametrize("h,hk,d,pt,prefix,own", [
    (8, 2, 128, 16, 0, [1]),
    (8, 2, 128, 16, 0, [0, 1, 700, 64, 65]),
    (8, 2, 128, 16, 0, [n % 50 for n in range(20)]),
    (32, 8, 128, 16, 1008, [3, 200, 0, 17]),
    (4, 4, 64, 32, 64, [1, 2, 3, 300, 31, 33]),
    (24, 4, 64, 32, 4096, [n * 7 % 300 for n in range(33)]),
    (16, 1, 128, 64, 5056, [n * 13 % 900 for n in range(40)]),
    (64, 1, 128, 16, 480, [5, 100, 0]),
    (5, 1, 64, 128, 2048, [9] * 70),
    (40, 8, 128, 1024, 3 * 1024, [1, 1025]),
    (2, 2, 128, 16, 16, [0] * 3),
    (12, 4, 128, 16, 320, [n % 50 for n in range(300)]),
])
def test_shared(h, hk, d, pt, prefix, own):
    table, pages = shared_tables(own, prefix, pt, 3)
    cache = filled_cache(pages, hk, pt, d, seed=4)
    kv_lens = [prefix + n for n in own]
    run_shared(cache, table, kv_lens, prefix, h, d, seed=5)
    run_shared(cache, table, kv_lens, prefix, h, d, seed=6, scale=0.4, strided=True, n_prefix=prefix // pt + 1)


def test_shared_prefix_inside_a_page_and_shorter_requests():
    """A prefix that ends inside a page (the rest of it in the requests' own rows), requests shorter than the prefix and empty ones."""
    pt, hk, h, d = 32, 2, 8, 128
    own = [500, 480, 490, 477, 333, 12, 0, 40]
    table, pages = tables(own, pt, 5)
    cache = filled_cache(pages, hk, pt, d, seed=6)
    for prefix in (1, 31, 33, 335, 476):
        # only whole requests share: those shorter than the prefix read its pages up to their length
        out = run_shared(cache, table, own, prefix, h, d, seed=prefix)
        assert (out[6] == 0).all()


@pytest.mark.parametrize("d,pt,prefix", [(128, 32, 1), (64, 32, 127), (128, 32, 129), (64, 16, 1000), (128, 1024, 3000), (64, 1024, 2049)])
def test_shared_prefix_of_many_rows(d, pt, prefix):
    """Over a thousand query rows to a key head (the tensor core kernel, in parts that may begin inside a long page): a prefix that
    ends inside a page or a tile, requests shorter than it, empty ones, and one part without a token."""
    hk, h, n = 2, 32, 70
    rng = random.Random(prefix)
    own = [rng.choice([0, prefix // 3, prefix, prefix + rng.randint(1, 300)]) for _ in range(n)]
    own[3], own[4] = prefix + 310, 0
    table, pages = tables(own, pt, 5)
    cache = filled_cache(pages, hk, pt, d, seed=6)
    out = run_shared(cache, table, own, prefix, h, d, seed=prefix)
    assert (out[4] == 0).all()
    run_shared(cache, table, own, prefix, h, d, seed=prefix + 1, scale=0.5, strided=True)


@pytest.mark.parametrize("n", [4, 70])
def test_shared_prefix_with_scales_that_are_not_finite(n):
    """Infinite and NaN value scales: in tokens of the prefix that only the longer requests see, and behind everyone's end."""
    hk, h, d, pt, prefix = 2, 32, 128, 32, 300
    own = [prefix + 5 if r % 2 else 200 for r in range(n)]
    table, pages = tables(own, pt, 5)
    cache = filled_cache(pages, hk, pt, d, seed=6)
    clean = run_shared(cache, table, own, prefix, h, d, seed=1)
    long = next(r for r in range(n) if own[r] > prefix)
    for t in (250, 299):  # behind the short ones' end
        s = spec.token_slots(table[long], pt, 300)[t].item()
        cache.v_scale[s // pt, :, s % pt] = math.inf if t == 250 else math.nan
    for r in range(n):
        last = own[r] % pt
        cache.v_scale[table[r, own[r] // pt].item(), :, last] = math.nan  # behind the end, in the last page
    q, out, w = bf16(n, h, d, seed=1), torch.zeros(n, h, d, dtype=torch.bfloat16, device=DEV), work(kv.attn_shared_workspace_bytes(cache, n, h))
    kv.shn_kv_attn_shared(q, cache, table[long, :10].contiguous(), ints([prefix]), table, ints(own), 1 / math.sqrt(d), out, w)
    assert status(w) == (0, 0)
    for r in range(n):
        if own[r] < prefix:
            assert torch.equal(out[r], clean[r])
        else:
            assert not torch.isfinite(out[r].float()).any()


def test_shared_bad_pages_of_a_prefix_of_many_rows():
    hk, h, d, pt, n, prefix = 2, 32, 128, 32, 70, 320
    own = [prefix + 3] * n
    table, pages = tables(own, pt, 5)
    cache = filled_cache(pages, hk, pt, d, seed=6)
    q, out, w = bf16(n, h, d, seed=1), torch.zeros(n, h, d, dtype=torch.bfloat16, device=DEV), work(kv.attn_shared_workspace_bytes(cache, n, h))
    for bad in (-1, pages, 2**31 - 1):
        front = table[0, :10].clone()
        front[4] = bad
        kv.shn_kv_attn_shared(q, cache, front, ints([prefix]), table, ints(own), 0.1, out, w)
        assert status(w)[0] == shn.SHN_ERR_INVALID_ARG and torch.isfinite(out.float()).all()
    kv.shn_kv_attn_shared(q, cache, table[0, :10].contiguous(), ints([prefix]), table, ints(own), 0.1, out, w)
    assert status(w) == (0, 0)


def test_shared_equals_prompt_of_one_token():
    own = [77, 1, 260]
    table, pages = tables(own, 16, 1)
    cache = filled_cache(pages, 2, 16, 128, seed=2)
    a = run_shared(cache, table, own, 0, 8, 128, seed=3)
    b = run_prompt(cache, table, [1, 1, 1], own, 8, 128, seed=3)
    assert (a.double() - b.double()).abs().max() <= 2 * BF16_HALF * a.double().abs().max()


def test_attention_reports_bad_pages_and_lengths():
    d, hk, h, pt = 128, 2, 4, 16
    table, pages = tables([40, 50], pt, 1)
    cache = filled_cache(pages, hk, pt, d, seed=2)
    q = bf16(3, h, d, seed=3)
    out = torch.full((3, h, d), 7.0, dtype=torch.bfloat16, device=DEV)
    w = work(kv.attn_shared_workspace_bytes(cache, 2, h))

    def prompt(table, cu, lens):
        out.fill_(7.0)
        kv.shn_kv_attn_prompt(q, cache, table, ints(cu), ints(lens), 0.1, out, w)
        return status(w)

    def shared(table, lens, prefix, n):
        out.fill_(7.0)
        kv.shn_kv_attn_shared(q[:2], cache, prefix, ints([n]), table, ints(lens), 0.1, out[:2], w)
        return status(w)

    assert prompt(table, [0, 1, 3], [40, 50])[0] == 0
    good = out.clone()
    for bad_page in (-1, pages, 2**31 - 1):
        bad = table.clone()
        bad[1, 1] = bad_page
        assert prompt(bad, [0, 1, 3], [40, 50]) == (shn.SHN_ERR_INVALID_ARG, 1)
        assert torch.equal(out[0], good[0]) and torch.isfinite(out.float()).all()
        assert shared(bad, [40, 50], None, 0) == (shn.SHN_ERR_INVALID_ARG, 1)
        assert torch.isfinite(out[:2].float()).all()
        assert shared(table, [40, 50], bad[1, :3].contiguous(), 48)[0] == shn.SHN_ERR_INVALID_ARG
        assert torch.isfinite(out[:2].float()).all()
    assert prompt(table, [0, 1, 3], [40, 16 * table.shape[1] + 1]) == (shn.SHN_ERR_INVALID_ARG, 1)
    assert prompt(table, [0, 1, 3], [-3, 50]) == (shn.SHN_ERR_INVALID_ARG, 0)
    assert (out[0] == 0).all() and torch.equal(out[1:], good[1:])
    assert prompt(table, [0, 1, 4], [40, 50])[0] == shn.SHN_ERR_INVALID_ARG
    assert torch.equal(out[0], good[0]) and (out[1:] == 7.0).all()
    assert prompt(table, [0, -1, 3], [40, 50])[0] == shn.SHN_ERR_INVALID_ARG
    assert (out == 7.0).all()
    assert shared(table, [40, 16 * table.shape[1] + 1], None, 0) == (shn.SHN_ERR_INVALID_ARG, 1)
    assert shared(table, [40, 50], table[1, :2].contiguous(), 33)[0] == shn.SHN_ERR_INVALID_ARG
    assert shared(table, [40, 50], None, -1)[0] == shn.SHN_ERR_INVALID_ARG
    assert shared(table, [40, 50], None, 0)[0] == 0


# ---- together --------------------------------------------------------------------------------------


def test_plan_store_attend_compress_and_decode_together():
    """A prompt step and decoding steps of a small batch as a server runs them: plan, store, attention; then the pages
    through the codec into another cache, which gives the same bits."""
    hk, h, d, pt, pages, n = 2, 8, 128, 16, 60, 3
    cache = kv.Cache.empty(pages, hk, pt, d, device=DEV)
    table, head, free = ints([[-1] * 12] * n), ints([0]), torch.randperm(pages, generator=gen(1), device=DEV).to(torch.int32)
    cs, wq = angles(512, d, 2), torch.ones(d, dtype=torch.bfloat16, device=DEV)
    ctx, w = ints([0] * n), work()
    ws = work(kv.attn_shared_workspace_bytes(cache, n, h))
    scale = 1 / math.sqrt(d)
    for step, new in enumerate([[100, 33, 1], [1, 1, 1], [1, 0, 1], [1, 1, 1]]):
        tokens = 140 if step == 0 else n
        _, cu, kv_len, pos, slots = plan_buffers(n, tokens)
        kv.shn_kv_plan(ctx, ints(new), pt, table, free, head, head, cu, kv_len, pos, slots, w)
        q, k, v = bf16(tokens, h, d, seed=step), bf16(tokens, hk, d, seed=10 + step), bf16(tokens, hk, d, seed=20 + step)
        qo, out = torch.empty_like(q), torch.zeros_like(q)
        kv.shn_kv_store(q, k, v, pos, slots, cache, qo, w, q_weight=wq, k_weight=wq, cos_sin=cs)
        kv.shn_kv_attn_prompt(qo, cache, table, cu, kv_len, scale, out, w)
        assert status(w) == (0, 0)
        total = sum(new)
        ref, tol = spec.cache_attention(qo[:total], cache, lambda r: table[r], kv_len.tolist(), cu.tolist(), scale)
        assert ((out[:total].double() - ref).abs() <= tol).all() and (out[total:] == 0).all()
        ctx = kv_len
    # the filled pages, compressed and decoded into another cache
    taken = sorted(free[:head.item()].tolist())
    p = shn.CodecParams(16, 7, 1024, 4)
    codec = shn.Codec(cache.segments(taken), p)
    other = kv.Cache.empty(pages, hk, pt, d, device=DEV)
    bytes_per_page = hk * pt * d
    for x, y in ((cache.k, other.k), (cache.v, other.v)):
        codec.compress(x.view(-1))
        assert codec.status("enc")[0] == 0
        flat = torch.empty(len(taken) * bytes_per_page, dtype=torch.uint8, device=DEV)
        codec.decode(codec.stream_buf, int(codec.out_bytes.item()), flat)
        assert codec.status("dec")[0] == 0
        y[taken] = flat.view(torch.int8).view(len(taken), hk, pt, d)
    other.k_scale.copy_(cache.k_scale), other.v_scale.copy_(cache.v_scale)
    q = bf16(n, h, d, seed=99)
    a, b = torch.empty_like(q), torch.empty_like(q)
    for c, o in ((cache, a), (other, b)):
        kv.shn_kv_attn_shared(q, c, None, ints([0]), table, ctx, scale, o, ws)
        assert status(ws) == (0, 0)
    assert torch.equal(a, b)
    # the same values as the codec's own fused dequantisation gives
    codec.compress(cache.k.view(-1))
    vals = torch.empty(len(taken) * bytes_per_page, dtype=torch.bfloat16, device=DEV)
    scales = cache.k_scale[taken].reshape(-1).contiguous()
    shn.shn_decode_bf16(codec.stream_buf, int(codec.out_bytes.item()), p, scales, cache.log2_group, codec.work_dec, vals)
    assert codec.status("dec")[0] == 0
    ko = torch.empty(len(taken) * pt, hk, d, dtype=torch.bfloat16, device=DEV)
    slots = (ints(taken)[:, None] * pt + torch.arange(pt, device=DEV)).flatten().to(torch.int32)
    kv.shn_kv_load(cache, slots, ko, None, w)
    assert torch.equal(ko.view(len(taken), pt, hk, d).transpose(1, 2).reshape(-1), vals)


def test_captured_step_follows_its_inputs():
    """plan, store, prompt and shared attention captured once; replayed with other lengths it gives what separate
    calls give, and a second graph has a workspace of its own."""
    hk, h, d, pt, n, pages = 2, 8, 64, 16, 4, 200
    cache = filled_cache(pages, hk, pt, d, seed=1)
    tokens = 64
    ctx, new, table, head = ints([0] * n), ints([1] * n), ints([[-1] * 40] * n), ints([0])
    free = torch.randperm(pages, generator=gen(2), device=DEV).to(torch.int32)
    nxt, cu, kv_len, pos, slots = plan_buffers(n, tokens)
    q, k, v = bf16(tokens, h, d, seed=3), bf16(tokens, hk, d, seed=4), bf16(tokens, hk, d, seed=5)
    out, one = torch.zeros_like(q), torch.zeros(n, h, d, dtype=torch.bfloat16, device=DEV)
    plen = ints([0])
    w = work(kv.attn_shared_workspace_bytes(cache, n, h))

    def step(w):
        kv.shn_kv_plan(ctx, new, pt, table, free, head, nxt, cu, kv_len, pos, slots, w)
        kv.shn_kv_store(None, k, v, None, slots, cache, None, w)
        kv.shn_kv_attn_prompt(q, cache, table, cu, kv_len, 0.1, out, w)
        kv.shn_kv_attn_shared(q[:n], cache, None, plen, table, kv_len, 0.1, one, w)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(w)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(w)
    for c, m in (([0] * 4, [30, 1, 0, 20]), ([5, 100, 16, 31], [1, 1, 1, 1]), ([0, 0, 0, 0], [0, 0, 0, 0]), ([200, 3, 90, 0], [7, 40, 2, 15])):
        table.fill_(-1)
        for r, x in enumerate(c):
            table[r, :-(-x // pt)] = torch.arange(-(-x // pt), dtype=torch.int32, device=DEV) + 40 * r
        free.copy_(torch.arange(160, 160 + pages, device=DEV).to(torch.int32) % pages)
        ctx.copy_(ints(c)), new.copy_(ints(m)), out.fill_(7.0), one.fill_(7.0)
        graph.replay()
        assert status(w) == (0, 0)
        got = [t.clone() for t in (out, one, cache.k, slots, kv_len)]
        out.fill_(7.0), one.fill_(7.0)
        step(work(w.numel()))
        for x, y in zip(got, (out, one, cache.k, slots, kv_len)):
            assert torch.equal(x, y)
        total = sum(m)
        assert (out[total:] == 7.0).all()
        ref, tol = spec.cache_attention(q[:total], cache, lambda r: table[r], kv_len.tolist(), cu.tolist(), 0.1)
        assert ((out[:total].double() - ref).abs() <= tol).all()


def test_two_streams_at_once_and_same_bits():
    """Calls on two streams at the same time, each with its own workspace, and repeated calls: the same bits."""
    own = [300, 1200, 40, 777]
    table, pages = tables(own, 32, 1)
    cache = filled_cache(pages, 4, 32, 128, seed=2)
    q = bf16(4, 16, 128, seed=3)
    nbytes = kv.attn_shared_workspace_bytes(cache, 4, 16)
    first = torch.empty_like(q)
    kv.shn_kv_attn_shared(q, cache, None, ints([0]), table, ints(own), 0.1, first, work(nbytes))
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs, works = [[torch.empty_like(q) for _ in range(8)] for _ in streams], [work(nbytes) for _ in streams]
    plen, lens = ints([0]), ints(own)
    torch.cuda.synchronize()
    for i in range(8):
        for s, o, w in zip(streams, outs, works):
            kv.shn_kv_attn_shared(q, cache, None, plen, table, lens, 0.1, o[i], w, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(x, first) for o in outs for x in o)


def test_binding_refuses():
    cache = filled_cache(4, 2, 16, 128)
    q, w = bf16(2, 4, 128), work(kv.attn_shared_workspace_bytes(cache, 2, 4))
    t, one = ints([[0, 1], [2, 3]]), ints([16, 16])
    out = torch.empty_like(q)
    ok = dict(q=q, cache=cache, prefix_pages=None, prefix_len=ints([0]), block_table=t, kv_len=one, scale=0.1, out=out, work=w)
    kv.shn_kv_attn_shared(**ok)
    for bad in (dict(q=q.half()), dict(q=q[:, :3]), dict(q=q[:1]), dict(out=out[:, :2]), dict(kv_len=one.long()), dict(block_table=t[:1]), dict(q=q.cpu()),
                dict(prefix_len=ints([0, 0])), dict(work=w[:256].cpu()), dict(q=q[..., :64]), dict(q=bf16(2, 128, 4).transpose(1, 2))):
        with pytest.raises((ValueError, shn.ShnError)):
            kv.shn_kv_attn_shared(**{**ok, **bad})
    with pytest.raises(shn.ShnError):
        kv.shn_kv_attn_shared(**{**ok, "work": work(256)[:128]})
    with pytest.raises(shn.ShnError):
        kv.Cache.empty(2, 2, 16, 96)
    with pytest.raises(ValueError):
        kv.Cache.empty(2, 2, 20, 64)
    with pytest.raises(ValueError):
        kv.Cache(cache.k, cache.v[:3], cache.k_scale, cache.v_scale)
