"""How far the attention calls may be off, as include/shn_kv.h says it: per query and head, against 64 bits,

    |out - exact| <= (r + score and sum errors) sum_j w_j |v_j|  +  (n f + 2^-24) vmax  +  2^-8 |exact|

with n the tokens the query sees and vmax = 127 times the largest value scale among them.

r: roundings to fp16, 2^-11 each. Prompts and large prefixes round a weight, its token's value scale and the product of that with the
INT8 value (r = 3 2^-11); single tokens only the product of weight and value scale (r = 2^-11).
f: fp16 ends at 2^-24, half a step of which is 2^-25. A weight enters as P = p 2^(e - E) with p <= 1 at the sequence's largest, its
value as v 2^-e below 254, and E is 6 below the exponent of the largest value scale that the query has seen: 2^-25 2^E 254 <=
2^-30 vmax a token, against a sum of weights of at least 1. (Single tokens: E is 5 below, and values enter as their integers, so that
127 stands for 254: the same.)
2^-24: a value scale relative to the largest of 32 tokens enters as fp16, too, off by at most 2^-25.
A score is a float32 sum of dim products (at most (dim + 8) 2^-24 of the sum of their magnitudes), which changes a weight's share by at
most twice that; sums over n tokens add (2 n + 64) 2^-24, which covers the exponential's 2^-22. The result is rounded to bfloat16,
2^-8 of itself.
"""
import math

import pytest
import torch

from entropy_coded_lossless_b200 import build as shn_build

shn_build.build()
from entropy_coded_lossless_b200 import kv, shn  # noqa: E402
from tests import test_gpu_kv as base  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    shn.lib()


PROMPT, SINGLE = 3 * 2.0**-11, 2.0**-11  # r


def exact(q, cache, slots_of, seen_of, scale, rounded=PROMPT, f=2.0**-30):
    """(result, tolerance) of queries q [rows, heads, dim]; row i sees the first seen_of[i] of the tokens at slots_of(i) (rows
    with the same slots object are done together)."""
    n, h, d = q.shape
    hk, pt = cache.kv_heads, cache.page_tokens
    out, tol = (torch.zeros(n, h, d, dtype=torch.float64, device=DEV) for _ in range(2))
    groups = {}
    for i in range(n):
        groups.setdefault(id(slots_of(i)), []).append(i)
    for rows in groups.values():
        sl = slots_of(rows[0]).long()
        at = torch.tensor(rows, device=DEV)
        seen = torch.tensor([seen_of[i] for i in rows], device=DEV)
        mask = torch.arange(len(sl), device=DEV)[None] >= seen[:, None]
        for head in range(h):
            k8, v8 = (getattr(cache, x)[sl // pt, head * hk // h, sl % pt].double() for x in ("k", "v"))
            ks, vs = (getattr(cache, x)[sl // pt, head * hk // h, sl % pt].double()[:, None] for x in ("k_scale", "v_scale"))
            k, v, x = k8 * ks, v8 * vs, q[at, head].double()
            s = (x @ k.T * scale).masked_fill(mask, -math.inf)
            w = torch.where(seen[:, None] > 0, torch.softmax(s, -1), torch.zeros_like(s))
            o = w @ v
            size = (x.abs() @ k.abs().T * abs(scale)).masked_fill(mask, 0.0).amax(-1, keepdim=True)
            vmax = 127 * vs.abs().T.expand(len(rows), -1).masked_fill(mask, 0.0).amax(-1, keepdim=True)
            rel = rounded * (1 + 2.0**-9) + 2 * (d + 8) * 2.0**-24 * size + (2 * seen[:, None] + 64) * 2.0**-24
            out[at, head] = o
            tol[at, head] = rel * (w @ v.abs()) + (seen[:, None] * f + 2.0**-24) * vmax + 2.0**-8 * o.abs() + 1e-35
    return out, tol


def check(out, ref, tol):
    bad = ~((out.double() - ref).abs() <= tol)
    assert not bad.any(), (bad.sum().item(), bad.nonzero()[:4].tolist(), out[bad][:4], ref[bad][:4], tol[bad][:4])


def prompt(cache, table, new, kv_lens, h, d, seed, scale, q=None):
    cu = [sum(new[:i]) for i in range(len(new) + 1)]
    q = base.bf16(cu[-1], h, d, seed=seed) if q is None else q
    out, w = torch.empty_like(q), base.work()
    kv.shn_kv_attn_prompt(q, cache, table, base.ints(cu), base.ints(kv_lens), scale, out, w)
    assert base.status(w) == (0, 0)
    slots = [base.spec.token_slots(table[r], cache.page_tokens, n) for r, n in enumerate(kv_lens)]
    owner = [r for r, n in enumerate(new) for _ in range(n)]
    seen = [max(0, kv_lens[r] - n + i + 1) for r, n in enumerate(new) for i in range(n)]
    check(out, *exact(q, cache, lambda i: slots[owner[i]], seen, scale))


def shared(cache, table, kv_lens, prefix, h, d, seed, scale, q=None, rounded=PROMPT, f=2.0**-30):
    """The prefix in the first pages of the longest request's row; a token is read from there below it, else from its own row."""
    pt, n = cache.page_tokens, len(kv_lens)
    front = table[max(range(n), key=lambda r: kv_lens[r]), :-(-prefix // pt)].contiguous()
    q = base.bf16(n, h, d, seed=seed) if q is None else q
    out, w = torch.empty_like(q), base.work(kv.attn_shared_workspace_bytes(cache, n, h))
    kv.shn_kv_attn_shared(q, cache, front if prefix else None, base.ints([prefix]), table, base.ints(kv_lens), scale, out, w)
    assert base.status(w) == (0, 0)
    slots = []
    for r, length in enumerate(kv_lens):
        sl = base.spec.token_slots(table[r], pt, length)
        m = min(prefix, length)
        sl[:m] = base.spec.token_slots(front, pt, m) if m else sl[:0]
        slots.append(sl)
    check(out, *exact(q, cache, lambda i: slots[i], kv_lens, scale, rounded, f))


def bounds(h, hk, n):
    """(rounded, f) of single tokens: these batches' prefixes go to the tensor cores from 65 groups of 8 (16) query rows on."""
    rows = 8 if h // hk <= 8 else 16
    return (PROMPT, 2.0**-30) if n * (h // hk) > 64 * rows else (SINGLE, 2.0**-30)


# (h, hk, new, kv_lens): one whose row tiles share their tokens among blocks, and one with more row tiles than SMs
FEW, MANY = (6, 2, [150, 3, 40], [1600, 3, 300]), (16, 16, [700, 900, 33], [700, 1200, 33])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [1, 2, 3, 8])
def test_few_tokens_whose_values_cancel(n, d):
    """Between few tokens of opposite values the results are small beside what they are made of: a rounding of the weights to
    bfloat16, or one more to fp16 for single tokens, would show."""
    pt, h, hk = 16, 16, 2
    table, pages = base.tables([n] * 60, pt, 1)
    cache = base.filled_cache(pages, hk, pt, d, seed=2)
    cache.v[:, :, 1::2] = -cache.v[:, :, ::2]  # a token and its opposite
    q = base.bf16(60 * n, h, d, seed=3)
    prompt(cache, table, [n] * 60, [n] * 60, h, d, 0, 0.002, q)
    shared(cache, table, [n] * 60, 0, h, d, 0, 0.002, q[:60], SINGLE, 2.0**-30)
    many = base.bf16(4000, h, d, seed=4)
    prompt(cache, table[:40], [100] * 40, [n] * 40, h, d, 0, 0.002, many)  # (most rows see nothing)


@pytest.mark.parametrize("h,hk,new,kv_lens", [FEW, MANY])
@pytest.mark.parametrize("d", [64, 128])
def test_prompts(h, hk, new, kv_lens, d):
    table, pages = base.tables(kv_lens, 32, 5)
    cache = base.filled_cache(pages, hk, 32, d, seed=6)
    prompt(cache, table, new, kv_lens, h, d, 7, 1 / math.sqrt(d))


@pytest.mark.parametrize("h,hk,n,prefix", [(8, 2, 5, 0), (8, 2, 5, 700), (32, 2, 70, 1500), (16, 1, 9, 300), (64, 1, 3, 64)])
@pytest.mark.parametrize("d", [64, 128])
def test_single_tokens(h, hk, n, prefix, d):
    lens = [prefix + 1 + r * 53 % 400 for r in range(n)]
    table, pages = base.tables(lens, 32, 5)
    cache = base.filled_cache(pages, hk, 32, d, seed=6)
    shared(cache, table, lens, prefix, h, d, 7, 1 / math.sqrt(d), None, *bounds(h, hk, n))


def one_strong_key(cache, table, n, at, d, nats):
    """Queries of ones; token `at` has the score `nats` and the others 0. Its values are zeros in the first half of the dimensions."""
    pt = cache.page_tokens
    cache.k.zero_(), cache.k_scale.fill_(nats / (127 * d))
    p, t = table[0, at // pt].item(), at % pt
    cache.k[p, :, t] = 127
    cache.v.fill_(127), cache.v_scale.fill_(1 / 127)
    cache.v[p, :, t, :d // 2] = 0


@pytest.mark.parametrize("log2_weight", [20, 24, 26, 29])
@pytest.mark.parametrize("d", [64, 128])
def test_many_weak_tokens_beside_a_strong_one(d, log2_weight):
    """Weights far below the strongest add up: 65,536 of 2^-26 are 2^-10 of the result, and all of it in half the dimensions."""
    n, pt, hk, h = 65536, 64, 1, 2
    table, pages = base.tables([n], pt, 1)
    cache = base.filled_cache(pages, hk, pt, d, seed=2)
    one_strong_key(cache, table, n, 5, d, log2_weight * math.log(2))
    q = torch.ones(300, h, d, dtype=torch.bfloat16, device=DEV)
    prompt(cache, table, [3], [n], h, d, 0, 1.0, q[:3])
    shared(cache, table, [n], 0, h, d, 0, 1.0, q[:1])
    both = table.repeat(300, 1)
    shared(cache, both, [n] * 300, n, h, d, 0, 1.0, q)  # (a large prefix of many rows)
    prompt(cache, both[:148], [2] * 148, [3000] * 148, h, d, 0, 1.0, q[:296])
    prompt(cache, both[:160], [1] * 160, [3000] * 160, h, d, 0, 1.0, q[:160])


@pytest.mark.parametrize("small", [0.3, 0.05, 1e-4, 1e-7, 1e-12, 1e-20])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("h,hk,new,kv_lens", [FEW, MANY, (4, 1, [40], [40])])
def test_tokens_that_a_row_does_not_see_do_not_touch_it(h, hk, new, kv_lens, d, small):
    """The first tokens of each sequence (and some at the border of what the queries see) have values far smaller than those behind
    them: a row that sees only these is as exact as if the others were not there."""
    pt = 16
    table, pages = base.tables(kv_lens, pt, 5)
    for first in (1, 13, 40, 70):
        cache = base.filled_cache(pages, hk, pt, d, seed=6)
        for r, n in enumerate(kv_lens):
            sl = base.spec.token_slots(table[r], pt, n)
            cut = max(first, n - new[r] + first)  # the row that sees so many tokens sees the small ones only
            for s in sl[:cut].tolist():
                cache.v_scale[s // pt, :, s % pt] *= small
        prompt(cache, table, new, kv_lens, h, d, 7, 1 / math.sqrt(d))


@pytest.mark.parametrize("small", [1e-4, 1e-7, 1e-12, 1e-20])
@pytest.mark.parametrize("h,hk,n,prefix", [(8, 2, 5, 700), (16, 1, 6, 300), (64, 1, 4, 90), (32, 2, 70, 1500)])
@pytest.mark.parametrize("d", [64, 128])
def test_tokens_of_a_prefix_that_a_request_does_not_see(h, hk, n, prefix, d, small):
    """Requests shorter than the prefix, whose later tokens have far larger values."""
    pt, cut = 16, prefix // 2 + 5
    lens = [prefix + 20 if r % 3 == 0 else cut - r % 7 for r in range(n)]
    table, pages = base.tables(lens, pt, 5)
    cache = base.filled_cache(pages, hk, pt, d, seed=6)
    for s in base.spec.token_slots(table[0], pt, cut).tolist():
        cache.v_scale[s // pt, :, s % pt] *= small
    shared(cache, table, lens, prefix, h, d, 7, 1 / math.sqrt(d), None, *bounds(h, hk, n))


@pytest.mark.parametrize("d", [64, 128])
def test_error_in_the_mean(d, monkeypatch):
    """Over many results the error is the result's own rounding to bfloat16 and the roundings to fp16, at most three for each token.
    These are independent of each other and across tokens, uniform within half a step of 2^-10 or less: at most 2^-11 / sqrt(3) of a
    token's part each, so that their squares add up to at most 2^-22 of the sum of the parts' squares, which for values of random
    signs is the result's. (Weights in bfloat16 would add 64 times that; 1.05: the sample's spread.)"""
    seen = []

    def mean(out, ref, tol):
        own = (ref.to(torch.bfloat16).double() - ref).norm() / ref.norm()
        seen.append((((out.double() - ref).norm() / ref.norm()).item(), own.item()))

    monkeypatch.setitem(globals(), "check", mean)
    pt, hk, h = 32, 16, 16
    for new, kv_lens in (([300, 40], [1500, 300]), ([900, 700], [900, 1000])):
        table, pages = base.tables(kv_lens, pt, 5)
        prompt(base.filled_cache(pages, hk, pt, d, seed=6), table, new, kv_lens, h, d, 7, 1 / math.sqrt(d))
    for h, hk, n, prefix in ((32, 8, 9, 700), (32, 2, 70, 1500)):
        lens = [prefix + 1 + r * 53 % 400 for r in range(n)]
        table, pages = base.tables(lens, pt, 5)
        shared(base.filled_cache(pages, hk, pt, d, seed=6), table, lens, prefix, h, d, 7, 1 / math.sqrt(d))
    assert len(seen) == 4
    for err, own in seen:
        assert err <= 1.05 * math.sqrt(own**2 + 2.0**-22), seen
