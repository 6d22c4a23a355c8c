"""The paged KV cache calls at sizes that fill the GPU: prompts of more row tiles than there are SMs over many tiles of tokens (the
kernel that does not share a row tile's tokens among blocks), and stores and loads in which a block takes several tokens."""
import math
import random

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


def fills_the_gpu(h, hk, new):
    """Row tiles of 256 rows, as many as these prompts can have: more than SMs, or the calls take another kernel."""
    tiles = (sum(new) * (h // hk) // 256 + min(len(new), sum(new))) * hk
    assert tiles > torch.cuda.get_device_properties(0).multi_processor_count


LONG = [
    (16, 16, 64, 32, [700, 900, 33, 1, 256], [0, 300, 2000, 5, 0]),
    (16, 8, 64, 16, [1500, 1, 700], [0, 900, 131]),
    (64, 1, 64, 128, [600, 77], [100, 640]),
    (12, 4, 64, 1024, [1300, 1100, 900, 80], [0, 1, 1023, 3000]),
    (16, 16, 128, 64, [700, 850, 40, 129], [0, 257, 1500, 0]),
    (32, 8, 128, 16, [1100, 333, 2], [0, 128, 1400]),
    (5, 1, 128, 32, [4000, 3700], [0, 600]),
    (40, 8, 128, 16, [600, 500], [7, 0]),
]


@pytest.mark.parametrize("h,hk,d,pt,new,ctx", LONG)
def test_long_prompts(h, hk, d, pt, new, ctx):
    fills_the_gpu(h, hk, new)
    kv_lens = [n + c for n, c in zip(new, ctx)]
    table, pages = base.tables(kv_lens, pt, 3, extra=1)
    cache = base.filled_cache(pages, hk, pt, d, seed=4)
    base.run_prompt(cache, table, new, kv_lens, h, d, seed=5, padding=2)
    base.run_prompt(cache, table, new, kv_lens, h, d, seed=6, scale=0.5, strided=True)  # a sharper softmax


@pytest.mark.parametrize("h,hk,d,pt,new,ctx", [LONG[0], LONG[5]])
def test_long_prompts_whose_scales_grow_and_fall(h, hk, d, pt, new, ctx):
    """Maxima that rise along the sequence (the softmax's reference), and value scales over many powers of two (the sums' range)."""
    fills_the_gpu(h, hk, new)
    kv_lens = [n + c for n, c in zip(new, ctx)]
    table, pages = base.tables(kv_lens, pt, 3)
    cache = base.filled_cache(pages, hk, pt, d, seed=4)
    order = torch.cat([base.spec.token_slots(table[r], pt, n) for r, n in enumerate(kv_lens)]).long()
    place = torch.cat([torch.arange(n, device=DEV) / n for n in kv_lens])  # 0 .. 1 along each sequence
    was = [cache.k_scale.clone(), cache.v_scale.clone()]

    def times(scale, by):
        flat = torch.ones(pages * pt, device=DEV)
        flat[order] = by
        scale *= flat.view(pages, 1, pt)

    for by_k, by_v in ((place * 4, None), ((1 - place) * 4, None), (None, 10.0 ** (12 * place - 6)), (None, 10.0 ** (6 - 12 * place))):
        cache.k_scale.copy_(was[0]), cache.v_scale.copy_(was[1])
        if by_k is not None:
            times(cache.k_scale, by_k)
        else:
            times(cache.v_scale, by_v)
        base.run_prompt(cache, table, new, kv_lens, h, d, seed=7)


@pytest.mark.parametrize("d", [64, 128])
def test_long_prompts_masked_empty_and_bad(d):
    """Rows that see nothing, masked places that hold NaN and infinities, a bad page, and the call captured and replayed."""
    hk, h, pt, new, kv_lens = 16, 16, 32, [1000, 700, 0, 300], [600, 900, 40, 300]
    fills_the_gpu(h, hk, new)
    table, pages = base.tables(kv_lens, pt, 8, extra=2)
    cache = base.filled_cache(pages, hk, pt, d, seed=9)
    clean = base.run_prompt(cache, table, new, kv_lens, h, d, seed=5)
    assert (clean[:400] == 0).all() and (clean[400] != 0).any()
    used = torch.zeros(pages * pt, dtype=torch.bool, device=DEV)
    for r, n in enumerate(kv_lens):
        used[base.spec.token_slots(table[r], pt, n)] = True
    last = base.spec.token_slots(table[1], pt, 900)[899].item()  # the last token of a sequence: one query sees it
    for s, x in ((cache.k_scale, math.nan), (cache.v_scale, math.inf)):
        s.masked_fill_(~used.view(pages, 1, pt), x)
        s[last // pt, :, last % pt] = x
    q, out, w = base.bf16(2000, h, d, seed=5), torch.zeros(2000, h, d, dtype=torch.bfloat16, device=DEV), base.work()
    args = (q, cache, table, base.ints([0, 1000, 1700, 1700, 2000]), base.ints(kv_lens), 1 / math.sqrt(d), out, w)
    kv.shn_kv_attn_prompt(*args)
    assert base.status(w) == (0, 0)
    keep = torch.arange(2000, device=DEV) != 1699
    assert torch.equal(out[keep], clean[keep]) and torch.isnan(out[1699]).all()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kv.shn_kv_attn_prompt(*args)
    first = out.clone()
    out.zero_()
    graph.replay()
    assert torch.equal(out.view(torch.int16), first.view(torch.int16)) and base.status(w) == (0, 0)
    table[1, 20] = pages
    kv.shn_kv_attn_prompt(*args)
    assert base.status(w) == (shn.SHN_ERR_INVALID_ARG, 1)
    others = torch.cat([torch.arange(1000), torch.arange(1700, 2000)]).to(DEV)
    assert torch.equal(out[others], clean[others])


def test_long_prompts_of_many_requests():
    """More requests than a block has threads, a few long ones among them."""
    rng = random.Random(1)
    new = [rng.choice([0, 1, 2, 5]) for _ in range(950)]
    kv_lens = [m + rng.choice([0, 0, 3, 40]) for m in new]
    new[500], kv_lens[500] = 900, 1500
    new[949], kv_lens[949] = 300, 300
    table, pages = base.tables(kv_lens, 16, 1)
    for d in (64, 128):
        base.run_prompt(base.filled_cache(pages, 2, 16, d, seed=2), table, new, kv_lens, 4, d, seed=3, padding=1)


@pytest.mark.parametrize("tokens,h,hk,d,pt,norm,rot,pairs", [
    (2500, 32, 8, 128, 32, True, 128, False), (5001, 6, 2, 64, 64, True, 32, True), (8192, 8, 8, 64, 16, False, 64, False), (8193, 16, 4, 128, 16, True, 64, True),
    (9001, 0, 7, 64, 128, True, 48, False), (9500, 40, 1, 128, 64, False, 0, False), (20011, 4, 2, 64, 32, True, 64, False),
])
def test_store_and_load_of_many_tokens(tokens, h, hk, d, pt, norm, rot, pairs):
    base.test_store_and_load(tokens, h, hk, d, pt, norm, rot, pairs)
