"""Batches of the paged KV cache calls that a serving loop meets between its ordinary ones: empty ones, and workspaces that
serve several sizes."""


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


def rows(n, h, d):
    return torch.full((n, h, d), 7.0, dtype=torch.bfloat16, device=DEV)


@pytest.mark.parametrize("prefix", [None, [0, 1]])
@pytest.mark.parametrize("h,hk", [(32, 8), (1, 1)])
def test_attention_of_no_requests(h, hk, prefix):
    """A step in which nobody decodes: the status word is set and nothing else happens."""
    cache = base.filled_cache(4, hk, 16, 128)
    none = base.ints([])
    pages = None if prefix is None else base.ints(prefix)
    q, out, w = rows(0, h, 128), rows(0, h, 128), base.work(kv.attn_shared_workspace_bytes(cache, 0, h))
    kv.shn_kv_attn_shared(q, cache, pages, base.ints([16]), none.view(0, 5), none, 0.1, out, w)
    assert base.status(w) == (0, 0)
    w = base.work(kv.attn_shared_workspace_bytes(cache, 9, h))
    kv.shn_kv_attn_shared(q, cache, pages, base.ints([16]), none.view(0, 5), none, 0.1, out, w)
    assert base.status(w) == (0, 0)
    w, some = base.work(), rows(3, h, 128)
    kv.shn_kv_attn_prompt(q, cache, none.view(0, 5), base.ints([0]), none, 0.1, out, w)
    assert base.status(w) == (0, 0)
    kv.shn_kv_attn_prompt(base.bf16(3, h, 128), cache, none.view(0, 5), base.ints([0]), none, 0.1, some, w)  # padding alone
    assert base.status(w) == (0, 0) and (some == 7.0).all()


def test_store_and_load_of_no_tokens():
    cache, w = base.filled_cache(4, 2, 16, 64), base.work()
    was, none = cache.k.clone(), base.ints([])
    kv.shn_kv_store(rows(0, 4, 64), rows(0, 2, 64), rows(0, 2, 64), none, none, cache, rows(0, 4, 64), w, cos_sin=base.angles(8, 64, 1))
    assert base.status(w) == (0, 0) and torch.equal(cache.k, was)
    w = base.work()
    kv.shn_kv_load(cache, none, rows(0, 2, 64), None, w)
    assert base.status(w) == (0, 0)


@pytest.mark.parametrize("h,hk,prefix", [(32, 8, 8192), (8, 2, 64), (6, 1, 4096)])
def test_a_shrinking_batch_keeps_its_workspace(h, hk, prefix):
    """The workspace of the largest batch, used again by smaller ones (whose prefix is cut into more parts)."""
    pt, d, most = 64, 128, 100
    own = [1 + n * 37 % 150 for n in range(most)]
    table, pages = base.shared_tables(own, prefix, pt, 3)
    cache = base.filled_cache(pages, hk, pt, d, seed=4)
    q, front = base.bf16(most, h, d, seed=5), table[0, :prefix // pt].contiguous()
    w = base.work(kv.attn_shared_workspace_bytes(cache, most, h))
    for n in (100, 65, 64, 33, 1, 64, 100):
        lens, a, b = base.ints([prefix + x for x in own[:n]]), rows(n, h, d), rows(n, h, d)
        fresh = base.work(kv.attn_shared_workspace_bytes(cache, n, h))
        for o, x in ((a, w), (b, fresh)):
            kv.shn_kv_attn_shared(q[:n], cache, front, base.ints([prefix]), table[:n], lens, 0.1, o, x)
            assert base.status(x) == (0, 0)
        assert torch.equal(a, b) and torch.isfinite(a).all()


@pytest.mark.parametrize("d", [64, 128])
def test_a_captured_step_with_room_for_a_long_prefix(d):
    """Which kernel the prefix takes is the room's: with room for a long one every length of it gives what a call without that room gives,
    no prefix at all among them, and lengths that the room cannot hold are reported."""
    pt, hk, h, n, room = 32, 2, 32, 70, 3200
    own = [r * 37 % 90 for r in range(n)]
    table, pages = base.shared_tables([room + x for x in own], 0, pt, 3)
    cache = base.filled_cache(pages, hk, pt, d, seed=4)
    q, plen, lens = base.bf16(n, h, d, seed=5), base.ints([0]), base.ints([0] * n)
    front, out = table[0, :room // pt].contiguous(), rows(n, h, d)
    shared = table.clone()
    shared[:, :room // pt] = front
    w = base.work(kv.attn_shared_workspace_bytes(cache, n, h))
    args = (q, cache, front, plen, shared, lens, 0.1, out, w)
    kv.shn_kv_attn_shared(*args)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kv.shn_kv_attn_shared(*args)
    for prefix in (0, 1, 31, 128, 1000, room):
        lens.copy_(base.ints([prefix + x for x in own])), plen.copy_(base.ints([prefix])), out.fill_(7.0)
        graph.replay()
        assert base.status(w) == (0, 0)
        ref, tol = base.spec.cache_attention(q, cache, lambda r: shared[r], [prefix + x for x in own], list(range(n + 1)), 0.1)
        assert ((out.double() - ref).abs() <= tol).all()
        assert (out[[r for r in range(n) if prefix + own[r] == 0]] == 0).all()
    for prefix, held in ((-1, 0), (room + 1, room)):
        plen.copy_(base.ints([prefix])), lens.copy_(base.ints([held + x for x in own]))
        graph.replay()
        assert base.status(w)[0] == shn.SHN_ERR_INVALID_ARG
        ref, tol = base.spec.cache_attention(q, cache, lambda r: shared[r], [held + x for x in own], list(range(n + 1)), 0.1)
        assert ((out.double() - ref).abs() <= tol).all()


def test_many_single_tokens():
    """Thousands of requests, more than any kernel has threads for, most of them short."""
    n, hk, h, d, pt = 5000, 2, 4, 64, 16
    lens = [r * 7 % 23 for r in range(n)]
    lens[4321] = 3000
    table, pages = base.tables(lens, pt, 1)
    cache = base.filled_cache(pages, hk, pt, d, seed=2)
    q, out, w = base.bf16(n, h, d, seed=3), rows(n, h, d), base.work(kv.attn_shared_workspace_bytes(cache, n, h))
    kv.shn_kv_attn_shared(q, cache, None, base.ints([0]), table, base.ints(lens), 0.1, out, w)
    assert base.status(w) == (0, 0)
    again = rows(n, h, d)
    kv.shn_kv_attn_prompt(q, cache, table, torch.arange(n + 1, dtype=torch.int32, device=DEV), base.ints(lens), 0.1, again, w)
    assert base.status(w) == (0, 0)
    some = [r for r in range(0, n, 250)] + [4321]
    ref, tol = base.spec.cache_attention(q[some], cache, lambda i: table[some[i]], [lens[r] for r in some], list(range(len(some) + 1)), 0.1)
    for o in (out, again):
        assert ((o[some].double() - ref).abs() <= tol).all()
        assert (o[[r for r in range(n) if lens[r] == 0]] == 0).all()
    # both hold each result to 2^-11 of its parts and half a step of bfloat16: together below 2^-6 of the largest value
    assert (out.double() - again.double()).abs().max() <= 2.0**-6 * out.double().abs().max()
