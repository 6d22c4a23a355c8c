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
