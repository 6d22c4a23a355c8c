"""Which request or token the paged KV cache calls name when several are wrong: the first, whatever the timing."""
import pytest
import torch

from entropy_coded_lossless_b200 import build as shn_build

shn_build.build()
from entropy_coded_lossless_b200 import kv, shn  # noqa: E402
from tests import test_gpu_kv as base  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"
BAD = shn.SHN_ERR_INVALID_ARG
ints, work, status = base.ints, base.work, base.status


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    shn.lib()


@pytest.mark.parametrize("n,new", [(2, 300), (40, 20), (500, 2)])
def test_plan_of_few_tokens_reports_the_first_bad_page(n, new):
    """Up to 1024 tokens (one block): of bad pages that are begun, and bad ones of the free list, the first request's."""
    pt = 16
    ctx, fresh = [5] * n, [new] * n
    each = -(-(5 + new) // pt) - 1  # pages a request takes
    for begun, taken in (((n - 1,), ()), ((0, n - 1), ()), ((n // 2, n - 1), (n - 1,)), ((), (0, n - 1)), ((n - 1,), (n // 2,)), ((1,), (n - 1, 0))):
        if not each:
            taken = ()
        table = [[r] + [-1] * each for r in range(n)]
        free = list(range(n, n + n * each + 3))
        for r in begun:
            table[r][0] = -2
        for r in taken:
            free[r * each + each - 1] = 2**31 - 1
        nxt, cu, kv_len, pos, slots = base.plan_buffers(n, 1024)
        w = work()
        for _ in range(5):
            kv.shn_kv_plan(ints(ctx), ints(fresh), pt, ints(table), ints(free), ints([0]), nxt, cu, kv_len, pos, slots, w)
            bad = begun + taken
            assert status(w) == ((BAD, min(bad)) if bad else (0, 0))
        assert nxt.item() == n * each and cu[-1].item() == n * new and kv_len.tolist() == [5 + new] * n
        assert (slots[:n * new] < 0).any().item() == bool(bad)


@pytest.mark.parametrize("n", [8193, 40000])
def test_store_and_load_of_many_tokens_report_the_first(n):
    cache, w, cs = base.filled_cache(2, 1, 16, 64), work(), base.angles(6, 64, 1)
    k, out = base.bf16(n, 1, 64, seed=n), torch.zeros(n, 1, 64, dtype=torch.bfloat16, device=DEV)
    none = torch.full((n,), -1, dtype=torch.int32, device=DEV)
    for first in (0, n // 3, n - 1):
        slots, positions = none.clone(), torch.zeros_like(none)
        slots[first:], positions[first:] = 32, 6
        for _ in range(3):
            kv.shn_kv_load(cache, slots, out, None, w)
            assert status(w) == (BAD, first)
            kv.shn_kv_store(None, k, k, None, slots, cache, None, w)
            assert status(w) == (BAD, first)
            kv.shn_kv_store(None, k, k, positions, none, cache, None, w, cos_sin=cs)
            assert status(w) == (BAD, first)
    assert not out.any()


@pytest.mark.parametrize("n,new", [(5, 3), (32, 1), (33, 1), (70, 5), (300, 1), (1000, 2)])
def test_prompts_report_the_first_bad_request(n, new):
    """Bad lengths, bad pages and bad ranges of queries, several at once."""
    hk, h, d, pt = 2, 4, 64, 16
    cache = base.filled_cache(8, hk, pt, d)
    q, w = base.bf16(n * new, h, d), work()
    out = torch.empty_like(q)
    table = torch.arange(n, device=DEV).remainder(8).to(torch.int32).view(n, 1).repeat(1, 2)
    for what in ("page", "length", "range", "page and length"):
        for bad in ((n - 1, 1), (n - 1, n // 2, n // 2 + 1), (0, n - 1)):
            t, lens, cu = table.clone(), [new + 2] * n, [i * new for i in range(n + 1)]
            for i, r in enumerate(bad):
                if what == "page" or (what == "page and length" and i % 2):
                    t[r] = 8
                elif what == "range":
                    cu[r + 1] = n * new + 1 + r  # request r's end, and the next one's beginning
                else:
                    lens[r] = -1
            for _ in range(3):
                kv.shn_kv_attn_prompt(q, cache, t, ints(cu), ints(lens), 0.1, out, w)
                assert status(w) == (BAD, min(bad)), (what, bad)


def test_refusals_of_arguments_that_are_no_tensors():
    """A stream that is none, an epsilon that is no number: refused, and the current device stays."""
    cache, w = base.filled_cache(2, 1, 16, 64), work()
    k, slots = base.bf16(2, 1, 64), ints([0, 1])
    was, before = cache.k.clone(), torch.cuda.current_device()

    class NoStream:
        cuda_stream = "x"

    with pytest.raises(ValueError):
        kv.shn_kv_load(cache, slots, k, None, w, stream=NoStream())
    with pytest.raises(ValueError):
        kv.shn_kv_store(None, k, k, None, slots, cache, None, w, stream=NoStream())
    with pytest.raises(ValueError):
        kv.shn_kv_store(None, k, k, None, slots, cache, None, w, eps="small")
    torch.cuda.synchronize()
    assert torch.equal(cache.k, was) and torch.cuda.current_device() == before
