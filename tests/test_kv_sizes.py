"""Host side of shn_kv_attn_shared's workspace (include/shn_kv.h): what the size query says for any number of requests. No
CUDA call; device pointers are stand-ins that are never dereferenced."""
import ctypes

import pytest

from entropy_coded_lossless_b200 import build as shn_build

shn_build.build()
from entropy_coded_lossless_b200 import kv, shn  # noqa: E402

P = 1 << 20  # 256-byte aligned


def cache(kv_heads=8, head_dim=128, page_tokens=32):
    return kv._CacheStruct(P, P, P, P, 64, kv_heads, page_tokens, head_dim)


def size(c, n, h):
    return kv._lib().shn_kv_attn_shared_workspace_bytes(ctypes.byref(c), n, h)


@pytest.mark.parametrize("hk,h", [(8, 32), (1, 1), (1024, 1024), (4, 24)])
def test_an_empty_batch_has_a_size(hk, h):
    assert size(cache(hk), 0, h) >= 256


def test_an_empty_batch_still_has_its_arguments_checked():
    c = cache()
    f = dict(q=None, qs=4096, reqs=0, h=32, c=ctypes.byref(c), prefix=None, n_prefix=0, plen=P, table=None, max_blocks=16, kv_len=None,
             scale=0.1, o=None, os=4096, work=P, work_bytes=256, stream=None)
    for over, code in ((dict(work=None), shn.SHN_ERR_INVALID_ARG), (dict(work=P + 64), shn.SHN_ERR_INVALID_ARG), (dict(plen=None), shn.SHN_ERR_INVALID_ARG),
                       (dict(work_bytes=255), shn.SHN_ERR_WORKSPACE), (dict(h=12), shn.SHN_ERR_INVALID_ARG)):
        assert kv._lib().shn_kv_attn_shared(*{**f, **over}.values()) == code


@pytest.mark.parametrize("hk,h,d", [(8, 32, 128), (1, 1, 128), (1, 64, 64), (4, 24, 64), (40, 40, 128), (148, 148, 64), (200, 400, 64), (1024, 1024, 128), (2, 34, 128)])
def test_a_workspace_serves_smaller_batches_too(hk, h, d):
    """A server sizes its workspace once, for its largest batch."""
    c = cache(hk, d)
    sizes = [size(c, n, h) for n in range(700)]
    assert all(a <= b for a, b in zip(sizes, sizes[1:])), next((n, a, b) for n, (a, b) in enumerate(zip(sizes, sizes[1:])) if a > b)
    assert size(c, 5000, h) >= sizes[-1]
