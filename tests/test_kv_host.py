"""Host side of the paged KV cache calls (include/shn_kv.h), no CUDA call: what they refuse before anything is
enqueued. Device pointers here are stand-ins that are never dereferenced."""
import ctypes

import pytest
import torch

from entropy_coded_lossless_b200 import build as shn_build

shn_build.build()  # the binding is an extension module: it is there before it is imported
from entropy_coded_lossless_b200 import kv, shn  # noqa: E402

BAD, UNSUP, WORK = shn.SHN_ERR_INVALID_ARG, shn.SHN_ERR_UNSUPPORTED, shn.SHN_ERR_WORKSPACE
P = 1 << 20  # 256-byte aligned


@pytest.fixture(scope="module")
def lib():
    shn_build.build()
    return kv._lib()


def cache(**over):
    f = dict(d_k=P, d_v=P, d_k_scale=P, d_v_scale=P, n_pages=64, kv_heads=8, page_tokens=32, head_dim=128)
    f.update(over)
    return kv._CacheStruct(*[f[n] for n, _ in kv._CacheStruct._fields_])


@pytest.mark.parametrize("over,code", [
    ({}, 0), (dict(head_dim=64), 0), (dict(page_tokens=16), 0), (dict(page_tokens=1024), 0), (dict(kv_heads=1), 0),
    (dict(head_dim=96), UNSUP), (dict(head_dim=256), UNSUP), (dict(page_tokens=8), BAD), (dict(page_tokens=48), BAD),
    (dict(page_tokens=2048), BAD), (dict(page_tokens=0), BAD), (dict(n_pages=0), BAD), (dict(kv_heads=0), BAD),
    (dict(kv_heads=1025), BAD), (dict(d_k=None), BAD), (dict(d_v=P + 8), BAD), (dict(d_k_scale=P + 2), BAD),
    (dict(n_pages=1 << 26), BAD), (dict(n_pages=(1 << 26) - 1), 0),
])
def test_cache_check(lib, over, code):
    assert lib.shn_kv_check_cache(ctypes.byref(cache(**over))) == code
    assert lib.shn_kv_check_cache(None) == BAD


def plan(lib, **over):
    f = dict(ctx=P, new=P, n=4, pt=32, table=P, max_blocks=16, free=P, n_free=64, head=P, next=P, cu=P, kv_len=P, pos=P, slots=P,
             max_tokens=128, work=P, work_bytes=256, stream=None)
    f.update(over)
    return lib.shn_kv_plan(*f.values())


@pytest.mark.parametrize("over,code", [
    (dict(pt=24), BAD), (dict(pt=8), BAD), (dict(ctx=None), BAD), (dict(table=None), BAD), (dict(free=None), BAD), (dict(head=None), BAD),
    (dict(next=None), BAD), (dict(cu=None), BAD), (dict(slots=None), BAD), (dict(max_tokens=1 << 31), BAD),
    (dict(max_blocks=1 << 26), BAD), (dict(work=None), BAD), (dict(work=P + 8), BAD), (dict(work_bytes=255), WORK),
])
def test_plan_refusals(lib, over, code):
    assert plan(lib, **over) == code


def store(lib, c=None, **over):
    f = dict(q=P, qs=4096, h=32, k=P, ks=1024, v=P, vs=1024, n=5, pos=P, slots=P, wq=None, wk=None, eps=1e-6, cs=P, npos=64, rot=128,
             pairs=0, cache=ctypes.byref(c if c is not None else cache()), qo=P, qos=4096, work=P, work_bytes=256, stream=None)
    f.update(over)
    return lib.shn_kv_store(*f.values())


@pytest.mark.parametrize("over,code", [
    (dict(qs=4095), BAD), (dict(qs=4088), BAD), (dict(ks=1016), BAD), (dict(q=P + 2), BAD), (dict(k=None), BAD), (dict(v=P + 8), BAD),
    (dict(qo=None), BAD), (dict(qo=P, qos=8192), BAD), (dict(slots=None), BAD), (dict(pos=None), BAD), (dict(rot=136), BAD),
    (dict(rot=24), BAD), (dict(rot=0), BAD), (dict(cs=None), BAD), (dict(cs=P + 4), BAD), (dict(pairs=2), BAD),
    (dict(wq=P + 2), BAD), (dict(wq=P, eps=-1.0), BAD), (dict(wk=P, eps=float("nan")), BAD), (dict(q=None), BAD), (dict(h=0), BAD),
    (dict(work_bytes=8), WORK), (dict(work=P + 128), BAD),
])
def test_store_refusals(lib, over, code):
    assert store(lib, **over) == code


def test_store_refuses_a_bad_cache(lib):
    assert store(lib, cache(head_dim=80)) == UNSUP
    assert store(lib, cache(page_tokens=20)) == BAD


@pytest.mark.parametrize("over,code", [
    (dict(slots=None), BAD), (dict(ks=1020), BAD), (dict(ks=512), BAD), (dict(v=P + 4), BAD), (dict(work=None), BAD), (dict(work_bytes=0), WORK),
    (dict(n=1 << 31), BAD),
])
def test_load_refusals(lib, over, code):
    f = dict(c=ctypes.byref(cache()), slots=P, n=7, k=P, ks=1024, v=P, vs=1024, work=P, work_bytes=256, stream=None)
    f.update(over)
    assert lib.shn_kv_load(*f.values()) == code


ATTN = [
    (dict(q=None), BAD), (dict(q=P + 8), BAD), (dict(qs=4090), BAD), (dict(os=1024), BAD), (dict(o=None), BAD), (dict(h=12), BAD), (dict(h=0), BAD),
    (dict(h=8 * 65), BAD), (dict(table=None), BAD), (dict(kv_len=None), BAD), (dict(max_blocks=1 << 27), BAD), (dict(work=None), BAD),
    (dict(work=P + 64), BAD), (dict(work_bytes=255), WORK),
]


@pytest.mark.parametrize("over,code", ATTN + [(dict(cu=None), BAD), (dict(n=1 << 27), BAD)])
def test_prompt_refusals(lib, over, code):
    f = dict(q=P, qs=4096, n=50, h=32, c=ctypes.byref(cache()), table=P, max_blocks=16, cu=P, kv_len=P, reqs=3, scale=0.1, o=P, os=4096,
             work=P, work_bytes=1 << 40, stream=None)
    f.update(over)
    assert lib.shn_kv_attn_prompt(*f.values()) == code


@pytest.mark.parametrize("over,code", ATTN + [(dict(prefix=None), BAD), (dict(plen=None), BAD), (dict(n_prefix=1 << 26), BAD)])
def test_shared_refusals(lib, over, code):
    f = dict(q=P, qs=4096, reqs=3, h=32, c=ctypes.byref(cache()), prefix=P, n_prefix=16, plen=P, table=P, max_blocks=16, kv_len=P, scale=0.1,
             o=P, os=4096, work=P, work_bytes=1 << 40, stream=None)
    f.update(over)
    assert lib.shn_kv_attn_shared(*f.values()) == code


def test_calls_refuse_outputs_that_are_inputs(lib):
    a, b = P + 4096, P + 8192
    assert plan(lib, new=a) == BAD and plan(lib, ctx=a) == BAD  # kv_len is the other one
    c = ctypes.byref(cache())
    assert lib.shn_kv_attn_prompt(a, 4096, 50, 32, c, P, 16, P, P, 3, 0.1, a, 4096, b, 1 << 40, None) == BAD
    assert lib.shn_kv_attn_shared(a, 4096, 3, 32, c, P, 16, P, P, 16, P, 0.1, a, 4096, b, 1 << 40, None) == BAD


def test_shared_workspace_query(lib):
    c = cache()
    one, many = (lib.shn_kv_attn_shared_workspace_bytes(ctypes.byref(c), n, 32) for n in (1, 300))
    assert 256 <= one <= many
    assert lib.shn_kv_attn_shared_workspace_bytes(ctypes.byref(c), 3, 12) == 0
    assert lib.shn_kv_attn_shared_workspace_bytes(ctypes.byref(c), 3, 8 * 65) == 0
    assert lib.shn_kv_attn_shared_workspace_bytes(ctypes.byref(cache(head_dim=100)), 3, 32) == 0


def test_binding_takes_no_cpu_tensors(lib):
    x = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        kv.shn_kv_plan(x, x, 16, x.view(4, 1), x, x, x, x, x, x, x, x)
    with pytest.raises(ValueError):
        kv.Cache(torch.zeros(2, 2, 16, 64, dtype=torch.int8), None, None, None)
