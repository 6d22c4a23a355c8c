"""What the cache attention does when a wait inside its tensor core kernel runs out: the library's KV sources built with no tries at
all, so that every wait gives up at once. Blocks end, give their tensor memory back and report; the context stays usable."""
import ctypes
import os
import subprocess

import pytest
import torch

from entropy_coded_lossless_b200 import build as shn_build

shn_build.build()
from entropy_coded_lossless_b200 import kv, shn  # noqa: E402
from tests import test_gpu_kv as base  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def hasty(tmp_path_factory):
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    kv._lib()
    folder = tmp_path_factory.mktemp("kv")
    sources = [s for s in shn_build.SOURCES if s.startswith("kv_")]
    objects = [str(folder / (s + ".o")) for s in sources]
    builds = [subprocess.Popen([shn_build.NVCC, *shn_build.FLAGS, "-DSHN_KV_WAIT_TRIES=0", "-I", os.path.join(shn_build.ROOT, "include"), "-c",
                                os.path.join(shn_build.CSRC, s), "-o", o]) for s, o in zip(sources, objects)]
    assert [b.wait() for b in builds] == [0] * len(builds)
    so = str(folder / "hasty.so")
    subprocess.check_call([shn_build.NVCC, "-shared", "-gencode", "arch=compute_100a,code=sm_100a", "-o", so, *objects, "-lcudart"])
    lib = ctypes.CDLL(so)
    for name in ("shn_kv_attn_prompt", "shn_kv_attn_shared"):
        fn, known = getattr(lib, name), getattr(kv._lib(), name)
        fn.restype, fn.argtypes = known.restype, known.argtypes
    return lib


def p(t):
    return t.data_ptr()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("h,hk,new,kv_lens", [
    (2, 1, [3], [3]),  # a block
    (2, 1, [3, 0, 5], [2500, 7, 900]),  # blocks of a cluster, which wait for each other in hardware
    (16, 16, [900, 700], [900, 1000]),  # more blocks than SMs: the later ones do not start on it
])
def test_prompt_whose_waits_run_out(hasty, h, hk, new, kv_lens, d):
    table, pages = base.tables(kv_lens, 32, 1)
    cache = base.filled_cache(pages, hk, 32, d, seed=2)
    cu = base.ints([sum(new[:i]) for i in range(len(new) + 1)])
    q, w, lens = base.bf16(sum(new), h, d, seed=3), base.work(), base.ints(kv_lens)
    out = torch.zeros_like(q)
    for _ in range(2):
        assert hasty.shn_kv_attn_prompt(p(q), h * d, sum(new), h, ctypes.byref(cache.c), p(table), table.shape[1], p(cu), p(lens), len(new), 0.1, p(out), h * d,
                                        p(w), w.numel(), None) == 0
        code, request = base.status(w)
        assert code == shn.SHN_ERR_TIMEOUT and new[request] > 0
    kv.shn_kv_attn_prompt(q, cache, table, cu, lens, 0.1, out, w)  # the library's own build, in the same context
    assert base.status(w) == (0, 0) and torch.isfinite(out).all()


@pytest.mark.parametrize("d", [64, 128])
def test_prefix_whose_waits_run_out(hasty, d):
    n, h, hk, prefix = 70, 32, 2, 320  # (over a thousand query rows to a key head: the tensor cores)
    table, pages = base.tables([prefix + 3] * n, 32, 1)
    cache = base.filled_cache(pages, hk, 32, d, seed=2)
    q, lens, plen, front = base.bf16(n, h, d, seed=3), base.ints([prefix + 3] * n), base.ints([prefix]), table[0, :10].contiguous()
    out, w = torch.zeros_like(q), base.work(kv.attn_shared_workspace_bytes(cache, n, h))
    for _ in range(2):
        assert hasty.shn_kv_attn_shared(p(q), h * d, n, h, ctypes.byref(cache.c), p(front), 10, p(plen), p(table), table.shape[1], p(lens), 0.1, p(out), h * d,
                                        p(w), w.numel(), None) == 0
        assert base.status(w)[0] == shn.SHN_ERR_TIMEOUT
    kv.shn_kv_attn_shared(q, cache, front, plen, table, lens, 0.1, out, w)
    assert base.status(w) == (0, 0) and torch.isfinite(out).all()
