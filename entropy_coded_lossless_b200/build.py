"""Build libshn.so (the CUDA kernels + C ABI) in-tree for sm_100a with nvcc, and _kv.so (the Python calls of the paged
KV cache over it) with g++ and torch's headers. Only the module ``kv`` needs the latter: where it cannot be built, build() warns.

    python -m entropy_coded_lossless_b200.build [--force]
"""
import os
import subprocess
import sys
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "libshn.so")
SOURCES = ["capi.cu", "histogram.cu", "build_tables.cu", "encode.cu", "decode.cu", "noalloc.cu", "offload.cu",
           "kv_capi.cu", "kv_plan.cu", "kv_store.cu", "kv_attn_tc.cu", "kv_decode.cu"]
HEADERS = [os.path.join(CSRC, "shn_internal.cuh"), os.path.join(ROOT, "include", "shn.h")]
# the paged KV cache's sources (kv_*.cu) alone include these
KV_HEADERS = [os.path.join(CSRC, "kv_internal.cuh"), os.path.join(CSRC, "kv_tc.cuh"),
              os.path.join(CSRC, "kv_decode.cuh"), os.path.join(ROOT, "include", "shn_kv.h")]
BINDING = os.path.join(HERE, "_kv.so")
BINDING_TORCH = os.path.join(HERE, "_build", "_kv.torch")  # the torch it was built for
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo", "-std=c++17",
         "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall", "--expt-relaxed-constexpr"]


def _stale(target, deps):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False) -> str:
    lib = build_lib(force, verbose)
    try:
        build_binding(force, verbose)
    except (ImportError, OSError, subprocess.CalledProcessError) as e:
        warnings.warn(f"_kv.so not built, so entropy_coded_lossless_b200.kv does not import ({e}); the codec does without it", RuntimeWarning,
                      stacklevel=2)
    return lib


def _torch_version():
    from importlib import metadata

    return metadata.version("torch")


def build_binding(force: bool = False, verbose: bool = False) -> str:
    src = os.path.join(CSRC, "kv_binding.cpp")
    version = _torch_version()
    if not force and not _stale(BINDING, [src, os.path.join(ROOT, "include", "shn_kv.h"), os.path.join(ROOT, "include", "shn.h")]):
        if os.path.exists(BINDING_TORCH) and open(BINDING_TORCH).read() == version:
            return BINDING
    if os.path.exists(BINDING):  # one that no longer fits is not left to be imported
        os.remove(BINDING)
    import sysconfig

    import torch
    from torch.utils import cpp_extension

    libs = [os.path.join(os.path.dirname(torch.__file__), "lib")]
    includes = cpp_extension.include_paths() + [sysconfig.get_paths()["include"], os.path.join(os.path.dirname(os.path.dirname(NVCC)), "include")]
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *[a for i in includes for a in ("-isystem", i)], src, "-o", BINDING, f"-L{HERE}", "-l:libshn.so", *[f"-L{d}" for d in libs], "-lc10", "-lc10_cuda",
           "-ltorch_cpu", "-ltorch_python", "-Wl,-rpath,$ORIGIN"]
    if verbose:
        print(" ".join(cmd))
    subprocess.check_call(cmd)
    os.makedirs(os.path.dirname(BINDING_TORCH), exist_ok=True)
    with open(BINDING_TORCH, "w") as f:
        f.write(version)
    return BINDING


def build_lib(force: bool = False, verbose: bool = False) -> str:
    srcs = [os.path.join(CSRC, s) for s in SOURCES]
    if not force and not _stale(LIB, srcs + HEADERS + KV_HEADERS):
        return LIB
    obj_dir = os.path.join(HERE, "_build")
    os.makedirs(obj_dir, exist_ok=True)
    objs = []
    for src in srcs:
        obj = os.path.join(obj_dir, os.path.basename(src) + ".o")
        deps = [src] + HEADERS + (KV_HEADERS if os.path.basename(src).startswith("kv_") else [])
        if force or _stale(obj, deps):
            cmd = [NVCC, *FLAGS, "-I", os.path.join(ROOT, "include"), "-c", src, "-o", obj]
            if verbose:
                cmd.insert(1, "-Xptxas=-v")
                print(" ".join(cmd))
            subprocess.check_call(cmd)
        objs.append(obj)
    subprocess.check_call([NVCC, "-shared", "-gencode", "arch=compute_100a,code=sm_100a", "-o", LIB, *objs,
                           "-lcudart"])
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
