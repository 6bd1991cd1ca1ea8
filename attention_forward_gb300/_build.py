"""Builds libfa_gb300.so in-tree from csrc/ with nvcc for sm_103a, and beside it
_fa_torch.so, the compiled part of the binding, with g++ against torch.

Each translation unit is compiled in its own nvcc process (in parallel), then
the objects are linked into one shared library against the shared CUDA
runtime, so the library and PyTorch use the same runtime instance when both
are loaded.  ``python -m attention_forward_gb300._build`` builds it.
"""
from __future__ import annotations

import hashlib
import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OBJ = os.path.join(PKG, "_objs")
LIB = os.path.join(PKG, "libfa_gb300.so")
PTXAS_LOG = os.path.join(OBJ, "ptxas.log")
TORCH_SOURCE = os.path.join(CSRC, "fa_torch.cpp")
TORCH_LIB = os.path.join(PKG, "_fa_torch.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                     "-Xptxas", "-v", "--expt-relaxed-constexpr",
                     f"-I{os.path.join(ROOT, 'include')}"]
SOURCES = ["fa_prefill_d128.cu", "fa_prefill_d64.cu", "fa_prefill_d64x3.cu", "fa_prefill_pair.cu",
           "fa_decode.cu", "fa_api.cu", "fa_noalloc.cu", "fa_diag.cu",
           "fa_score_d128_bf16.cu", "fa_score_d128_f16.cu",
           "fa_score_d64_bf16.cu", "fa_score_d64_f16.cu", "fa_score_docs.cu", "fa_score_api.cu",
           "fa_cache.cu", "fa_cache_attn.cu", "fa_cache_api.cu", "fa_merge.cu",
           "fa_paged_copy.cu", "fa_paged_attn_d64.cu", "fa_paged_attn_d128.cu",
           "fa_paged_attn_latent.cu", "fa_paged_api.cu", "fa_expanded.cu"]


def nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found")
    return cand


def _cuda_lib_dir() -> str:
    return os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))),
                        "lib64")


def _fingerprint() -> str:
    h = hashlib.sha256()
    for name in sorted(os.listdir(CSRC)):
        if name.endswith(".cpp"):  # the binding's, which has its own fingerprint
            continue
        with open(os.path.join(CSRC, name), "rb") as f:
            h.update(name.encode() + f.read())
    with open(os.path.join(ROOT, "include", "fa.h"), "rb") as f:
        h.update(f.read())
    h.update(" ".join(NVCC_FLAGS).encode())
    return h.hexdigest()


def _compile(src: str, obj_dir: str = OBJ, defines=()) -> tuple[str, str]:
    obj = os.path.join(obj_dir, os.path.splitext(src)[0] + ".o")
    cmd = [nvcc(), *NVCC_FLAGS, *[f"-D{d}" for d in defines], "-c",
           os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    return obj, r.stdout + r.stderr


def build_binding(force: bool = False) -> str:
    """Compile _fa_torch.so unless an up-to-date build exists (for this torch and this
    Python)."""
    import sysconfig

    import torch

    at = os.path.dirname(os.path.abspath(torch.__file__))
    include = [os.path.join(at, "include"),
               os.path.join(at, "include", "torch", "csrc", "api", "include"),
               sysconfig.get_paths()["include"],
               os.path.join(os.path.dirname(_cuda_lib_dir()), "include")]
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *[f"-I{d}" for d in include], TORCH_SOURCE]
    libs = ["-L" + os.path.join(at, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    h = hashlib.sha256(" ".join([*cmd, *libs, torch.__version__, sys.version]).encode())
    for name in (TORCH_SOURCE, os.path.join(ROOT, "include", "fa.h")):
        with open(name, "rb") as f:
            h.update(f.read())
    os.makedirs(OBJ, exist_ok=True)
    stamp = os.path.join(OBJ, "fingerprint_torch")
    if (not force and os.path.exists(TORCH_LIB) and os.path.exists(stamp)
            and open(stamp).read() == h.hexdigest()):
        return TORCH_LIB
    tmp = TORCH_LIB + f".tmp{os.getpid()}"
    r = subprocess.run([*cmd, "-o", tmp, *libs], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for fa_torch.cpp:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, TORCH_LIB)
    with open(stamp, "w") as f:
        f.write(h.hexdigest())
    return TORCH_LIB


def build(force: bool = False, verbose: bool = False, defines=(),
          variant: str | None = None) -> str:
    """Compile and link the library, and the binding's compiled part, unless up-to-date
    builds exist.

    ``variant`` with ``defines`` (macro names, optionally NAME=VALUE) builds
    another copy of the same sources with those macros set, into
    ``_variants/libfa_gb300_<variant>.so``: the alternative arms of paired
    measurements (bench.py --paired).  The in-tree library is unaffected."""
    defines = tuple(defines)
    obj_dir, lib = OBJ, LIB
    if variant is not None:
        obj_dir = os.path.join(PKG, "_variants", f"objs_{variant}")
        lib = os.path.join(PKG, "_variants", f"libfa_gb300_{variant}.so")
    os.makedirs(obj_dir, exist_ok=True)
    stamp = os.path.join(obj_dir, "fingerprint")
    fp = _fingerprint() + " ".join(defines)
    if (not force and os.path.exists(lib) and os.path.exists(stamp)
            and open(stamp).read() == fp):
        if variant is None:
            build_binding()
        return lib
    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        binding = ex.submit(build_binding, force) if variant is None else None
        results = list(ex.map(lambda s: _compile(s, obj_dir, defines), SOURCES))
        if binding is not None:
            binding.result()
    with open(os.path.join(obj_dir, "ptxas.log"), "w") as f:
        for (obj, log), src in zip(results, SOURCES):
            f.write(f"==== {src}\n{log}\n")
    tmp = lib + f".tmp{os.getpid()}"
    cmd = [nvcc(), *ARCH, "-shared", "--cudart", "shared", "-o", tmp,
           *[o for o, _ in results], f"-L{_cuda_lib_dir()}",
           "-Xlinker", f"-rpath,{_cuda_lib_dir()}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib)
    with open(stamp, "w") as f:
        f.write(fp)
    if verbose:
        print(open(os.path.join(obj_dir, "ptxas.log")).read())
    return lib


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
