"""Build the sm_100a codec library (``libhq.so``) in-tree with nvcc, and the
extension through which Python calls the serving operators
(``_hq_torch-<python>-<torch>.so``) with g++.

Each ``csrc/*.cu`` file is compiled to an object in parallel, then linked
into ``kv_quantization_tile_b200/libhq.so`` with the CUDA runtime linked
statically; ``csrc/hq_torch.cpp`` is compiled against torch's headers and linked
to that library.  The build is skipped when both are newer than every source
and header; an extension built for another torch or Python has another name, so
it is neither loaded nor taken for this one.
"""
from __future__ import annotations

import glob
import os
import re
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OBJ = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libhq.so")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2",
                "--expt-relaxed-constexpr", "-I", os.path.join(ROOT, "include")]


def ext_path() -> str:
    """The extension for this Python and this torch, whose binary interfaces it uses."""
    import torch
    key = f"{sysconfig.get_config_var('SOABI')}-torch-{torch.__version__}-abi{int(torch._C._GLIBCXX_USE_CXX11_ABI)}"
    return os.path.join(PKG, f"_hq_torch-{re.sub('[^A-Za-z0-9.+-]', '_', key)}.so")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return (_sources() + [os.path.join(CSRC, "hq_torch.cpp")] + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
            + glob.glob(os.path.join(ROOT, "include", "*.h")) + [os.path.abspath(__file__)])


def stale() -> bool:
    ext = ext_path()
    if not (os.path.exists(LIB) and os.path.exists(ext)):
        return True
    t = min(os.path.getmtime(LIB), os.path.getmtime(ext))
    return any(os.path.getmtime(p) > t for p in _deps())


def _compile(src: str, extra: list[str]) -> str:
    obj = os.path.join(OBJ, os.path.basename(src)[:-3] + ".o")
    cmd = [NVCC, *FLAGS, *extra, "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    if r.stderr.strip():
        sys.stderr.write(r.stderr)
    return obj


def _run(cmd: list[str], what: str):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")


def _compile_ext() -> str:
    import torch
    from torch.utils import cpp_extension
    obj = os.path.join(OBJ, "hq_torch.o")
    inc = [*cpp_extension.include_paths(), os.path.join(os.path.dirname(os.path.dirname(NVCC)), "include"),
           sysconfig.get_paths()["include"]]
    _run(["g++", "-O2", "-fPIC", "-std=c++17", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
          *[f"-isystem{p}" for p in inc], "-c", os.path.join(CSRC, "hq_torch.cpp"), "-o", obj], "g++ for hq_torch.cpp")
    return obj


def _link_ext(obj: str):
    from torch.utils import cpp_extension
    ext = ext_path()
    tmp = ext + f".tmp{os.getpid()}"
    _run(["g++", "-shared", "-o", tmp, obj, LIB, *[f"-L{p}" for p in cpp_extension.library_paths()], "-lc10", "-lc10_cuda",
          "-ltorch_cpu", "-ltorch_python", "-Wl,-rpath,$ORIGIN"], "link of the extension")
    os.replace(tmp, ext)


def build(force: bool = False, ptxas_verbose: bool = False) -> str:
    """Compile (if stale) and return the path of libhq.so."""
    if not force and not stale():
        return LIB
    os.makedirs(OBJ, exist_ok=True)
    extra = ["-Xptxas", "-v"] if ptxas_verbose else []
    srcs = _sources()
    with ThreadPoolExecutor(max(1, min(len(srcs) + 1, os.cpu_count() or 1))) as ex:
        ext = ex.submit(_compile_ext)
        objs = list(ex.map(lambda s: _compile(s, extra), srcs))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [NVCC, *ARCH, "-shared", "-cudart", "static", "-Xlinker", "-soname=libhq.so", "-o", tmp, *objs]
    _run(cmd, "nvcc link")
    os.replace(tmp, LIB)
    _link_ext(ext.result())
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, ptxas_verbose="-v" in sys.argv))
