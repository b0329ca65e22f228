"""Build the C-ABI shared library libdflash_attn.so in-tree with nvcc (sm_103a), and
the Python entry of the serving operators (_dflash_binding.so) with g++ against
the installed torch.

Each translation unit compiles in parallel; the link steps produce
``dflash_block_draft_gb300/_lib/libdflash_attn.so`` and, linked to it,
``_lib/_dflash_binding.so``.  Object files go to
``dflash_block_draft_gb300/_build/``.  Both are git-ignored.

The library needs nvcc alone.  Where torch, Python's headers or the C++ compiler are
missing, it is built without the binding, which is said on stderr; the serving
operators' Python functions then raise, the C ABI is whole.
"""
from __future__ import annotations

import concurrent.futures as cf
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OBJ_DIR = os.path.join(HERE, "_build")
LIB_DIR = os.path.join(HERE, "_lib")
LIB_PATH = os.path.join(LIB_DIR, "libdflash_attn.so")
BINDING_PATH = os.path.join(LIB_DIR, "_dflash_binding.so")

SOURCES = ["api.cu", "attn_simt.cu", "attn_tc.cu", "mask_scan.cu", "dense_noalloc.cu",
           "attn_decode.cu", "attn_bwd.cu", "attn_bwd_tc.cu", "attn_latent.cu", "api_serving.cu", "qk_norm_rope.cu",
           "attn_paged.cu", "attn_paged_tc.cu", "verify.cu", "sample.cu", "tree_accept.cu", "cache_move.cu", "pages.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
              "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the DFlash CUDA library cannot be built")


def _deps():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [os.path.join(INCLUDE, "dflash_attn.h"), __file__]
    return max(os.path.getmtime(f) for f in files)


def _compiled_against() -> str:
    """The Python and torch that a binding compiled now fits (torch itself is not imported)."""
    with open(os.path.join(_torch_dir(), "version.py")) as f:
        return f"{sysconfig.get_config_var('SOABI')}\n{_torch_dir()}\n{f.read()}"


def _stamp() -> str:
    return os.path.join(OBJ_DIR, "binding.for")


def _binding_fits() -> bool:
    try:
        with open(_stamp()) as f:
            return f.read() == _compiled_against()
    except OSError:
        return False


def up_to_date() -> bool:
    newest = _deps()
    lacks = binding_lacks()
    need = [LIB_PATH] if lacks else [LIB_PATH, BINDING_PATH]
    return all(os.path.exists(p) and os.path.getmtime(p) >= newest for p in need) and bool(lacks or _binding_fits())


def _torch_dir() -> str | None:
    spec = importlib.util.find_spec("torch")
    return list(spec.submodule_search_locations)[0] if spec and spec.submodule_search_locations else None


def _cxx() -> str:
    return os.environ.get("CXX", "g++")


def binding_lacks() -> str | None:
    """What the binding needs and this machine does not have, or None."""
    if _torch_dir() is None:
        return "torch"
    if not os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        return "Python.h"
    if shutil.which(_cxx().split()[0]) is None:
        return f"the C++ compiler {_cxx()}"
    return None


def _run(cmd, what):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    return r


def _compile_binding() -> str:
    torch = _torch_dir()
    obj = os.path.join(OBJ_DIR, "binding.o")
    inc = [os.path.join(torch, "include"), os.path.join(torch, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include"), INCLUDE]
    _run([*_cxx().split(), "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-w",
          *[f"-I{d}" for d in inc], "-c", os.path.join(CSRC, "binding.cpp"), "-o", obj], "g++ on binding.cpp")
    return obj


def _link_binding(obj: str) -> None:
    torch = os.path.join(_torch_dir(), "lib")
    tmp = BINDING_PATH + f".{os.getpid()}.tmp"
    _run([*_cxx().split(), "-shared", "-o", tmp, obj, f"-L{LIB_DIR}", "-ldflash_attn", f"-L{torch}",
          "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{torch}"],
         "link of the binding")
    os.replace(tmp, BINDING_PATH)
    with open(_stamp(), "w") as f:
        f.write(_compiled_against())


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Compile and link the library and the binding if stale (or force).  Returns the library's path."""
    if not force and not extra_flags and up_to_date():
        return LIB_PATH
    os.makedirs(OBJ_DIR, exist_ok=True)
    os.makedirs(LIB_DIR, exist_ok=True)
    cc = nvcc()

    def compile_one(src):
        obj = os.path.join(OBJ_DIR, os.path.splitext(src)[0] + ".o")
        cmd = [cc, *ARCH, *NVCC_FLAGS, *extra_flags, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            sys.stderr.write(r.stdout + r.stderr)
        return obj

    lacks = binding_lacks()
    with cf.ThreadPoolExecutor(max_workers=min(len(SOURCES) + 1, os.cpu_count() or 4)) as ex:
        binding = None if lacks else ex.submit(_compile_binding)
        objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB_PATH + f".{os.getpid()}.tmp"
    cmd = [cc, *ARCH, "-shared", "-o", tmp, *objs, "-ldl", "-lrt",
           "-lpthread"]
    _run(cmd, "link")
    os.replace(tmp, LIB_PATH)
    linked = False
    try:
        if lacks:
            sys.stderr.write(f"{lacks} not found: built without the Python binding of the serving operators\n")
        else:
            _link_binding(binding.result())
            linked = True
    finally:
        if not linked and os.path.exists(BINDING_PATH):
            os.remove(BINDING_PATH)  # it speaks to an older library
    return LIB_PATH


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True,
                extra_flags=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else ()))
