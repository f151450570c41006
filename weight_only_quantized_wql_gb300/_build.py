"""Build libwql.so in-tree with nvcc for sm_103a, and the compiled half of the
Python binding with g++ (no cmake).

Each .cu file is compiled in its own nvcc process (in parallel), then linked
with ``nvcc -shared``; ``binding.cpp`` against the torch that is installed.  The
results land in ``_build/libwql.so`` and ``_build/_wql_torch.so`` beside this
file; each is rebuilt only when a source or header of its own is newer, the
binding also when another torch or Python is installed.  The library needs
neither torch nor Python's headers (``--library``: it alone).
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "libwql.so")
BINDING = os.path.join(BUILD, "_wql_torch.so")
BINDING_SRC = os.path.join(CSRC, "binding.cpp")
BINDING_FOR = os.path.join(BUILD, "_wql_torch.for")     # the torch and Python it was built for
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2",
              "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def _nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found; the CUDA toolkit is required to build libwql")
    return path


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _library_inputs() -> list[str]:
    return (sources() + glob.glob(os.path.join(CSRC, "*.cuh")) +
            glob.glob(os.path.join(CSRC, "*.h")) + [os.path.join(INCLUDE, "wql.h")])


def _newer_than(target: str, inputs: list[str]) -> bool:
    if not os.path.exists(target):
        return False
    t = os.path.getmtime(target)
    return all(os.path.getmtime(p) <= t for p in inputs)


def _built_for() -> str:
    import torch
    return f"torch {torch.__version__}, {sysconfig.get_config_var('SOABI')}"


def library_up_to_date() -> bool:
    return _newer_than(LIB, _library_inputs())


def binding_up_to_date() -> bool:
    if not _newer_than(BINDING, [BINDING_SRC, os.path.join(INCLUDE, "wql.h")]):
        return False
    if not os.path.exists(BINDING_FOR):
        return False
    with open(BINDING_FOR) as f:
        return f.read() == _built_for()


def up_to_date() -> bool:
    return library_up_to_date() and binding_up_to_date()


def _run(what: str, cmd: list[str], verbose: bool = False) -> None:
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr[-4000:]}")
    if verbose and (r.stdout or r.stderr):
        print(r.stdout, r.stderr, flush=True)


def _link(what: str, target: str, cmd: list[str]) -> None:
    tmp = target + f".tmp{os.getpid()}"
    _run(what, [*cmd, "-o", tmp])
    os.replace(tmp, target)


def _compile_binding() -> str:
    import torch
    torch_inc = os.path.join(os.path.dirname(torch.__file__), "include")
    obj = os.path.join(BUILD, "binding.o")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_nvcc()))), "include")
    inc = [torch_inc, os.path.join(torch_inc, "torch", "csrc", "api", "include"), cuda,
           sysconfig.get_paths()["include"], INCLUDE]
    _run(f"g++ on {BINDING_SRC}",
         ["g++", "-O2", "-std=c++17", "-fPIC", "-c", BINDING_SRC, "-o", obj,
          f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
          "-DTORCH_EXTENSION_NAME=_wql_torch", *(f"-I{i}" for i in inc)])
    return obj


def _link_binding(obj: str) -> None:
    import torch
    torch_lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    # the library beside it is found by name, so that both are one instance
    _link("link of the binding", BINDING,
          ["g++", "-shared", obj, f"-L{BUILD}", "-l:libwql.so", "-Wl,-rpath,$ORIGIN",
           f"-L{torch_lib}", "-ltorch", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python", "-lc10",
           "-lc10_cuda"])
    with open(BINDING_FOR, "w") as f:
        f.write(_built_for())


def build(force: bool = False, verbose: bool = False, extra_flags: list[str] | None = None,
          library: bool = True, binding: bool = True) -> str:
    """Build what is stale of the library and of the compiled half of the Python
    binding.  The library is linked first; a binding that cannot be built raises
    after that."""
    library = library and (force or not library_up_to_date())
    binding = binding and (force or not binding_up_to_date())
    if not library and not binding:
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    flags = NVCC_FLAGS + list(extra_flags or [])

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        _run(f"nvcc on {src}", [nvcc, *ARCH, *flags, "-c", src, "-o", obj], verbose)
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(9, len(sources()) + 1)) as ex:
        binding_obj = ex.submit(_compile_binding) if binding else None
        objs = list(ex.map(compile_one, sources())) if library else []
    if library:
        _link("link", LIB, [nvcc, *ARCH, "-shared", "--cudart", "static", *objs])
    if binding_obj is not None:
        _link_binding(binding_obj.result())
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose=True, binding="--library" not in sys.argv))
