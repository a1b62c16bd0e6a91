"""Compile the sm_103a shared library in place (nvcc, no cmake).

``build()`` writes ``libsdpa_gb300.so`` next to this file.  Each translation
unit is compiled by its own nvcc process, in parallel, for exactly one target:
``-gencode arch=compute_103a,code=sm_103a``.  Then ``_sdpa_binding.so``, the
paged operators' binding on torch tensors (g++ with torch's headers; its
compilation runs beside the others).  The library, a C ABI, needs no torch:
where there is none, it is all that is built.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sysconfig
import tempfile

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(os.path.dirname(PKG), "include")
LIB_NAME = "libsdpa_gb300.so"
LIB_PATH = os.path.join(PKG, LIB_NAME)
BINDING_PATH = os.path.join(PKG, "_sdpa_binding.so")
BINDING_SOURCE = "sdpa_binding.cpp"

SOURCES = ["sdpa_fwd_sm103a.cu", "sdpa_fwd64_sm103a.cu", "sdpa_sparse_sm103a.cu",
           "sdpa_cache_sm103a.cu", "sdpa_paged_sm103a.cu", "sdpa_paged_tc_sm103a.cu",
           "sdpa_pages_sm103a.cu", "sdpa_norm_sm103a.cu", "sdpa_norm64_sm103a.cu",
           "sdpa_api.cpp", "sdpa_paged_api.cpp", "sdpa_pages_api.cpp"]
GENCODE = ["-gencode", "arch=compute_103a,code=sm_103a"]
COMMON = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC",
          "-Xcompiler", "-fvisibility=hidden", "-I", INCLUDE, "-I", CSRC]


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the sm_103a library cannot be built")
    return cand


def _inputs():
    """Sources of the library (the header last)."""
    deps = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f != BINDING_SOURCE]
    deps.append(os.path.join(INCLUDE, "sdpa.h"))
    return deps


def _have_torch() -> bool:
    try:
        import torch  # noqa: F401
    except ImportError:
        return False
    return True


def binding_key() -> str:
    """What a binding belongs to: its code reads torch's and Python's objects as the headers lay them out."""
    import torch

    # (the suffix names Python's version and the machine)
    return (f"{sysconfig.get_config_var('EXT_SUFFIX')}, torch {torch.__version__} {torch.version.git_version}, C++ ABI "
            f"{int(torch._C._GLIBCXX_USE_CXX11_ABI)}")


def binding_key_path() -> str:
    return BINDING_PATH + ".built_for"


def binding_built_for() -> str | None:
    """The key of the binding that is there (None: it does not say)."""
    try:
        with open(binding_key_path(), encoding="utf-8") as f:
            return f.read()
    except OSError:
        return None


def _binding_commands(obj: str, out: str):
    """Compiler and linker commands of the binding."""
    import torch
    from torch.utils.cpp_extension import include_paths

    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    cuda = os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include")
    inc = [x for p in (*include_paths(), cuda, sysconfig.get_paths()["include"]) for x in ("-isystem", p)]
    cxx = shutil.which("g++") or "g++"
    abi = "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch._C._GLIBCXX_USE_CXX11_ABI)
    return ([cxx, "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", abi, *inc, "-c", os.path.join(CSRC, BINDING_SOURCE), "-o", obj],
            [cxx, "-shared", "-o", out, obj, "-L" + PKG, "-l:" + LIB_NAME, "-L" + lib, "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python",
             "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + lib])


def _newer(built: str, inputs) -> bool:
    return os.path.exists(built) and all(os.path.getmtime(d) <= os.path.getmtime(built) for d in inputs)


def _library_up_to_date() -> bool:
    return _newer(LIB_PATH, _inputs())


def _binding_up_to_date() -> bool:
    return binding_built_for() == binding_key() and \
        _newer(BINDING_PATH, [os.path.join(CSRC, BINDING_SOURCE), os.path.join(INCLUDE, "sdpa.h")])


def up_to_date() -> bool:
    return _library_up_to_date() and (not _have_torch() or _binding_up_to_date())


def _finish(proc, cmd, what: str) -> None:
    out, _ = proc.communicate()
    if proc.returncode != 0:
        raise RuntimeError(f"{what} failed ({' '.join(cmd)}):\n{out.decode()}")


def _start(cmd, verbose: bool):
    if verbose:
        print(" ".join(cmd))
    return subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)


def _install(made: str, path: str) -> None:
    shutil.copyfile(made, path + ".tmp")
    os.replace(path + ".tmp", path)


def build(force: bool = False, verbose: bool = False) -> str:
    """Build ``libsdpa_gb300.so`` and, with torch, the binding, each if one of its
    sources is newer (the binding also if it belongs to another torch or Python);
    return the library's path."""
    library = force or not _library_up_to_date()
    binding = _have_torch() and (force or not _binding_up_to_date())
    if not library and not binding:
        return LIB_PATH
    with tempfile.TemporaryDirectory(prefix="sdpa_build_") as tmp:
        procs, objs = [], []
        if binding:
            made = os.path.join(tmp, "binding.so")
            compile_binding, link_binding = _binding_commands(os.path.join(tmp, "binding.o"), made)
            binding_proc = _start(compile_binding, verbose)
        if library:
            nvcc = _nvcc()
            for src in SOURCES:
                obj = os.path.join(tmp, os.path.splitext(src)[0] + ".o")
                cmd = [nvcc, *GENCODE, *COMMON, "-c", os.path.join(CSRC, src), "-o", obj]
                procs.append((_start(cmd, verbose), cmd))
                objs.append(obj)
            for p, cmd in procs:
                _finish(p, cmd, "nvcc")
            tmp_lib = os.path.join(tmp, LIB_NAME)
            link = [nvcc, *GENCODE, "-shared", "-o", tmp_lib, *objs]
            _finish(_start(link, verbose), link, "link")
            _install(tmp_lib, LIB_PATH)
        if binding:
            _finish(binding_proc, compile_binding, "g++")
            _finish(_start(link_binding, verbose), link_binding, "link")
            key = os.path.join(tmp, "key")
            with open(key, "w", encoding="utf-8") as f:
                f.write(binding_key())
            # (one that is cut short here says nothing, and is made again)
            if os.path.exists(binding_key_path()):
                os.unlink(binding_key_path())
            _install(made, BINDING_PATH)
            _install(key, binding_key_path())
    return LIB_PATH


if __name__ == "__main__":
    print(build(force=True, verbose=True))
