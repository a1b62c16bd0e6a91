"""Compile the sm_103a shared library in place (nvcc, no cmake).

``build()`` writes ``libsdpa_gb300.so`` next to this file.  Each translation
unit is compiled by its own nvcc process, in parallel, for exactly one target:
``-gencode arch=compute_103a,code=sm_103a``.  Then ``_sdpa_binding.so``, the
paged operators' binding on torch tensors (g++ with torch's headers; its
compilation runs beside the others).
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
    deps = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    deps.append(os.path.join(INCLUDE, "sdpa.h"))
    return deps


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


def up_to_date() -> bool:
    if not os.path.exists(LIB_PATH) or not os.path.exists(BINDING_PATH):
        return False
    t = min(os.path.getmtime(LIB_PATH), os.path.getmtime(BINDING_PATH))
    return all(os.path.getmtime(d) <= t for d in _inputs())


def build(force: bool = False, verbose: bool = False) -> str:
    """Build ``libsdpa_gb300.so`` and the binding if any source is newer; return the library's path."""
    if not force and up_to_date():
        return LIB_PATH
    nvcc = _nvcc()
    with tempfile.TemporaryDirectory(prefix="sdpa_build_") as tmp:
        procs, objs = [], []
        binding, link_binding = _binding_commands(os.path.join(tmp, "binding.o"), os.path.join(tmp, "binding.so"))
        binding_proc = subprocess.Popen(binding, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
        for src in SOURCES:
            obj = os.path.join(tmp, os.path.splitext(src)[0] + ".o")
            cmd = [nvcc, *GENCODE, *COMMON, "-c", os.path.join(CSRC, src), "-o", obj]
            if verbose:
                print(" ".join(cmd))
            procs.append((subprocess.Popen(cmd, stdout=subprocess.PIPE,
                                           stderr=subprocess.STDOUT), cmd))
            objs.append(obj)
        for p, cmd in procs:
            out, _ = p.communicate()
            if p.returncode != 0:
                raise RuntimeError(f"nvcc failed ({' '.join(cmd)}):\n{out.decode()}")
        tmp_lib = os.path.join(tmp, LIB_NAME)
        link = [nvcc, *GENCODE, "-shared", "-o", tmp_lib, *objs]
        r = subprocess.run(link, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}{r.stderr}")
        shutil.copyfile(tmp_lib, LIB_PATH + ".tmp")
        os.replace(LIB_PATH + ".tmp", LIB_PATH)
        out, _ = binding_proc.communicate()
        if binding_proc.returncode != 0:
            raise RuntimeError(f"g++ failed ({' '.join(binding)}):\n{out.decode()}")
        r = subprocess.run(link_binding, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}{r.stderr}")
        shutil.copyfile(os.path.join(tmp, "binding.so"), BINDING_PATH + ".tmp")
        os.replace(BINDING_PATH + ".tmp", BINDING_PATH)
    return LIB_PATH


if __name__ == "__main__":
    print(build(force=True, verbose=True))
