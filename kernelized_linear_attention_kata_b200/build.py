"""Build the KATA CUDA library (libkata.so) in-tree for sm_100a with nvcc.

    python -m kernelized_linear_attention_kata_b200.build [--force] [--verbose]

The library is a plain C-ABI shared object (see include/kata.h); nothing in
it depends on PyTorch. The CUDA runtime is linked statically, the driver API
(needed for TMA descriptors) is resolved at run time through the runtime's
driver entry-point query, so the .so runs on any machine with the driver.
After it, and not needed by it, _binding-<torch><python>.so marshals the gated delta
rule's calls for Python (csrc/binding.cpp, built against the installed torch).
"""

from __future__ import annotations

import argparse
import glob
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB_PATH = os.path.join(PKG_DIR, "libkata.so")
BINDING_SRC = os.path.join(CSRC, "binding.cpp")

ARCH_FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "--expt-relaxed-constexpr",
              "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden"]


def nvcc_path() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the KATA CUDA library cannot be built")


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps() -> list[str]:
    return (sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
            + glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)])


def up_to_date() -> bool:
    if not os.path.exists(LIB_PATH):
        return False
    t = os.path.getmtime(LIB_PATH)
    return all(os.path.getmtime(p) <= t for p in _deps())


def binding_path() -> str:
    """Where the binding for this torch and this Python lies: it holds their inline
    code and runs with no other, so both are in its name."""
    import torch
    abi = int(torch._C._GLIBCXX_USE_CXX11_ABI)
    return os.path.join(PKG_DIR, f"_binding-torch{torch.__version__}-abi{abi}{sysconfig.get_config_var('EXT_SUFFIX')}")


def build_binding(force: bool = False, verbose: bool = False) -> str:
    path = binding_path()
    deps = [BINDING_SRC, os.path.abspath(__file__), *glob.glob(os.path.join(INCLUDE, "*.h"))]
    if not force and os.path.exists(path) and all(os.path.getmtime(p) <= os.path.getmtime(path) for p in deps):
        return path
    import torch
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc_path())))
    includes = [INCLUDE, os.path.join(root, "include"),
                os.path.join(root, "include", "torch", "csrc", "api", "include"),
                sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    tmp = path + ".tmp"
    # the system's g++, as nvcc uses it: the C++ runtime has to be the one torch uses
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *(f"-I{p}" for p in includes), BINDING_SRC, "-o", tmp, f"-L{os.path.join(root, 'lib')}",
           "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    if verbose:
        print(" ".join(cmd), flush=True)
    done = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
    if done.returncode != 0:
        raise RuntimeError(f"binding failed to build:\n{done.stdout.decode(errors='replace')}")
    os.replace(tmp, path)
    return path


def build(force: bool = False, verbose: bool = False, extra: list[str] | None = None) -> str:
    """The library, then the binding. A binding that cannot be built (no torch, no
    Python headers, another compiler) is a warning: every other call works without."""
    path = build_library(force, verbose, extra)
    try:
        build_binding(force, verbose)
    except (ImportError, OSError, RuntimeError) as e:
        warnings.warn(f"the gated delta rule cannot be called from Python, its binding was not built: {e}",
                      RuntimeWarning, stacklevel=2)
    return path


def build_library(force: bool = False, verbose: bool = False, extra: list[str] | None = None) -> str:
    if not force and up_to_date():
        return LIB_PATH
    nvcc = nvcc_path()
    objdir = os.path.join(PKG_DIR, "_build")
    os.makedirs(objdir, exist_ok=True)
    objs = []
    procs = []
    for src in sources():
        obj = os.path.join(objdir, os.path.basename(src) + ".o")
        cmd = [nvcc, *ARCH_FLAGS, *NVCC_FLAGS, "-I", INCLUDE, "-I", CSRC, "-c",
               src, "-o", obj, *(extra or [])]
        if verbose:
            print(" ".join(cmd), flush=True)
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
        objs.append(obj)
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        text = out.decode(errors="replace")
        if p.returncode != 0:
            failed.append((src, text))
        elif verbose and text.strip():
            print(text)
    if failed:
        msg = "\n".join(f"--- {s}\n{t}" for s, t in failed)
        raise RuntimeError(f"nvcc failed:\n{msg}")
    tmp = LIB_PATH + ".tmp"
    cmd = [nvcc, *ARCH_FLAGS, "-shared", "-o", tmp, *objs, "-cudart", "static", "-ldl", "-lrt",
           "-lpthread"]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__)
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    ap.add_argument("--ptxas-info", action="store_true", help="print registers / spills per kernel")
    a = ap.parse_args(argv)
    extra = ["-Xptxas", "-v"] if a.ptxas_info else None
    path = build(force=a.force or a.ptxas_info, verbose=a.verbose or a.ptxas_info, extra=extra)
    print(path)


if __name__ == "__main__":
    sys.exit(main())
