"""Build libttq.so (the HIP kernels and the C ABI) for gfx950 with hipcc, and
_binding.so (the serving operators' Python binding, host code only) with g++.

Both are built in-tree, next to this file, so they travel with the source
tree.  `python -m test_activation_aware_amd.build` or build() runs it; it
always recompiles.  Each source is compiled to an object of its own (in
parallel, under _build/), then the objects are linked.

The binding needs g++ and torch's headers, which the library does not: where
it does not compile, build() leaves the library, removes an earlier build's
binding and warns; the serving functions then raise when they are called."""
from __future__ import annotations

import concurrent.futures
import glob
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libttq.so")
BINDING = os.path.join(PKG, "_binding.so")
OBJDIR = os.path.join(PKG, "_build")

HIPCC_FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++17",
    "-fPIC",
    # packed fp32 VALU forms are kept out of the generated code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wno-unused-command-line-argument",
]


def hipcc() -> str:
    path = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(path):
        raise RuntimeError("hipcc not found; the TTQ HIP library cannot be built")
    return path


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.hip"))) + [os.path.join(CSRC, "api.cpp")]


def _compile_binding() -> tuple:
    import torch
    from torch.utils import cpp_extension
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    include = [*cpp_extension.include_paths(), os.path.join(rocm, "include"), sysconfig.get_paths()["include"]]
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = BINDING + ".tmp"
    # torch's own libraries are loaded before the module is imported
    cmd = ["g++", "-std=c++17", "-O2", "-fPIC", "-shared", "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM=1",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *[f"-I{i}" for i in include],
           os.path.join(CSRC, "binding.cpp"), "-o", tmp, "-L", libs, "-ltorch_python", "-ltorch_cpu", "-lc10",
           "-lc10_hip"]
    proc = subprocess.run(cmd, capture_output=True, text=True)
    if proc.returncode == 0:
        os.replace(tmp, BINDING)
    return BINDING, proc.returncode, " ".join(cmd), proc.stderr


def _compile(src: str) -> tuple:
    obj = os.path.join(OBJDIR, os.path.basename(src) + ".o")
    cmd = [hipcc(), *HIPCC_FLAGS, "-I", os.path.join(ROOT, "include"), "-c", "-o", obj, src]
    proc = subprocess.run(cmd, capture_output=True, text=True)
    errs = "\n".join(l for l in proc.stderr.splitlines() if "packed-fp32-ops" not in l)
    return obj, proc.returncode, " ".join(cmd), errs


def build(verbose: bool = False, jobs: int = 0) -> str:
    os.makedirs(OBJDIR, exist_ok=True)
    srcs = sources()
    jobs = jobs or min(16, len(srcs), os.cpu_count() or 1)
    with concurrent.futures.ThreadPoolExecutor(jobs) as ex:
        binding = ex.submit(_compile_binding)
        results = list(ex.map(_compile, srcs))
        try:
            binding = binding.result()
        except Exception as e:  # no g++, no torch
            binding = (BINDING, 1, "", f"{type(e).__name__}: {e}")
    for obj, rc, cmd, errs in results:
        if verbose:
            print(cmd, flush=True)
        if rc != 0:
            raise RuntimeError(f"the compiler failed ({rc}) on {obj}:\n{errs}")
        if verbose and errs.strip():
            print(errs, file=sys.stderr)
    tmp = LIB + ".tmp"
    cmd = [hipcc(), "--offload-arch=gfx950", "-shared", "-fPIC", "-o", tmp, *[r[0] for r in results]]
    if verbose:
        print(" ".join(cmd), flush=True)
    proc = subprocess.run(cmd, capture_output=True, text=True)
    if proc.returncode != 0:
        raise RuntimeError(f"link failed ({proc.returncode}):\n{proc.stderr}")
    os.replace(tmp, LIB)
    _, rc, cmd, errs = binding
    if verbose and cmd:
        print(cmd, flush=True)
    if rc != 0:
        if os.path.exists(BINDING):
            os.remove(BINDING)  # an earlier one may not fit this library
        warnings.warn(f"{LIB} is built; the serving operators' {os.path.basename(BINDING)} is not: {errs}",
                      RuntimeWarning, stacklevel=2)
    elif verbose and errs.strip():
        print(errs, file=sys.stderr)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
    sys.exit(0 if os.path.exists(BINDING) else 1)
