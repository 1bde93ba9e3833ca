"""Build libls_sampler.so in-tree with nvcc for sm_103a.

    python -m logits_sampling_gb300.build [--force]

Compiles logits_sampling_gb300/csrc/*.cu and csrc/ops/*.cu into logits_sampling_gb300/libls_sampler.so
(-gencode arch=compute_103a,code=sm_103a, -O3, -lineinfo, no fast-math).  The
build is skipped when the library is newer than every source and header.

The Python calls of include/ls_row_ops.h and ls_token_ops.h (csrc/py) are a small
extension module over torch's C++ tensors, _row_ops_c.so, compiled beside it
with g++ against the installed torch's headers.  _row_ops_c.for says which torch
and Python that was: with others it is compiled again, and not loaded.

VARIANTS holds test-only builds of the same sources with other compile-time
constants (never loaded by the package itself): ``reselect`` puts the top-p
candidate bound above every cut, so every top-p row takes the re-select over
all of its entries -- the path that otherwise runs only when rounding beats
the bound's slack.
"""
import glob
import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libls_sampler.so")
BINDING = os.path.join(PKG, "_row_ops_c.so")
BINDING_FOR = os.path.join(PKG, "_row_ops_c.for")
BINDING_SOURCE = os.path.join(CSRC, "py", "row_ops_py.cpp")
ARCH_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a"]
VARIANTS = {"reselect": ["-DLS_TOPP_SLACK=-64.0f"]}


def variant_path(name):
    return os.path.join(PKG, f"libls_sampler_{name}.so")


def _nvcc():
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libls_sampler.so")


def _binding_command(out):
    """The compiler's command line for the extension module."""
    torch = os.path.dirname(importlib.util.find_spec("torch").origin)  # no import: only its headers are needed
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_nvcc()))), "include")
    include = [os.path.join(torch, "include"), os.path.join(torch, "include", "torch", "csrc", "api", "include"), cuda,
               sysconfig.get_paths()["include"]]
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", *[a for i in include for a in ("-isystem", i)], "-I",
            INCLUDE, BINDING_SOURCE, "-o", out, "-L", os.path.join(torch, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu",
            "-ltorch_python"]


def binding_target():
    """The torch and the Python that an extension module is for: it is linked against their ABIs."""
    try:
        version = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        import torch
        version = torch.__version__
    return f"torch {version}, {sys.implementation.cache_tag}"


def binding_built_for():
    """What binding_target() was when the extension module was compiled, "" when unknown."""
    if not os.path.exists(BINDING_FOR):
        return ""
    with open(BINDING_FOR) as f:
        return f.read().strip()


def _binding_up_to_date():
    if binding_built_for() != binding_target():
        return False
    t = os.path.getmtime(BINDING) if os.path.exists(BINDING) else 0
    inputs = glob.glob(os.path.join(CSRC, "py", "*")) + glob.glob(os.path.join(INCLUDE, "*.h"))
    return all(os.path.getmtime(p) <= t for p in inputs + [os.path.abspath(__file__)])


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "ops", "*.cu")))


def _inputs():
    return sources() + sorted(glob.glob(os.path.join(CSRC, "**", "*.cuh"), recursive=True)) + sorted(
        glob.glob(os.path.join(INCLUDE, "*.h"))) + [os.path.abspath(__file__)]


def up_to_date(lib=LIB):
    if not os.path.exists(lib):
        return False
    t = os.path.getmtime(lib)
    return all(os.path.getmtime(p) <= t for p in _inputs())


def build(force=False, verbose=False, variant=None):
    """Compile the shared library (or a test-only variant of VARIANTS);
    returns its path.  Each translation unit (one per kernel mode and cluster
    size, plus the C ABI) compiles in its own nvcc process, in parallel; the
    objects are then linked."""
    lib = LIB if variant is None else variant_path(variant)
    extra = [] if variant is None else VARIANTS[variant]
    if variant is None and (force or not _binding_up_to_date()):
        tmp = f"{BINDING}.tmp{os.getpid()}"
        binding = subprocess.Popen(_binding_command(tmp))
    else:
        binding = None
    try:
        _build_library(lib, extra, force, verbose, variant)
    finally:
        failed = binding is not None and binding.wait() != 0
    if failed:
        raise subprocess.CalledProcessError(1, "g++", f"compiling {BINDING_SOURCE} failed")
    if binding is not None:
        os.replace(tmp, BINDING)
        with open(tmp, "w") as f:
            f.write(binding_target() + "\n")
        os.replace(tmp, BINDING_FOR)
    return lib


def _build_library(lib, extra, force, verbose, variant):
    if not force and up_to_date(lib):
        return
    tag = f".{variant or 'main'}.tmp{os.getpid()}"
    objs, procs = [], []
    for src in sources():
        obj = os.path.join(PKG, os.path.basename(src)[:-3] + tag + ".o")
        cmd = [_nvcc(), *ARCH_FLAGS, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", *extra,
               "-I", INCLUDE, "-I", CSRC, "-c", src, "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
            print(" ".join(cmd))
        objs.append(obj)
        procs.append(subprocess.Popen(cmd))
    failed = [p.args[-3] for p in procs if p.wait() != 0]
    try:
        if failed:
            raise subprocess.CalledProcessError(1, "nvcc", f"compiling {failed} failed")
        tmp = lib + tag
        subprocess.run([_nvcc(), *ARCH_FLAGS, "-shared", *objs, "-o", tmp, "-lcudart"], check=True)
        os.replace(tmp, lib)
    finally:
        for o in objs:
            if os.path.exists(o):
                os.remove(o)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
    if "--variants" in sys.argv:
        for name in VARIANTS:
            print(build(force="--force" in sys.argv, variant=name))
