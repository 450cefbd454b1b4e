"""Build the CUDA library in-tree for sm_100a.

    python -m structured_sparse_attention_fibonacci_b200.build [--force] [--ptxas-v]

Compiles csrc/*.cu with nvcc (one object per source, in parallel) and links
them into two plain C-ABI shared libraries next to this file, which the Python
binding loads with ctypes:
  libsparse_attn.so         the library;
  libsparse_attn_bounds.so  the same sources compiled with SA_DEBUG_BOUNDS:
                            every staged row a kernel reads is checked against
                            the rows its shared-memory ring holds, and every
                            staging round against the ring's size; a violation
                            sets bit 1 of the device error word (no trap), so
                            the parity tests can run under it in place of a
                            memory checker;
and csrc/sa_binding.cpp with nvcc's host compiler, against the installed torch:
  _binding.so               extension module behind paged.py's calls;
  _binding.built_for        the torch and the Python that it was built for: another
                            one's classes and interface may differ, so it is built
                            again for them.
"""
import concurrent.futures as cf
import glob
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libsparse_attn.so")
LIB_BOUNDS = os.path.join(HERE, "libsparse_attn_bounds.so")
BINDING = os.path.join(HERE, "_binding.so")
BINDING_FOR = os.path.join(HERE, "_binding.built_for")
BINDING_SRC = os.path.join(CSRC, "sa_binding.cpp")
OBJ_DIR = os.path.join(HERE, "_build")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
    "--expt-relaxed-constexpr",
]

VARIANTS = {LIB: [], LIB_BOUNDS: ["-DSA_DEBUG_BOUNDS"]}


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _built_for():
    """The installed torch and Python, as far as compiled code depends on them."""
    import torch
    return (f"torch {torch.__version__} cxx11_abi {int(torch._C._GLIBCXX_USE_CXX11_ABI)} "
            f"{sysconfig.get_config_var('SOABI')}\n")


def _stale(lib):
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    if lib == BINDING:
        if not os.path.exists(BINDING_FOR):
            return True
        with open(BINDING_FOR) as f:
            if f.read() != _built_for():
                return True
        deps = (BINDING_SRC, os.path.join(INCLUDE, "sparse_attn.h"), os.path.abspath(__file__))
        return any(os.path.getmtime(d) > t for d in deps)
    deps = sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
    deps += glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)]
    return any(os.path.getmtime(d) > t for d in deps)


def _compile(nvcc, src, obj, extra, verbose):
    cmd = [nvcc, *NVCC_FLAGS, *extra, "-I", INCLUDE, "-I", CSRC, "-c", src, "-o", obj]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.check_call(cmd)
    return obj


def _build_binding(nvcc, verbose):
    import torch
    base = os.path.dirname(torch.__file__)
    tmp = BINDING + f".tmp{os.getpid()}"
    cmd = [nvcc, "-gencode", "arch=compute_100a,code=sm_100a", "-O2", "-std=c++17", "-shared",
           "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-isystem", os.path.join(base, "include"),
           "-isystem", os.path.join(base, "include", "torch", "csrc", "api", "include"),
           "-isystem", sysconfig.get_path("include"), "-I", INCLUDE, BINDING_SRC,
           "-L", os.path.join(base, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda",
           "-cudart", "none", "-o", tmp]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.check_call(cmd)
    if os.path.exists(BINDING_FOR):
        os.remove(BINDING_FOR)      # an interrupted build leaves a stale one
    os.replace(tmp, BINDING)
    with open(tmp, "w") as f:
        f.write(_built_for())
    os.replace(tmp, BINDING_FOR)


def build(force: bool = False, verbose: bool = False, extra=(), variants=None) -> str:
    """Compile the stale libraries (all with force); returns the main library's path."""
    nvcc = os.environ.get("NVCC", "nvcc")
    todo = [lib for lib in (variants or VARIANTS) if force or _stale(lib)]
    binding = force or _stale(BINDING)
    if not todo and not binding:
        return LIB
    os.makedirs(OBJ_DIR, exist_ok=True)
    jobs = []
    with cf.ThreadPoolExecutor(max_workers=max(1, min(16, os.cpu_count() or 1))) as ex:
        if binding:
            jobs.append(ex.submit(_build_binding, nvcc, verbose))
        for lib in todo:
            tag = os.path.splitext(os.path.basename(lib))[0]
            objs = []
            for src in sources():
                obj = os.path.join(OBJ_DIR, f"{tag}.{os.path.basename(src)}.o")
                objs.append(obj)
                jobs.append(ex.submit(_compile, nvcc, src, obj, [*VARIANTS[lib], *extra], verbose))
            jobs.append((lib, objs))
        futures = [j for j in jobs if not isinstance(j, tuple)]
        for f in futures:
            f.result()
    for j in jobs:
        if isinstance(j, tuple):
            lib, objs = j
            tmp = lib + f".tmp{os.getpid()}"
            subprocess.check_call([nvcc, "-gencode", "arch=compute_100a,code=sm_100a", "-shared",
                                   *objs, "-o", tmp])
            os.replace(tmp, lib)
    return LIB


if __name__ == "__main__":
    extra = ["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else []
    print(build(force="--force" in sys.argv or bool(extra), verbose=True, extra=extra))
