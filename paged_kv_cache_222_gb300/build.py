"""Build libpkv.so (the C-ABI library) in-tree with nvcc for sm_103a, and
_binding.so, the compiled Python entry of its most frequent calls.

Each CUDA translation unit is compiled in parallel, then linked into a shared
library next to this file.  CUDA's runtime is linked statically and the driver
entry point for tensor-map encoding is looked up at run time, so the library
loads on a machine without a GPU driver (only calls that reach the GPU need
one).  Rebuilds only when a source or header is newer than the library, or the
Python or PyTorch that the binding was built against is another.

The library needs neither Python's nor PyTorch's headers: where the binding
does not compile, the library is built all the same and the compiler's message
printed; the calls that need the binding then raise.

    python -m paged_kv_cache_222_gb300.build [--force] [--verbose]
"""

import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG, "_build")
LIB_PATH = os.path.join(PKG, "libpkv.so")
BINDING_PATH = os.path.join(PKG, "_binding.so")

SOURCES = ["api.cu", "append.cu", "decode.cu", "cascade.cu", "multi_query.cu", "blocks.cu", "chunk.cu", "chunk_tc.cu", "rotary.cu",
           "compact.cu", "block_manager.cpp"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc():
    exe = shutil.which("nvcc")
    if exe is None and os.path.exists("/usr/local/cuda/bin/nvcc"):
        exe = "/usr/local/cuda/bin/nvcc"
    if exe is None:
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libpkv.so")
    return exe


def _inputs():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)]
    files.append(os.path.abspath(__file__))
    return files


def _newest(path):
    """No source is newer than the built file."""
    return os.path.exists(path) and all(os.path.getmtime(f) <= os.path.getmtime(path) for f in _inputs())


def _binding_against():
    """What the binding is built against: another Python or PyTorch needs another."""
    import torch
    return f"{sys.version}\n{torch.__version__}\n{os.path.dirname(torch.__file__)}\n"


def _stamp_path():
    return BINDING_PATH + ".against"


def _binding_up_to_date():
    if not _newest(BINDING_PATH) or not os.path.exists(_stamp_path()):
        return False
    with open(_stamp_path()) as f:
        return f.read() == _binding_against()


def up_to_date():
    return _newest(LIB_PATH) and _binding_up_to_date()


def _binding_command(out):
    """g++ command of the Python extension module against the installed PyTorch."""
    import sysconfig

    import torch
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    inc = [INCLUDE, os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
           os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    return ([shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared",
             f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"] + [f"-I{i}" for i in inc]
            + [os.path.join(CSRC, "binding.cpp"), "-o", out, "-L" + os.path.join(root, "lib"), "-ltorch_python",
               "-ltorch_cuda", "-ltorch_cpu", "-ltorch", "-lc10_cuda", "-lc10"])


def _start(cmd, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    return subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)


def _start_binding(out, verbose):
    """The running compiler, or the reason there is none."""
    try:
        return _start(_binding_command(out), verbose), ""
    except (ImportError, OSError) as e:
        return None, f"{type(e).__name__}: {e}"


def _finish_binding(started, tmp, verbose):
    proc, text = started
    if proc is not None:
        text = proc.communicate()[0].decode(errors="replace")
        if proc.returncode == 0:
            if verbose:
                sys.stdout.write(text)
            os.replace(tmp, BINDING_PATH)
            with open(_stamp_path(), "w") as f:
                f.write(_binding_against())
            return
    for stale in (BINDING_PATH, _stamp_path()):  # of other sources or another PyTorch
        if os.path.exists(stale):
            os.remove(stale)
    print(f"the compiled binding was not built (libpkv.so does not need it):\n{text}", file=sys.stderr, flush=True)


def build(force=False, verbose=False, ptxas_verbose=False):
    """Compile and link libpkv.so, and the binding where it compiles; returns the
    library's path."""
    lib, binding = force or not _newest(LIB_PATH), force or not _binding_up_to_date()
    if not lib and not binding:
        return LIB_PATH
    os.makedirs(BUILD_DIR, exist_ok=True)
    binding_tmp = BINDING_PATH + ".tmp"
    started = _start_binding(binding_tmp, verbose) if binding else None
    try:
        if lib:
            _build_library(verbose, ptxas_verbose)
    finally:
        if binding:
            _finish_binding(started, binding_tmp, verbose or ptxas_verbose)
    return LIB_PATH


def _build_library(verbose, ptxas_verbose):
    cc = nvcc()
    common = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                     "-I", INCLUDE, "-I", CSRC, "--expt-relaxed-constexpr"]
    if ptxas_verbose:
        common += ["-Xptxas", "-v"]
    procs = []
    objs = []
    for src in SOURCES:
        obj = os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".o")
        objs.append(obj)
        procs.append((src, _start([cc] + common + ["-c", os.path.join(CSRC, src), "-o", obj], verbose)))
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        text = out.decode(errors="replace")
        if p.returncode != 0:
            failed.append((src, text))
        elif verbose or ptxas_verbose:
            sys.stdout.write(text)
    if failed:
        msg = "\n".join(f"--- {s}\n{t}" for s, t in failed)
        raise RuntimeError(f"compilation failed:\n{msg}")
    tmp = LIB_PATH + ".tmp"
    p = _start([cc] + ARCH + ["-shared", "-o", tmp] + objs + ["-cudart", "static"], verbose)
    out, _ = p.communicate()
    if p.returncode != 0:
        raise RuntimeError("link failed:\n" + out.decode(errors="replace"))
    os.replace(tmp, LIB_PATH)


if __name__ == "__main__":
    force = "--force" in sys.argv
    verbose = "--verbose" in sys.argv
    print(build(force=force, verbose=verbose, ptxas_verbose="--ptxas" in sys.argv))
