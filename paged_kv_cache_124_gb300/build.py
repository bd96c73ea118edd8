"""Build the C-ABI library libpa_gb300.so for sm_103a, and the binding's native
module _step_calls.so, in tree.

The library needs nvcc alone: each translation unit under csrc/ is compiled in
parallel and the objects are linked into paged_kv_cache_124_gb300/libpa_gb300.so.
The module, csrc/binding/, is compiled beside them by the host's C++ compiler
against PyTorch's headers and linked to the library.  Each is built again when
one of its own sources or headers is newer, the module also for another
PyTorch.

    python -m paged_kv_cache_124_gb300.build [--force] [--library]

--library: the library alone, for clients of the C ABI (no PyTorch).
"""

import concurrent.futures
import os
import platform
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OBJ_DIR = os.path.join(ROOT, "_build", "obj")
LIB = os.path.join(PKG, "libpa_gb300.so")
BINDING = os.path.join(CSRC, "binding", "step_calls.cpp")
MODULE = os.path.join(PKG, "_step_calls.so")
TORCH_STAMP = os.path.join(OBJ_DIR, "torch_version")      # PyTorch's version that the module was built for
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
COMMON = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC]


def _nvcc():
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found; the CUDA 13 toolkit is required to build libpa_gb300.so")
    return cand


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cu", ".cpp")))


def _public_headers():
    return [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE) if f.endswith(".h")]


def _library_inputs():
    hdrs = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    return sources() + hdrs + _public_headers() + [os.path.abspath(__file__)]


def _module_inputs():
    return [BINDING] + _public_headers() + [os.path.abspath(__file__)]


# ELF e_machine of a shared object built for this host (x86-64 or AArch64)
_ELF_MACHINE = {"x86_64": 62, "amd64": 62, "aarch64": 183, "arm64": 183}


def elf_matches_host(header, machine=None):
    """True if `header` (the first 20 bytes of a file) starts a 64-bit
    little-endian ELF object for this host's machine."""
    want = _ELF_MACHINE.get((machine or platform.machine()).lower())
    return (len(header) >= 20 and header[:4] == b"\x7fELF" and header[4] == 2 and header[5] == 1 and
            want is not None and int.from_bytes(header[18:20], "little") == want)


def _current(built, inputs):
    """The file exists, was built for this host's machine, and is newer than
    its inputs."""
    if not os.path.exists(built):
        return False
    with open(built, "rb") as f:
        if not elf_matches_host(f.read(20)):
            return False
    t = os.path.getmtime(built)
    return all(os.path.getmtime(p) <= t for p in inputs)


def library_up_to_date():
    return _current(LIB, _library_inputs())


def module_up_to_date():
    """As the library, and built for this PyTorch."""
    if not _current(MODULE, _module_inputs()) or not os.path.exists(TORCH_STAMP):
        return False
    import torch

    with open(TORCH_STAMP) as f:
        return f.read() == torch.__version__


def _compile(src, verbose):
    obj = os.path.join(OBJ_DIR, os.path.basename(src) + ".o")
    cmd = [_nvcc(), *ARCH, *COMMON, "-c", src, "-o", obj]
    if src.endswith(".cu") and verbose:
        cmd += ["-Xptxas", "-v"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("nvcc failed for %s:\n%s\n%s" % (src, " ".join(cmd), r.stderr))
    return obj, r.stderr


def _run(what, cmd):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("%s failed:\n%s\n%s" % (what, " ".join(cmd), r.stderr))


def _cxx():
    cand = shutil.which("g++") or shutil.which("c++")
    if cand is None:
        raise RuntimeError("no C++ compiler found; g++ is required to build _step_calls.so")
    return cand


def _compile_binding():
    import torch

    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    obj = os.path.join(OBJ_DIR, os.path.basename(BINDING) + ".o")
    _run("the binding's compilation",
         [_cxx(), "-O2", "-std=c++17", "-fPIC", "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch._C._GLIBCXX_USE_CXX11_ABI,
          "-I", INCLUDE, "-isystem", inc, "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"),
          "-isystem", sysconfig.get_paths()["include"], "-c", BINDING, "-o", obj])
    return obj


def _link_binding(obj):
    import torch

    _run("the binding's link",
         [_cxx(), "-shared", "-o", MODULE + ".tmp", obj, LIB, "-Wl,-rpath,$ORIGIN", "-L",
          os.path.join(os.path.dirname(torch.__file__), "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10"])
    os.replace(MODULE + ".tmp", MODULE)
    with open(TORCH_STAMP, "w") as f:
        f.write(torch.__version__)


def build_library(force=False, verbose=False):
    """Compile csrc/ into libpa_gb300.so (sm_103a).  Returns its path."""
    if not force and library_up_to_date():
        return LIB
    os.makedirs(OBJ_DIR, exist_ok=True)
    with concurrent.futures.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        results = list(ex.map(lambda s: _compile(s, verbose), sources()))
    if verbose:
        for _, log in results:
            if log:
                sys.stderr.write(log)
    tmp = LIB + ".tmp"
    _run("link", [_nvcc(), *ARCH, "-shared", "-Xlinker", "-soname=" + os.path.basename(LIB), "-o", tmp] +
         [o for o, _ in results])
    os.replace(tmp, LIB)
    return LIB


def build(force=False, verbose=False):
    """The library, and the binding's module beside it.  Returns the library's path."""
    if not force and module_up_to_date():
        return build_library(verbose=verbose)
    os.makedirs(OBJ_DIR, exist_ok=True)
    with concurrent.futures.ThreadPoolExecutor(max_workers=1) as ex:
        binding = ex.submit(_compile_binding)
        build_library(force, verbose)
        _link_binding(binding.result())
    return LIB


if __name__ == "__main__":
    print((build_library if "--library" in sys.argv else build)(force="--force" in sys.argv, verbose="-v" in sys.argv))
