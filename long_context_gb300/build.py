"""Build step for the native library ``libcpattn.so`` (sm_103a).

Compiles the CUDA/C++ sources under ``csrc/`` in parallel with nvcc and links
them into ``long_context_gb300/libcpattn.so``, and ``csrc/binding.cpp`` with the
host compiler into the CPython module ``_binding.so`` beside it (against the
installed PyTorch's headers).  The CUDA runtime is linked
statically and the driver is reached through the runtime's entry-point query,
so the library loads on a machine without a GPU (the host-only planner can run
there) and needs only the NVIDIA driver on a GPU machine.
"""

from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libcpattn.so")
BINDING = os.path.join(PKG, "_binding.so")
BINDING_FOR = os.path.join(BUILD, "binding.for")
BINDING_SRC = os.path.join(CSRC, "binding.cpp")

SOURCES = ["plan.cpp", "api.cu", "schedule.cu", "merge.cu", "attn_fwd.cu", "attn_bwd.cu",
           "dcp.cu", "decode.cu", "noalloc.cu", "ulysses.cu", "norm_rope.cu", "paged_sched.cu",
           "paged_rows.cu", "paged_tile.cu", "paged_fp4.cu", "paged_fp4_rows.cu", "serve_api.cu"]
HEADERS = ["kernels.h", "ptx.cuh", "work.cuh", "debug.cuh", "paged_plan.cuh", "seq.cuh",
           "fp4.cuh"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc():
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        raise RuntimeError("nvcc not found: the CUDA 13 toolkit is required")
    return nvcc


def _flags(verbose_ptxas=False):
    f = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                "-I", INCLUDE, "-I", CSRC, "--expt-relaxed-constexpr"]
    if verbose_ptxas:
        f += ["-Xptxas", "-v"]
    return f


def _stale():
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = [os.path.join(CSRC, s) for s in SOURCES + HEADERS]
    deps.append(os.path.join(INCLUDE, "cpattn.h"))
    deps.append(os.path.abspath(__file__))
    return any(os.path.getmtime(d) > t for d in deps)


def _build_variant(name, define, force):
    lib = os.path.join(PKG, "lib%s.so" % name)
    build()
    if not force and os.path.exists(lib) and os.path.getmtime(lib) >= os.path.getmtime(LIB):
        return lib
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    flags = _flags() + ["-D%s=1" % define]

    def compile_one(src):
        obj = os.path.join(BUILD, name + "_" + src + ".o")
        r = subprocess.run([nvcc] + flags + ["-c", os.path.join(CSRC, src), "-o", obj],
                           capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed on %s:\n%s" % (src, r.stderr))
        return obj

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    tmp = lib + ".tmp"
    r = subprocess.run([nvcc] + ARCH + ["-shared", "-cudart", "static", "-o", tmp] + objs,
                       capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s" % r.stderr)
    os.replace(tmp, lib)
    return lib


def build_fault_injection(force=False):
    """Test-only variant ``libcpattn_fault.so`` built with
    ``-DCPATTN_FAULT_INJECT_DROP_P``: the first CTA of the attention kernels
    (forward, backward, paged tiles) skips one hand-off, or does not start a copy that
    it waits for (few rows over the 4-bit cache), so that a bounded device wait runs
    out.  Used by the failure detection tests; never loaded by the
    package."""
    return _build_variant("cpattn_fault", "CPATTN_FAULT_INJECT_DROP_P", force)


def build_debug(force=False):
    """Debug variant ``libcpattn_debug.so`` built with ``-DCPATTN_DEBUG``: the
    attention kernels (forward, backward, schedule) check every global index
    and TMA coordinate they derive and report a violation as
    CPATTN_ERR_DEVICE_BOUNDS in the workspace error word (never a trap).
    Same C ABI as libcpattn.so.  The norm + rotation and paged-cache kernels have no
    such checks, and the binding's calls of them (``_binding.so`` is linked to
    libcpattn.so) do not reach this library when ``cpattn._lib`` is swapped for it."""
    return _build_variant("cpattn_debug", "CPATTN_DEBUG", force)


def _run(cmd, what):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("%s failed:\n%s\n%s" % (what, r.stdout, r.stderr))


def _torch_dir():
    import importlib.util
    spec = importlib.util.find_spec("torch")
    return os.path.dirname(spec.origin) if spec else None


def _binding_for():
    """What ``_binding.so`` is bound to -- the Python and the PyTorch that load it --
    or None where no PyTorch with CUDA is installed: then there is no binding, and
    the calls that need it say so."""
    root = _torch_dir()
    if root is None or not os.path.exists(os.path.join(root, "lib", "libc10_cuda.so")):
        return None
    with open(os.path.join(root, "version.py")) as f:
        return "%s\n%s\n%s" % (sys.version, root, f.read())


def _compile_binding():
    root = _torch_dir()
    obj = os.path.join(BUILD, "binding.cpp.o")
    inc = [os.path.join(root, "include"),
           os.path.join(root, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(os.path.dirname(os.path.dirname(
               os.path.realpath(_nvcc()))), "include"), INCLUDE]
    _run(["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-c", BINDING_SRC, "-o", obj]
         + [x for p in inc for x in ("-isystem" if p != INCLUDE else "-I", p)], "g++ binding.cpp")
    return obj


def _link_binding(obj):
    lib = os.path.join(_torch_dir(), "lib")
    tmp = BINDING + ".tmp"
    _run(["g++", "-shared", "-o", tmp, obj, "-L" + PKG, "-l:libcpattn.so", "-Wl,-rpath,$ORIGIN",
          "-L" + lib, "-Wl,-rpath," + lib, "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu",
          "-ltorch", "-lc10_cuda", "-lc10"], "linking _binding.so")
    os.replace(tmp, BINDING)
    with open(BINDING_FOR, "w") as f:
        f.write(_binding_for())


def _binding_stale():
    want = _binding_for()
    if want is None:
        return False
    if not os.path.exists(BINDING) or not os.path.exists(BINDING_FOR):
        return True
    with open(BINDING_FOR) as f:
        if f.read() != want:
            return True
    deps = [BINDING_SRC, os.path.join(INCLUDE, "cpattn.h"), os.path.abspath(__file__)]
    return any(os.path.getmtime(d) > os.path.getmtime(BINDING) for d in deps)


def build(force=False, verbose_ptxas=False, quiet=True):
    """Compile and link ``libcpattn.so`` and, where PyTorch with CUDA is installed,
    ``_binding.so`` unless they are up to date.  The library does not depend on the
    binding: an error of the latter is raised when the former is in place."""
    os.makedirs(BUILD, exist_ok=True)
    binding = _binding_for() is not None and (force or _binding_stale())
    if not force and not _stale():
        if binding:
            _link_binding(_compile_binding())
        return LIB
    nvcc = _nvcc()
    flags = _flags(verbose_ptxas)

    def compile_one(src):
        obj = os.path.join(BUILD, src + ".o")
        cmd = [nvcc] + flags + ["-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed on %s:\n%s\n%s" % (src, r.stdout, r.stderr))
        return obj, r.stderr

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        obj = ex.submit(_compile_binding) if binding else None
        results = list(ex.map(compile_one, SOURCES))
    if not quiet or verbose_ptxas:
        for _, log in results:
            if log.strip():
                sys.stderr.write(log)
    objs = [o for o, _ in results]
    tmp = LIB + ".tmp"
    cmd = [nvcc] + ARCH + ["-shared", "-cudart", "static", "-o", tmp] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s\n%s" % (r.stdout, r.stderr))
    os.replace(tmp, LIB)
    if binding:
        _link_binding(obj.result())
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose_ptxas="-v" in sys.argv, quiet=False)
    print(LIB)
