"""Build librf.so (the CUDA kernels and the C ABI) in-tree with nvcc.

Every translation unit in ``csrc/`` is compiled for sm_103a only
(``-gencode arch=compute_103a,code=sm_103a``), in parallel, into ``_build/``
at the repository root; the shared library lands in ``lib/librf.so`` next to
this file. The CUDA runtime is linked statically, and the driver's tensor-map
encoder is looked up at run time, so the library loads on a machine without a
GPU driver (only the kernels need one). The paged serving calls have a native
binding (csrc/serving_binding.cpp, compiled against the installed torch's
headers), ``lib/_rf_serving.so``, which calls librf.so next to it.

Usage:  python -m online_softmax_attention_rf_gb300.build [--force] [-v]
"""

import concurrent.futures
import importlib.util
import json
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIBDIR = os.path.join(HERE, "lib")
BUILD_DIR = os.path.join(ROOT, "_build")
LIB_PATH = os.path.join(LIBDIR, "librf.so")
BINDING_SRC = os.path.join(CSRC, "serving_binding.cpp")
BINDING_PATH = os.path.join(LIBDIR, "_rf_serving.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
CFLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-I", CSRC, "-I", INCLUDE,
          "-Xptxas", "-warn-spills"]


def _nvcc():
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        raise RuntimeError("nvcc not found")
    return nvcc


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _headers():
    hs = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".h", ".cuh"))]
    return hs + [os.path.join(INCLUDE, "rf.h")]


def _stale(target, deps):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _compile(src, verbose, extra):
    obj = os.path.join(BUILD_DIR, os.path.basename(src)[:-3] + ".o")
    cmd = [_nvcc(), *ARCH, *CFLAGS, *extra, "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("nvcc failed for %s:\n%s\n%s" % (src, " ".join(cmd), r.stderr))
    if verbose and r.stderr.strip():
        print(r.stderr, file=sys.stderr)
    return obj


def _run(cmd, what):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("%s failed:\n%s\n%s" % (what, " ".join(cmd), r.stderr))


def _torch_dir():
    """Directory of the installed torch, found without importing it."""
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.submodule_search_locations:
        raise RuntimeError("the binding of the paged serving calls needs torch")
    return spec.submodule_search_locations[0]


def _binding_lacks():
    """What the binding needs and this machine does not have, or None. Users of the
    C library need none of it."""
    try:
        t = _torch_dir()
    except RuntimeError:
        return "torch"
    for what, path in (("torch's headers", os.path.join(t, "include", "ATen")),
                       ("Python.h", os.path.join(sysconfig.get_paths()["include"], "Python.h"))):
        if not os.path.exists(path):
            return "%s (%s)" % (what, path)
    return None if shutil.which("g++") else "g++"


def _binding_commands(obj, tmp):
    """The binding's compile and link commands."""
    t = _torch_dir()
    gxx = shutil.which("g++") or "g++"
    tlib = os.path.join(t, "lib")
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    dirs = [os.path.join(t, "include"), os.path.join(t, "include", "torch", "csrc", "api", "include"),
            sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    return ([gxx, "-O2", "-std=c++17", "-fPIC", "-I", INCLUDE,
             *[f for d in dirs for f in ("-isystem", d)], "-c", BINDING_SRC, "-o", obj],
            [gxx, "-shared", "-o", tmp, obj, "-L", LIBDIR, "-l:librf.so", "-L", tlib,
             "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10", "-Wl,-rpath,$ORIGIN",
             "-Wl,-rpath," + tlib])


def _binding_made_with(commands):
    """What a built binding depends on besides its sources: the commands (they
    name torch's, Python's and CUDA's directories), torch's version and Python's
    binary interface. A binding made with something else is built again."""
    with open(os.path.join(_torch_dir(), "version.py")) as f:
        version = f.read()
    return json.dumps([commands, version, sysconfig.get_config_var("SOABI")], indent=1)


def _read(path):
    if not os.path.exists(path):
        return None
    with open(path) as f:
        return f.read()


def build(force=False, verbose=False, extra_flags=()):
    """Compile what changed and link lib/librf.so, then the binding of the paged
    serving calls; returns librf.so's path. Where the binding cannot be built
    (no torch, Python.h or g++) the library is, with a warning; those calls of
    api.py then raise."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    os.makedirs(LIBDIR, exist_ok=True)
    hdrs = _headers()
    todo = []
    objs = []
    for src in sources():
        obj = os.path.join(BUILD_DIR, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        if force or _stale(obj, [src, *hdrs]):
            todo.append(src)
    binding_obj = os.path.join(BUILD_DIR, "serving_binding.o")
    binding_tmp, binding_stamp = BINDING_PATH + ".tmp", os.path.join(BUILD_DIR, "serving_binding.json")
    lacks = _binding_lacks()
    binding = False
    if lacks is None:
        commands = _binding_commands(binding_obj, binding_tmp)
        made_with = _binding_made_with(commands)
        binding = force or made_with != _read(binding_stamp) or \
            _stale(binding_obj, [BINDING_SRC, os.path.join(INCLUDE, "rf.h")])
    with concurrent.futures.ThreadPoolExecutor(max_workers=len(todo) + 1) as ex:
        jobs = [ex.submit(_compile, s, verbose, list(extra_flags)) for s in todo]
        if binding:
            binding_job = ex.submit(_run, commands[0], "g++ for %s" % BINDING_SRC)
        for j in jobs:
            j.result()
    if force or todo or _stale(LIB_PATH, objs):
        tmp = LIB_PATH + ".tmp"
        cmd = [_nvcc(), *ARCH, "-shared", "-Xcompiler", "-fPIC", "-o", tmp, *objs]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("link failed:\n%s\n%s" % (" ".join(cmd), r.stderr))
        os.replace(tmp, LIB_PATH)
    if lacks is not None:
        warnings.warn("_rf_serving.so, the binding of the paged serving calls, is not built: no "
                      + lacks)
        return LIB_PATH
    if binding:
        binding_job.result()
    if binding or _stale(BINDING_PATH, [binding_obj]):
        _run(commands[1], "link of %s" % BINDING_PATH)
        os.replace(binding_tmp, BINDING_PATH)
        with open(binding_stamp, "w") as f:
            f.write(made_with)
    return LIB_PATH


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
