"""Build libgbnms.so in-tree with nvcc for sm_103a (GB300).

Each translation unit compiles in its own nvcc process (in parallel), then
nvcc links the shared library.  The C++ half of the Python binding (g++, torch's
headers) compiles beside them; without torch, or with one for CPUs alone, it is
left out.  -fmad=false keeps every binary32 product and sum individually rounded
(the kernels also use explicit _rn intrinsics); no fast-math flag is ever passed.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.util
import os
import shutil
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "libgbnms.so")
# Instruction-throughput probe for the roofline denominators (bench.py only).
PROBE_SRC = os.path.join(PKG, "probe", "alu_probe.cu")
PROBE_LIB = os.path.join(BUILD, "libgbprobe.so")


def _torch_folder():
    spec = importlib.util.find_spec("torch")
    return spec.submodule_search_locations[0] if spec and spec.submodule_search_locations else None


def _torch_version() -> str:
    # From its file: importing torch takes seconds.
    try:
        with open(os.path.join(_torch_folder() or "", "version.py")) as f:
            return next(line.split("=")[-1].strip().strip("'\"") for line in f if line.startswith("__version__"))
    except (OSError, StopIteration):
        return "none"


# Tensor functions of block.py: for the torch and the interpreter that they are compiled against, and no others.
BINDING_SRC = os.path.join(PKG, "binding", "block_binding.cpp")
BINDING_LIB = os.path.join(BUILD, "gbblock-torch%s-%s.so" % (_torch_version(), sysconfig.get_config_var("SOABI")))

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-fmad=false", "-Xcompiler", "-fPIC",
              "-Xcompiler", "-Wall", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for c in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _with_binding() -> bool:
    torch = _torch_folder()
    return torch is not None and os.path.exists(os.path.join(torch, "lib", "libc10_cuda.so"))


def _binding_command(out: str):
    torch = _torch_folder()
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    includes = [INCLUDE, os.path.join(torch, "include"), os.path.join(torch, "include", "torch", "csrc", "api", "include"),
                sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    lib = os.path.join(torch, "lib")
    return [os.environ.get("CXX") or "g++", "-O2", "-std=c++17", "-Wall", "-fPIC", "-shared", "-fvisibility=hidden",
            *(f for i in includes for f in ("-isystem" if i != INCLUDE else "-I", i)), BINDING_SRC, "-o", out, "-L", lib,
            "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda", f"-Wl,-rpath,{lib}"]


def _stale() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(PROBE_LIB):
        return True
    if os.path.getmtime(PROBE_SRC) > os.path.getmtime(PROBE_LIB):
        return True
    if _with_binding():
        if not os.path.exists(BINDING_LIB):
            return True
        if any(os.path.getmtime(d) > os.path.getmtime(BINDING_LIB) for d in
               [BINDING_SRC, __file__] + glob.glob(os.path.join(INCLUDE, "*.h"))):
            return True
    t = os.path.getmtime(LIB)
    deps = sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
    deps += glob.glob(os.path.join(INCLUDE, "*.h")) + [__file__]
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Compile (if stale) and return the path of libgbnms.so."""
    if not force and not _stale():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    objs = []
    cmds = []
    for src in sources():
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        cmds.append([cc, *ARCH, *NVCC_FLAGS, *extra_flags, "-c", src, "-o", obj])

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("%s failed:\n%s\n%s" % (os.path.basename(cmd[0]), " ".join(cmd), r.stderr))
        return r.stderr

    probe_tmp = PROBE_LIB + ".tmp%d" % os.getpid()
    # The probe has no binary32 contraction concern (its instructions are
    # inline PTX) and builds straight to its own shared library.
    cmds.append([cc, *ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", *extra_flags,
                 "-shared", PROBE_SRC, "-o", probe_tmp])
    binding_tmp = BINDING_LIB + ".tmp%d" % os.getpid()
    with_binding = _with_binding()
    if with_binding:
        cmds.append(_binding_command(binding_tmp))
    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(cmds), os.cpu_count() or 1))) as ex:
        for out in ex.map(run, cmds):
            if verbose and out:
                print(out)
    os.replace(probe_tmp, PROBE_LIB)
    if with_binding:
        os.replace(binding_tmp, BINDING_LIB)
    tmp = LIB + ".tmp%d" % os.getpid()
    run([cc, *ARCH, "-shared", "-o", tmp, *objs])
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose=True,
                extra_flags=["-Xptxas", "-v"] if "--ptxas" in sys.argv else []))
