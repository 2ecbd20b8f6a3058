"""Build the moeq4k CUDA library in-tree for sm_103a.

Each ``csrc/*.cu`` translation unit is compiled by nvcc in parallel into
``_build/``; the objects are linked into ``libmoeq4k.so`` next to this file.
``csrc/binding.cpp`` becomes the extension module ``_binding`` beside it, against
the headers of Python and of the installed PyTorch; it is built again for another
PyTorch, and where there is none the library is built alone.
"""
from __future__ import annotations

import glob
import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libmoeq4k.so")
BINDING_SRC = os.path.join(CSRC, "binding.cpp")
BINDING = os.path.join(PKG, "_binding" + sysconfig.get_config_var("EXT_SUFFIX"))
BINDING_FOR = os.path.join(BUILD, "binding_for")  # the PyTorch that BINDING was built against

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "--expt-relaxed-constexpr",
              "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden"]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found: the moeq4k library cannot be built")
    return path


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _headers():
    return glob.glob(os.path.join(INCLUDE, "*.h"))


def torch_version():
    """The installed PyTorch (version and place, without importing it), or None."""
    spec = importlib.util.find_spec("torch")
    if spec is None:
        return None
    return f"{importlib.metadata.version('torch')} {spec.origin}"


def _newer(out, deps) -> bool:
    return os.path.exists(out) and all(os.path.getmtime(d) <= os.path.getmtime(out) for d in deps)


def library_up_to_date() -> bool:
    return _newer(LIB, _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + _headers())


def binding_up_to_date() -> bool:
    version = torch_version()
    if version is None:
        return True
    if not os.path.exists(BINDING_FOR) or open(BINDING_FOR).read() != version:
        return False
    return _newer(BINDING, [BINDING_SRC] + _headers())


def up_to_date() -> bool:
    return library_up_to_date() and binding_up_to_date()


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    library = force or not library_up_to_date()
    binding = torch_version() is not None and (force or not binding_up_to_date())
    if not library and not binding:
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()

    def compile_one(src, flags):
        obj = os.path.join(BUILD, os.path.splitext(os.path.basename(src))[0] + ".o")
        cmd = [cc, *NVCC_FLAGS, *flags, "-I", INCLUDE, "-I", CSRC, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr)
        return obj

    def compile_binding():
        import torch
        include = os.path.join(os.path.dirname(torch.__file__), "include")
        return compile_one(BINDING_SRC, ["-I", include, "-I", os.path.join(include, "torch", "csrc", "api", "include"),
                                         "-I", sysconfig.get_paths()["include"],
                                         f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"])

    def link(out, flags):
        tmp = out + f".tmp{os.getpid()}"
        r = subprocess.run([cc, "-shared", "-o", tmp, *flags], capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, out)

    srcs = _sources() if library else []
    with ThreadPoolExecutor(max_workers=max(1, min(len(srcs) + 1, os.cpu_count() or 4))) as ex:
        module = ex.submit(compile_binding) if binding else None
        objs = list(ex.map(lambda src: compile_one(src, [*ARCH, *extra_flags]), srcs))
        if library:
            link(LIB, [*ARCH, *objs, "-lcuda"])
        if module is not None:
            # the library beside the module, whatever the directory; PyTorch's are loaded before it
            link(BINDING, [module.result(), "-L", PKG, f"-l:{os.path.basename(LIB)}", "-Xlinker", "-rpath=$ORIGIN",
                           "-L", os.path.join(os.path.dirname(importlib.util.find_spec("torch").origin), "lib"),
                           "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10"])
            with open(BINDING_FOR, "w") as f:
                f.write(torch_version())
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose=True))
