"""Build the CUDA library ``libsimcomm.so`` (sm_100a) in the package directory with nvcc, and the binding's helper
``_marshal`` (the checks of a call's tensors; its file's name says which Python and torch it is for) with g++. The library needs neither Python nor torch; where the helper cannot be
built that is said, and the binding does without it.

    python -m collective_communication_primitives_b200.build [--force] [-v]

Every ``csrc/*.cu`` is compiled to its own object (in parallel, under ``_build/``), then the objects
are linked into the shared library. No relocatable device code: each translation unit's kernels and
device symbols are its own.
"""
import glob
import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libsimcomm.so")
MARSHAL_SRC = os.path.join(CSRC, "marshal.cpp")
OBJ_DIR = os.path.join(ROOT, "_build", "simcomm")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = [
    *ARCH,
    "-O3", "-std=c++17", "-lineinfo",
    "-fmad=false",                 # sums are plain adds; the AVG scale is a separate multiply
    "-Xcompiler", "-fPIC",
    "-Xcompiler", "-Wall",
    "--expt-relaxed-constexpr",
]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _headers():
    return glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(INCLUDE, "*.h"))


def _nvcc():
    nvcc = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return nvcc if os.path.exists(nvcc) else "nvcc"


def _obj(src):
    return os.path.join(OBJ_DIR, os.path.splitext(os.path.basename(src))[0] + ".o")


def _newer(target, deps):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(f) > t for f in deps)


def marshal_path():
    """The helper's file. It reads tensors where this interpreter's torch holds them, so the name has what that depends on: a
    helper of another Python or torch is another file, which is neither loaded nor taken for this one. Raises ImportError
    without torch."""
    import sysconfig

    import torch
    for_ = f"{sysconfig.get_config_var('SOABI')}-torch-{torch.__version__}-abi{int(torch.compiled_with_cxx11_abi())}"
    return os.path.join(PKG, f"_marshal.{for_}.so")


def _marshal_stale():
    try:
        return _newer(marshal_path(), [MARSHAL_SRC])
    except (ImportError, OSError):  # no torch, or one whose own libraries are missing
        return False  # nothing to build it for


def _stale():
    return _newer(LIB, sources() + _headers()) or _marshal_stale()


def build_marshal(verbose: bool = False):
    """The helper is built against the headers of the torch that this interpreter imports."""
    import sysconfig

    import torch
    path = marshal_path()
    root = os.path.dirname(torch.__file__)
    inc = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_path("include"), os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")]
    cmd = ["g++", "-O2", "-std=c++20", "-fPIC", "-shared", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}"]
    for d in inc:
        cmd += ["-isystem", d]
    cmd += ["-o", path + ".tmp", MARSHAL_SRC, "-L", os.path.join(root, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10"]
    if verbose:
        print(" ".join(cmd))
    subprocess.run(cmd, check=True)
    os.replace(path + ".tmp", path)


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not _stale():
        return LIB
    os.makedirs(OBJ_DIR, exist_ok=True)
    nvcc, hdrs = _nvcc(), _headers()

    def compile_one(src):
        obj = _obj(src)
        if not force and not _newer(obj, [src] + hdrs):
            return obj
        cmd = [nvcc, *NVCC_FLAGS, "-I", INCLUDE, "-I", CSRC, "-c", "-o", obj + ".tmp", src]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        subprocess.run(cmd, check=True)
        os.replace(obj + ".tmp", obj)
        return obj

    with ThreadPoolExecutor(max_workers=max(1, min(len(sources()) + 1, os.cpu_count() or 1))) as ex:
        helper = ex.submit(build_marshal, verbose) if force or _marshal_stale() else None
        objs = list(ex.map(compile_one, sources()))
        if force or _newer(LIB, objs):
            subprocess.run([nvcc, *ARCH, "-shared", "-o", LIB + ".tmp", *objs], check=True)
            os.replace(LIB + ".tmp", LIB)
        try:
            if helper is not None:
                helper.result()
        except (ImportError, OSError, subprocess.CalledProcessError) as e:  # no torch, no g++, no headers
            print("the helper _marshal was not built, the binding looks at tensors in Python:", e, file=sys.stderr)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
