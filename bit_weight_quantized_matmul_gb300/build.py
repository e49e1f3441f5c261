"""Build libwq.so (sm_103a) in-tree with nvcc: one object per translation unit,
compiled in parallel, then linked as a shared library with the CUDA runtime
linked statically (the library loads without libcudart.so or libcuda.so; the
tensor-map encoder is resolved at run time through the runtime's driver entry
point).  Beside it _wq_calls.so (g++), through which wq.py makes the KV cache
calls of torch tensors."""
import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libwq.so")
CALLS = os.path.join(PKG, "_wq_calls.so")
CALLS_FOR = os.path.join(BUILD, "wq_calls.for")      # what it was compiled against
HEADER = os.path.join(os.path.dirname(PKG), "include", "wq.h")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-Xptxas", "-v"]


def nvcc():
    p = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(p):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libwq.so")
    return p


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + [HEADER]


def _newer(made, deps):
    return os.path.exists(made) and all(os.path.getmtime(d) <= os.path.getmtime(made) for d in deps)


def calls_for():
    """What _wq_calls.so is compiled against, and works with alone: this torch, its ABI and this interpreter."""
    import torch
    return f"torch {torch.__version__}, CXX11 ABI {int(torch._C._GLIBCXX_USE_CXX11_ABI)}, {sysconfig.get_config_var('SOABI')}"


def lib_up_to_date():
    return _newer(LIB, _deps())


def calls_up_to_date():
    if not _newer(CALLS, [os.path.join(CSRC, "wq_calls.cpp"), HEADER]) or not os.path.exists(CALLS_FOR):
        return False
    with open(CALLS_FOR) as f:
        return f.read() == calls_for()


def up_to_date():
    return lib_up_to_date() and calls_up_to_date()


def build_calls():
    """_wq_calls.so against this interpreter's and this torch's headers."""
    import torch
    os.makedirs(BUILD, exist_ok=True)
    root = os.path.dirname(torch.__file__)
    include = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
               sysconfig.get_paths()["include"], os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")]
    tmp = CALLS + ".tmp"
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           f'-DWQ_CALLS_FOR="{calls_for()}"']
    cmd += ["-I" + i for i in include] + [os.path.join(CSRC, "wq_calls.cpp"), "-o", tmp, "-L" + os.path.join(root, "lib")]
    r = subprocess.run(cmd + ["-ltorch_python", "-ltorch_cpu", "-lc10"], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on wq_calls.cpp:\n{r.stderr}")
    os.replace(tmp, CALLS)
    with open(CALLS_FOR, "w") as f:
        f.write(calls_for())


def build(force=False, verbose=False):
    if not force and lib_up_to_date():
        if not calls_up_to_date():
            build_calls()
            if verbose:
                print(f"built {CALLS}", file=sys.stderr)
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        cmd = [cc] + ARCH + FLAGS + ["-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stderr}")
        with open(obj + ".ptxas.txt", "w") as f:
            f.write(r.stderr)
        return obj

    srcs = _sources()
    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(srcs), os.cpu_count() or 4))) as ex:
        calls = ex.submit(build_calls)
        objs = list(ex.map(compile_one, srcs))
        calls.result()
    tmp = LIB + ".tmp"
    cmd = [cc] + ARCH + ["-shared", "-cudart", "static", "-o", tmp] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)
    if verbose:
        print(f"built {LIB}", file=sys.stderr)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True)
