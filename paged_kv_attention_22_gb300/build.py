"""Build libpkv.so (the CUDA kernels and the C ABI) in place, for sm_103a only.

Each translation unit is compiled by nvcc in parallel, then linked into one
shared library next to this file. The CUDA runtime is linked statically, so the
library needs only the driver at run time; it builds the same way on x86_64
and aarch64 hosts.

Beside it goes _marshal.so, the compiled part of the Python binding, built by
g++ against the installed torch (and rebuilt when torch changes).
"""
import os
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD_DIR = os.path.join(HERE, "_build")
LIBRARY = os.path.join(HERE, "libpkv.so")
MARSHAL = os.path.join(HERE, "_marshal.so")
MARSHAL_TORCH = os.path.join(BUILD_DIR, "marshal_torch_version")  # what MARSHAL was built against
SOURCES = ["kv_store.cu", "decode.cu", "prefill.cu", "api.cu", "decode_noalloc.cu",
           "q4_cache.cu", "q4_decode.cu", "api_q4.cu", "evict.cu", "api_evict.cu",
           "block_manager.cpp"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-I" + os.path.join(ROOT, "include")]


def _nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _cuda_home() -> str:
    return os.environ.get("CUDA_HOME", "/usr/local/cuda")


def _marshal_command(torch_dir: str):
    lib = os.path.join(torch_dir, "lib")
    include = [os.path.join(ROOT, "include"), sysconfig.get_paths()["include"],
               os.path.join(torch_dir, "include"),
               os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
               os.path.join(_cuda_home(), "include")]
    return (["g++", "-O2", "-std=c++17", "-fPIC", "-shared", os.path.join(CSRC, "marshal.cpp")]
            + ["-I" + d for d in include] + ["-L" + lib, "-L" + HERE, "-Wl,-rpath,$ORIGIN"]
            + ["-l:libpkv.so", "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"])


def _torch():
    import torch
    return os.path.dirname(torch.__file__), torch.__version__


def _needs_rebuild() -> bool:
    if not os.path.exists(LIBRARY) or not os.path.exists(MARSHAL) \
            or not os.path.exists(MARSHAL_TORCH):
        return True
    with open(MARSHAL_TORCH) as f:
        if f.read() != _torch()[1]:
            return True
    lib_time = min(os.path.getmtime(LIBRARY), os.path.getmtime(MARSHAL))
    deps = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    include = os.path.join(ROOT, "include")
    deps += [os.path.join(include, f) for f in os.listdir(include)]
    deps.append(os.path.abspath(__file__))
    return any(os.path.getmtime(d) > lib_time for d in deps)


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    if not force and not _needs_rebuild():
        return LIBRARY
    os.makedirs(BUILD_DIR, exist_ok=True)
    nvcc = _nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".o")
        cmd = [nvcc, *ARCH, *FLAGS, *extra_flags, "-c", os.path.join(CSRC, src), "-o", obj]
        proc = subprocess.run(cmd, capture_output=True, text=True)
        return src, obj, cmd, proc

    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as pool:
        # the object first: linking it needs the library
        marshal_obj = os.path.join(BUILD_DIR, "marshal.o")
        torch_dir, torch_version = _torch()
        cmd = [a for a in _marshal_command(torch_dir) if not a.startswith(("-l", "-L", "-Wl", "-shared"))]
        marshal = pool.submit(subprocess.run, cmd + ["-c", "-o", marshal_obj], capture_output=True,
                              text=True)
        results = list(pool.map(compile_one, SOURCES))
        marshal = marshal.result()
    errors = []
    for src, obj, cmd, proc in results:
        if verbose or proc.returncode != 0:
            sys.stderr.write(" ".join(cmd) + "\n" + proc.stdout + proc.stderr)
        if proc.returncode != 0:
            errors.append(src)
    if errors:
        raise RuntimeError("nvcc failed for " + ", ".join(errors))
    tmp = LIBRARY + ".tmp"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp] + [r[1] for r in results]
    proc = subprocess.run(cmd, capture_output=True, text=True)
    if proc.returncode != 0:
        raise RuntimeError("link failed:\n" + proc.stdout + proc.stderr)
    os.replace(tmp, LIBRARY)
    if marshal.returncode != 0:
        raise RuntimeError("g++ failed for marshal.cpp:\n" + marshal.stdout + marshal.stderr)
    tmp = MARSHAL + ".tmp"
    cmd = [marshal_obj if a.endswith("marshal.cpp") else a for a in _marshal_command(torch_dir)]
    proc = subprocess.run(cmd + ["-o", tmp], capture_output=True, text=True)
    if proc.returncode != 0:
        raise RuntimeError("link failed:\n" + proc.stdout + proc.stderr)
    os.replace(tmp, MARSHAL)
    with open(MARSHAL_TORCH, "w") as f:
        f.write(torch_version)
    return LIBRARY


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv,
                extra_flags=["-Xptxas", "-v"] if "--ptxas" in sys.argv else []))
