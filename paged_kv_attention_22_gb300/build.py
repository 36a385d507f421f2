"""Build libpkv.so (the CUDA kernels and the C ABI) in place, for sm_103a only.

Each translation unit is compiled by nvcc in parallel, then linked into one
shared library next to this file. The CUDA runtime is linked statically, so the
library needs only the driver at run time; it builds the same way on x86_64
and aarch64 hosts.

Beside it goes _marshal.so, the compiled part of the Python binding, built by
g++ against the installed torch (and rebuilt when torch changes). The library
needs neither torch nor Python's headers: build_library() makes it alone, and
build() has it in place before anything that concerns _marshal.so can fail.
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
MARSHAL_SOURCE = "marshal.cpp"
MARSHAL_TORCH = os.path.join(BUILD_DIR, "marshal_torch_version")  # what MARSHAL was built against
SOURCES = ["kv_store.cu", "decode.cu", "prefill.cu", "api.cu", "decode_noalloc.cu",
           "q4_cache.cu", "q4_decode.cu", "api_q4.cu", "evict.cu", "api_evict.cu",
           "heads.cu", "api_heads.cu", "chunk.cu",
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
    return (["g++", "-O2", "-std=c++17", "-fPIC", "-shared", os.path.join(CSRC, MARSHAL_SOURCE)]
            + ["-I" + d for d in include] + ["-L" + lib, "-L" + HERE, "-Wl,-rpath,$ORIGIN"]
            + ["-l:libpkv.so", "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"])


def _torch():
    import torch
    return os.path.dirname(torch.__file__), torch.__version__


def _older(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    made = os.path.getmtime(target)
    include = os.path.join(ROOT, "include")
    deps = [os.path.join(CSRC, f) for f in deps] + [os.path.join(include, f) for f in os.listdir(include)]
    return any(os.path.getmtime(d) > made for d in deps + [os.path.abspath(__file__)])


def _library_stale() -> bool:
    return _older(LIBRARY, [f for f in os.listdir(CSRC) if f != MARSHAL_SOURCE])


def _marshal_stale() -> bool:
    if _older(MARSHAL, [MARSHAL_SOURCE]) or not os.path.exists(MARSHAL_TORCH):
        return True
    with open(MARSHAL_TORCH) as f:
        return f.read() != _torch()[1]


def _link(cmd, target: str) -> None:
    tmp = target + ".tmp"
    proc = subprocess.run(cmd + ["-o", tmp], capture_output=True, text=True)
    if proc.returncode != 0:
        raise RuntimeError("link failed:\n" + proc.stdout + proc.stderr)
    os.replace(tmp, target)


def build_library(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """libpkv.so, if it is missing or older than its sources."""
    if not force and not _library_stale():
        return LIBRARY
    os.makedirs(BUILD_DIR, exist_ok=True)
    nvcc = _nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".o")
        cmd = [nvcc, *ARCH, *FLAGS, *extra_flags, "-c", os.path.join(CSRC, src), "-o", obj]
        proc = subprocess.run(cmd, capture_output=True, text=True)
        return src, obj, cmd, proc

    with ThreadPoolExecutor(max_workers=len(SOURCES)) as pool:
        results = list(pool.map(compile_one, SOURCES))
    errors = []
    for src, obj, cmd, proc in results:
        if verbose or proc.returncode != 0:
            sys.stderr.write(" ".join(cmd) + "\n" + proc.stdout + proc.stderr)
        if proc.returncode != 0:
            errors.append(src)
    if errors:
        raise RuntimeError("nvcc failed for " + ", ".join(errors))
    _link([nvcc, *ARCH, "-shared"] + [r[1] for r in results], LIBRARY)
    return LIBRARY


def _compile_marshal(force: bool):
    """marshal.o and the command that links it (which needs the library), or None."""
    if not force and not _marshal_stale():
        return None
    os.makedirs(BUILD_DIR, exist_ok=True)
    torch_dir, torch_version = _torch()
    obj = os.path.join(BUILD_DIR, "marshal.o")
    cmd = [a for a in _marshal_command(torch_dir) if not a.startswith(("-l", "-L", "-Wl", "-shared"))]
    proc = subprocess.run(cmd + ["-c", "-o", obj], capture_output=True, text=True)
    if proc.returncode != 0:
        raise RuntimeError("g++ failed for marshal.cpp:\n" + proc.stdout + proc.stderr)
    return [obj if a.endswith(MARSHAL_SOURCE) else a for a in _marshal_command(torch_dir)], torch_version


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Both, the two compilations side by side."""
    with ThreadPoolExecutor(max_workers=1) as pool:
        marshal = pool.submit(_compile_marshal, force)
        build_library(force, verbose, extra_flags)
    made = marshal.result()
    if made is not None:
        _link(made[0], MARSHAL)
        with open(MARSHAL_TORCH, "w") as f:
            f.write(made[1])
    return LIBRARY


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv,
                extra_flags=["-Xptxas", "-v"] if "--ptxas" in sys.argv else []))
