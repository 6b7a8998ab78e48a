"""Builds libpkv.so (the CUDA kernels + C ABI) in-tree for sm_103a with nvcc.

Each translation unit compiles in parallel to an object file under
``paged_kv_cache_248_gb300/_build/``; the objects link into
``paged_kv_cache_248_gb300/libpkv.so``; ``binding.c`` becomes the CPython module ``_native`` of this Python's ABI.
No cmake, no torch extension machinery.
Run ``python -m paged_kv_cache_248_gb300._build`` or call :func:`build`.
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
OUT_DIR = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libpkv.so")
NATIVE = os.path.join(PKG, "_native" + sysconfig.get_config_var("EXT_SUFFIX"))  # CPython module over libpkv (binding.c)
INCLUDE = os.path.join(ROOT, "include")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "--expt-relaxed-constexpr", "-Xcompiler", "-fPIC,-fvisibility=hidden",
              f"-I{INCLUDE}"]


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libpkv")
    return cand


CXX_FLAGS = ["-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", f"-I{INCLUDE}"]


def sources() -> list[str]:
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cu", ".cpp")))


def _headers_mtime() -> float:
    hs = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    hs += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE) if f.endswith(".h")]
    return max(os.path.getmtime(h) for h in hs)


def build(force: bool = False, verbose: bool = False, extra_flags: list[str] | None = None) -> str:
    nvcc = _nvcc()
    os.makedirs(OUT_DIR, exist_ok=True)
    hdr = _headers_mtime()
    srcs = sources()
    flags = NVCC_FLAGS + (extra_flags or [])

    def compile_one(src: str) -> str:
        obj = os.path.join(OUT_DIR, os.path.splitext(os.path.basename(src))[0] + ".o")
        if (not force and os.path.exists(obj) and os.path.getmtime(obj) >= os.path.getmtime(src)
                and os.path.getmtime(obj) >= hdr):
            return obj
        if src.endswith(".cpp"):  # host-only C++ (block manager)
            cmd = [shutil.which("g++") or "g++", *CXX_FLAGS, "-c", src, "-o", obj + ".tmp"]
        else:
            cmd = [nvcc, *ARCH, *flags, "-c", src, "-o", obj + ".tmp"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout, r.stderr, file=sys.stderr)
        os.replace(obj + ".tmp", obj)
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(len(srcs), os.cpu_count() or 4)) as ex:
        objs = list(ex.map(compile_one, srcs))
    if force or not os.path.exists(LIB) or any(os.path.getmtime(o) > os.path.getmtime(LIB) for o in objs):
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB)
    src = os.path.join(CSRC, "binding.c")
    cmd = [shutil.which("gcc") or "gcc", "-O2", "-shared", "-fPIC", f"-I{INCLUDE}",
           f"-I{sysconfig.get_paths()['include']}", src, "-ldl"]
    record = os.path.join(OUT_DIR, "_native.cmd")  # the command that made the module: another Python's differs
    made_by = open(record).read() if os.path.exists(record) else ""
    if (force or made_by != " ".join(cmd) or not os.path.exists(NATIVE)
            or os.path.getmtime(NATIVE) < max(os.path.getmtime(src), hdr)):
        tmp = NATIVE + f".tmp{os.getpid()}"
        r = subprocess.run([*cmd, "-o", tmp], capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"gcc failed for binding.c:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, NATIVE)
        with open(record, "w") as f:
            f.write(" ".join(cmd))
    untagged = os.path.join(PKG, "_native.so")  # of a build before the module carried its ABI: any Python would load it
    if os.path.exists(untagged):
        os.remove(untagged)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
