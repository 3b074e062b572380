"""Build liblola.so in place: one nvcc per translation unit (in parallel), sm_103a only; then the Python
binding's marshalling module beside it."""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "liblola.so")
SOURCES = ["lola_capi.cu", "lola_phi.cu", "lola_select.cu", "lola_chunk.cu", "lola_output.cu", "lola_output_tc.cu",
           "lola_decode.cu", "lola_noalloc.cu", "lola_relsre.cu",
           "lola_fixed.cu", "lola_hola.cu", "lola_hola_tc.cu", "lola_attn.cu",
           "lola_attn_tc.cu", "lola_append.cu", "lola_paged.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA 13 toolkit is required to build liblola.so")


def _flags(verbose_ptxas: bool) -> list[str]:
    f = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC]
    if verbose_ptxas:
        f += ["-Xptxas", "-v"]
    return f


def pymod() -> str | None:
    """The binding's marshalling module (csrc/lola_py.cpp) for this torch, whose C++ interface it is compiled
    against; None without torch."""
    try:
        import torch
    except ImportError:
        return None
    return os.path.join(PKG, f"_lola_py-{torch.__version__}.so")


def _stale() -> bool:
    built = [p for p in (LIB, pymod()) if p]
    if not all(os.path.exists(p) for p in built):
        return True
    t = min(os.path.getmtime(p) for p in built)
    deps = [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [os.path.join(INCLUDE, "lola.h"), __file__]
    return any(os.path.getmtime(p) > t for p in deps)


def build(force: bool = False, verbose_ptxas: bool = False, jobs: int | None = None) -> str:
    """Compile every translation unit and link liblola.so; returns its path."""
    if not force and not _stale():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    flags = _flags(verbose_ptxas)

    def one(src: str) -> tuple[str, str]:
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        cmd = [cc, *flags, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stderr

    def binding() -> list[str] | None:
        if pymod() is None:
            return None
        import torch
        lib = os.path.join(os.path.dirname(torch.__file__), "lib")
        inc = os.path.join(os.path.dirname(torch.__file__), "include")
        obj = os.path.join(BUILD, "lola_py.o")
        cmd = [cc, "-O2", "-std=c++17", "-w", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", sysconfig.get_paths()["include"],
               "-I", inc, "-I", os.path.join(inc, "torch", "csrc", "api", "include"), "-c", os.path.join(CSRC, "lola_py.cpp"),
               "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"compiling the binding's module failed:\n{r.stdout}\n{r.stderr}")
        return [obj, "-L", lib, "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda", "-Xlinker", f"-rpath,{lib}"]

    with ThreadPoolExecutor(max_workers=jobs or len(SOURCES) + 1) as ex:
        py = ex.submit(binding)
        results = list(ex.map(one, SOURCES))
        py_link = py.result()
    if verbose_ptxas:
        for _, log in results:
            sys.stderr.write(log)
    tmp = LIB + f".{os.getpid()}.tmp"
    r = subprocess.run([cc, *ARCH, "-shared", "-o", tmp, *[o for o, _ in results]], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    if py_link is None:
        return LIB
    tmp = pymod() + f".{os.getpid()}.tmp"
    r = subprocess.run([cc, "-shared", "-o", tmp, *py_link, "-cudart", "none", "-L", PKG, "-l:liblola.so",
                        "-Xlinker", "-rpath,$ORIGIN"], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"building the binding's module failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, pymod())
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose_ptxas="-v" in sys.argv)
    print(LIB)
