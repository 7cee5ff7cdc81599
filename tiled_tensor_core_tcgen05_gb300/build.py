"""Build the CUDA library libtg_gemm.so in-tree for sm_103a (GB300).

Each translation unit under csrc/ is compiled in parallel with nvcc
(-gencode arch=compute_103a,code=sm_103a), then linked into one shared
library next to this file. No torch extension machinery: the library exports
a plain C ABI (include/tg_gemm.h). Beside it a small CPython module,
_tg_torch.so, holds the tensor forms of a serving step's calls
(csrc/tg_torch.cpp, against torch's headers): it is left out where torch is not
installed, which the library does not need, and built again for another torch.
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
OBJDIR = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libtg_gemm.so")
BINDING = os.path.join(PKG, "_tg_torch.so")
BINDING_FOR = os.path.join(OBJDIR, "tg_torch.for")
# the debug build (device-side bounds checks, TG_DEBUG=1): same sources, its own objects
OBJDIR_DEBUG = os.path.join(PKG, "_build_debug")
LIB_DEBUG = os.path.join(PKG, "libtg_gemm_debug.so")
SOURCES = ["tg_api.cu", "k_tiled.cu", "k_tiled2.cu", "k_splitk.cu", "k_w4.cu", "k_w4r.cu", "k_attn.cu", "k_softmax.cu", "k_rope.cu", "k_kv.cu", "k_kv_attn.cu", "k_kv_tile.cu", "k_kv_shared.cu", "k_pages.cu", "k_sample.cu", "k_fill.cu", "k_epilogue.cu", "k_pad.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
CFLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC,
          "--expt-relaxed-constexpr"]


def nvcc() -> str:
    home = os.environ.get("CUDA_HOME") or os.environ.get("CUDA_PATH") or "/usr/local/cuda"
    cand = os.path.join(home, "bin", "nvcc")
    if os.path.exists(cand):
        return cand
    found = shutil.which("nvcc")
    if not found:
        raise RuntimeError("nvcc not found: set CUDA_HOME")
    return found


def _inputs() -> list[str]:
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files.append(os.path.join(INCLUDE, "tg_gemm.h"))
    files.append(os.path.abspath(__file__))
    return files


def _newest(made: str, inputs: list[str]) -> bool:
    return os.path.exists(made) and all(os.path.getmtime(f) <= os.path.getmtime(made) for f in inputs)


def up_to_date(lib: str = LIB) -> bool:
    return _newest(lib, _inputs())


def torch_dir() -> str | None:
    """Where torch (with CUDA) is installed."""
    import importlib.util
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.origin:
        return None
    d = os.path.dirname(spec.origin)
    return d if os.path.exists(os.path.join(d, "lib", "libc10_cuda.so")) else None


def binding_for(torch_dir: str) -> str:
    """What the module is built for: the interpreter and torch's place and version."""
    with open(os.path.join(torch_dir, "version.py")) as f:
        return f"{sys.version}\n{torch_dir}\n{f.read()}"


def binding_up_to_date(torch_dir: str) -> bool:
    if not _newest(BINDING, [os.path.join(CSRC, "tg_torch.cpp"), os.path.join(INCLUDE, "tg_gemm.h"), os.path.abspath(__file__)]):
        return False
    try:
        with open(BINDING_FOR) as f:
            return f.read() == binding_for(torch_dir)
    except FileNotFoundError:
        return False


def compile_binding(objdir: str, torch_dir: str) -> str:
    """The CPython module's object file."""
    include = os.path.join(torch_dir, "include")
    obj = os.path.join(objdir, "tg_torch.o")
    home = os.path.dirname(os.path.dirname(nvcc()))
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-c", os.path.join(CSRC, "tg_torch.cpp"), "-o", obj, "-I", INCLUDE,
           "-isystem", include, "-isystem", os.path.join(include, "torch", "csrc", "api", "include"),
           "-I", os.path.join(home, "include"), "-I", sysconfig.get_paths()["include"]]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for tg_torch.cpp:\n{r.stdout}\n{r.stderr}")
    return obj


def link_binding(obj: str, torch_dir: str) -> None:
    """Links the module with the library next to it and with torch."""
    lib = os.path.join(torch_dir, "lib")
    tmp = BINDING + f".tmp{os.getpid()}"
    cmd = ["g++", "-shared", obj, "-o", tmp, LIB, "-L", lib, "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10",
           "-lc10_cuda", "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{lib}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed for tg_torch.cpp:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING)
    with open(BINDING_FOR, "w") as f:
        f.write(binding_for(torch_dir))


def build(force: bool = False, verbose: bool = False, extra: list[str] | None = None, debug: bool = False) -> str:
    """Compile and link libtg_gemm.so (or, with debug=True, libtg_gemm_debug.so with the
    device-side bounds checks); returns its path. Skips work when up to date."""
    lib_path = LIB_DEBUG if debug else LIB
    objdir = OBJDIR_DEBUG if debug else OBJDIR
    torch = None if debug else torch_dir()
    want_lib = force or bool(extra) or not up_to_date(lib_path)
    want_binding = torch is not None and (force or not binding_up_to_date(torch))
    if not want_lib and not want_binding:
        return lib_path
    os.makedirs(objdir, exist_ok=True)
    cc = nvcc()
    flags = CFLAGS + ARCH + (["-DTG_DEBUG=1"] if debug else []) + (extra or [])

    def compile_one(src: str) -> str:
        obj = os.path.join(objdir, src.replace(".cu", ".o"))
        cmd = [cc, "-c", os.path.join(CSRC, src), "-o", obj] + flags
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr, flush=True)
        return obj

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        binding = ex.submit(compile_binding, objdir, torch) if want_binding else None
        objs = list(ex.map(compile_one, SOURCES)) if want_lib else []
    if want_lib:
        tmp = lib_path + f".tmp{os.getpid()}"
        cmd = [cc, "-shared", "-o", tmp, "-Xlinker", f"-soname={os.path.basename(lib_path)}"] + objs + ARCH + ["-lineinfo"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, lib_path)
    if binding is not None:
        link_binding(binding.result(), torch)
    return lib_path


if __name__ == "__main__":
    v = "-v" in sys.argv
    extra = ["-Xptxas", "-v"] if "--ptxas" in sys.argv else None
    print(build(force=True, verbose=v or bool(extra), extra=extra, debug="--debug" in sys.argv))
