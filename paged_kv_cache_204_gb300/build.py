"""Build the CUDA library in-tree: every .cu under csrc/ is compiled for
sm_103a (and every .cpp, host-only code, by nvcc's host compiler) in
parallel and linked into _build/libpkv.so (CUDA runtime linked statically,
so the library loads beside any PyTorch build). csrc/torch_binding.cxx becomes
the Python extension _build/_pkv_torch.so, compiled against this machine's
PyTorch and linked to libpkv.so; it is built again when either it or that
PyTorch has changed.

Run by its path, `python paged_kv_cache_204_gb300/build.py`: importing the package
needs the library."""
from __future__ import annotations

import glob
import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT_DIR = os.path.join(HERE, "_build")
LIB = os.path.join(OUT_DIR, "libpkv.so")
BINDING_SRC = os.path.join(CSRC, "torch_binding.cxx")
BINDING = os.path.join(OUT_DIR, "_pkv_torch.so")
BINDING_ABI = BINDING + ".abi"  # the PyTorch and the Python it was built for

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
              "-I", INCLUDE, "-I", CSRC]


def _nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cpp")))


def _headers() -> list[str]:
    return glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)]


def _newer(made: str, sources: list[str]) -> bool:
    return os.path.exists(made) and all(os.path.getmtime(d) <= os.path.getmtime(made) for d in sources)


def library_up_to_date() -> bool:
    return _newer(LIB, _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
                  + _headers())


def binding_abi() -> str:
    """What the Python extension is bound to: this PyTorch and this Python."""
    import sysconfig
    import torch
    return f"torch {torch.__version__} {sysconfig.get_config_var('SOABI')}"


def binding_for() -> str | None:
    """The binding_abi() that the extension was built for; None if there is none."""
    if not os.path.exists(BINDING) or not os.path.exists(BINDING_ABI):
        return None
    with open(BINDING_ABI) as f:
        return f.read()


def binding_up_to_date() -> bool:
    return _newer(BINDING, [BINDING_SRC] + _headers()) and binding_for() == binding_abi()


def up_to_date() -> bool:
    return library_up_to_date() and binding_up_to_date()


def _binding_flags() -> tuple[list[str], list[str]]:
    """Compiler and linker flags of the Python extension."""
    import sysconfig
    import torch
    home = os.path.dirname(torch.__file__)
    cuda = os.path.join(os.path.dirname(os.path.dirname(_nvcc())) or "/usr/local/cuda", "include")
    inc = [os.path.join(home, "include"), os.path.join(home, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], cuda, INCLUDE]
    libs = os.path.join(home, "lib")
    return ([f"-I{i}" for i in inc] + [f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"],
            [f"-L{libs}", "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python", f"-Wl,-rpath,{libs}", LIB,
             "-Wl,-rpath,$ORIGIN"])


def _run(what: str, cmd: list[str]) -> str:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stderr}")
    return r.stderr


def _compile_binding(obj: str) -> list[str]:
    """The extension's object file; returns the flags it is linked with."""
    cflags, ldflags = _binding_flags()
    _run(f"g++ on {BINDING_SRC}", ["g++", "-O2", "-std=c++17", "-fPIC", *cflags, "-c", BINDING_SRC, "-o", obj])
    return ldflags


def _link_binding(obj: str, ldflags: list[str]) -> None:
    tmp = BINDING + f".tmp{os.getpid()}"
    _run("link", ["g++", "-shared", "-o", tmp, obj, *ldflags])
    if os.path.exists(BINDING_ABI):
        os.remove(BINDING_ABI)
    os.replace(tmp, BINDING)
    with open(BINDING_ABI, "w") as f:
        f.write(binding_abi())


def build(force: bool = False, verbose_ptxas: bool = False, jobs: int | None = None) -> str:
    """Build what is not up to date: the library and the Python extension. The library is in
    place even where the extension does not compile, which then raises."""
    library, extension = force or not library_up_to_date(), force or not binding_up_to_date()
    if not library and not extension:
        return LIB
    os.makedirs(OUT_DIR, exist_ok=True)
    srcs = _sources() if library else []
    binding_obj = os.path.join(OUT_DIR, "torch_binding.cxx.o")
    nvcc = _nvcc()
    extra = ["-Xptxas", "-v"] if verbose_ptxas else []

    def compile_one(src: str) -> tuple[str, str]:
        obj = os.path.join(OUT_DIR, os.path.basename(src) + ".o")
        return obj, _run(f"nvcc on {src}", [nvcc, *ARCH, *NVCC_FLAGS, *extra, "-c", src, "-o", obj])

    with ThreadPoolExecutor(max_workers=jobs or min(len(srcs) + 1, os.cpu_count() or 4)) as ex:
        binding = ex.submit(_compile_binding, binding_obj) if extension else None
        results = list(ex.map(compile_one, srcs))
        if library:
            if verbose_ptxas:
                for _, log in results:
                    sys.stderr.write(log)
            tmp = LIB + f".tmp{os.getpid()}"
            _run("link", [nvcc, *ARCH, "-shared", "-cudart", "static", "-Xlinker", "-soname=libpkv.so", "-o", tmp]
                 + [o for o, _ in results])
            os.replace(tmp, LIB)
        if binding is not None:
            _link_binding(binding_obj, binding.result())
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose_ptxas="-v" in sys.argv))
