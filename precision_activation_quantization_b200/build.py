"""Build libpqg.so in-tree with nvcc for sm_100a, and its tensor binding.

    python -m precision_activation_quantization_b200.build [--force] [--verbose]

Each translation unit under csrc/ compiles in parallel to an object in _build/,
and then everything links into precision_activation_quantization_b200/libpqg.so
against the static CUDA runtime.  csrc/pqg_torch.cpp, which marshals torch tensors
for the C ABI, becomes _pqg_torch.so beside it.  No fast-math: the codes and scales must be
bit-exact, so every division and reciprocal has to round correctly.
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import os
import shutil
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libpqg.so")
BINDING = os.path.join(PKG, "_pqg_torch.so")
BINDING_SRC = os.path.join(CSRC, "pqg_torch.cpp")
BINDING_ABI = BINDING[:-3] + ".abi"   # the torch and python that BINDING was built for

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                     "-Xcompiler", "-fvisibility=hidden", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libpqg.so")
    return path


def sources() -> list[str]:
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _inputs() -> list[str]:
    deps = [os.path.join(CSRC, f) for f in os.listdir(CSRC)
            if f.endswith((".cu", ".cuh", ".h"))]
    deps.append(os.path.join(INCLUDE, "pqg.h"))
    deps.append(os.path.abspath(__file__))
    return deps


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(d) <= t for d in _inputs())


def _compile(src: str, verbose: bool, defines=(), build_dir: str = BUILD) -> str:
    obj = os.path.join(build_dir, os.path.basename(src)[:-3] + ".o")
    cmd = ([nvcc()] + NVCC_FLAGS + [f"-D{d}" for d in defines]
           + (["-Xptxas", "-v"] if verbose else []) + ["-c", src, "-o", obj])
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{res.stderr}")
    if verbose and res.stderr:
        print(res.stderr)
    return obj


def build(force: bool = False, verbose: bool = False, defines=(), out: str = LIB) -> str:
    """Compile and link libpqg.so unless it is newer than every source.

    ``defines`` (e.g. ``["PQG_ITEMS_PLAIN=4"]``) set the build-time tuning
    macros; with ``out`` they build a variant library elsewhere."""
    if not force and not defines and out == LIB and up_to_date():
        return LIB
    build_dir = BUILD if not defines else os.path.join(BUILD, "_".join(defines).replace("=", ""))
    os.makedirs(build_dir, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        objs = list(ex.map(lambda s: _compile(s, verbose, defines, build_dir), sources()))
    tmp = out + f".tmp{os.getpid()}"
    cmd = [nvcc()] + ARCH + ["-shared", "-cudart", "static", "-o", tmp] + objs
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stderr}")
    os.replace(tmp, out)
    return out


def binding_abi() -> str:
    """What a built binding depends on beside its sources."""
    import torch
    return f"torch {torch.__version__}, {sysconfig.get_config_var('SOABI')}\n"


def binding_up_to_date() -> bool:
    deps = [BINDING_SRC, os.path.join(INCLUDE, "pqg.h"), os.path.abspath(__file__)]
    if not os.path.exists(BINDING) or not os.path.exists(BINDING_ABI):
        return False
    with open(BINDING_ABI, encoding="utf-8") as f:
        if f.read() != binding_abi():
            return False
    return all(os.path.getmtime(d) <= os.path.getmtime(BINDING) for d in deps)


def build_binding(force: bool = False) -> str:
    """Compile _pqg_torch.so against the installed torch unless it is newer than
    its sources and was built for the same torch and python."""
    if not force and binding_up_to_date():
        return BINDING
    import torch
    home = os.path.dirname(os.path.abspath(torch.__file__))
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    include = [os.path.join(home, "include"),
               os.path.join(home, "include", "torch", "csrc", "api", "include"),
               os.path.join(cuda, "include"), sysconfig.get_paths()["include"], INCLUDE]
    tmp = BINDING + f".tmp{os.getpid()}"
    cmd = (["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}"]
           + [f"-isystem{d}" for d in include] + ["-o", tmp, BINDING_SRC]
           + ["-L" + os.path.join(home, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu",
              "-ltorch_cuda", "-ltorch_python", "-ldl"])
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"g++ failed on {BINDING_SRC}:\n{res.stderr}")
    os.replace(tmp, BINDING)
    with open(BINDING_ABI, "w", encoding="utf-8") as f:
        f.write(binding_abi())
    return BINDING


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true", help="print ptxas register/spill info")
    args = ap.parse_args()
    print(build(force=args.force, verbose=args.verbose))
    print(build_binding(force=args.force))


if __name__ == "__main__":
    main()
