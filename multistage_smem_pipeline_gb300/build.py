"""Build the C-ABI library libgemm_tn_f16.so in-tree with nvcc for sm_103a.

    python -m multistage_smem_pipeline_gb300.build [--force]

Each translation unit under csrc/ is compiled in parallel, then linked into
multistage_smem_pipeline_gb300/lib/libgemm_tn_f16.so (the CUDA runtime is
linked statically; the driver's cuTensorMapEncodeTiled is fetched at run time
through the runtime's entry-point query, so no -lcuda is needed).  The Python
binding of moe_fp4.h and linear.h, csrc/experts_binding.cpp, is compiled beside them against
the installed torch's headers and linked to the library; without a torch the
library alone is built.
"""
from __future__ import annotations

import glob
import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OBJ_DIR = os.path.join(PKG, "_build")
LIB_DIR = os.path.join(PKG, "lib")
LIB = os.path.join(LIB_DIR, "libgemm_tn_f16.so")
BINDING_SRC = os.path.join(CSRC, "experts_binding.cpp")   # includes linear_binding.h
BINDING = os.path.join(LIB_DIR, "_experts.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2",
                     "-I" + INCLUDE, "-I" + CSRC]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libgemm_tn_f16.so")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + [f for folder, kind in ((CSRC, "*.cuh"), (CSRC, "*.h"), (INCLUDE, "*.h"))
                         for f in glob.glob(os.path.join(folder, kind))]


def _has_torch() -> bool:
    """The binding is left out where there is none to compile it against."""
    return importlib.util.find_spec("torch") is not None


def _built_for() -> str:
    """What the binding's object code depends on beside its sources: torch and Python."""
    try:
        version = importlib.metadata.version("torch")   # without the second that importing it takes
    except importlib.metadata.PackageNotFoundError:
        import torch
        version = torch.__version__
    return f"torch {version}, {sysconfig.get_config_var('SOABI')}\n"


def _stamp() -> str:
    return os.path.splitext(BINDING)[0] + ".built_for"


def _read(path: str) -> str:
    if not os.path.exists(path):
        return ""
    with open(path) as f:
        return f.read()


def up_to_date() -> bool:
    wanted = [LIB] + ([BINDING] if _has_torch() else [])
    if not all(os.path.exists(w) for w in wanted):
        return False
    if BINDING in wanted and _read(_stamp()) != _built_for():
        return False
    t = min(os.path.getmtime(w) for w in wanted)
    return all(os.path.getmtime(d) <= t for d in _deps() + [BINDING_SRC])


def _binding_command(out: str) -> list[str]:
    """Compiles the binding of moe_fp4.h to an object file."""
    import torch
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-I" + inc,
            "-I" + os.path.join(inc, "torch", "csrc", "api", "include"),
            "-I" + sysconfig.get_paths()["include"], "-I" + cuda, "-I" + INCLUDE,
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
            "-c", BINDING_SRC, "-o", out]


def _link_binding(obj: str) -> None:
    import torch
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = BINDING + f".{os.getpid()}.tmp"
    subprocess.check_call(["g++", "-shared", "-o", tmp, obj, "-L" + libs, "-lc10", "-lc10_cuda",
                           "-ltorch_cpu", "-ltorch_cuda", "-ltorch", "-ltorch_python", "-L" + LIB_DIR,
                           "-l:libgemm_tn_f16.so", "-Wl,-rpath,$ORIGIN"])
    os.replace(tmp, BINDING)
    with open(_stamp(), "w") as f:
        f.write(_built_for())


def _start(cmd: list[str]) -> subprocess.Popen:
    return subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)


def _finish(procs, verbose: bool) -> list[str]:
    """Waits for compilers; what those that failed said."""
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        if p.returncode != 0:
            failed.append(f"{os.path.basename(src)}:\n{out}")
        elif verbose and out:
            sys.stdout.write(out)
    return failed


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(OBJ_DIR, exist_ok=True)
    os.makedirs(LIB_DIR, exist_ok=True)
    exe = nvcc()
    procs = []
    objs = []
    for src in _sources():
        obj = os.path.join(OBJ_DIR, os.path.basename(src) + ".o")
        objs.append(obj)
        cmd = [exe] + NVCC_FLAGS + (["-Xptxas", "-v"] if verbose else []) + ["-c", src, "-o", obj]
        procs.append((src, _start(cmd)))
    binding_obj = os.path.join(OBJ_DIR, "experts_binding.cpp.o")
    binding, binding_failed = [], []
    if _has_torch():
        try:
            binding.append((BINDING_SRC, _start(_binding_command(binding_obj))))
        except Exception as e:  # an installed torch that does not import
            binding_failed.append(f"{os.path.basename(BINDING_SRC)}: {e!r}")
    failed = _finish(procs, verbose)
    binding_failed += _finish(binding, verbose)
    if failed:
        raise RuntimeError("compilation failed:\n" + "\n".join(failed + binding_failed))
    tmp = LIB + f".{os.getpid()}.tmp"
    subprocess.check_call([exe] + ARCH + ["-shared", "-o", tmp, "-Xlinker",
                                          "-soname=libgemm_tn_f16.so"] + objs)
    os.replace(tmp, LIB)
    if binding_failed:
        raise RuntimeError("compilation of the binding failed:\n" + "\n".join(binding_failed))
    if binding:
        _link_binding(binding_obj)
    else:
        print("no torch: the Python binding of moe_fp4.h is left out", file=sys.stderr)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
