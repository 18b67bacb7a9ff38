"""Build ``libattn_res.so`` for sm_103a and the compiled binding ``_mx.so`` of
its microscaled entry points, in-tree.

Twelve translation units: the C ABI (attn_res_api.cu; attn_res_mx_api.cu with
the microscaled row kernels), the microscaled product (attn_res_mx_product.cu)
and the mixture's kernel specialisations for each num_blocks value
(attn_res_inst.cu compiled nine times with -DATTN_RES_S=0..8), compiled in
parallel and linked into one shared object with the CUDA runtime linked
statically; and mx_binding.cpp, host code against the installed PyTorch, linked
to it.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OBJ_DIR = os.path.join(PKG, "_build")
LIB_DIR = os.path.join(PKG, "_lib")
LIB = os.path.join(LIB_DIR, "libattn_res.so")
BINDING = os.path.join(LIB_DIR, "_mx.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                     "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    exe = shutil.which("nvcc")
    if exe:
        return exe
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    if os.path.exists(cand):
        return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libattn_res")


def _sources():
    deps = [os.path.join(CSRC, f) for f in os.listdir(CSRC)
            if f.endswith((".cu", ".cuh", ".cpp"))] + [os.path.join(INCLUDE, "attn_res.h")]
    units = [(n, os.path.join(CSRC, n + ".cu"), [])
             for n in ("attn_res_mx_product", "attn_res_api", "attn_res_mx_api")]
    for s in range(9):
        units.append((f"attn_res_inst_s{s}", os.path.join(CSRC, "attn_res_inst.cu"),
                      [f"-DATTN_RES_S={s}"]))
    return units, deps


def _binding_cmd(obj: str):
    """The host compiler's command for mx_binding.cpp, and the linker's."""
    import sysconfig

    import torch
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    inc = [os.path.join(root, "include"), os.path.join(cuda, "include"),
           sysconfig.get_paths()["include"]]
    comp = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-I", INCLUDE]
    for p in inc:
        comp += ["-isystem", p]
    link = ["-L", LIB_DIR, "-lattn_res", "-L", os.path.join(root, "lib"), "-lc10", "-lc10_cuda",
            "-ltorch", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python", "-Wl,-rpath,$ORIGIN"]
    return comp + ["-c", os.path.join(CSRC, "mx_binding.cpp"), "-o", obj], ["g++", "-shared", obj] + link


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """Compile (if stale) and return the path of the shared object."""
    units, deps = _sources()
    if not force and not ptxas_info and not _stale(LIB, deps) and not _stale(BINDING, deps):
        return LIB
    os.makedirs(OBJ_DIR, exist_ok=True)
    os.makedirs(LIB_DIR, exist_ok=True)
    exe = nvcc()

    binding_obj = os.path.join(OBJ_DIR, "mx_binding.o")
    binding_compile, binding_link = _binding_cmd(binding_obj)

    def compile_one(u):
        if u is None:
            name, cmd, obj = "mx_binding", binding_compile, binding_obj
            r = subprocess.run(cmd, capture_output=True, text=True)
            if r.returncode != 0:
                raise RuntimeError(f"g++ failed for {name}:\n{r.stdout}\n{r.stderr}")
            return None, r.stderr
        name, src, extra = u
        obj = os.path.join(OBJ_DIR, name + ".o")
        cmd = [exe] + NVCC_FLAGS + extra + (["-Xptxas", "-v"] if ptxas_info else []) + \
            ["-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {name}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stderr

    workers = min(len(units) + 1, max(1, os.cpu_count() or 1))
    with cf.ThreadPoolExecutor(workers) as ex:
        results = list(ex.map(compile_one, units + [None]))
    if verbose or ptxas_info:
        for _, log in results:
            if log:
                sys.stderr.write(log)
    objs = [o for o, _ in results if o is not None]
    for target, cmd in ((LIB, [exe] + ARCH + ["-shared"] + objs), (BINDING, binding_link)):
        tmp = target + f".tmp{os.getpid()}"
        r = subprocess.run(cmd + ["-o", tmp], capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, target)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True,
                ptxas_info="--ptxas-info" in sys.argv))
