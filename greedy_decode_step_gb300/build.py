"""Build libdec.so (sm_103a) in place with nvcc: one object per translation
unit, compiled in parallel, then linked against the shared CUDA runtime; and
with the host compiler the extension module ``_binding`` against torch."""
from __future__ import annotations

import contextlib
import os
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libdec.so")
BINDING = os.path.join(HERE, "_binding.so")
UNITS = ["api.cu", "gemv_qkv.cu", "gemv_glu.cu", "gemv_resid.cu", "gemv_head.cu", "attn.cu", "step.cu", "prefill.cu",
         "select.cu", "tcgemm.cu", "kv4.cu", "long_attn.cu", "blocks.cu", "long_api.cu", "fp8.cu", "fp8_gemm.cu",
         "moe_route.cu", "moe.cu", "fp8_api.cu"]
HEADERS = ["dec_common.cuh", "dec_kernels.cuh", "dec_attn.cuh", "dec_step.cuh", "dec_launch.cuh", "dec_long.cuh",
           "dec_host.cuh", "dec_tc.cuh", "dec_fp8.cuh", "dec_moe.cuh"]
ARCH = "-gencode=arch=compute_103a,code=sm_103a"


def nvcc() -> str:
    home = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    path = os.path.join(home, "bin", "nvcc")
    return path if os.path.exists(path) else "nvcc"


def _flags():
    return [ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2", "-I", CSRC, "-I", INCLUDE,
            "--expt-relaxed-constexpr"]


def _binding_key() -> str:
    """What the binding's object depends on beside its sources: the versions of torch and Python."""
    import torch
    return f"{torch.__version__}_{sysconfig.get_config_var('SOABI')}"


def _binding_job(force: bool):
    """The compile command of binding.cpp, or None, and its object (one per torch and Python)."""
    import torch
    src, header = os.path.join(CSRC, "binding.cpp"), os.path.join(INCLUDE, "libdec.h")
    obj = os.path.join(BUILD, f"binding_{_binding_key()}.o")
    root = os.path.join(os.path.dirname(torch.__file__), "include")
    cuda = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")
    paths = [root, os.path.join(root, "torch", "csrc", "api", "include"), sysconfig.get_paths()["include"], cuda, INCLUDE]
    cmd = ["g++", "-O2", "-fPIC", "-std=c++17", *(f"-I{p}" for p in paths), "-c", src, "-o", obj]
    return (cmd if force or _stale(obj, [src, header, __file__]) else None), obj


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    """Compile the CUDA sources into ``libdec.so`` next to this file."""
    os.makedirs(BUILD, exist_ok=True)
    headers = [os.path.join(CSRC, h) for h in HEADERS] + [os.path.join(INCLUDE, "libdec.h")]
    objs = []
    jobs = []
    for u in UNITS:
        src = os.path.join(CSRC, u)
        obj = os.path.join(BUILD, u.replace(".cu", ".o"))
        objs.append(obj)
        if force or _stale(obj, [src, __file__] + headers):
            jobs.append([nvcc(), *_flags(), *extra, "-c", src, "-o", obj])

    binding_cmd, binding_obj = _binding_job(force)
    if binding_cmd:
        jobs.insert(0, binding_cmd)

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"{os.path.basename(cmd[0])} failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            sys.stderr.write(r.stdout + r.stderr)

    with ThreadPoolExecutor(max_workers=min(len(jobs) + 1, os.cpu_count() or 1)) as ex:
        list(ex.map(run, jobs))
    if force or jobs or _stale(LIB, objs):
        tmp = LIB + f".tmp{os.getpid()}"
        cuda_lib = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "lib64")
        run([nvcc(), ARCH, "-shared", "-cudart", "shared", "-o", tmp, *objs, "-Xlinker", f"-rpath,{cuda_lib}"])
        os.replace(tmp, LIB)
    # the linked module has one name, so a note beside it says which object it was linked from
    note = os.path.join(BUILD, "binding_linked")
    linked = None
    if os.path.exists(note):
        with open(note) as f:
            linked = f.read()
    if force or jobs or linked != os.path.basename(binding_obj) or _stale(BINDING, [binding_obj, LIB]):
        import torch
        tmp = BINDING + f".tmp{os.getpid()}"
        libs = os.path.join(os.path.dirname(torch.__file__), "lib")
        # torch is imported first, so its libraries are found by name; libdec.so lies beside the module
        run(["g++", "-shared", "-o", tmp, binding_obj, "-L", HERE, "-l:libdec.so", "-L", libs, "-ltorch_python",
             "-ltorch_cpu", "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN"])
        with contextlib.suppress(FileNotFoundError):  # another process may build as well
            os.remove(note)
        os.replace(tmp, BINDING)
        with open(note, "w") as f:
            f.write(os.path.basename(binding_obj))
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True,
                extra=["-Xptxas", "-v"] if "--ptxas" in sys.argv else []))
