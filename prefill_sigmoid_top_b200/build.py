"""Build libmoe_b200.so in-tree with nvcc for sm_100a (run: python -m prefill_sigmoid_top_b200.build)."""
from __future__ import annotations

import concurrent.futures as cf
import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libmoe_b200.so")
SOURCES = ["api.cu", "router.cu", "router_screen.cu", "align.cu", "finalize.cu", "gemm_bf16.cu", "gemm_persistent.cu",
           "gemm_pair.cu", "nvfp4.cu", "nvfp4_pair.cu", "layer_fused.cu", "measure.cu", "tp_finalize.cu",
           "router_group.cu", "int8.cu", "int8_gemm.cu", "int8_few.cu",
           "int8_pair.cu"]
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo", "-std=c++17", "-DNDEBUG", "-Xcompiler", "-fPIC",
         "-Xcompiler", "-fvisibility=hidden", "-I", os.path.join(ROOT, "include"), "-I", CSRC]


def _stale(out: str, deps: list[str]) -> bool:
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(d) > t for d in deps)


def binding_path() -> str:
    """The binding for this interpreter and this torch: it is compiled against the headers of both and fits no others,
    so each pair has a file of its own and one that was built before an upgrade is not loaded after it."""
    import torch
    return os.path.join(PKG, f"_binding.{sysconfig.get_config_var('SOABI')}.torch-{torch.__version__}.so")


def build_binding(force: bool = False) -> str:
    """Compile the CPython extension that marshals the short calls (csrc/binding.cpp), against libmoe_b200.so beside it."""
    src, header = os.path.join(CSRC, "binding.cpp"), os.path.join(ROOT, "include", "moe_b200.h")
    path = binding_path()
    if force or _stale(path, [src, header]):
        import torch
        tdir = os.path.dirname(torch.__file__)
        tmp = path + f".tmp{os.getpid()}"
        cxx = os.environ.get("CXX", "g++")
        cmd = [
            cxx, "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", sysconfig.get_paths()["include"],
            "-isystem", os.path.join(tdir, "include"),
            "-isystem", os.path.join(tdir, "include", "torch", "csrc", "api", "include"),
            "-isystem", os.path.join(os.path.dirname(os.path.dirname(NVCC)), "include"),
            "-I", os.path.join(ROOT, "include"), src, "-o", tmp, "-L", PKG, "-l:libmoe_b200.so",
            "-L", os.path.join(tdir, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda",
            "-Wl,-rpath,$ORIGIN"]
        try:
            subprocess.check_call(cmd)
        except (OSError, subprocess.CalledProcessError) as e:
            raise RuntimeError(f"the Python binding was not built: {cxx} failed on {src} (it takes the headers of Python "
                               f"and torch, which the C library does not): {e}") from e
        os.replace(tmp, path)
    return path


TRACE_LIB = os.path.join(PKG, "libmoe_b200_trace.so")


def build(force: bool = False, verbose: bool = False, extra_flags: list[str] | None = None,
          trace: bool = False) -> str:
    """Compile the library (nvcc alone; build_binding compiles what Python calls it through); trace=True
    builds the timeline variant instead (-DMOE_PAIR_TRACE for the 2-SM pair GEMMs, -DMOE_LAYER_TRACE for
    the single-launch layer, into libmoe_b200_trace.so; see pair_trace.py and layer_trace.py), never
    loaded by the package."""
    build_dir = BUILD + ("_trace" if trace else "")
    lib = TRACE_LIB if trace else LIB
    os.makedirs(build_dir, exist_ok=True)
    headers = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".h", ".cuh"))]
    inc = os.path.join(ROOT, "include")
    headers += [os.path.join(inc, f) for f in os.listdir(inc) if f.endswith(".h")]
    flags = FLAGS + (["-DMOE_PAIR_TRACE", "-DMOE_LAYER_TRACE"] if trace else []) + (extra_flags or [])
    jobs = []
    objs = []
    for src in SOURCES:
        path = os.path.join(CSRC, src)
        obj = os.path.join(build_dir, src.replace(".cu", ".o"))
        objs.append(obj)
        if force or _stale(obj, [path, *headers]):
            jobs.append([NVCC, *flags, "-c", path, "-o", obj])
    with cf.ThreadPoolExecutor(max_workers=min(8, max(1, len(jobs)))) as ex:
        for cmd, res in zip(jobs, ex.map(lambda c: subprocess.run(c, capture_output=True, text=True), jobs)):
            if verbose or res.returncode != 0:
                sys.stderr.write(res.stdout + res.stderr)
            if res.returncode != 0:
                raise RuntimeError(f"nvcc failed: {' '.join(cmd)}")
    if force or jobs or _stale(lib, objs):
        tmp = lib + f".tmp{os.getpid()}"
        subprocess.check_call([NVCC, "-gencode", "arch=compute_100a,code=sm_100a", "-shared", *objs, "-o", tmp])
        os.replace(tmp, lib)
    return lib


def main(argv: list[str]) -> int:
    """Both, the library first: a C program needs that alone, so a binding that cannot be built here is reported and
    leaves it in place."""
    force, trace = "--force" in argv, "--trace" in argv
    print(build(force=force, verbose="-v" in argv, trace=trace))
    if not trace:
        try:
            print(build_binding(force))
        except RuntimeError as e:
            print(e, file=sys.stderr)
    return 0


if __name__ == "__main__":
    sys.exit(main(sys.argv[1:]))
