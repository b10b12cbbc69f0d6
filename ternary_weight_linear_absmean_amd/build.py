"""Build libbitlinear.so in-tree with hipcc for gfx950.

    python -m ternary_weight_linear_absmean_amd.build [-v] [-j N]

Each source is compiled to an object (in parallel), then linked into
``ternary_weight_linear_absmean_amd/libbitlinear.so``.  Device code is built
with FMA contraction off (every fp32 step of the quantisers and the rescale
is one IEEE rounding), without packed-fp32 instructions, and with the leading
kernel arguments preloaded into SGPRs.  Beside it ``_calls.so``, the Python
binding's short way into the calls on the paged caches (host code): it takes a C++
compiler, Python's and torch's headers, and where it cannot be built the binding does
without it.
"""
import concurrent.futures as cf
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(ROOT, "_build")
LIB = os.path.join(HERE, "libbitlinear.so")
CALLS = os.path.join(HERE, "_calls.so")

SOURCES = ["api.cpp", "quant.hip", "gemv.hip", "gemm.hip", "gemm_skinny.hip", "ffn.hip",
           "stack.hip", "stack_persistent.hip", "backward.hip", "t5.hip",
           "kv8.hip", "kv8_attention.hip", "kv4.hip",
           "kv4_attention.hip", "kv_read.hip", "w4.hip"]
ARCH = "gfx950"

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
FLAGS = [f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC",
         "-ffp-contract=off", "-fno-fast-math", "-fvisibility=hidden",
         "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
         # kernarg preload: the leading kernel arguments (up to 16 dwords) are
         # placed in SGPRs at wave launch, so a kernel reads them without a
         # scalar load round trip (the fused decode kernel passes its job
         # boundaries there; the few-token product gains ~0.15 us per launch)
         "-mllvm", "-amdgpu-kernarg-preload-count=16",
         "-Wall", "-Wno-unused-function",
         "-I", INCLUDE, "-I", CSRC]


def _compile(src, verbose):
    obj = os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".o")
    cmd = [HIPCC, *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
    if src.endswith(".cpp"):
        cmd[1:1] = ["-x", "hip"]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    err = "\n".join(l for l in r.stderr.splitlines()
                    if "packed-fp32-ops" not in l and l.strip())
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed on {src}:\n{err}")
    if err and verbose:
        print(err, flush=True)
    return obj


def _compile_calls(verbose):
    import torch

    torch_dir = os.path.dirname(torch.__file__)
    rocm = os.path.dirname(os.path.dirname(HIPCC))
    tmp = CALLS + ".tmp"
    built_for = f"torch {torch.__version__}, Python {sys.version_info[0]}.{sys.version_info[1]}"
    # NDEBUG: without it pybind11's headers bring a thread-local counter.  A library with
    # thread-local storage that is loaded into a running program and never touches it makes
    # every other library's access to its own take the slow way (glibc 2.35): 1 us a launch.
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-DNDEBUG",
           "-D__HIP_PLATFORM_AMD__", "-DUSE_ROCM", f'-DBUILT_FOR="{built_for}"', "-I", INCLUDE,
           "-I", sysconfig.get_paths()["include"], "-I", os.path.join(torch_dir, "include"),
           "-I", os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
           "-I", os.path.join(rocm, "include"), os.path.join(CSRC, "torch_calls.cpp"), "-o", tmp,
           "-L", os.path.join(torch_dir, "lib"), "-lc10", "-lc10_hip", "-ltorch_cpu", "-ltorch_hip", "-ltorch_python"]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed on torch_calls.cpp:\n{r.stderr}")
    os.replace(tmp, CALLS)


def build_calls(verbose: bool = False):
    """_calls.so's path, or None, with the reason on stderr and no file of an earlier
    build left, where it cannot be built."""
    try:
        _compile_calls(verbose)
        return CALLS
    except (ImportError, OSError, RuntimeError) as e:
        if os.path.exists(CALLS):
            os.remove(CALLS)
        print(f"_calls.so is not built, calls on the paged caches go through ctypes: {e}", file=sys.stderr, flush=True)
        return None


def build(verbose: bool = False, jobs: int = 8) -> str:
    os.makedirs(BUILD_DIR, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=max(1, min(jobs, len(SOURCES) + 1))) as ex:
        calls = ex.submit(build_calls, verbose)
        objs = list(ex.map(lambda s: _compile(s, verbose), SOURCES))
        calls.result()
    tmp = LIB + ".tmp"
    cmd = [HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp, *objs]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    jobs = 8
    if "-j" in sys.argv:
        jobs = int(sys.argv[sys.argv.index("-j") + 1])
    print(build(verbose="-v" in sys.argv, jobs=jobs))
