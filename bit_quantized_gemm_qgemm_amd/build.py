"""Build libqgemm.so in-tree with hipcc for gfx950, and the module _binding, the
native half of the Python binding, with the host compiler (left out, with a
warning, where there is no g++ or no Python headers: the library does not need it).

    python -m bit_quantized_gemm_qgemm_amd.build [-v]

Every call compiles from source (no up-to-date check), so the library always
matches the sources it sits next to.
"""

import concurrent.futures
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG_DIR, "csrc")
ROOT = os.path.dirname(PKG_DIR)
INCLUDE = os.path.join(ROOT, "include")
LIB_NAME = "libqgemm.so"
LIB_PATH = os.path.join(PKG_DIR, LIB_NAME)
BINDING_PATH = os.path.join(PKG_DIR, "_binding" + sysconfig.get_config_var("EXT_SUFFIX"))
BUILD_DIR = os.path.join(ROOT, "_build")

SOURCES = ["decode_gemm.hip", "tile_gemm.hip", "tile_wo256.hip", "tile_mx256.hip", "quantize.hip",
           "prepack.hip", "probes.hip", "kv_cache.hip", "paged_attention.hip",
           "api.cpp"]

HIPCC_FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-Wall",
    "-Wno-unused-command-line-argument",
    # packed fp32 VALU ops stay off: the compiler would otherwise form them
    # from plain float code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I", INCLUDE,
    "-I", CSRC,
]


def _hipcc():
    exe = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(exe):
        raise RuntimeError("hipcc not found; a ROCm toolchain is required to build libqgemm")
    return exe


def _run(cmd, what, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"{what}:\n{res.stdout}\n{res.stderr}")


def _compile(src, verbose):
    obj = os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".o")
    lang = ["-x", "hip"] if src.endswith(".cpp") else []
    cmd = [_hipcc(), *HIPCC_FLAGS, *lang, "-c", os.path.join(CSRC, src), "-o", obj]
    _run(cmd, f"hipcc failed on {src}", verbose)
    return obj


def _binding_needs():
    """What the binding's build lacks on this machine, or None."""
    if shutil.which("g++") is None:
        return "g++"
    if not os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        return "Python.h"
    return None


def _compile_binding(verbose):
    import torch

    obj = os.path.join(BUILD_DIR, "binding.o")
    _run(["g++", "-O2", "-std=c++17", "-fPIC", "-Wall",
          f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", INCLUDE,
          "-isystem", os.path.join(os.path.dirname(torch.__file__), "include"),
          "-isystem", sysconfig.get_paths()["include"],
          "-c", os.path.join(CSRC, "binding.cpp"), "-o", obj], "g++ failed on binding.cpp", verbose)
    return obj


def _link_binding(obj, verbose):
    """By library names only: importing torch has loaded its libraries, and
    libqgemm.so lies next to the binding."""
    import torch

    tmp = BINDING_PATH + ".tmp"
    _run(["g++", "-shared", "-fPIC", obj, "-L", PKG_DIR, "-l:" + LIB_NAME,
          "-L", os.path.join(os.path.dirname(torch.__file__), "lib"), "-ltorch_python", "-ltorch_cpu",
          "-lc10", "-Wl,-rpath,$ORIGIN", "-o", tmp], "link of the binding failed", verbose)
    os.replace(tmp, BINDING_PATH)


def build(verbose=False):
    """Compile every HIP source for gfx950 and link libqgemm.so in the package,
    then the binding next to it."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    jobs = min(len(SOURCES), max(1, (os.cpu_count() or 2)))
    with concurrent.futures.ThreadPoolExecutor(max_workers=jobs) as ex:
        missing = _binding_needs()
        binding = None if missing else ex.submit(_compile_binding, verbose)
        objs = list(ex.map(lambda s: _compile(s, verbose), SOURCES))
    tmp = LIB_PATH + ".tmp"
    _run([_hipcc(), "--offload-arch=gfx950", "-shared", "-fPIC", *objs, "-o", tmp], "link failed",
         verbose)
    os.replace(tmp, LIB_PATH)
    if not missing:
        _link_binding(binding.result(), verbose)
        return LIB_PATH
    if os.path.exists(BINDING_PATH):   # of an earlier build, with other sources
        os.remove(BINDING_PATH)
    warnings.warn(f"{missing} not found: built without the native binding", RuntimeWarning)
    return LIB_PATH


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
