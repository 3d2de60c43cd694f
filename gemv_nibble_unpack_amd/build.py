"""Build the HIP library in-tree for gfx950 (cross-compiles without a GPU).

    python -m gemv_nibble_unpack_amd.build
"""
from __future__ import annotations

import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
SOURCES = ["quant.hip", "prepack.hip", "matmul.hip", "gemm_launch.hip", "probe.hip", "noalloc.hip",
           "graph.hip", "gemm16.hip"]
# the decoder-layer operators, beside csrc: the traffic records of the matmul
# kernels carry a hash over csrc, which these sources do not change
LAYER_CSRC = os.path.join(HERE, "csrc_layer")
LAYER_SOURCES = ["norm.hip", "append.hip", "attn.hip", "attn_many.hip"]
# the MXFP4 operators
MX_CSRC = os.path.join(HERE, "csrc_mx")
MX_SOURCES = ["mx_quant.hip", "mx_rows.hip", "mx_gemm.hip", "moe.hip"]
OUT = os.path.join(HERE, "libgemv_nibble_unpack.so")
# the Python marshalling of the decoder-layer and MXFP4 operators: host code, built
# against torch's headers, linked to OUT beside it
BIND_SOURCE = os.path.join(LAYER_CSRC, "bind.cpp")
BIND_OUT = os.path.join(HERE, "_layer_bind.so")
OBJ_DIR = os.path.join(HERE, "_build")
ARCH = os.environ.get("W4_OFFLOAD_ARCH", "gfx950")

FLAGS = [
    "-O3", "-std=c++17", f"--offload-arch={ARCH}", "-fPIC", "-shared",
    # correctly rounded float32 division: the quantizers decide codes with '/'
    "-fhip-fp32-correctly-rounded-divide-sqrt", "-fno-fast-math",
    # no packed-FP32 VALU instructions in device code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    # leading scalar kernel arguments arrive preloaded in SGPRs (up to the
    # user-SGPR limit) instead of through a kernel-argument fetch
    "-mllvm", "-amdgpu-kernarg-preload-count=16",
    "-Wall", "-Wno-unused-command-line-argument", *os.environ.get("W4_EXTRA_FLAGS", "").split(),
]


def hipcc():
    for c in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("hipcc not found")


def _run(cmd, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    noise = "packed-fp32-ops' is not a recognized feature"
    err = "\n".join(l for l in res.stderr.splitlines() if noise not in l)
    if res.returncode != 0:
        raise RuntimeError(f"hipcc failed ({res.returncode}):\n{err}")
    if err.strip() and verbose:
        print(err, file=sys.stderr)


def build(verbose=True, jobs=None):
    """Compile every HIP source (in parallel, one object each) and link the
    package's shared library. Each translation unit carries its own device
    code; no device function is called across units.

    The Python marshalling of the decoder-layer operators is built beside it
    where torch, Python's headers and a host C++ compiler are there; the library
    needs none of them and is in its place before an error of the marshalling is
    raised."""
    os.makedirs(OBJ_DIR, exist_ok=True)
    inc = ["-I", os.path.join(ROOT, "include"), "-I", CSRC]
    srcs = ([os.path.join(CSRC, s) for s in SOURCES] +
            [os.path.join(LAYER_CSRC, s) for s in LAYER_SOURCES] +
            [os.path.join(MX_CSRC, s) for s in MX_SOURCES])
    objs = [os.path.join(OBJ_DIR, os.path.splitext(os.path.basename(s))[0] + ".o") for s in srcs]
    cflags = [f for f in FLAGS if f != "-shared"]
    cmds = [[hipcc(), *cflags, *inc, "-c", s, "-o", o] for s, o in zip(srcs, objs)]
    missing = bind_missing()
    jobs = jobs or min(len(cmds) + 1, max(1, (os.cpu_count() or 1)))
    with ThreadPoolExecutor(max_workers=jobs) as ex:
        units = [ex.submit(_run, c, verbose) for c in cmds]
        bind = None if missing else ex.submit(_build_bind_object, verbose)
        for f in units:
            f.result()
        tmp = OUT + ".tmp"
        _run([hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", *objs, "-o", tmp], verbose)
        undefined_kernels(tmp)
        os.replace(tmp, OUT)
        if os.path.exists(BIND_OUT):
            os.remove(BIND_OUT)        # never one of another library
        if missing:
            print(f"{os.path.basename(BIND_OUT)} not built: {missing}", file=sys.stderr)
            return OUT
        _run(bind_link(bind.result(), BIND_OUT + ".tmp"), verbose)
        os.replace(BIND_OUT + ".tmp", BIND_OUT)
    return OUT


def _cxx():
    for c in (os.environ.get("CXX"), shutil.which("g++"), shutil.which("c++")):
        if c and shutil.which(c):
            return c
    return None


def _torch_dir():
    spec = importlib.util.find_spec("torch")          # its place, without importing it
    return os.path.dirname(spec.origin) if spec and spec.origin else None


def bind_missing():
    """What the marshalling module cannot be built for, or None."""
    if _torch_dir() is None:
        return "torch is not installed"
    if not os.path.exists(os.path.join(_torch_dir(), "include", "c10", "hip", "HIPStream.h")):
        return "torch is no ROCm build with headers"
    if not os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        return "Python.h is not installed"
    if _cxx() is None:
        return "no host C++ compiler found"
    return None


def _torch_abi():
    """torch's _GLIBCXX_USE_CXX11_ABI, asked of it in a process of its own."""
    r = subprocess.run([sys.executable, "-c", "import torch; print(int(torch.compiled_with_cxx11_abi()))"],
                       capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"torch cannot be imported:\n{r.stderr}")
    return int(r.stdout.split()[-1])


def _build_bind_object(verbose):
    obj = os.path.join(OBJ_DIR, "bind.o")
    _run(bind_compile(obj, _torch_abi()), verbose)
    return obj


def bind_compile(obj, abi):
    """The command that compiles the marshalling module (host code only)."""
    inc = os.path.join(_torch_dir(), "include")
    return [_cxx(), "-O2", "-std=c++17", "-fPIC", "-Wall", "-D__HIP_PLATFORM_AMD__", "-DUSE_ROCM",
            f"-D_GLIBCXX_USE_CXX11_ABI={abi}", "-I", os.path.join(ROOT, "include"), "-isystem", inc,
            "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"), "-isystem",
            os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "include"), "-I",
            sysconfig.get_paths()["include"], "-c", BIND_SOURCE, "-o", obj]


def bind_link(obj, out):
    return [_cxx(), "-shared", "-fPIC", obj, "-o", out, f"-L{HERE}", f"-l:{os.path.basename(OUT)}",
            "-Wl,-rpath,$ORIGIN", f"-L{os.path.join(_torch_dir(), 'lib')}", "-ltorch_python",
            "-ltorch_hip", "-ltorch_cpu", "-lc10_hip", "-lc10"]


def undefined_kernels(path):
    """Fail if the library references a kernel it does not define: clang drops
    a kernel's host stub without an error when the host pass cannot
    instantiate it, which would only surface when the library is loaded."""
    nm = shutil.which("nm") or "/usr/bin/nm"
    if not os.path.exists(nm):
        return
    res = subprocess.run([nm, "-C", "--undefined-only", path], capture_output=True, text=True)
    bad = [l.strip() for l in res.stdout.splitlines() if "w4::" in l]
    if bad:
        raise RuntimeError("kernels referenced but not defined:\n" + "\n".join(bad))


if __name__ == "__main__":
    print(build())
