"""Build libtq2.so in-tree with hipcc for gfx950.

Flags: -O3, no fast-math (IEEE division and rounding are part of the
definition of pack and of the int8 quantizer), packed-fp32 ops disabled,
code object v5.  Output: ternary_packed_weight_amd/libtq2.so, and beside it
_tq2call.so, the binding's native part (host code against torch's headers).
"""
import os
import subprocess
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libtq2.so")
CALL_LIB = os.path.join(HERE, "_tq2call.so")
PROBE_LIB = os.path.join(HERE, "libtq2probe.so")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
SOURCES = [os.path.join(CSRC, f) for f in ("tq2_kernels.hip", "tq2_api.cpp", "tq2_kv4.hip", "tq2_kv4_api.cpp")]
FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-shared",
    "-mcode-object-version=5",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-command-line-argument",
    "-I", os.path.join(ROOT, "include"), "-I", CSRC,
]


def _hipcc(sources, out, verbose, extra=()):
    tmp = out + ".tmp"
    cmd = [HIPCC, *FLAGS, *extra, *sources, "-o", tmp]
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("hipcc failed:\n" + res.stdout + res.stderr)
    errs = [l for l in res.stderr.splitlines() if "error" in l]
    if errs:
        raise RuntimeError("\n".join(errs))
    # a kernel whose host-side stub was dropped links without complaint and
    # only fails at load time: refuse undefined symbols of our own namespace
    und = subprocess.run(["nm", "-D", "--undefined-only", tmp], capture_output=True, text=True)
    own = [l.split()[-1] for l in und.stdout.splitlines() if "_ZN3tq2" in l]
    if und.returncode != 0 or own:
        raise RuntimeError(f"{out}: undefined library symbols: {own or und.stderr}")
    os.replace(tmp, out)
    return out


def _call(verbose):
    """_tq2call.so: torch's and Python's symbols come from the process that imports it."""
    import torch
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = CALL_LIB + ".tmp"
    cmd = ["g++", "-std=c++17", "-O2", "-fPIC", "-shared", "-Wall", "-I", os.path.join(ROOT, "include"),
           "-D__HIP_PLATFORM_AMD__", "-DUSE_ROCM", "-I", os.path.join(os.path.dirname(os.path.dirname(HIPCC)), "include"),
           "-I", sysconfig.get_paths()["include"], "-I", inc, f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           os.path.join(CSRC, "tq2_call.cpp"), "-L", lib, "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_hip", "-o", tmp]
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        if os.path.exists(CALL_LIB):  # of other sources than the library beside it
            os.remove(CALL_LIB)
        raise RuntimeError("g++ failed:\n" + res.stdout + res.stderr)
    os.replace(tmp, CALL_LIB)


def build(verbose: bool = False, extra=()) -> str:
    """Build libtq2.so (the library), libtq2probe.so (bench calibration) and
    _tq2call.so (the binding's native part).  The last one needs g++ and torch's
    headers; where it cannot be built the others are there, and enough."""
    _hipcc(SOURCES, LIB, verbose, extra)
    _hipcc([os.path.join(CSRC, "tq2_probes.hip")], PROBE_LIB, verbose, extra)
    _call(verbose)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
