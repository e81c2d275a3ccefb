"""Build libkvcodec.so and the modules around it in-tree with hipcc for gfx950 (no GPU needed)."""

import glob
import os
import subprocess
import sys
import sysconfig
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB_PATH = os.path.join(PKG, "libkvcodec.so")

# -ffp-contract=off: the codec's float steps are defined operation by
# operation; no multiply-add may be fused behind our back.
# -packed-fp32-ops off: no packed fp32 instructions are generated.
HIPCC_FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
    "-ffp-contract=off", "-fno-fast-math",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-function",
    "-I", INCLUDE, "-I", CSRC,
]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.hip"))) + sorted(glob.glob(os.path.join(CSRC, "*.cpp")))


# streaming bandwidth probes of the benchmark (not part of the codec ABI)
PROBE_SRC = os.path.join(PKG, "probe", "stream_probe.hip")
PROBE_LIB = os.path.join(PKG, "libkvprobe.so")


def _hipcc(srcs, out, verbose, extra=(), cwd=None):
    hipcc = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
    tmp = out + ".tmp"
    cmd = [hipcc] + HIPCC_FLAGS + ([] if "-c" in extra else ["-shared"]) + list(extra) + list(srcs) + ["-o", tmp]
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True, cwd=cwd)
    errs = "\n".join(l for l in res.stderr.splitlines()
                     if "packed-fp32-ops" not in l and l.strip())
    if res.returncode != 0:
        sys.stderr.write(errs + "\n")
        raise RuntimeError(f"hipcc failed ({res.returncode})")
    if verbose and errs:
        print(errs)
    os.replace(os.path.join(cwd or "", tmp), os.path.join(cwd or "", out))
    return out


# Python module of the operators of kvattend.h: tensors in, C calls out
BINDING_SRC = os.path.join(PKG, "binding", "kvattend_py.cpp")
BINDING_LIB = os.path.join(PKG, "_kvattend.so")


def _binding(verbose):
    try:
        import torch
    except ImportError as e:
        print(f"{os.path.basename(BINDING_LIB)} left out, it needs torch: {e}", flush=True)
        return
    base = os.path.dirname(torch.__file__)
    _hipcc([BINDING_SRC], BINDING_LIB, verbose,
           ["-isystem", os.path.join(base, "include"), "-I", sysconfig.get_paths()["include"],
            "-L" + os.path.join(base, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10"])


def build(verbose=False, extra=()):
    """libkvcodec.so (the codec), libkvprobe.so (the benchmark's probes) and _kvattend.so (a binding, which
    alone needs torch), every source compiled anew, a few at a time. The library is linked whatever becomes of the
    other two."""
    with tempfile.TemporaryDirectory() as tmp, ThreadPoolExecutor(6) as pool:
        # named without the folder, whose path would get into the library: the same sources give the same bytes
        compiled = [os.path.basename(s) + ".o" for s in sources()]
        # the slowest first
        order = sorted(zip(sources(), compiled), key=lambda x: -os.path.getsize(x[0]))
        others = [pool.submit(_binding, verbose)]
        objects = [pool.submit(_hipcc, [s], o, verbose, ["-c"] + list(extra), tmp) for s, o in order]
        others.append(pool.submit(_hipcc, [PROBE_SRC], PROBE_LIB, verbose))
        for j in objects:
            j.result()
        _hipcc(compiled, LIB_PATH, verbose, extra, tmp)
        for j in others:
            j.result()
    return LIB_PATH


if __name__ == "__main__":
    print(build(verbose=True))
