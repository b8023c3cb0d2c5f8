"""Build libkda.so (HIP, gfx950) in-tree.

Every .hip translation unit is compiled in parallel with hipcc for gfx950, then
linked with the host API into ``libkda.so`` next to this file.  Packed fp32
arithmetic is disabled for all device code (``-packed-fp32-ops`` off).  The token
mixers' binding (``_mixers.so``, host code against torch's headers) is built beside it.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
ROOT = os.path.dirname(HERE)
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libkda.so")
PEAKS_LIB = os.path.join(HERE, "libkda_peaks.so")
BINDING = os.path.join(HERE, "_mixers.so")
BUILD_DIR = os.path.join(ROOT, "_build")

ARCH = os.environ.get("KDA_OFFLOAD_ARCH", "gfx950")
COMMON = ["-O3", "-std=c++17", "-fPIC", f"-I{INCLUDE}", f"-I{CSRC}", "-Wall",
          "-Wno-unused-function"]
DEVICE = [f"--offload-arch={ARCH}", "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
          "-munsafe-fp-atomics"]


def _hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found")


def _compile(src: str) -> str:
    obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
    cmd = [_hipcc(), *COMMON]
    if src.endswith(".hip"):
        cmd += ["-x", "hip", *DEVICE]
    cmd += ["-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"compile failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    return obj


def _link(objs, out):
    tmp = out + ".tmp"
    cmd = [_hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, out)


def build_binding() -> str | None:
    """_mixers.so from csrc/binding/: a Python extension that links to torch, which is imported
    before it, and is handed libkda's entry points at run time.  Without torch there is nothing to
    build it against (None): the C library does not need it."""
    try:
        import torch
    except ImportError:
        return None
    top = os.path.dirname(torch.__file__)
    tmp = BINDING + ".tmp"
    cmd = ["g++", "-std=c++17", "-O2", "-fPIC", "-shared", "-Wall", "-D__HIP_PLATFORM_AMD__", "-DUSE_ROCM",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f"-I{INCLUDE}",
           "-isystem", sysconfig.get_paths()["include"], "-isystem", os.path.join(top, "include"),
           "-isystem", os.path.join(top, "include", "torch", "csrc", "api", "include"), "-isystem", "/opt/rocm/include",
           os.path.join(CSRC, "binding", "mixers_binding.cpp"), "-o", tmp, "-L" + os.path.join(top, "lib"),
           "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_hip"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"compile failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING)
    return BINDING


def build(verbose: bool = False) -> str:
    """libkda.so from csrc/*.hip and csrc/*.cpp, the token mixers' binding, and the benchmark's
    bandwidth probes (libkda_peaks.so, from csrc/bench/) beside it."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    srcs = sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC)
                  if f.endswith(".hip") or f.endswith(".cpp"))
    probe_srcs = sorted(os.path.join(CSRC, "bench", f) for f in os.listdir(os.path.join(CSRC, "bench"))
                        if f.endswith(".hip"))
    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs) + len(probe_srcs))) as ex:
        binding = ex.submit(build_binding)
        objs = list(ex.map(_compile, srcs))
        probe_objs = list(ex.map(_compile, probe_srcs))
        binding = binding.result()
    _link(objs, LIB)
    _link(probe_objs, PEAKS_LIB)
    if verbose:
        print(f"built {LIB}, {binding or 'no binding (torch is not installed)'} and {PEAKS_LIB}")
    return LIB


def build_sanitized(out_dir: str | None = None) -> str:
    """libkda.so with its host code (argument validation, planning, launch set-up in
    csrc/*.cpp) built by g++ under AddressSanitizer and UndefinedBehaviorSanitizer, linked with
    the device objects of the regular build (run build() first).  Load it with gcc's libasan and
    libubsan preloaded; the device code is unchanged."""
    out_dir = out_dir or os.path.join(BUILD_DIR, "asan")
    os.makedirs(out_dir, exist_ok=True)
    probes = {os.path.basename(f) + ".o" for f in os.listdir(os.path.join(CSRC, "bench"))}
    objs = sorted(os.path.join(BUILD_DIR, f) for f in os.listdir(BUILD_DIR)
                  if f.endswith(".hip.o") and f not in probes)
    if not objs:
        raise RuntimeError("no device objects in _build: run build() first")
    san = ["-fsanitize=address,undefined", "-fno-omit-frame-pointer"]
    host_objs = []
    for src in sorted(f for f in os.listdir(CSRC) if f.endswith(".cpp")):
        obj = os.path.join(out_dir, src[:-len(".cpp")] + ".o")
        cmd = ["g++", "-std=c++17", "-O1", "-g", "-fPIC", *san, "-D__HIP_PLATFORM_AMD__",
               "-I/opt/rocm/include", f"-I{INCLUDE}", f"-I{CSRC}", "-c",
               os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"compile failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
        host_objs.append(obj)
    lib = os.path.join(out_dir, "libkda.so")
    cmd = ["g++", "-shared", *san, "-o", lib, *host_objs, *objs, "-L/opt/rocm/lib", "-lamdhip64",
           "-Wl,-rpath,/opt/rocm/lib"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    return lib


if __name__ == "__main__":
    if sys.argv[1:] == ["sanitized"]:
        print(build_sanitized())
    else:
        build(verbose=True)
    sys.exit(0)
