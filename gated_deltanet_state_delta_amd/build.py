"""Build libgdn.so (HIP, gfx950) and the binding's _calls.so in-tree.

Every translation unit under csrc/ is compiled with hipcc for gfx950 into
_build/, in parallel, and linked into gated_deltanet_state_delta_amd/libgdn.so.
Packed-fp32 VALU instructions are disabled for all device code.  Beside it,
binding/calls.cpp (host code only) becomes the CPython module _calls; where
that fails (no g++, no headers of torch or Python) there is only the library.

    python -m gated_deltanet_state_delta_amd.build [--jobs N]
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import hashlib
import os
import re
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build", "libgdn")
LIB = os.path.join(PKG, "libgdn.so")
CALLS = os.path.join(PKG, "_calls.so")
ARCH = "gfx950"

DEVICE_FLAGS = ["-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops"]
# Per-file device flags.  The pair-role prefill runs one wave per SIMD, so its
# speed depends on latency hiding inside each wave: its MFMA accumulators stay
# in VGPRs (its state is scaled and converted by VALU code every chunk, and
# accumulators in AGPRs would cost a copy each way), and the machine
# scheduler that groups memory operations into clauses is used, with the
# target's own register-pressure trackers.  On B4 x S4096: about 18% faster
# than the default strategy; 1% faster than the iterative ILP strategy, and
# the trackers 1.2% more (outputs bit-identical); the plain max-ILP strategy
# is 6% slower.
# The decode kernel at value width 128 (the single-step pool decode of
# Hv32 x 128 x 128 states) takes the memory-clause scheduler with the
# register-pressure trackers: 168.1-169.4 -> 165.9-167.0 us median over
# three alternating same-box runs (the iterative ILP scheduler used before
# had been 2.2% ahead of the default; the memory-clause scheduler without
# the trackers is slower); a scheduler flag on the multi-token width-64
# form made it 2.5% slower, so that one keeps the default.
FILE_FLAGS = {"gdn_prefill_pair.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form",
                                     "-mllvm", "-amdgpu-sched-strategy=max-memory-clause",
                                     "-mllvm", "-amdgpu-use-amdgpu-trackers"],
              "gdn_decode_dv128.hip": ["-mllvm", "-amdgpu-sched-strategy=max-memory-clause",
                                       "-mllvm", "-amdgpu-use-amdgpu-trackers"]}
COMMON = ["--offload-arch=" + ARCH, "-O3", "-std=c++17", "-fPIC", "-Wall",
          "-Wno-unused-function", "-Wno-unused-variable", "-I", os.path.join(ROOT, "include")]


def hipcc() -> str:
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    cand = os.path.join(rocm, "bin", "hipcc")
    return cand if os.path.exists(cand) else (shutil.which("hipcc") or "hipcc")


def header_digest() -> str:
    """What gdn_header_digest returns: include/libgdn.h without comments and blanks, digested."""
    with open(os.path.join(ROOT, "include", "libgdn.h")) as f:
        text = re.sub(r"/\*.*?\*/|//[^\n]*", " ", f.read(), flags=re.S)
    return hashlib.sha256(" ".join(text.split()).encode()).hexdigest()[:16]


def _digest_flag() -> str:
    return '-DGDN_HEADER_DIGEST="%s"' % header_digest()


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC)
                  if f.endswith(".hip") or f.endswith(".cpp"))


def _compile(src: str) -> str:
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    extra = FILE_FLAGS.get(os.path.basename(src), [])
    cmd = [hipcc()] + COMMON + DEVICE_FLAGS + extra + ["-c", src, "-o", obj]
    if src.endswith(".cpp"):
        cmd = [hipcc()] + COMMON + [_digest_flag(), "-x", "hip"] + DEVICE_FLAGS + ["-c", src, "-o", obj]
    res = subprocess.run(cmd, capture_output=True, text=True)
    noise = "is not a recognized feature for this target"
    err = "\n".join(l for l in res.stderr.splitlines() if noise not in l)
    if res.returncode != 0:
        raise RuntimeError("hipcc failed for %s:\n%s" % (src, err))
    if err.strip():
        sys.stderr.write(err + "\n")
    return obj


def _build_calls(tmp: str) -> None:
    import sysconfig

    import torch
    from torch.utils import cpp_extension
    # NDEBUG: without it a header adds a thread-local variable to the module, and
    # with one loaded late every access to other libraries' ones goes a slow way
    # (pages_extend 15.5 -> 17.9 us on the host).
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-DNDEBUG", "-D__HIP_PLATFORM_AMD__=1",
           _digest_flag(), "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch._C._GLIBCXX_USE_CXX11_ABI]
    for d in cpp_extension.include_paths() + [sysconfig.get_paths()["include"]]:
        cmd += ["-isystem", d]
    # torch's libraries are loaded before the module, so it carries no path to them
    cmd += [os.path.join(PKG, "binding", "calls.cpp"), "-L" + os.path.join(os.path.dirname(torch.__file__), "lib"),
            "-ltorch_python", "-ltorch_cpu", "-lc10", "-o", tmp]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(res.stderr)
    if res.stderr.strip():
        sys.stderr.write(res.stderr)


def _link(objs, tmp: str) -> None:
    cmd = [hipcc(), "--offload-arch=" + ARCH, "-shared", "-fPIC", "-o", tmp] + objs
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("link failed:\n" + res.stderr)


def build(jobs: int | None = None) -> str:
    os.makedirs(BUILD, exist_ok=True)
    srcs = sources()
    jobs = jobs or min(len(srcs), max(1, min(16, os.cpu_count() or 1)))
    lib, calls = (path + ".tmp%d" % os.getpid() for path in (LIB, CALLS))
    try:
        with cf.ThreadPoolExecutor(max_workers=jobs) as ex:
            module = ex.submit(_build_calls, calls)
            objs = list(ex.map(_compile, srcs))
        _link(objs, lib)
        # both together: they belong to one header
        os.replace(lib, LIB)
        if module.exception() is None:
            os.replace(calls, CALLS)
        else:  # the library needs neither g++ nor torch, and works without the module
            sys.stderr.write("binding/calls.cpp was not built, calls go the general way in Python:\n%s\n" % module.exception())
            if os.path.exists(CALLS):
                os.remove(CALLS)
    finally:
        for tmp in (lib, calls):
            if os.path.exists(tmp):
                os.remove(tmp)
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--jobs", type=int, default=None)
    print(build(ap.parse_args().jobs))
