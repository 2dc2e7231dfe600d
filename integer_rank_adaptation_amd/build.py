"""Build libintlora.so (all HIP kernels + the C ABI) for gfx950, in-tree, and the Python module
_tensor_list (host code on torch's headers).

Each source is compiled to an object in parallel, then the objects are linked.
"""
from __future__ import annotations

import concurrent.futures
import os
import subprocess
import sys
import sysconfig
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libintlora.so")
TENSOR_LIST = os.path.join(HERE, "_tensor_list.so")
SOURCES = ["capi.hip", "merge.hip", "linear.hip", "ste.hip", "fplinear.hip", "gated.hip", "adapters.hip", "gradclip.hip"]

# -ffp-contract=off: no implicit multiply-add fusion (every fp32 step is the IEEE
# operation written); packed fp32 instructions are disabled for all device code.
FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
    "-ffp-contract=off", "-fno-fast-math",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-function",
]


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc"):
        if cand and os.path.exists(cand):
            return cand
    return "hipcc"


def tensor_list_cmd(out: str):
    import torch

    tdir = os.path.dirname(torch.__file__)
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            "-isystem", os.path.join(tdir, "include"),
            "-isystem", os.path.join(tdir, "include", "torch", "csrc", "api", "include"),
            "-isystem", sysconfig.get_paths()["include"], os.path.join(CSRC, "tensor_list.cpp"), "-o", out,
            "-L" + os.path.join(tdir, "lib"), "-ltorch_python", "-ltorch_cpu", "-ltorch", "-lc10"]


def _run(cmd):
    res = subprocess.run(cmd, capture_output=True, text=True)
    msgs = [l for l in (res.stdout + res.stderr).splitlines() if "packed-fp32-ops" not in l]
    return res.returncode, msgs


def build(verbose: bool = False) -> str:
    with tempfile.TemporaryDirectory(prefix="intlora_build_") as tmpd:
        jobs = []
        for src in SOURCES:
            obj = os.path.join(tmpd, src.replace(".hip", ".o"))
            jobs.append((obj, [hipcc(), *FLAGS, "-I", os.path.join(ROOT, "include"), "-c", os.path.join(CSRC, src),
                               "-o", obj]))
        ext = TENSOR_LIST + ".tmp%d" % os.getpid()
        jobs.append((ext, tensor_list_cmd(ext)))
        with concurrent.futures.ThreadPoolExecutor(max_workers=len(jobs)) as ex:
            results = list(ex.map(lambda j: _run(j[1]), jobs))
        for (obj, cmd), (rc, msgs) in zip(jobs, results):
            if verbose:
                print(" ".join(cmd))
            if rc != 0:
                sys.stderr.write("\n".join(msgs) + "\n")
                raise RuntimeError(os.path.basename(cmd[0]) + " failed compiling " + os.path.basename(obj))
            if verbose and msgs:
                print("\n".join(msgs))
        tmp = LIB + ".tmp%d" % os.getpid()
        link = [hipcc(), "--offload-arch=gfx950", "-shared", "-fPIC", "-o", tmp] + [o for o, _ in jobs if o != ext]
        rc, msgs = _run(link)
        if rc != 0:
            sys.stderr.write("\n".join(msgs) + "\n")
            raise RuntimeError("linking libintlora.so failed")
        os.replace(tmp, LIB)
        os.replace(ext, TENSOR_LIST)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
