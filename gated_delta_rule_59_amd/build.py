"""Build libkda (the HIP kernels and the C ABI) for gfx950 into this package directory.

    python -m gated_delta_rule_59_amd.build

hipcc compiles every source under csrc/ and links one shared library, libkda.so. Where torch is
installed, the host compiler builds csrc/torch/marshal.cpp, which marshals torch tensors into it, as
_marshal.so; the library needs neither.
"""
from __future__ import annotations

import glob
import importlib.util
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
LIB = os.path.join(HERE, "libkda.so")
ARCH = os.environ.get("KDA_OFFLOAD_ARCH", "gfx950")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

# -packed-fp32-ops: no packed fp32 VALU instructions are generated.
FLAGS = ["-O3", "-std=c++17", "-fPIC", f"--offload-arch={ARCH}", "-munsafe-fp-atomics",
         "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
         "-Wall", "-Wno-unused-function", "-I", INCLUDE]


MARSHAL = os.path.join(HERE, "_marshal.so")
CXX = os.environ.get("CXX", "g++")


def marshal_command(out: str):
    """The compiler's command line for the marshalling module; None without torch."""
    import sysconfig

    torch = importlib.util.find_spec("torch")
    if torch is None:
        return None
    root = os.path.dirname(torch.origin)
    dirs = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
            sysconfig.get_paths()["include"], "/opt/rocm/include"]
    lib = os.path.join(root, "lib")
    return [CXX, "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-D__HIP_PLATFORM_AMD__",
            "-DUSE_ROCM", "-Wall", "-Wno-attributes", "-I", INCLUDE, *[f"-isystem{d}" for d in dirs],
            os.path.join(CSRC, "torch", "marshal.cpp"), "-o", out, "-L", lib, "-ltorch_python", "-ltorch",
            "-ltorch_cpu", "-lc10", "-lc10_hip", f"-Wl,-rpath,{lib}"]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.hip")) + glob.glob(os.path.join(CSRC, "*.cpp")))


def build(verbose: bool = False, jobs: int = 8) -> str:
    objdir = os.path.join(HERE, "_build")
    os.makedirs(objdir, exist_ok=True)
    procs, objs = [], []
    marshal = MARSHAL + ".tmp%d" % os.getpid()
    marshal_cmd = marshal_command(marshal)
    marshal_proc = marshal_cmd and _start(marshal_cmd, verbose)
    for src in sources():
        obj = os.path.join(objdir, os.path.basename(src) + ".o")
        objs.append(obj)
        procs.append((src, _start([HIPCC, *FLAGS, "-x", "hip", "-c", src, "-o", obj], verbose)))
        if len(procs) >= jobs:
            _wait(procs.pop(0))
    for p in procs:
        _wait(p)
    tmp = LIB + ".tmp%d" % os.getpid()
    subprocess.run([HIPCC, f"--offload-arch={ARCH}", "-shared", "-o", tmp, *objs], check=True)
    os.replace(tmp, LIB)
    # after the library, which does not wait for it
    if marshal_proc:
        _wait(("csrc/torch/marshal.cpp", marshal_proc))
        os.replace(marshal, MARSHAL)
    else:
        sys.stderr.write("torch is not installed: _marshal.so is not built\n")
    return LIB


def _start(cmd, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    return subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)


def _wait(item):
    src, p = item
    out, _ = p.communicate()
    text = out.decode(errors="replace")
    lines = [l for l in text.splitlines() if "packed-fp32-ops" not in l and l.strip()]
    if p.returncode != 0:
        sys.stderr.write(text)
        raise RuntimeError(f"the compiler failed for {src}")
    if lines:
        sys.stderr.write("\n".join(lines) + "\n")


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
