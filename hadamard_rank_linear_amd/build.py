"""Build the gfx950 HIP library libhlq.so and the Python module _hlq_torch.so
in-tree with hipcc and the host's C++ compiler.

The library needs hipcc alone; the module, which the training step's operators
are called through from Python, also needs torch.  Each source compiles to an
object of its own (in parallel), then one link."""
from __future__ import annotations

import concurrent.futures
import importlib.util
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
OBJ = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libhlq.so")
EXT = os.path.join(HERE, "_hlq_torch.so")
# (source, object, extra flags): the transform kernels build once per block size
SOURCES = [("hlq_tr.hip", f"hlq_tr{n}", [f"-DHLQ_TR_N={n}"]) for n in (16, 32, 64, 128)] + [
    ("hlq_gemm.hip", "hlq_gemm", []), ("hlq_lqs.hip", "hlq_lqs", []),
    ("hlq_acbp.hip", "hlq_acbp", []), ("hlq_noalloc.hip", "hlq_noalloc", []),
    ("hlq_ablation.hip", "hlq_ablation", []),
    ("hlq_norm.hip", "hlq_norm", []), ("hlq_logprob.hip", "hlq_logprob", []),
    ("hlq_clip.hip", "hlq_clip", []),
    ("hlq_api.cpp", "hlq_api", []), ("hlq_train_api.cpp", "hlq_train_api", [])]

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
CXX = os.environ.get("CXX", "g++")

# Numerics flags: no FMA contraction (the transforms must round every add),
# IEEE division, denormals kept; packed fp32 instructions disabled.
FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
    "-ffp-contract=off", "-fhip-fp32-correctly-rounded-divide-sqrt",
    "-fno-gpu-flush-denormals-to-zero",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wno-unused-command-line-argument",
]


def _run(cmd, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError("build failed: " + " ".join(cmd[-3:]))


def _ext_command(out):
    """The binding's native half: host code against torch's C++ API."""
    import torch
    home = os.path.dirname(os.path.abspath(torch.__file__))
    inc = [os.path.join(home, "include"), os.path.join(home, "include/torch/csrc/api/include"),
           "/opt/rocm/include", sysconfig.get_paths()["include"]]
    lib = os.path.join(home, "lib")
    return [CXX, "-O2", "-std=c++17", "-fPIC", "-shared", "-D__HIP_PLATFORM_AMD__=1",
            "-DUSE_ROCM=1", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            *[f for i in inc for f in ("-isystem", i)], "-o", out,
            os.path.join(CSRC, "hlq_torch.cpp"), "-L", lib, "-ltorch_python", "-ltorch",
            "-ltorch_cpu", "-ltorch_hip", "-lc10", "-lc10_hip", "-ldl"]


def build(verbose: bool = False) -> str:
    os.makedirs(OBJ, exist_ok=True)
    inc = ["-I", os.path.join(ROOT, "include")]
    objs, cmds = [], []
    for src, name, extra in SOURCES:
        o = os.path.join(OBJ, name + ".o")
        objs.append(o)
        cmds.append([HIPCC, *FLAGS, *extra, *inc, "-c", "-o", o, os.path.join(CSRC, src)])
    ext = None
    with concurrent.futures.ThreadPoolExecutor(max_workers=len(cmds) + 1) as ex:
        if importlib.util.find_spec("torch") is not None:
            ext = ex.submit(lambda: _run(_ext_command(EXT + ".tmp"), verbose))
        for f in [ex.submit(_run, c, verbose) for c in cmds]:
            f.result()
    tmp = LIB + ".tmp"
    _run([HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", "-o", tmp, *objs], verbose)
    os.replace(tmp, LIB)
    if ext is None:
        sys.stderr.write("torch is not installed: built without _hlq_torch.so, the Python "
                         "binding of the training step's operators\n")
    else:
        ext.result()
        os.replace(EXT + ".tmp", EXT)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
