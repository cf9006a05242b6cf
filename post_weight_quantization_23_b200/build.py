"""Build libgptq_b200.so in-tree with nvcc for sm_100a.

    python -m post_weight_quantization_23_b200.build [--verbose-ptxas]

Every .cu under csrc/ is compiled for sm_100a and linked into one shared
library next to this file.  csrc_py/ops.cpp, the Python entry of the adapter,
checkpoint and input-gradient operators, becomes the extension module _ops beside
it (g++ against torch's headers; it calls the library's C ABI).
"""
import argparse
import glob
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libgptq_b200.so")
OBJ = os.path.join(HERE, "_build")
OPS_SRC = os.path.join(HERE, "csrc_py", "ops.cpp")
OPS = os.path.join(HERE, "_ops" + sysconfig.get_config_var("EXT_SUFFIX"))

NVCC_FLAGS = [
    "-O3", "-std=c++17", "-lineinfo",
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-Xcompiler", "-fPIC,-O2,-fvisibility=hidden",
    "--expt-relaxed-constexpr",
]


def nvcc():
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def build(verbose_ptxas=False, force=False, jobs=None):
    os.makedirs(OBJ, exist_ok=True)
    srcs = sources()
    headers = glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(
        os.path.join(HERE, "..", "include", "*.h"))
    newest_hdr = max((os.path.getmtime(h) for h in headers), default=0)
    objs, procs = [], []
    for s in srcs:
        o = os.path.join(OBJ, os.path.basename(s)[:-3] + ".o")
        objs.append(o)
        if (not force and os.path.exists(o) and os.path.getmtime(o) >= os.path.getmtime(s)
                and os.path.getmtime(o) >= newest_hdr):
            continue
        cmd = [nvcc(), *NVCC_FLAGS, "-c", s, "-o", o]
        if verbose_ptxas:
            cmd += ["-Xptxas", "-v"]
        procs.append((s, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    failed = False
    for s, p in procs:
        out = p.communicate()[0].decode()
        if out.strip():
            print(f"--- {os.path.basename(s)}\n{out}", file=sys.stderr)
        if p.returncode != 0:
            failed = True
    if failed:
        raise RuntimeError("nvcc failed")
    if (force or procs or not os.path.exists(LIB)
            or os.path.getmtime(LIB) < max(os.path.getmtime(o) for o in objs)):
        cmd = [nvcc(), "-shared", "-gencode", "arch=compute_100a,code=sm_100a", *objs,
               "-o", LIB]
        subprocess.run(cmd, check=True)
    build_ops(force)
    return LIB


def build_ops(force=False):
    deps = [OPS_SRC, os.path.join(HERE, "..", "include", "gptq.h"), os.path.abspath(__file__)]
    if (not force and os.path.exists(OPS)
            and os.path.getmtime(OPS) >= max(os.path.getmtime(d) for d in deps)):
        return OPS
    import torch
    from torch.utils.cpp_extension import include_paths
    tlib = os.path.join(os.path.dirname(torch.__file__), "lib")
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    incs = [*include_paths(), os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *[f"-I{i}" for i in incs], OPS_SRC, "-o", OPS, "-L" + HERE, "-l:" + os.path.basename(LIB),
           "-Wl,-rpath,$ORIGIN", "-L" + tlib, "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]
    subprocess.run(cmd, check=True)
    return OPS


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--verbose-ptxas", action="store_true")
    ap.add_argument("--force", action="store_true")
    a = ap.parse_args()
    print(build(a.verbose_ptxas, a.force))
