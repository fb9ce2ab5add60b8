"""Build the sm_100a shared library libmoe_b200.so in-tree with nvcc.

    python -m mixture_experts_layer_46_b200.build [--force] [--verbose]

Every .cu under csrc/ is compiled for sm_100a (-gencode arch=compute_100a,
code=sm_100a, -lineinfo) into one object each, in parallel, then linked into
mixture_experts_layer_46_b200/libmoe_b200.so with the CUDA runtime linked
statically; csrc/moe_torch.cpp becomes the Python module _moe_torch.so beside it.  Objects go to _build/ (git-ignored).

The tuned kernel-configuration table (configs/b200_tuned.csv, written by
tune.py) is turned into a C array, _build/moe_config_table.inc, that the
library compiles in as its built-in table.
"""

from __future__ import annotations

import argparse
import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libmoe_b200.so")
BINDING = os.path.join(PKG, "_moe_torch.so")
BINDING_FOR = os.path.join(BUILD, "moe_torch.built_for")  # the torch and Python whose headers it was compiled with
INCLUDE = os.path.join(ROOT, "include")

CONFIG_CSV = os.path.join(PKG, "configs", "b200_tuned.csv")
CONFIG_INC = os.path.join(BUILD, "moe_config_table.inc")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-I", INCLUDE, "-I", CSRC, "-I", BUILD]

# columns of the tuning table that select the kernels (the rest are the tuner's notes)
CONFIG_COLUMNS = ("wdtype", "H", "I", "E", "k", "t_lo", "t_hi", "tile", "pair", "g1_256",
                  "g2_single", "tiny", "prefetch", "fused", "split", "g1_il")


def read_config_csv(path: str = CONFIG_CSV):
    """Rows of the tuning table as dicts of ints (wdtype: 0 = bf16, 4 = MXFP4)."""
    import csv

    rows = []
    if not os.path.exists(path):
        return rows
    with open(path, newline="") as f:
        for r in csv.DictReader(line for line in f if not line.startswith("#")):
            row = {}
            for c in CONFIG_COLUMNS:
                v = (r.get(c) or "0").strip()
                row[c] = {"bf16": 0, "mxfp4": 4}[v] if c == "wdtype" else int(v)
            rows.append(row)
    return rows


def write_config_inc() -> None:
    """The C array of the built-in configuration table (rewritten only when it changes)."""
    rows = read_config_csv()
    lines = ["// generated by build.py from configs/b200_tuned.csv: do not edit",
             f"constexpr int kNumBuiltinConfigs = {len(rows)};",
             "const moe_config_t kBuiltinConfigs[] = {"]
    for r in rows:
        lines.append("    {" + ", ".join(str(r[c]) for c in CONFIG_COLUMNS) + "},")
    if not rows:
        lines.append("    {0, 0, 0, 0, 0, 0, -1, 32, 0, 0, 0, 0, 0, 0, 0, 0},  // placeholder, never matched")
    lines.append("};")
    text = "\n".join(lines) + "\n"
    if os.path.exists(CONFIG_INC):
        with open(CONFIG_INC) as f:
            if f.read() == text:
                return
    with open(CONFIG_INC, "w") as f:
        f.write(text)


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA library cannot be built")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _headers():
    return sorted(glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) +
                  glob.glob(os.path.join(INCLUDE, "*.h")) + [CONFIG_INC])


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False, ptxas_verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    write_config_inc()
    cc = nvcc()
    headers = _headers()
    jobs = []
    objs = []
    for src in _sources():
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        if force or _stale(obj, [src] + headers):
            cmd = [cc, *ARCH, *FLAGS, "-c", src, "-o", obj]
            if ptxas_verbose:
                cmd += ["-Xptxas", "-v"]
            jobs.append(cmd)

    def run(cmd):
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        return cmd, r

    with cf.ThreadPoolExecutor(max_workers=min(8, max(1, len(jobs)))) as ex:
        for cmd, r in ex.map(run, jobs):
            if r.returncode != 0 or verbose or ptxas_verbose:
                sys.stderr.write(r.stdout + r.stderr)
            if r.returncode != 0:
                raise RuntimeError("nvcc failed: " + " ".join(cmd))
    if force or jobs or _stale(LIB, objs):
        # export only the C ABI (moe_*); the static CUDA runtime stays private
        vmap = os.path.join(BUILD, "exports.map")
        with open(vmap, "w") as f:
            f.write("{ global: moe_*; local: *; };\n")
        cmd = [cc, *ARCH, "-shared", "-cudart", "static", "-o", LIB, *objs, "-ldl", "-lrt",
               "-lpthread", "-Xlinker", "--version-script=" + vmap]
        if verbose:
            print(" ".join(cmd), flush=True)
        subprocess.run(cmd, check=True)
    build_binding(force, verbose)
    return LIB


def build_binding(force: bool = False, verbose: bool = False) -> str:
    """The Python module over the operators around the forward (csrc/moe_torch.cpp)."""
    import sysconfig

    import torch

    src = os.path.join(CSRC, "moe_torch.cpp")
    built_for = f"torch {torch.__version__}, {sys.implementation.cache_tag}"
    same = False
    if os.path.exists(BINDING_FOR):
        with open(BINDING_FOR) as f:
            same = f.read() == built_for
    if same and not (force or _stale(BINDING, [src, os.path.join(INCLUDE, "moe.h")])):
        return BINDING
    base = os.path.dirname(torch.__file__)
    inc = [os.path.join(base, "include"), os.path.join(base, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include"), INCLUDE]
    lib = os.path.join(base, "lib")
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
    for d in inc:
        cmd += ["-isystem" if d != INCLUDE else "-I", d]
    cmd += [src, "-o", BINDING, "-L" + lib, "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python", "-L" + PKG,
            "-l:" + os.path.basename(LIB), "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + lib]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    with open(BINDING_FOR, "w") as f:
        f.write(built_for)
    return BINDING


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    ap.add_argument("--ptxas-verbose", action="store_true")
    a = ap.parse_args()
    print(build(force=a.force, verbose=a.verbose, ptxas_verbose=a.ptxas_verbose))
