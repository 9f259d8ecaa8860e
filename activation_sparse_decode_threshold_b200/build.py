"""Build libpi_ffn.so (sm_100a) in-tree with nvcc, and _pi_torch.so, the
binding's native part, with g++ against torch's headers.  The library needs
nothing of torch: where torch is not installed it is built alone.  The native
part is built again when torch or Python is another than it was built for.

Usage: python -m activation_sparse_decode_threshold_b200.build [--force] [--verbose]
"""
from __future__ import annotations

import argparse
import os
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor
from importlib import metadata

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
OUT = os.path.join(HERE, "libpi_ffn.so")
EXT = os.path.join(HERE, "_pi_torch.so")
OBJ = os.path.join(ROOT, "_build")
EXT_FOR = os.path.join(OBJ, "pi_torch.for")   # what the native part was built for
SOURCES = ["pi_decode_f16.cu", "pi_decode_bf16.cu", "pi_decode_i4f16.cu", "pi_decode_i4bf16.cu",
           "pi_decode_f16i8.cu", "pi_decode_bf16i8.cu", "pi_decode_i4i8.cu",
           "pi_decode_f32.cu", "pi_host.cu", "pi_decode.cu", "pi_repack.cu", "pi_prefill.cu", "pi_noalloc.cu", "pi_batch.cu",
           "pi_attn.cu", "pi_int4.cu", "pi_kv.cu", "pi_paged.cu"]
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-Xcompiler", "-fvisibility=hidden"]


def _nvcc() -> str:
    for c in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if c and (os.path.isabs(c) and os.path.exists(c) or not os.path.isabs(c)):
            return c
    return "nvcc"


def _deps_newer(target: str, sources: list[str]) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    for s in sources:
        if os.path.getmtime(s) > t:
            return True
    return False


def _ext_target() -> str | None:
    """What the native part's binary interface depends on (torch is not imported for it); None without torch."""
    try:
        return f"torch {metadata.version('torch')} python {sysconfig.get_config_var('SOABI')}\n"
    except metadata.PackageNotFoundError:
        return None


def _read(path: str) -> str:
    try:
        with open(path) as f:
            return f.read()
    except OSError:
        return ""


def _ext_cmd(src: str) -> list[str]:
    import torch
    base = os.path.dirname(torch.__file__)
    cuda = os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include")
    if not os.path.isdir(cuda):
        cuda = "/usr/local/cuda/include"
    inc = [sysconfig.get_paths()["include"], os.path.join(base, "include"),
           os.path.join(base, "include", "torch", "csrc", "api", "include"), cuda]
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            *[a for d in inc for a in ("-isystem", d)], src, "-o", EXT + ".tmp", "-L" + os.path.join(base, "lib"),
            "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10"]


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    os.makedirs(OBJ, exist_ok=True)
    headers = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".h", ".cuh"))]
    headers.append(os.path.join(ROOT, "include", "pi_ffn.h"))
    nvcc = _nvcc()
    objs = []
    jobs = []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(OBJ, src.replace(".cu", ".o"))
        objs.append(o)
        if force or _deps_newer(o, [s] + headers):
            cmd = [nvcc, *ARCH, *FLAGS, "-c", s, "-o", o]
            if ptxas_info:
                cmd += ["-Xptxas", "-v"]
            jobs.append(cmd)

    def run(cmd):
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0 or verbose or ptxas_info:
            sys.stderr.write(r.stdout + r.stderr)
        if r.returncode != 0:
            raise RuntimeError(f"{os.path.basename(cmd[0])} failed: {' '.join(cmd)}")

    def library():
        with ThreadPoolExecutor(max_workers=min(os.cpu_count() or 4, max(1, len(jobs)))) as ex:
            list(ex.map(run, jobs))
        if force or jobs or not os.path.exists(OUT):
            run([nvcc, *ARCH, "-shared", "-o", OUT + ".tmp", *objs, "-lcudart"])
            os.replace(OUT + ".tmp", OUT)

    def native_part():
        target = _ext_target()
        if target is None:
            sys.stderr.write("torch is not installed: the binding's native part is not built\n")
            return
        ext_src = os.path.join(CSRC, "pi_torch.cpp")
        if force or _read(EXT_FOR) != target or _deps_newer(EXT, [ext_src, os.path.join(ROOT, "include", "pi_ffn.h")]):
            run(_ext_cmd(ext_src))
            os.replace(EXT + ".tmp", EXT)
            with open(EXT_FOR, "w") as f:
                f.write(target)

    with ThreadPoolExecutor(max_workers=2) as ex:
        parts = [ex.submit(library), ex.submit(native_part)]
    for part in parts:   # the library first: it is there whatever becomes of the native part
        part.result()
    return OUT


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    ap.add_argument("--ptxas-info", action="store_true")
    a = ap.parse_args()
    print(build(a.force, a.verbose, a.ptxas_info))
