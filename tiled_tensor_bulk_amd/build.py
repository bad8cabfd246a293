"""Build libtmap.so and libtkv.so (gfx950) in-tree with hipcc, and _tkv.so with g++.

    python -m tiled_tensor_bulk_amd.build [--jobs N]

Each translation unit is compiled in parallel into tiled_tensor_bulk_amd/_build
and linked into tiled_tensor_bulk_amd/libtmap.so (the tile copies) or
libtkv.so (the 4-bit cache and its operators); _tkv.so is libtkv's calls on torch
tensors.  Cross-compiles without a GPU.
"""
from __future__ import annotations

import argparse
import os
import shutil
import subprocess
import sys
import time

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libtmap.so")
TKV_LIB = os.path.join(PKG, "libtkv.so")
TORCH_LIB = os.path.join(PKG, "_tkv.so")
ROOT = os.path.dirname(PKG)

SOURCES = (["tmap_host.cpp"] + [f"tmap_{m}_r{r}.hip" for m in ("load", "store", "roundtrip") for r in (2, 5)]
           + [f"tmap_band_{m}.hip" for m in ("load", "store", "roundtrip")]
           + [f"tmap_corner_{m}.hip" for m in ("load", "store", "roundtrip")]
           + [f"tmap_corner4_{m}.hip" for m in ("load", "store", "roundtrip")] + ["tmap_noalloc.hip"])
TKV_SOURCES = (["tkv_host.cpp"] + [f"tkv_attend_d{d}.hip" for d in (256, 128, 96, 64)]
               + ["tkv_combine.hip", "tkv_evict.hip", "tkv_move.hip"])
ARCH = "gfx950"


def hipcc() -> str:
    for p in ("/opt/rocm/bin/hipcc", shutil.which("hipcc") or ""):
        if p and os.path.exists(p):
            return p
    raise RuntimeError("hipcc not found")


def common_flags():
    return [f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC", "-Wall",
            # packed fp32 instructions are kept out of every device build
            "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
            "-I", os.path.join(ROOT, "include")]


def torch_command(out: str):
    """g++'s command for _tkv.so: host code only."""
    import sysconfig

    import torch

    at = os.path.dirname(torch.__file__)
    rocm = os.path.dirname(os.path.dirname(os.path.realpath(hipcc())))
    return (["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-Wall",
             "-D__HIP_PLATFORM_AMD__", "-DUSE_ROCM", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
             f"-I{at}/include", f"-I{at}/include/torch/csrc/api/include", f"-I{rocm}/include",
             f"-I{sysconfig.get_paths()['include']}", os.path.join(CSRC, "tkv_torch.cpp"), "-o", out, f"-L{PKG}",
             "-l:libtkv.so", f"-L{at}/lib"]
            + [f"-l{n}" for n in ("torch_python", "torch", "torch_cpu", "torch_hip", "c10", "c10_hip")]
            + ["-Wl,-rpath,$ORIGIN"])


def build(jobs: int = 7, verbose: bool = False, incremental: bool = False) -> str:
    """Compile every translation unit (or, with incremental=True, only those
    older than a source or header) and link the libraries."""
    os.makedirs(BUILD, exist_ok=True)
    cc = hipcc()
    procs = []
    t0 = time.time()
    newest_hdr = max(os.path.getmtime(os.path.join(d, f)) for d in (CSRC, os.path.join(ROOT, "include"))
                     for f in os.listdir(d) if f.endswith(".h"))
    pending = []
    for src in TKV_SOURCES + SOURCES:
        obj = os.path.join(BUILD, src + ".o")
        if (incremental and os.path.exists(obj)
                and os.path.getmtime(obj) > max(newest_hdr, os.path.getmtime(os.path.join(CSRC, src)))):
            continue
        pending.append(src)
    running = []
    while pending or running:
        while pending and len(running) < max(1, jobs):
            src = pending.pop(0)
            obj = os.path.join(BUILD, src + ".o")
            cmd = [cc, *common_flags(), "-c", os.path.join(CSRC, src), "-o", obj]
            if verbose:
                print(" ".join(cmd), flush=True)
            running.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
        src, p = running.pop(0)
        out, _ = p.communicate()
        text = out.decode(errors="replace")
        # hipcc's host pass does not know the packed-fp32 feature name: harmless
        lines = [l for l in text.splitlines() if "packed-fp32-ops" not in l]
        if p.returncode != 0:
            sys.stderr.write("\n".join(lines) + "\n")
            raise RuntimeError(f"compiling {src} failed")
        if verbose and lines:
            print("\n".join(lines))
    for lib, sources in ((LIB, SOURCES), (TKV_LIB, TKV_SOURCES)):
        tmp = lib + ".tmp"
        objs = [os.path.join(BUILD, src + ".o") for src in sources]
        subprocess.check_call([cc, f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp, *objs])
        os.replace(tmp, lib)
    subprocess.check_call(torch_command(TORCH_LIB + ".tmp"))
    os.replace(TORCH_LIB + ".tmp", TORCH_LIB)
    if verbose:
        print(f"built {LIB}, {TKV_LIB} and {TORCH_LIB} in {time.time() - t0:.1f}s", flush=True)
    return LIB


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--jobs", type=int, default=7)
    ap.add_argument("-v", "--verbose", action="store_true")
    ap.add_argument("--incremental", action="store_true", help="recompile only out-of-date units")
    a = ap.parse_args()
    build(jobs=a.jobs, verbose=a.verbose, incremental=a.incremental)


if __name__ == "__main__":
    main()
