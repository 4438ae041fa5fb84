"""Build libsgmv.so (the C-ABI library) in-tree with hipcc for gfx950.

Usage: ``python segmented_gather_gemm_sgmv_amd/build.py``.

The kernel file is compiled once per rank (-DSGMV_RANK=8, 16, 32, 64) and
once more for the rank dispatch and helper kernels; these objects, the paged
cache's and the C ABI's compile in parallel, then link into one shared library,
against which the Python extension that marshals the paged-cache calls is
linked.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import tempfile
from pathlib import Path
from typing import Optional

PKG = Path(__file__).resolve().parent
ROOT = PKG.parent
CSRC = PKG / "csrc"        # SGMV
CSRC_KV = PKG / "csrc_kv"  # the paged key/value cache
INCLUDE = ROOT / "include"
LIBRARY = PKG / "libsgmv.so"
BINDING = PKG / "_kv_binding.so"  # the paged-cache calls' argument marshalling (g++, torch's headers)

KERNELS = CSRC / "sgmv_kernels.hip"
API = CSRC / "sgmv_api.cpp"
HOST = CSRC / "sgmv_host.cpp"  # host-only entry points (no HIP): also built alone with the sanitizers
KV = [CSRC_KV / n for n in ("kv_api.cpp", "kv_tables.hip", "kv_rope.hip", "kv_attention.hip")]
SOURCES = [KERNELS, API, HOST, *KV]
RANKS = (8, 16, 32, 64)
ARCH = "gfx950"

# Packed fp32 instructions are disabled: hipcc would otherwise form them from
# ordinary float code. The host pass does not know the feature and says so.
FLAGS = ["-O3", "-std=c++17", "-fPIC", f"--offload-arch={ARCH}",
         "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
         "-Wall", "-Wno-unused-function"]
NOISE = "-packed-fp32-ops' is not a recognized feature"


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), shutil.which("hipcc"), "/opt/rocm/bin/hipcc"):
        if cand and Path(cand).exists():
            return cand
    raise FileNotFoundError("hipcc not found (ROCm is required to build libsgmv.so)")


def _messages(res) -> list:
    return [ln for ln in (res.stdout + res.stderr).splitlines() if NOISE not in ln]


def _run(cmd, what: str, verbose: bool) -> None:
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"{what} failed:\n" + "\n".join(_messages(res)))


def build_binding(library: Path = LIBRARY, verbose: bool = False) -> Optional[Path]:
    """Compile the Python extension that marshals the paged-cache calls (no
    device code), linked against `library` next to it. Without g++ or torch
    (which the library itself does not need) it is left out: the package's
    other calls work, those of the paged cache raise."""
    import importlib.util
    import sysconfig

    missing = [n for n, there in (("g++", shutil.which("g++")), ("torch", importlib.util.find_spec("torch"))) if not there]
    if missing:
        BINDING.unlink(missing_ok=True)  # one of an earlier build would not go with this library
        print(f"{BINDING.name} is left out: no {' and no '.join(missing)}", file=sys.stderr, flush=True)
        return None
    import torch
    from torch.utils.cpp_extension import include_paths, library_paths
    inc = [f"-I{p}" for p in [INCLUDE, sysconfig.get_paths()["include"]] + list(include_paths())]
    libs = [f"-L{p}" for p in [library.parent] + list(library_paths())]
    tmp_out = BINDING.with_suffix(".so.tmp")
    _run(["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
          f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *inc, str(CSRC_KV / "kv_binding.cpp"),
          "-o", str(tmp_out), *libs, f"-l:{library.name}", "-lc10", "-ltorch_cpu", "-ltorch_python",
          "-Wl,-rpath,$ORIGIN"], "g++", verbose)
    os.replace(tmp_out, BINDING)
    return BINDING


def build(output: Path = LIBRARY, extra_flags=(), verbose: bool = False, jobs: int = 0) -> Path:
    """Compile every HIP/C++ source into one shared library (always rebuilds)."""
    cc = hipcc()
    inc = [f"-I{INCLUDE}", f"-I{CSRC}"]
    jobs = jobs or min(8, os.cpu_count() or 1)
    with tempfile.TemporaryDirectory(prefix="sgmv_build_") as tmp:
        units = [(KERNELS, [f"-DSGMV_RANK={r}"], Path(tmp) / f"kernels_r{r}.o") for r in RANKS]
        units += [(KERNELS, [], Path(tmp) / "kernels_dispatch.o"), (API, [], Path(tmp) / "api.o"),
                  (HOST, [], Path(tmp) / "host.o")]
        units += [(src, [], Path(tmp) / f"{src.stem}.o") for src in KV]
        pending = list(units)
        running = []
        failed = []
        while pending or running:
            while pending and len(running) < jobs:
                src, defs, obj = pending.pop(0)
                cmd = [cc, *FLAGS, *extra_flags, *defs, *inc, "-c", str(src), "-o", str(obj)]
                if verbose:
                    print(" ".join(cmd), flush=True)
                running.append((cmd, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.PIPE,
                                                      text=True)))
            cmd, proc = running.pop(0)
            out, err = proc.communicate()
            res = subprocess.CompletedProcess(cmd, proc.returncode, out, err)
            msgs = _messages(res)
            if proc.returncode != 0:
                failed.append(" ".join(cmd) + "\n" + "\n".join(msgs))
            elif verbose and msgs:
                print("\n".join(msgs))
        if failed:
            raise RuntimeError("hipcc failed:\n" + "\n\n".join(failed))
        tmp_out = output.with_suffix(".so.tmp")
        cmd = [cc, "-shared", "-fPIC", f"--offload-arch={ARCH}", *extra_flags,
               *[str(u[2]) for u in units], "-o", str(tmp_out)]
        _run(cmd, "hipcc link", verbose)
    os.replace(tmp_out, output)
    if output == LIBRARY:
        build_binding(output, verbose)
    return output


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
