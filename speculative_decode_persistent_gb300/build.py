"""In-tree build of libmk.so (nvcc, sm_103a only) and of the Python side of its
operators, _bind (g++, against torch's headers).

Each translation unit compiles in its own process, in parallel, then one
link step produces speculative_decode_persistent_gb300/libmk.so.
"""
from __future__ import annotations

import importlib.metadata
import importlib.util
import os
import platform
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(HERE, "_build")
SO = os.path.join(HERE, "libmk.so")
SOURCES = ["mk_kernel.cu", "mk_api.cu", "mk_pack.cu", "ops/kv_rows.cu", "ops/kv_move.cu", "ops/rope_rows.cu", "ops/tree.cu",
           "ops/attend.cu", "ops/attend_f16.cu", "ops/attend_q8.cu", "ops/attend_tree_f16.cu", "ops/attend_tree_q8.cu"]
BIND = os.path.join(HERE, "_bind.so")
BIND_SOURCE = os.path.join(CSRC, "ops", "bind.cpp")
BIND_KEY = os.path.join(BUILD, "bind.key")  # what BIND was built for
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC,
         "--expt-relaxed-constexpr"]


def _stale(out: str, deps: list[str]) -> bool:
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(d) > t for d in deps)


def _bind_key() -> str:
    """What a built BIND goes with beside its sources: torch's binary interface, Python's, the machine."""
    spec = importlib.util.find_spec("torch")
    try:
        version = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:  # not installed as a package: its files' time
        version = str(spec and os.path.getmtime(spec.origin))
    return "\n".join((platform.machine(), str(sysconfig.get_config_var("SOABI")), str(spec and spec.origin), version))


def _bind_stale(headers: list[str]) -> bool:
    if _stale(BIND, [BIND_SOURCE] + [h for h in headers if h.endswith(".h")]) or not os.path.exists(BIND_KEY):
        return True
    with open(BIND_KEY) as f:
        return f.read() != _bind_key()


def _bind_command(out: str) -> list[str]:
    import torch
    home = os.path.dirname(os.path.abspath(torch.__file__))
    cuda = os.path.dirname(os.path.dirname(os.path.abspath(NVCC)))
    include = [INCLUDE, os.path.join(home, "include"), sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    return ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *(f"-I{d}" for d in include), BIND_SOURCE, "-o", out,
            f"-L{os.path.join(home, 'lib')}", "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    headers = [os.path.join(d, f) for d in (CSRC, os.path.join(CSRC, "ops"), INCLUDE) for f in os.listdir(d)
               if f.endswith((".cuh", ".h"))]
    objs, jobs = [], []
    for src in SOURCES:
        path = os.path.join(CSRC, src)
        obj = os.path.join(BUILD, os.path.basename(src).replace(".cu", ".o"))
        objs.append(obj)
        if force or _stale(obj, [path] + headers):
            cmd = [NVCC, *ARCH, *FLAGS, "-c", path, "-o", obj]
            if ptxas_info:
                cmd.insert(1, "-Xptxas=-v")
            jobs.append(cmd)

    tmp_bind = BIND + f".tmp{os.getpid()}"
    bind = force or _bind_stale(headers)
    if bind:
        jobs.append(_bind_command(tmp_bind))

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        return cmd, r

    with ThreadPoolExecutor(max_workers=max(1, len(jobs))) as ex:
        for cmd, r in ex.map(run, jobs):
            if verbose or ptxas_info or r.returncode:
                sys.stderr.write(r.stdout + r.stderr)
            if r.returncode:
                raise RuntimeError("compiler failed: " + " ".join(cmd))
    if bind:
        os.replace(tmp_bind, BIND)
        with open(BIND_KEY, "w") as f:
            f.write(_bind_key())
    if force or _stale(SO, objs):
        tmp = SO + f".tmp{os.getpid()}"
        cmd = [NVCC, *ARCH, "-shared", "-o", tmp, *objs, "-lcudart"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode:
            sys.stderr.write(r.stdout + r.stderr)
            raise RuntimeError("link failed")
        os.replace(tmp, SO)
    return SO


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv)
    print(SO)
