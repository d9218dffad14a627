"""Build libpml.so in-tree: every CUDA translation unit under csrc/ compiled
for sm_103a in parallel, then linked into one shared library next to this
file; beside it the Python module _calls (csrc/binding.cpp), against this
interpreter's PyTorch, which the serving operators' calls need and the library
does not.  Rebuilds each only when a source, header, flag or (for _calls) the
interpreter or PyTorch changed."""
from __future__ import annotations

import hashlib
import os
import shutil
import subprocess
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG, "_build")
LIB_PATH = os.path.join(PKG, "libpml.so")
CALLS_PATH = os.path.join(PKG, "_calls.so")

SOURCES = ["api.cu", "schedule.cu", "fp8_logits.cu", "fp8_logits_h8.cu", "fp8_logits_h16.cu",
           "fp8_logits_h32.cu", "fp8_logits_h64.cu", "bf16_scores.cu", "nvfp4_scores.cu",
           "topk.cu", "mxfp4_logits.cu", "noalloc.cu", "api_serving.cu", "rope.cu",
           "index_quant.cu", "pages.cu", "paged_attention.cu", "paged_attention_d64.cu",
           "paged_attention_d128.cu"]
NVCC_FLAGS = [
    "-gencode", "arch=compute_103a,code=sm_103a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC,-O2",
    "--expt-relaxed-constexpr",
]


def _nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _fingerprint(extra_flags) -> str:
    h = hashlib.sha256()
    for d in (CSRC, INCLUDE):
        for name in sorted(os.listdir(d)):
            if name.endswith((".cu", ".cuh", ".h", ".cpp")):
                with open(os.path.join(d, name), "rb") as f:
                    h.update(name.encode() + f.read())
    h.update(" ".join(NVCC_FLAGS + list(extra_flags)).encode())
    return h.hexdigest()


def _stamped(stamp: str, made: str, fp: str) -> bool:
    """Whether `made` is there and was made from what `fp` says."""
    if not (os.path.exists(made) and os.path.exists(stamp)):
        return False
    with open(stamp) as f:
        return f.read().strip() == fp


def _write(stamp: str, fp: str) -> None:
    with open(stamp, "w") as f:
        f.write(fp)


def _build_calls(nvcc: str, fp: str, force: bool) -> None:
    import torch
    stamp = os.path.join(BUILD_DIR, "stamp_calls")
    fp += f" {sysconfig.get_config_var('SOABI')} {torch.__version__}"
    if not force and _stamped(stamp, CALLS_PATH, fp):
        return
    home = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(shutil.which(nvcc) or nvcc)))
    tmp = CALLS_PATH + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           os.path.join(CSRC, "binding.cpp"), "-o", tmp, "-I", INCLUDE,
           "-isystem", sysconfig.get_path("include"), "-isystem", os.path.join(home, "include"),
           "-isystem", os.path.join(cuda, "include"), "-L", os.path.join(home, "lib"),
           "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on binding.cpp:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, CALLS_PATH)
    _write(stamp, fp)


def build(force: bool = False, extra_flags=(), verbose: bool = False) -> str:
    """Compile and link libpml.so and _calls; returns the library's path.  A
    failure of _calls is raised with the library in place."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    stamp = os.path.join(BUILD_DIR, "stamp")
    fp = _fingerprint(extra_flags)
    nvcc = _nvcc()

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD_DIR, src.replace(".cu", ".o"))
        cmd = [nvcc, *NVCC_FLAGS, *extra_flags, "-I", INCLUDE, "-I", CSRC, "-c",
               os.path.join(CSRC, src), "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr, flush=True)
        return obj

    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        calls = ex.submit(_build_calls, nvcc, fp, force)
        if force or not _stamped(stamp, LIB_PATH, fp):
            objs = list(ex.map(compile_one, SOURCES))
            tmp = LIB_PATH + f".tmp{os.getpid()}"
            cmd = [nvcc, "-shared", "-gencode", "arch=compute_103a,code=sm_103a", *objs, "-o", tmp]
            r = subprocess.run(cmd, capture_output=True, text=True)
            if r.returncode != 0:
                raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
            os.replace(tmp, LIB_PATH)
            _write(stamp, fp)
        calls.result()
    return LIB_PATH


if __name__ == "__main__":
    print(build(force=True, verbose=True))
