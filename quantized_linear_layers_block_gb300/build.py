"""Build the CUDA library libtl_gb300.so in-tree (sm_103a only), and _tensors.so, the Python module that hands
torch tensors to it (only where a torch with CUDA and Python's headers are installed; the library needs neither).

Usage: python -m quantized_linear_layers_block_gb300.build   (or build() from Python)

Each CUDA translation unit under csrc/ is compiled in parallel with
`nvcc -gencode arch=compute_103a,code=sm_103a -lineinfo -O3`, then linked
into a shared library next to this file; tensors.cpp by nvcc's host compiler against torch's headers. Objects go to
_build/ at the repository root; both are git-ignored.
"""

from __future__ import annotations

import concurrent.futures
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OBJDIR = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libtl_gb300.so")
TENSORS = os.path.join(PKG, "_tensors.so")
SOURCES = ["tl_api.cu", "pack.cu", "rotate_quant.cu", "decode.cu", "decode_fused_m.cu", "prefill.cu", "codec.cu",
           "decode_f32.cu", "decode_tc.cu", "kv_append.cu", "paged_attention_bf16.cu", "paged_attention_f16.cu",
           "paged_attention_f8.cu", "lora.cu", "tree_plan.cu", "tree_attention_bf16.cu", "tree_attention_f16.cu",
           "tree_attention_f8.cu", "verify_tree.cu", "kv_compact.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2", "-I", os.path.join(ROOT, "include")]


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libtl_gb300.so")
    return cand


def _torch_dir() -> str | None:
    """Where torch is installed, if _tensors.so can be built against it: with CUDA, and Python's headers at hand."""
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.origin:
        return None
    d = os.path.dirname(spec.origin)
    need = [os.path.join(d, "lib", "libc10_cuda.so"), os.path.join(d, "include", "c10", "cuda", "CUDAGuard.h"),
            os.path.join(sysconfig.get_paths()["include"], "Python.h")]
    return d if all(os.path.exists(f) for f in need) else None


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    if _torch_dir() is not None and (not os.path.exists(TENSORS) or os.path.getmtime(TENSORS) < t):
        return True
    deps = [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [os.path.join(ROOT, "include", "tl.h"), __file__]
    return any(os.path.getmtime(d) > t for d in deps if os.path.exists(d))


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile and link the library if any source is newer; return its path."""
    if not force and not _stale():
        return LIB
    nvcc = _nvcc()
    os.makedirs(OBJDIR, exist_ok=True)

    def compile_one(src: str) -> str:
        obj = os.path.join(OBJDIR, src.replace(".cu", ".o"))
        cmd = [nvcc, *ARCH, *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose:
            sys.stdout.write(r.stdout + r.stderr)
        return obj

    torch_dir = _torch_dir()

    def compile_tensors() -> str | None:
        """The object, or None where there is nothing to build against. Errors are raised when the library is linked."""
        if torch_dir is None:
            return None
        obj = os.path.join(OBJDIR, "tensors.o")
        cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include")
        dirs = [sysconfig.get_paths()["include"], os.path.join(torch_dir, "include"),
                os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"), cuda]
        cmd = [nvcc, "-O2", "-std=c++17", "-Xcompiler", "-fPIC,-fvisibility=hidden", *(f"-I{d}" for d in dirs),
               "-c", os.path.join(CSRC, "tensors.cpp"), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for tensors.cpp:\n{r.stdout}\n{r.stderr}")
        return obj

    with concurrent.futures.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        tensors = ex.submit(compile_tensors)
        objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB + ".tmp"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs, "-lcudart_static", "-ldl", "-lpthread", "-lrt"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    tensors_obj = tensors.result()
    if tensors_obj is not None:
        tmp = TENSORS + ".tmp"
        libs = os.path.join(torch_dir, "lib")
        cmd = [nvcc, "-shared", "-cudart", "none", "-o", tmp, tensors_obj, f"-L{libs}", "-ltorch_python", "-ltorch_cpu", "-lc10_cuda",
               "-lc10", f"-L{PKG}", "-l:libtl_gb300.so", "-Xlinker", "-rpath,$ORIGIN", "-Xlinker", f"-rpath,{libs}"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link of _tensors.so failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, TENSORS)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
