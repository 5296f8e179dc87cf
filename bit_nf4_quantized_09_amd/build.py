"""Compile the gfx950 HIP library libqlora_nf4.so in-tree with hipcc, and the binding of decoder.py with g++."""
import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
OUT_DIR = os.path.join(HERE, "_lib")
LIB = os.path.join(OUT_DIR, "libqlora_nf4.so")
PROBE_SOURCE = "hbm_probe.hip"      # the HBM ceiling probes: a library of their own
BINDING_SOURCE = "decoder_binding.cpp"   # the Python calls of decoder.py: a CPython extension over the library
BINDING = os.path.join(OUT_DIR, "qlora_decoder_binding.so")
PROBE_LIB = os.path.join(OUT_DIR, "libnf4_hbm_probe.so")
SOURCES = ["api.hip", "codec.hip", "lora.hip", "fused.hip", "gemv.hip", "adamw.hip", "codebook.hip", "lowrank.hip",
           "decoder_api.hip", "rope.hip", "kv_append.hip", "kv_attention.hip", "head_loss.hip",
           "step_api.hip", "block_norm.hip", "gradients.hip", "logits.hip"]
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
    "-ffp-contract=off",                                  # no silent multiply-add fusion
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I", os.path.join(ROOT, "include"),
]


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(OUT_DIR, src.replace(".hip", ".o"))
    cmd = [HIPCC] + FLAGS + ["-c", os.path.join(CSRC, src), "-o", obj]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    errs = "\n".join(l for l in r.stderr.splitlines() if "packed-fp32-ops" not in l)
    if r.returncode != 0:
        raise RuntimeError("hipcc failed for %s:\n%s" % (src, errs))
    if errs.strip() and verbose:
        print(errs, flush=True)
    return obj


def _binding_lacks(cxx: str):
    """What the binding needs and is not here (None: nothing): the library needs none of it."""
    import sysconfig

    if shutil.which(cxx) is None:
        return "the C++ compiler %s" % cxx
    python = os.path.join(sysconfig.get_paths()["include"], "Python.h")
    if not os.path.exists(python):
        return python
    try:
        import torch
    except ImportError:
        return "torch"
    headers = os.path.join(os.path.dirname(torch.__file__), "include", "torch", "csrc")
    return None if os.path.isdir(headers) else headers


def _build_binding(verbose: bool) -> None:
    """The CPython extension (torch's headers and libraries; next to the library, which it loads).  Without what it needs
    the library stands alone: its linears and its C entry points work, decoder.py's calls say that they are not built."""
    import sysconfig

    cxx = os.environ.get("CXX", "g++")
    lacks = _binding_lacks(cxx)
    if lacks is not None:
        if os.path.exists(BINDING):
            os.remove(BINDING)               # (one of another build would not fit this library)
        warnings.warn("the binding of decoder.py is not built: %s is missing" % lacks)
        return
    import torch

    root = os.path.dirname(torch.__file__)
    tmp = BINDING + ".tmp%d" % os.getpid()
    cmd = [cxx, "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-Wno-unknown-pragmas",
           "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch._C._GLIBCXX_USE_CXX11_ABI,
           "-isystem", os.path.join(root, "include"), "-isystem", os.path.join(root, "include", "torch", "csrc", "api", "include"),
           "-isystem", sysconfig.get_paths()["include"], os.path.join(CSRC, BINDING_SOURCE), "-o", tmp,
           "-L" + OUT_DIR, "-lqlora_nf4", "-Wl,-rpath,$ORIGIN",
           "-L" + os.path.join(root, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10"]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("%s failed for %s:\n%s" % (cxx, BINDING_SOURCE, r.stderr))
    if r.stderr.strip() and verbose:
        print(r.stderr, flush=True)
    os.replace(tmp, BINDING)


def build(verbose: bool = False) -> str:
    os.makedirs(OUT_DIR, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        objs = list(ex.map(lambda s: _compile(s, verbose), SOURCES + [PROBE_SOURCE]))
    probe_obj = objs.pop()
    tmp = PROBE_LIB + ".tmp%d" % os.getpid()
    subprocess.run([HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", probe_obj, "-o", tmp], check=True)
    os.replace(tmp, PROBE_LIB)
    tmp = LIB + ".tmp%d" % os.getpid()
    cmd = [HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC"] + objs + ["-o", tmp]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)
    _build_binding(verbose)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
