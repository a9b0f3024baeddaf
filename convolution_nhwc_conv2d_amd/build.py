"""Build libcnhwc.so (the HIP kernels + C ABI) in-tree with hipcc for gfx950, and
_seq.so beside it (the sequence operators' calls on torch tensors).

Every source is compiled on every call (the build check must really compile),
in parallel, then linked into convolution_nhwc_conv2d_amd/.
"""
import importlib.util
import os
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
ROOT = os.path.dirname(PKG)
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libcnhwc.so")
OBJDIR = os.path.join(PKG, "_build")
SOURCES = ["select.cpp", "api.cpp", "gemm.hip", "gemm_lds.hip", "wino_gemm.hip", "winograd.hip", "winograd_h.hip",
           "unfold.hip", "noalloc.hip", "gemm_patch.hip", "layer_norm.hip", "causal_conv.hip", "scan.hip",
           "rms_norm.hip", "rotary.hip", "linear_attention.hip", "linear_attention_f32.hip", "linear_attention_f16.hip",
           "linear_attention_bf16.hip"]
EXT = os.path.join(PKG, "_seq.so")
EXT_SOURCE = "seq_torch.cpp"
TORCH = importlib.util.find_spec("torch").submodule_search_locations[0]
ARCH = "gfx950"

COMMON = ["-O3", "-std=c++17", "-fPIC", f"--offload-arch={ARCH}", "-I", INCLUDE, "-I", CSRC,
          # packed fp32 VALU forms stay off (only ordinary fp32 instructions are emitted)
          "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
          "-Wall", "-Wno-unused-function"]
# The extension is host code; torch's headers name their platform by USE_ROCM.
EXT_FLAGS = ["-O2", "-std=c++17", "-fPIC", "-I", INCLUDE, "-isystem", os.path.join(TORCH, "include"), "-isystem",
             os.path.join(TORCH, "include", "torch", "csrc", "api", "include"), "-isystem",
             sysconfig.get_paths()["include"], "-DUSE_ROCM", "-Wall"]


def _hipcc():
    for c in ("/opt/rocm/bin/hipcc", "hipcc"):
        if os.path.exists(c) or c == "hipcc":
            return c


def _compile(src, verbose):
    obj = os.path.join(OBJDIR, os.path.splitext(src)[0] + ".o")
    cmd = [_hipcc()] + (EXT_FLAGS if src == EXT_SOURCE else COMMON) + ["-c", os.path.join(CSRC, src), "-o", obj]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    msgs = "\n".join(l for l in (r.stdout + r.stderr).splitlines() if "packed-fp32-ops" not in l)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{msgs}")
    if msgs.strip() and verbose:
        print(msgs, flush=True)
    return obj


def build(verbose: bool = False) -> str:
    # the Winograd matrices header is generated from exact rationals
    subprocess.run([sys.executable, os.path.join(CSRC, "gen_winograd.py")], check=True,
                   capture_output=not verbose)
    os.makedirs(OBJDIR, exist_ok=True)
    with ThreadPoolExecutor(max_workers=min(8, len(SOURCES) + 1)) as ex:
        *objs, ext = ex.map(lambda s: _compile(s, verbose), SOURCES + [EXT_SOURCE])
    _link(LIB, objs, verbose)
    _link(EXT, [ext, LIB, "-Wl,-rpath,$ORIGIN", "-L" + os.path.join(TORCH, "lib"), "-ltorch_python", "-ltorch_cpu",
                "-lc10", "-lc10_hip"], verbose)
    return LIB


def _link(target, inputs, verbose):
    tmp = target + ".tmp"
    # the library goes by its file name alone, which the extension finds beside itself
    name = ["-Wl,-soname," + os.path.basename(target)]
    cmd = [_hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp] + name + inputs
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, target)


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
