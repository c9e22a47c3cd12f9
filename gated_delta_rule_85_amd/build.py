"""Build libgdr.so (the HIP kernels and the C ABI of include/gdr.h) for gfx950, and
_gdr_torch.so, the compiled part of the Python binding (host code only).

Each .hip source is compiled with hipcc into an object in _build/, then
linked into gated_delta_rule_85_amd/libgdr.so.  Packed-fp32 instruction
selection is switched off for the device code.  The binding is compiled with
g++ against torch's headers and linked to libgdr.so.
"""
import importlib.util
import os
import subprocess
import sys
import sysconfig
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OUT = os.path.join(PKG, "libgdr.so")
BINDING = os.path.join(PKG, "_gdr_torch.so")
BUILD = os.path.join(ROOT, "_build")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"
FLAGS = ["--offload-arch=" + ARCH, "-O3", "-std=c++17", "-fPIC", "-Wall",
         "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
         "-I" + os.path.join(ROOT, "include")]
# MFMA operands and results in VGPRs rather than AGPRs (fewer copies in the
# register-resident loops of every kernel that keeps its work in registers).
VGPR_FORM = ["-mllvm", "-amdgpu-mfma-vgpr-form=1"]
# The scans run one wave per SIMD, so nothing hides an LDS read's latency but
# the wave's own later instructions: the ILP-seeking scheduler issues the
# operand reads well ahead of their MFMAs (the default one waits on each).
ILP = ["-mllvm", "-amdgpu-sched-strategy=iterative-ilp"]
# The backward's chunk-local kernel (also one wave per SIMD, at the register
# limit) spills under the iterative ILP scheduler; with the max-ILP one and
# VGPR-form MFMAs it spills nothing (default scheduler: 17 registers) and runs 8%
# faster.  On the scans the max-ILP scheduler costs 30%.
MAX_ILP = ["-mllvm", "-amdgpu-sched-strategy=max-ilp"]
# Linear attention's scans place their reads of LDS by hand, a step ahead; within a step the max-ILP
# scheduler gains 1 to 2% over the default one.
# The reverse scan runs eight waves (two per SIMD, 256 registers each); the ILP
# scheduler's schedule of it does not survive register allocation in this
# compiler, and the default scheduler with its operand reads pipelined by hand
# serves it.
SOURCES = {"gdr_api.hip": VGPR_FORM, "gdr_prep.hip": VGPR_FORM, "gdr_scan.hip": VGPR_FORM + ILP,
           "gdr_bwd.hip": VGPR_FORM, "gdr_bwd_scan.hip": VGPR_FORM,
           "gdr_bwd_mfma.hip": VGPR_FORM + MAX_ILP, "gdr_noalloc.hip": [],
           "gdr_step.hip": [], "gdr_tree.hip": VGPR_FORM, "gdr_copy.hip": [], "gdr_pool_api.hip": [],
           "gdr_la_scan.hip": VGPR_FORM + MAX_ILP, "gdr_la_bwd.hip": [], "gdr_la_api.hip": [],
           "gdr_norm.hip": [], "gdr_norm_bwd.hip": [], "gdr_norm_api.hip": []}


def _compile(src):
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [HIPCC] + FLAGS + SOURCES[src] + ["-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    err = "\n".join(l for l in r.stderr.splitlines() if "packed-fp32-ops" not in l)
    if r.returncode != 0:
        raise RuntimeError("hipcc failed for %s:\n%s" % (src, err))
    if err.strip():
        sys.stderr.write(err + "\n")
    return obj


def _compile_binding():
    """The binding's object (torch is found without importing it)."""
    torch = os.path.dirname(importlib.util.find_spec("torch").origin)
    obj = os.path.join(BUILD, "gdr_torch.o")
    include = [os.path.join(ROOT, "include"), "/opt/rocm/include", os.path.join(torch, "include"),
               os.path.join(torch, "include", "torch", "csrc", "api", "include"), sysconfig.get_paths()["include"]]
    r = subprocess.run(["g++", "-O2", "-std=c++17", "-fPIC", "-Wall", "-D__HIP_PLATFORM_AMD__"] + ["-I" + i for i in include]
                       + ["-c", os.path.join(CSRC, "gdr_torch.cpp"), "-o", obj], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("g++ failed for gdr_torch.cpp:\n%s" % r.stderr)
    return obj, ["-L" + os.path.join(torch, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10"]


def build(verbose=False):
    os.makedirs(BUILD, exist_ok=True)
    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        binding = ex.submit(_compile_binding)
        objs = list(ex.map(_compile, SOURCES))
        binding, torch_libs = binding.result()
    # both are linked before either takes its place: a failure leaves the old pair
    with tempfile.TemporaryDirectory(dir=BUILD) as tmp:
        lib, bind = (os.path.join(tmp, os.path.basename(f)) for f in (OUT, BINDING))
        subprocess.run([HIPCC, "--offload-arch=" + ARCH, "-shared", "-fPIC", "-o", lib] + objs, check=True)
        subprocess.run(["g++", "-shared", "-o", bind, binding, "-L" + tmp, "-lgdr", "-Wl,-rpath,$ORIGIN"] + torch_libs,
                       check=True)
        os.replace(lib, OUT)
        os.replace(bind, BINDING)
    if verbose:
        print(OUT)
    return OUT


if __name__ == "__main__":
    build(verbose=True)
