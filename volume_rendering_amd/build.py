"""Builds libnerf_mi355x.so in-tree with hipcc for gfx950, and the checked
library libnerf_mi355x_checked.so (the same sources with -DNERF_CHECK: the
kernels record failed index-range checks, read back by nerf_check_flags).

    python -m volume_rendering_amd.build          # build both (always recompiles)

Every HIP source is compiled with fused multiply-add contraction off (the
bit-reproducible steps are written as explicitly rounded float32/float64
operations) and with packed fp32 instructions disabled.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libnerf_mi355x.so")
LIB_CHECKED = os.path.join(PKG, "libnerf_mi355x_checked.so")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"

SOURCES = ["render_nerf_bf16.hip", "render_nerf_f32.hip", "render_hash.hip", "mlp_bf16.hip", "mlp_f32.hip",
           "kernels.hip", "kilo.hip", "abi.cpp", "pack.cpp", "layouts.cpp", "noalloc.hip", "train.hip", "hash_train.hip",
           "route.hip", "experts.hip", "distill.hip", "experts_abi.cpp", "gate.hip", "routed_mlp.hip", "scan.hip",
           "scan_grad.hip", "scan_plan.cpp", "clip.hip", "fields_abi.cpp"]

COMMON = ["-O3", "-std=c++17", "-fPIC", "-ffp-contract=off", f"-I{INCLUDE}", f"-I{CSRC}", "-Wall",
          "-Wno-unused-function"]
# matrix-instruction accumulators in architectural VGPRs (operands stay in
# AGPRs where the kernels place them), so epilogues read results directly
DEVICE = [f"--offload-arch={ARCH}", "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
          "-mllvm", "-amdgpu-mfma-vgpr-form"]
# sources built without the VGPR-form option: the INR step's kernels (whose
# small MFMA accumulators may live in AGPRs) make that pass of this compiler
# fail on the larger decoder shapes; the experts' products (64 to 128 accumulators
# a lane) build and run alike either way (1024 -> 4096 gradients 618 us, 333 -> 517
# forward 187 and 185 with it, float32 1024 -> 1024 394 and 391)
DEVICE_AGPR_FORM = {"hash_train.hip", "experts.hip"}


def _compile(src: str, checked: bool = False) -> str:
    obj = os.path.join(BUILD, "checked" if checked else "", os.path.splitext(src)[0] + ".o")
    path = os.path.join(CSRC, src)
    cmd = [HIPCC] + COMMON + (["-DNERF_CHECK"] if checked else [])
    if src.endswith(".hip"):
        dev = DEVICE if src not in DEVICE_AGPR_FORM else [a for a in DEVICE if a not in ("-mllvm",
                                                                                       "-amdgpu-mfma-vgpr-form")]
        cmd += dev + ["-x", "hip"]
    cmd += ["-c", path, "-o", obj]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{' '.join(cmd)}\n{res.stdout}\n{res.stderr}")
    # the host pass does not know the packed-fp32 feature; that warning is harmless
    noise = [l for l in res.stderr.splitlines() if "packed-fp32-ops" not in l and l.strip()]
    if noise:
        sys.stderr.write(f"[{src}]\n" + "\n".join(noise) + "\n")
    return obj


def build(verbose: bool = True, checked: bool = False) -> str:
    """Builds one library (the checked one with checked=True); returns its path."""
    lib = LIB_CHECKED if checked else LIB
    os.makedirs(os.path.join(BUILD, "checked") if checked else BUILD, exist_ok=True)
    srcs = [s for s in SOURCES if os.path.exists(os.path.join(CSRC, s))]
    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        objs = list(ex.map(lambda src: _compile(src, checked), srcs))
    tmp = lib + ".tmp"
    cmd = [HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp] + objs
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{' '.join(cmd)}\n{res.stdout}\n{res.stderr}")
    # a kernel whose host-side launch stub the compiler did not emit (e.g. a
    # target-only builtin in code the host pass also sees) links fine and
    # fails only when the library is loaded: refuse such a library here
    und = subprocess.run(["nm", "-D", "--undefined-only", tmp], capture_output=True, text=True)
    missing = [l.split()[-1] for l in und.stdout.splitlines() if "__device_stub__" in l]
    if missing:
        raise RuntimeError("kernels without host launch stubs:\n" + "\n".join(missing))
    os.replace(tmp, lib)
    if verbose:
        print(f"built {lib}")
    return lib


def build_all(verbose: bool = True) -> None:
    build(verbose)
    build(verbose, checked=True)


if __name__ == "__main__":
    build_all()
