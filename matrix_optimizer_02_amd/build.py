"""Builds libdmuon_ns.so in-tree for gfx950 with hipcc.

    python -m matrix_optimizer_02_amd.build      (or __graft_entry__.build())

Every HIP source is compiled with packed-fp32 instructions disabled
(-target-feature -packed-fp32-ops); the planner is plain C++ built with g++.
"""

from __future__ import annotations

import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
ROOT = os.path.dirname(PKG)
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libdmuon_ns.so")

HIP_SOURCES = ["api.hip", "clip.hip", "head.hip", "k_adamw.hip", "k_diag.hip", "k_elementwise.hip", "k_gemm_bf16.hip",
               "k_gemm_f32.hip", "k_head_gemm.hip", "k_head_probs.hip", "k_head_rows.hip", "k_head_stream.hip",
               "k_head_wide.hip", "k_head_x3.hip", "k_resident.hip", "tune.hip"]
CXX_SOURCES = ["head_layout.cpp", "plan.cpp"]
ARCH = "gfx950"


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found")


HIP_FLAGS = [f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC", "-Wall", "-fvisibility=hidden",
             "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
             "-ffp-contract=fast"]


def _run(cmd, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError(f"build step failed: {' '.join(cmd[:3])} ...")
    return res


HEADERS = ["dmuon_ns.h", "dmuon_head.h", "dmuon_logprobs.h", "dmuon_clip.h"]


def exported_symbols(header: str = "dmuon_ns.h"):
    """Names of the functions a header of include/ declares with DMUON_API."""
    import re

    with open(os.path.join(INCLUDE, header)) as f:
        text = f.read()
    return re.findall(r"^DMUON_API\s+[\w\s\*]*?\b(\w+)\s*\(", text, flags=re.M)


# Sources whose accumulators are registers that only their assembly text names.
ASM_ACCUMULATORS = ["k_head_wide.hip"]


def check_accumulators(assembly: str, what: str) -> None:
    """Refuses device assembly in which anything but the products and the reads of
    their sums touches an accumulation register: the sums lie there without the
    compiler's knowledge, and what it kept or moved there itself would be lost, or
    would overwrite them."""
    import re

    n = r"(?:0x[0-9a-f]+|\d+)"
    products, refused = 0, []
    for line in assembly.splitlines():
        code = line.split(";")[0].split("//")[0].strip()
        if code.startswith(".") or not re.search(r"\ba(\d+\b|\[)", code):
            continue
        if re.fullmatch(rf"v_mfma_\w+ (a\[{n}:{n}\]), v\[\d+:\d+\], v\[\d+:\d+\], (\1|0)", code):
            products += 1
        elif not re.fullmatch(rf"v_accvgpr_read_b32 v\d+, a(\d+|\[{n}\])", code):
            refused.append(code)
    if refused:
        raise RuntimeError(f"{what}: the compiler uses accumulation registers, which hold the kernel's sums: "
                           + "; ".join(refused[:8]))
    if products == 0:
        raise RuntimeError(f"{what}: no product found")


def _device_assembly(bdir: str, src: str) -> str:
    """What -save-temps=obj left of a source's device code."""
    with open(os.path.join(bdir, f"{os.path.splitext(src)[0]}-hip-amdgcn-amd-amdhsa-{ARCH}.s")) as f:
        return f.read()


def compile_hip(src: str, obj: str, extra_flags=(), verbose: bool = False) -> None:
    """One HIP source of csrc/ to an object file."""
    temps = ["-save-temps=obj"] if src in ASM_ACCUMULATORS else []
    _run([hipcc(), *HIP_FLAGS, *extra_flags, *temps, f"-I{INCLUDE}", "-c", os.path.join(CSRC, src), "-o", obj], verbose)
    if temps:
        check_accumulators(_device_assembly(os.path.dirname(obj), src), src)


def build(verbose: bool = False, extra_flags=(), out: str = None, build_dir: str = None) -> str:
    """Compile every source and link libdmuon_ns.so; returns the library path.
    ``extra_flags`` (e.g. -D tuning macros) go to every hipcc compile; ``out``
    and ``build_dir`` redirect the library and the object files."""
    lib = out or LIB
    bdir = build_dir or BUILD
    os.makedirs(bdir, exist_ok=True)
    objs = []
    cc = hipcc()
    for src in HIP_SOURCES:
        obj = os.path.join(bdir, src + ".o")
        compile_hip(src, obj, extra_flags, verbose)
        objs.append(obj)
    for src in CXX_SOURCES:
        obj = os.path.join(bdir, src + ".o")
        _run(["g++", "-O2", "-std=c++17", "-fPIC", "-Wall", "-fvisibility=hidden", f"-I{INCLUDE}", "-c",
              os.path.join(CSRC, src), "-o", obj], verbose)
        objs.append(obj)
    version_script = os.path.join(bdir, "exports.map")
    with open(version_script, "w") as f:
        names = [s for h in HEADERS for s in exported_symbols(h)]
        f.write("{ global: " + " ".join(s + ";" for s in names) + " local: *; };\n")
    tmp = lib + ".tmp"
    _run([cc, f"--offload-arch={ARCH}", "-shared", "-fPIC", *objs,
          f"-Wl,--version-script={version_script}", "-o", tmp], verbose)
    os.replace(tmp, lib)
    return lib


if __name__ == "__main__":
    print(build(verbose=True))
