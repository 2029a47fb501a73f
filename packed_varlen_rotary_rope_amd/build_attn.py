"""Build the HIP library libattn.so (packed and paged attention kernels, the cache append and its
pages, the rotation with several axes) for gfx950 with hipcc (in-tree). It links against
librope_qk.so beside it, whose inverse frequencies the rotations use; build that first (build.py).

Usage: python packed_varlen_rotary_rope_amd/build_attn.py  (run as a script: importing the
package itself needs the libraries)
"""
from __future__ import annotations

import os
import subprocess
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
# sources and their flags: the attention is compiled once for each form of its scores, the longest
# compilations first
SRCS = [(os.path.join(PKG, "csrc", name), [f"-DATTN_MODS={mods}"])
        for name in ("attn_bwd.hip", "attn_paged.hip", "attn_fwd.hip") for mods in (3, 2, 1, 0)]
SRCS += [(os.path.join(PKG, "csrc", name), []) for name in
         ("rope_axes.hip", "attn_plan.hip", "kv_append.hip", "kv_pages.hip")]
LIB_PATH = os.path.join(PKG, "libattn.so")
ARCH = "gfx950"

HIPCC_FLAGS = [
    f"--offload-arch={ARCH}",
    "-O3",
    "-std=c++17",
    "-fPIC",
    # every product and sum is rounded as written (the append's rotation relies on it)
    "-ffp-contract=off",
    # no packed fp32 instructions (v_pk_fma_f32 and friends) in device code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wno-unused-command-line-argument",
    "-I", os.path.join(ROOT, "include"),
]


def hipcc() -> str:
    return os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "bin", "hipcc")


def build(extra_flags=(), out: str = LIB_PATH) -> str:
    """Compile each source to an object, then link the library."""
    import tempfile
    tmp = out + ".tmp"
    with tempfile.TemporaryDirectory() as d:
        def compile_one(item):
            number, (src, flags) = item
            obj = os.path.join(d, f"{number}_{os.path.basename(src)}.o")
            subprocess.run([hipcc(), *HIPCC_FLAGS, *flags, *extra_flags, "-c", "-o", obj, src], check=True)
            return obj

        with ThreadPoolExecutor(8) as pool:
            objs = list(pool.map(compile_one, enumerate(SRCS)))
        subprocess.run([hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp, *objs,
                        "-L", PKG, "-l:librope_qk.so", "-Wl,-rpath,$ORIGIN"], check=True)
    os.replace(tmp, out)
    return out


if __name__ == "__main__":
    print(build())
