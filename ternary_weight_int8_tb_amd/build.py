"""Build libtb.so, the HIP library of this package, for gfx950 (in-tree)."""

from __future__ import annotations

import os
import subprocess
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
SOURCES = ("tb.hip", "tb_norm.hip", "tb_mx.hip", "tb_moe.hip", "tb_kv.hip", "tb_attn.hip")   # libtb.so, one object each
PROBE_SRC = os.path.join(PKG, "csrc", "probe.hip")
PROBE_LIB = os.path.join(PKG, "libtb_probe.so")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libtb.so")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

FLAGS = [
    "-O3", "--offload-arch=gfx950", "-std=c++17", "-fPIC",
    # one IEEE rounding per fp32 operation: no fused multiply-add, correctly rounded division
    "-ffp-contract=off", "-fhip-fp32-correctly-rounded-divide-sqrt",
    # no packed fp32 instructions (v_pk_*_f32)
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    # leading scalar kernel arguments arrive preloaded in SGPRs (no kernel-argument fetch
    # before the first loads); the code object keeps a fallback for firmware without it
    "-mllvm", "-amdgpu-kernarg-preload-count=16",
    "-Wall", "-Wno-unused-command-line-argument",
]


def _compile(src: str, out: str, args: list[str]) -> str:
    subprocess.run([HIPCC, *FLAGS, *args, "-I", INCLUDE, src, "-o", out + ".tmp"], check=True)
    os.replace(out + ".tmp", out)
    return out


def build(out: str = LIB, extra: list[str] | None = None) -> str:
    """Build libtb.so (the path) and libtb_probe.so (benchmark probes)."""
    obj_dir = os.path.join(PKG, "_build")
    os.makedirs(obj_dir, exist_ok=True)
    args = ["-c", *(extra or [])]
    with ThreadPoolExecutor() as pool:
        probe = pool.submit(_compile, PROBE_SRC, PROBE_LIB, ["-shared"])
        objs = list(pool.map(lambda s: _compile(os.path.join(CSRC, s), os.path.join(obj_dir, s + ".o"), args),
                             SOURCES))
        probe.result()
    subprocess.run([HIPCC, "--offload-arch=gfx950", "-fPIC", "-shared", *objs, "-o", out + ".tmp"], check=True)
    os.replace(out + ".tmp", out)
    return out


if __name__ == "__main__":
    print(build())
