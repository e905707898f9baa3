"""Build libkdaconv.so in-tree with hipcc for gfx950.

    python -m packed_varlen_causal_depthwise_amd.build
"""

from __future__ import annotations

import concurrent.futures
import os
import pathlib
import shutil
import subprocess
import tempfile

PKG = pathlib.Path(__file__).resolve().parent
ROOT = PKG.parent
SOURCES = [PKG / "csrc" / name for name in (
    "kdaconv.hip",
    "delta_rule.hip",
    "delta_rule_bf16.hip",
    "delta_rule_f16.hip",
    "delta_rule_f32.hip",
    "norms.hip",
)]
HEADERS = [ROOT / "include" / "kdaconv.h", *sorted((PKG / "csrc").glob("*.h"))]
LIBRARY = PKG / "libkdaconv.so"
ARCH = "gfx950"

FLAGS = [
    f"--offload-arch={ARCH}",
    "-O3",
    "-std=c++17",
    "-fPIC",
    # Packed FP32 instructions stay off: the compiler must not form them.
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    # Exact IEEE binary32 semantics: no contraction, no flushing of subnormals.
    "-ffp-contract=off",
    "-fno-fast-math",
    "-fno-gpu-flush-denormals-to-zero",
    "-Wall",
]


def hipcc() -> str:
    return shutil.which("hipcc") or "/opt/rocm/bin/hipcc"


def build(output: pathlib.Path = LIBRARY, extra_flags=()) -> pathlib.Path:
    """Compiles each source to an object, several at a time, and links them."""
    tmp = output.with_name(output.name + f".tmp{os.getpid()}")
    with tempfile.TemporaryDirectory() as work:
        objects = [pathlib.Path(work) / (src.stem + ".o") for src in SOURCES]

        def compile_one(src, obj):
            subprocess.run([hipcc(), *FLAGS, *extra_flags, "-I", str(ROOT / "include"), "-c",
                            "-o", str(obj), str(src)], check=True)

        with concurrent.futures.ThreadPoolExecutor(max_workers=min(8, len(SOURCES))) as pool:
            list(pool.map(compile_one, SOURCES, objects))
        subprocess.run([hipcc(), f"--offload-arch={ARCH}", "-fPIC", "-shared", "-o", str(tmp),
                        *map(str, objects)], check=True)
    os.replace(tmp, output)
    return output


if __name__ == "__main__":
    print(build())
