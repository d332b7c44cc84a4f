"""Build libbpe.so in-tree for gfx950 with hipcc.

    python -m byte_level_bpe_pretokenize_amd.build
"""
from __future__ import annotations

import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libbpe.so")
SOURCES = [os.path.join(CSRC, f)
           for f in ("bpe_encode.hip", "bpe_decode.hip", "bpe_train.hip", "bpe_noalloc.hip",
                     "bpe_api.cpp", "bpe_tables.cpp", "bpe_text.cpp")]
# the operators on token IDs (include/bpe_lm.h)
SOURCES += [os.path.join(PKG, "csrc_lm", f)
            for f in ("lm_embed.hip", "lm_logits.hip", "lm_blocks.hip", "lm_api.cpp", "lm_layout.cpp")]
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-shared",
    "-Wall",
    # no packed fp32 instructions anywhere in device code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I", os.path.join(ROOT, "include"),
]


def build(verbose: bool = False) -> str:
    tmp = LIB + ".tmp"
    cmd = [HIPCC, *FLAGS, *SOURCES, "-o", tmp]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
