"""Compile liblora4.so for gfx950 with hipcc (in-tree, next to this file).

    python -m lora_fine_tuning_amd.build
"""

import os
import shutil
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "liblora4.so")
SOURCES = [os.path.join(HERE, "csrc", "lora4.hip")]   # includes every csrc/*.hpp
# the kernels of the feed-forward operators, attention and the loss, compiled
# beside it (lora4.hip includes them itself where it is compiled alone)
FFN_SOURCES = [os.path.join(HERE, "csrc", name) for name in ("ffn.hip", "attn.hip", "loss.hip")]
# measured roofline denominators (MFMA rate, HBM read bandwidth), beside the library
PROBE_LIB = os.path.join(HERE, "libpeakprobe.so")
PROBE_SOURCES = [os.path.join(HERE, "csrc", "peak_probe.hip")]

FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-shared",
    # packed fp32 VALU forms are kept out of the generated code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    # IEEE fp32 division: the NF4 encoder divides by the block absmax
    "-fhip-fp32-correctly-rounded-divide-sqrt",
    "-ffp-contract=off",
    "-fvisibility=hidden",
]


def hipcc():
    for cand in (os.environ.get("HIPCC"), shutil.which("hipcc"), "/opt/rocm/bin/hipcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found")


def _run(cmd, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError("hipcc failed")


def _compile(sources, out, verbose):
    _run([hipcc(), *FLAGS, "-I", os.path.join(ROOT, "include"), "-I", os.path.join(HERE, "csrc"),
          *sources, "-o", out + ".tmp"], verbose)
    os.replace(out + ".tmp", out)


def _object(source, obj, verbose):
    flags = [f for f in FLAGS if f != "-shared"]
    _run([hipcc(), *flags, "-DLORA4_FFN_SEPARATE", "-c", "-I", os.path.join(ROOT, "include"),
          "-I", os.path.join(HERE, "csrc"), source, "-o", obj], verbose)
    return obj


def build(verbose=False):
    """Compile the library and the peak probe; returns the library's path.
    Always recompiles."""
    _compile(PROBE_SOURCES, PROBE_LIB, verbose)
    with tempfile.TemporaryDirectory() as tmp, ThreadPoolExecutor(4) as pool:
        objs = list(pool.map(lambda s: _object(s, os.path.join(tmp, os.path.basename(s) + ".o"), verbose),
                             SOURCES + FFN_SOURCES))
        _compile(objs, LIB, verbose)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
