"""Build libccl.so in-tree with hipcc for gfx950.

One shared library holds the host compiler, the plan runtime, the C entry points, the
executor kernel, and the kernels of the products, the row exchange and the layer's operators
around them. Host sources are plain C++17; the kernel source is HIP. Every file is compiled
with packed-fp32 instructions disabled.
"""

from __future__ import annotations

import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIBDIR = os.path.join(HERE, "lib")
LIB = os.path.join(LIBDIR, "libccl.so")
BUILD = os.path.join(ROOT, "_build")

HOST_SOURCES = ["compiler.cpp", "simulate.cpp", "capi.cpp", "tune.cpp", "specialize.cpp", "products.cpp", "layers.cpp"]
DEVICE_SOURCES = ["executor.hip", "static_scratch.hip", "hop_probe.hip", "products.hip", "product_tile_bf16.hip",
                  "product_tile_f32.hip", "product_rows.hip", "exchange.hip", "select.hip", "norm.hip", "loss.hip",
                  "loss_tile_bf16.hip", "loss_tile_f32.hip"]
ARCH = "gfx950"
COMMON = ["-O3", "-std=c++17", "-fPIC", "-Wall", "-Wno-unused-result", "-I", os.path.join(ROOT, "include"), "-I", "/opt/rocm/include"]
DEVICE_FLAGS = [f"--offload-arch={ARCH}", "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
                "-fno-gpu-rdc", "-mcode-object-version=5"]


def hipcc() -> str:
    for c in ("/opt/rocm/bin/hipcc", "hipcc"):
        if os.path.isabs(c) and os.path.exists(c):
            return c
    return "hipcc"


def _run(cmd):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("build failed:\n" + " ".join(cmd) + "\n" + r.stdout + r.stderr)
    return r.stdout + r.stderr


EMBED = "embedded_executor.cpp"  # generated: the executor's device source as text


def write_embedded_source() -> str:
    """The device code that plan-specialized kernels are compiled from at run time: the
    public header, the device ABI and the executor's device code, without their
    #include lines (the runtime compiler has no system headers beyond <stdint.h>)."""
    parts = []
    for path in (os.path.join(ROOT, "include", "ccl.h"), os.path.join(CSRC, "device_abi.h"),
                 os.path.join(CSRC, "executor_device.h")):
        with open(path) as fh:
            text = fh.read()
        parts.append("\n".join(line for line in text.split("\n") if not line.lstrip().startswith("#include")))
    body = "\n".join(parts)
    delim = "CCLSRC"
    if (")" + delim + '"') in body:
        raise RuntimeError("embedded source contains the raw-string delimiter")
    out = os.path.join(BUILD, EMBED)
    with open(out, "w") as fh:
        fh.write("// generated by build.py\nnamespace ccl {\nextern const char kEmbeddedExecutorSource[];\n"
                 f"const char kEmbeddedExecutorSource[] = R\"{delim}(" + body + f"){delim}\";\n}}  // namespace ccl\n")
    return out


def build(verbose: bool = False) -> str:
    os.makedirs(LIBDIR, exist_ok=True)
    os.makedirs(BUILD, exist_ok=True)
    cc = hipcc()
    embedded = write_embedded_source()
    jobs = [[cc, *COMMON, "-x", "c++", "-c", embedded, "-o", embedded + ".o"]]
    for s in HOST_SOURCES:
        jobs.append([cc, *COMMON, "-x", "c++", "-D__HIP_PLATFORM_AMD__", "-c", os.path.join(CSRC, s),
                     "-o", os.path.join(BUILD, s + ".o")])
    for s in DEVICE_SOURCES:
        jobs.append([cc, *COMMON, *DEVICE_FLAGS, "-c", os.path.join(CSRC, s), "-o", os.path.join(BUILD, s + ".o")])
    with ThreadPoolExecutor(max_workers=min(8, len(jobs))) as ex:
        outs = list(ex.map(_run, jobs))
    objs = [os.path.join(BUILD, s + ".o") for s in HOST_SOURCES + DEVICE_SOURCES] + [embedded + ".o"]
    tmp = LIB + ".tmp"
    outs.append(_run([cc, "-shared", "-fPIC", f"--offload-arch={ARCH}", "-Wl,--no-undefined", *objs,
                      "-L/opt/rocm/lib", "-lhiprtc", "-o", tmp]))
    os.replace(tmp, LIB)
    if verbose:
        for o in outs:
            if o.strip():
                print(o, file=sys.stderr)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
