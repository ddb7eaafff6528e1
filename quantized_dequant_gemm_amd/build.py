"""Ahead-of-time build of libqdg.so for gfx950 with hipcc.

Every kernel instance is a template specialisation compiled here, once.
The streaming family's source text is also embedded in the library, so that
qdg_plan_jit can compile an instance at run time with hipRTC. Run
``python -m quantized_dequant_gemm_amd.build`` or call ``build()``. The
shared object lands next to this file.
"""

import concurrent.futures as cf
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
OUT_DIR = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libqdg.so")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

SOURCES = ["api.cpp", "jit.cpp", "preprocess.hip", "actquant.hip", "moe_align.hip", "stream_gemm.hip", "tile_gemm.hip", "wstream_gemm.hip", "qtile_gemm.hip",
           "wstream8_gemm.hip", "noalloc.cpp", "api_ops.cpp", "moe_route.hip", "gemm_i8.hip", "api_layer.cpp", "row_ops.hip", "lora.hip"]

COMMON = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-Wall", "-Wno-unused-function",
    "-Wno-unused-variable", "-Wno-unused-but-set-variable",
    # no packed fp32 arithmetic anywhere in device code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I", os.path.join(ROOT, "include"),
]


# the sources a run-time compiled kernel is built from (one file per family,
# and the headers they include)
JIT_TEXTS = [("kJitStreamSrc", os.path.join(CSRC, "stream_gemm.hip")),
             ("kJitTileSrc", os.path.join(CSRC, "tile_gemm.hip")),
             ("kJitWstreamSrc", os.path.join(CSRC, "wstream_gemm.hip")),
             ("kJitQtileSrc", os.path.join(CSRC, "qtile_gemm.hip")),
             ("kJitWstream8Src", os.path.join(CSRC, "wstream8_gemm.hip")),
             ("kJitDeviceHdr", os.path.join(CSRC, "qdg_device.h")),
             ("kJitInternalHdr", os.path.join(CSRC, "qdg_internal.h")),
             ("kJitQdgHdr", os.path.join(ROOT, "include", "qdg.h"))]


def _write_jit_sources():
    out = ["// Generated by build.py: source texts for run-time compilation."]
    for name, path in JIT_TEXTS:
        text = open(path, encoding="utf-8").read()
        assert ")QDGJIT\"" not in text
        out.append(f'static const char {name}[] = R"QDGJIT({text})QDGJIT";')
    path = os.path.join(OUT_DIR, "jit_sources.inc")
    data = "\n".join(out) + "\n"
    if not os.path.exists(path) or open(path, encoding="utf-8").read() != data:
        with open(path, "w", encoding="utf-8") as f:
            f.write(data)


def _compile(src):
    obj = os.path.join(OUT_DIR, os.path.basename(src) + ".o")
    lang = ["-x", "hip"]
    cmd = [HIPCC] + COMMON + ["-I", OUT_DIR] + lang + ["-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    warn = "\n".join(l for l in r.stderr.splitlines() if "packed-fp32-ops" not in l and l.strip())
    return obj, warn


def build(verbose=False, jobs=None):
    os.makedirs(OUT_DIR, exist_ok=True)
    _write_jit_sources()
    srcs = [s for s in SOURCES if os.path.exists(os.path.join(CSRC, s))]
    jobs = jobs or min(len(srcs), max(1, (os.cpu_count() or 4) - 1), 8)
    with cf.ThreadPoolExecutor(jobs) as ex:
        results = list(ex.map(_compile, srcs))
    if verbose:
        for (o, w) in results:
            if w:
                print(w, file=sys.stderr)
    objs = [o for o, _ in results]
    tmp = LIB + ".tmp"
    cmd = [HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", "-o", tmp] + objs + [
        "-L/opt/rocm/lib", "-lhiprtc", "-Wl,-rpath,/opt/rocm/lib"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
