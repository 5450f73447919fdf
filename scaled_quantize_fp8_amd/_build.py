"""Build libfp8linear.so (the FP8 linear path) and libfp8probe.so (its
measurement kernels) in-tree with hipcc for gfx950."""

from __future__ import annotations

import hashlib
import os
import shutil
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB_NAME = "libfp8linear.so"
LIB_PATH = os.path.join(HERE, LIB_NAME)
SOURCES = [os.path.join(CSRC, f) for f in ("fp8l_api.hip", "fp8l_grouped.hip", "fp8l_i8.hip", "fp8l_mx4.hip",
                                           "fp8l_route.hip", "fp8l_version.hip")]
OBJ_DIR = os.path.join(HERE, "_build")  # objects; not tracked
PROBE_LIB_PATH = os.path.join(HERE, "libfp8probe.so")
PROBE_SOURCES = [os.path.join(CSRC, "fp8l_probe.hip")]


def source_hash() -> str:
    """SHA-256 over the library's sources and its public header (file names
    and bytes, in sorted order).  The build compiles it into the library
    (fp8_source_hash), so a library built from other sources is detected."""
    h = hashlib.sha256()
    files = sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC)
                   if f.endswith((".hip", ".hpp", ".h")))
    files.append(os.path.join(ROOT, "include", "fp8linear.h"))
    for path in files:
        h.update(os.path.relpath(path, ROOT).encode())
        with open(path, "rb") as f:
            h.update(f.read())
    return h.hexdigest()


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), shutil.which("hipcc"), "/opt/rocm/bin/hipcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found")


def _flags(source: str) -> list[str]:
    return [
        "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
        # packed fp32 VALU forms stay off (see the library's design notes)
        "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
        "-I", os.path.join(ROOT, "include"),
        *([f'-DFP8L_SOURCE_HASH="{source_hash()}"'] if "version" in os.path.basename(source) else []),
    ]


def compile_command(source: str, out: str, extra: list[str] | None = None) -> list[str]:
    return [hipcc(), *_flags(source), *(extra or []), "-c", source, "-o", out]


def link_command(objects: list[str], out: str) -> list[str]:
    return [hipcc(), "--offload-arch=gfx950", "-shared", "-fPIC", *objects, "-o", out]


def _run_all(jobs: list[tuple[str, list[str]]], verbose: bool) -> None:
    """Run the commands in parallel; raise with the output of those that failed."""
    procs = [(name, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT,
                                     text=True)) for name, cmd in jobs]
    failed = []
    for name, proc in procs:
        text, _ = proc.communicate()
        msgs = [ln for ln in text.splitlines() if "packed-fp32-ops" not in ln and ln.strip()]
        if proc.returncode != 0:
            failed.append(f"hipcc failed for {name}:\n" + "\n".join(msgs))
        elif verbose and msgs:
            print("\n".join(msgs))
    if failed:
        raise RuntimeError("\n".join(failed))


def build(verbose: bool = False) -> str:
    """Compile both libraries (always recompiles; the translation units are
    compiled in parallel).  Returns the path of libfp8linear.so."""
    libs = {LIB_PATH: SOURCES, PROBE_LIB_PATH: PROBE_SOURCES}
    os.makedirs(OBJ_DIR, exist_ok=True)
    obj = {src: os.path.join(OBJ_DIR, os.path.basename(src) + ".o")
           for srcs in libs.values() for src in srcs}
    _run_all([(os.path.basename(src), compile_command(src, o)) for src, o in obj.items()], verbose)
    _run_all([(os.path.basename(lib), link_command([obj[s] for s in srcs], lib + ".tmp"))
              for lib, srcs in libs.items()], verbose)
    for lib in libs:
        os.replace(lib + ".tmp", lib)
    return LIB_PATH


if __name__ == "__main__":
    print(build(verbose=True))
