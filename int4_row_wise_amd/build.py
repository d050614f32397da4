"""Build libqemb.so, libqemb_attention.so and libqemb_serving.so (the HIP C-ABI
libraries) in-tree for gfx950.

    python -m int4_row_wise_amd.build

hipcc cross-compiles on a machine without a GPU.  Flags: no fast-math and no
floating-point contraction (the quantizer must round exactly as its rules
say), packed-fp32 instructions disabled.
"""
from __future__ import annotations

import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
SRC = os.path.join(CSRC, "qemb.hip")  # the translation unit; it includes the csrc/*.inc parts
HEADER = os.path.join(ROOT, "include", "qemb.h")
LIB = os.path.join(HERE, "libqemb.so")
LIB_HASH = LIB + ".srchash"  # source sha256 recorded at build time
# the gather floor (a measurement aid for bench.py, not part of the C ABI)
FLOOR_SRC = os.path.join(CSRC, "gather_floor.hip")
FLOOR_LIB = os.path.join(HERE, "libqemb_floor.so")
# attention over a paged key-value cache: a translation unit and library of its own
ATTN_DIR = os.path.join(CSRC, "attention")
ATTN_SRC = os.path.join(ATTN_DIR, "attention.hip")
ATTN_HEADER = os.path.join(ROOT, "include", "qemb_attention.h")
ATTN_LIB = os.path.join(HERE, "libqemb_attention.so")
# what stands around the attention in a serving loop: another one
SERVING_DIR = os.path.join(CSRC, "serving")
SERVING_SRC = os.path.join(SERVING_DIR, "serving.hip")
SERVING_HEADER = os.path.join(ROOT, "include", "qemb_serving.h")
SERVING_LIB = os.path.join(HERE, "libqemb_serving.so")

HIPCC_FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-ffp-contract=off",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-fPIC", "-shared", "-Wall",
]


def hipcc() -> str:
    for c in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", "hipcc"):
        if c and (os.path.isabs(c) and os.path.exists(c) or not os.path.isabs(c)):
            return c
    return "hipcc"


def _compile(src: str, lib: str) -> tuple:
    """Start hipcc on one translation unit: (process, temporary output, library)."""
    tmp = lib + ".tmp%d" % os.getpid()
    cmd = [hipcc(), *HIPCC_FLAGS, "-I", os.path.join(ROOT, "include"), "-o", tmp, src]
    return subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True), tmp, lib


def _finish(job: tuple, verbose: bool) -> None:
    proc, tmp, lib = job
    out, _ = proc.communicate()
    out = "\n".join(l for l in out.splitlines() if "packed-fp32-ops" not in l)
    if proc.returncode != 0:
        raise RuntimeError("hipcc failed:\n" + out)
    if out.strip() and verbose:
        print(out)
    os.replace(tmp, lib)


def _record(lib: str, sha: str) -> None:
    with open(lib + ".srchash", "w") as f:
        f.write(sha + "\n")


def _newer(lib: str, sources: list) -> bool:
    return os.path.exists(lib) and os.path.getmtime(lib) >= max(os.path.getmtime(f) for f in sources)


def build_attention(verbose: bool = False) -> str:
    """Compile csrc/attention/attention.hip into libqemb_attention.so."""
    sha = attention_source_sha256()
    _finish(_compile(ATTN_SRC, ATTN_LIB), verbose)
    _record(ATTN_LIB, sha)
    return ATTN_LIB


def build_serving(verbose: bool = False) -> str:
    """Compile csrc/serving/serving.hip into libqemb_serving.so."""
    sha = serving_source_sha256()
    _finish(_compile(SERVING_SRC, SERVING_LIB), verbose)
    _record(SERVING_LIB, sha)
    return SERVING_LIB


def build(force: bool = True, verbose: bool = False) -> str:
    """Compile csrc/qemb.hip into int4_row_wise_amd/libqemb.so, and beside it
    the gather floor, the attention library and the serving library."""
    if (not force and _newer(LIB, source_files() + [HEADER]) and _newer(ATTN_LIB, attention_source_files())
            and _newer(SERVING_LIB, serving_source_files())):
        return LIB
    # the hash of the sources as compiled: taken before the compiler reads
    # them, so an edit made while it runs cannot be recorded for this build
    src_hash = source_sha256()
    attn_hash = attention_source_sha256()
    serving_hash = serving_source_sha256()
    # the small libraries compile beside the large one
    jobs = [_compile(FLOOR_SRC, FLOOR_LIB), _compile(ATTN_SRC, ATTN_LIB), _compile(SERVING_SRC, SERVING_LIB), _compile(SRC, LIB)]
    try:
        for job in jobs:
            _finish(job, verbose)
    finally:
        for proc, _, _ in jobs:
            if proc.poll() is None:
                proc.kill()
    _record(LIB, src_hash)
    _record(ATTN_LIB, attn_hash)
    _record(SERVING_LIB, serving_hash)
    return LIB


def source_files() -> list:
    """The kernel sources: qemb.hip, the parts it includes and the gather
    floor, in a fixed order."""
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".hip", ".inc")))


def source_sha256() -> str:
    """sha256 over the kernel sources the library is built from (each file's
    name and bytes, in sorted order)."""
    return _sha256(source_files())


def attention_source_files() -> list:
    """The attention library's sources: its own, the shared helpers and the headers."""
    own = [os.path.join(ATTN_DIR, f) for f in os.listdir(ATTN_DIR) if f.endswith((".hip", ".inc"))]
    return sorted(own) + [os.path.join(CSRC, "common.inc"), ATTN_HEADER, HEADER]


def attention_source_sha256() -> str:
    """sha256 over the attention library's sources, as source_sha256."""
    return _sha256(attention_source_files())


def serving_source_files() -> list:
    """The serving library's sources: its own, the shared helpers and the headers."""
    own = [os.path.join(SERVING_DIR, f) for f in os.listdir(SERVING_DIR) if f.endswith((".hip", ".inc"))]
    return sorted(own) + [os.path.join(ATTN_DIR, "rows.inc"), os.path.join(CSRC, "common.inc"), SERVING_HEADER, ATTN_HEADER, HEADER]


def serving_source_sha256() -> str:
    """sha256 over the serving library's sources, as source_sha256."""
    return _sha256(serving_source_files())


def _sha256(paths: list) -> str:
    import hashlib
    h = hashlib.sha256()
    for path in paths:
        h.update(os.path.basename(path).encode() + b"\0")
        with open(path, "rb") as f:
            h.update(f.read())
    return h.hexdigest()


def built_source_sha256() -> str | None:
    """The source hash recorded when libqemb.so was last built, if any."""
    return recorded_hash(LIB)


def recorded_hash(lib: str) -> str | None:
    """The source hash recorded when a library was last built, if any."""
    try:
        with open(lib + ".srchash") as f:
            return f.read().strip()
    except OSError:
        return None


def ensure_built() -> str:
    """Build only if no library exists yet (used by tests, smoke and bench)."""
    if not os.path.exists(LIB):
        return build(force=True)
    if not os.path.exists(ATTN_LIB):
        build_attention()
    if not os.path.exists(SERVING_LIB):
        build_serving()
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose="-v" in sys.argv))
