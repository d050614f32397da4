"""Checks on the gfx950 assembly of the serving library (CPU only), those that
test_isa_checks.py makes of the table library: no packed-fp32 instruction, no
scalar-cache write, no select on an SCC that arithmetic left; no scratch."""
from __future__ import annotations

import os
import re
import shutil
import subprocess
import tempfile

import pytest

from int4_row_wise_amd import build as qbuild
from tests import test_isa_checks as checks


@pytest.fixture(scope="module")
def asm():
    hipcc = qbuild.hipcc()
    if shutil.which(hipcc) is None and not os.path.exists(hipcc):
        pytest.skip("hipcc not available")
    flags = [f for f in qbuild.HIPCC_FLAGS if f not in ("-fPIC", "-shared")]
    with tempfile.TemporaryDirectory() as d:
        out = os.path.join(d, "serving.s")
        cmd = [hipcc, *flags, "--cuda-device-only", "-S", "-I", os.path.join(qbuild.ROOT, "include"), "-o", out, qbuild.SERVING_SRC]
        r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
        assert r.returncode == 0, r.stdout[-2000:]
        with open(out) as f:
            return f.read()


def test_no_packed_fp32(asm):
    checks.test_no_packed_fp32(asm)


def test_no_scalar_cache_writes(asm):
    checks.test_no_scalar_cache_writes(asm)


def test_no_stale_scc_select(asm):
    checks.test_no_stale_scc_select(asm)


def test_no_scratch(asm):
    """No kernel spills to scratch memory."""
    sizes = re.findall(r"\.private_segment_fixed_size:\s*(\d+)", asm)
    assert sizes and all(int(s) == 0 for s in sizes), sizes
