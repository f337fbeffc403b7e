"""Range-checked buffer accesses, in the assembly of kernels built here: the check is certain for the vector offset (with
the instruction's own) only as long as the scalar offset does not pass the resource's size. Where a resource may be
shorter than a step that the code takes (rows past the last token, columns past the experts), the step has to be in the
vector offset: no access of these kernels has a scalar offset."""

import ctypes
import os
import re
import shutil
import subprocess

import pytest

from mxfp4_block_scaled_amd import build

ACCESS = re.compile(r"^\s*(buffer_(?:load|store)_\w+)\s+(.*)$")


def accesses(source, tmp_path):
    """(instruction, scalar offset) of every buffer access by kernel; scratch has descriptors of its own."""
    if not shutil.which(build.HIPCC) and not os.path.exists(build.HIPCC):
        pytest.skip("no hipcc")
    out = str(tmp_path / "kernels.s")
    subprocess.run([build.HIPCC, *build.FLAGS, "--offload-device-only", "-S", "-x", "hip",
                    os.path.join(build.CSRC, source), "-o", out], check=True, capture_output=True)
    found, kernel = {}, None
    for line in open(out):
        if line.startswith("_Z") and ":" in line:
            kernel = line.split(":")[0]
        m = ACCESS.match(line.split(";")[0])
        if m:  # data, vector offset (or "off"), resource, scalar offset and flags
            found.setdefault(kernel, []).append((m[1], m[2].split(",")[-1].split()[0], line.strip()))
    return found


def test_the_router_steps_in_vector_offsets(tmp_path):
    found = accesses("route_loss.hip", tmp_path)
    kernels = [k for k in found if "balance_kernel" in k or "route_backward_kernel" in k]
    assert sum("balance_kernel" in k for k in kernels) == 30 and sum("route_backward_kernel" in k for k in kernels) == 10
    for k in kernels:
        assert len(found[k]) >= 2
        for name, scalar, line in found[k]:
            assert scalar in ("0", "null"), (k, line)


def test_held_steps_stay_inside(tmp_path):
    """Row (or rank, or k) steps that loads of the ragged FP4-weight kernels take through a scalar offset: below the
    size whatever the fragment asks for, and the step itself where it is inside."""
    src, so = tmp_path / "held.cpp", str(tmp_path / "held.so")
    src.write_text('#include "w4a16_plan.hpp"\nextern "C" int held(int r, int n) { return mxf::w16_held_step(r, n); }\n')
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-Wno-unknown-pragmas", "-I", build.CSRC, str(src), "-o", so],
                   check=True)
    held = ctypes.CDLL(so).held
    for n in range(1, 140):
        for r in range(0, 136):
            assert 0 <= held(r, n) < n and (held(r, n) == r or r >= n)
