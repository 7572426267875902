"""Static properties of the fused linear kernels' gfx950 code (host only).

The direct-load kernels wait for their loads by explicit counts.  A
vector-memory wait that the compiler puts right before an LDS read waits for
loads still in flight into other stages; none may stand among the MFMAs.  And
every direct load writes LDS at M0, which must be set.
"""
from __future__ import annotations

import os
import re
import subprocess

import pytest

from tiling_roofline_analysis_amd import build


@pytest.fixture(scope="module", params=["linear_bf16.hip", "linear_f32.hip"])
def kernels(request, tmp_path_factory):
    out = str(tmp_path_factory.mktemp("isa") / "k.s")
    cmd = [build.hipcc(), *build.FLAGS, "--cuda-device-only", "-S",
           os.path.join(build.CSRC, request.param), "-o", out]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    with open(out) as fh:
        text = fh.read()
    found = {}
    for m in re.finditer(r"^(_Z\S+):\s*;\s*@\1\n(.*?)^\.Lfunc_end", text, re.M | re.S):
        lines = [x.split(";")[0].strip() for x in m.group(2).splitlines()]
        found[m.group(1)] = [x for x in lines if x and not x.startswith(".")]
    return request.param, found


def direct(found):
    dma = re.compile(r"^buffer_load_dword(x4)? .* lds$")
    return {n: b for n, b in found.items() if any(dma.match(x) for x in b)}


def test_the_direct_kernels_are_there(kernels):
    src, found = kernels
    got = direct(found)
    tiles = [n for n in got if "linear_tile" in n]
    wide = [n for n in got if "linear_wide" in n]
    # three tile sizes, shallow and deep, by three forms plain and two gated; in
    # binary32 also two tile sizes whose lanes load 4 bytes
    assert len(tiles) == (40 if src == "linear_f32.hip" else 30)
    # the 256 x 256 kernel: 16 bits only
    assert len(wide) == (0 if src == "linear_f32.hip" else 5)


def test_fragment_reads_wait_for_no_other_stage(kernels):
    _, found = kernels
    memory = re.compile(r"(ds_|global_|buffer_|s_barrier|s_endpgm)")
    for name, body in direct(found).items():
        last = max(i for i, x in enumerate(body) if x.startswith("v_mfma"))
        for i, x in enumerate(body[:last]):
            if x.startswith("s_waitcnt") and "vmcnt" in x:
                after = next(y for y in body[i + 1:] if memory.match(y))
                assert not after.startswith("ds_read"), f"{name}: '{x}' before '{after}'"


def test_m0_is_set(kernels):
    _, found = kernels
    for name, body in direct(found).items():
        assert any(re.match(r"s_\w+ m0,", x) for x in body), name


@pytest.fixture(scope="module", params=["linear_bf16.hip", "linear_f32.hip"])
def ir(request, tmp_path_factory):
    out = str(tmp_path_factory.mktemp("ir") / "k.ll")
    cmd = [build.hipcc(), *build.FLAGS, "--cuda-device-only", "-emit-llvm", "-S",
           os.path.join(build.CSRC, request.param), "-o", out]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    with open(out) as fh:
        text = fh.read()
    return {m.group(1): m.group(2) for m in
            re.finditer(r"^define [^\n]*amdgpu_kernel void @(\w+)\(.*?\{\n(.*?)^\}", text,
                        re.M | re.S)}


def test_lanes_meet_between_the_sums_writes_and_reads(ir):
    # the epilogue's lanes read what other lanes of the wave wrote to LDS: a fence of
    # the wave stands between, and in the 256 x 256 kernel, which does so twice, also
    # before the next write
    kernels = {n: b for n, b in ir.items() if "linear_tile" in n or "linear_wide" in n}
    assert len(kernels) >= 40
    for name, body in kernels.items():
        fences = len(re.findall(r'fence syncscope\("wavefront"\) acq_rel', body))
        assert fences >= (3 if "linear_wide" in name else 1), name
