"""Static properties of the gfx950 code of the norms, of quantizing and of the products on
8-bit matrices (host only).

The products wait for their direct loads by explicit counts.  A vector-memory wait that the
compiler puts right before an LDS read waits for loads still in flight into other stages;
none may stand among the MFMAs.  Every direct load writes LDS at M0, which must be set.
"""
from __future__ import annotations

import concurrent.futures
import os
import re
import subprocess

import pytest

from tiling_roofline_analysis_amd import build

SOURCES = ("scaled_bf16.hip", "scaled_f32.hip", "quantize.hip", "norm.hip")


def assembled(src, to):
    out = os.path.join(to, src + ".s")
    cmd = [build.hipcc(), *build.FLAGS, "--cuda-device-only", "-S", os.path.join(build.CSRC, src),
           "-o", out]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    with open(out) as fh:
        return fh.read()


@pytest.fixture(scope="module")
def texts(tmp_path_factory):
    to = str(tmp_path_factory.mktemp("isa"))
    with concurrent.futures.ThreadPoolExecutor(len(SOURCES)) as ex:
        return dict(zip(SOURCES, ex.map(lambda s: assembled(s, to), SOURCES)))


def kernels(text):
    found = {}
    for m in re.finditer(r"^(_Z\S+):\s*;\s*@\1\n(.*?)^\.Lfunc_end", text, re.M | re.S):
        lines = [x.split(";")[0].strip() for x in m.group(2).splitlines()]
        found[m.group(1)] = [x for x in lines if x and not x.startswith(".")]
    return found


def products(texts):
    for src in SOURCES[:2]:
        for name, body in kernels(texts[src]).items():
            if "scaled_tile" in name or "scaled_wide" in name:
                yield src, name, body


def test_the_kernels_are_there(texts):
    count = {}
    for src, name, _ in products(texts):
        kind = "tile" if "scaled_tile" in name else "wide"
        count[src, kind] = count.get((src, kind), 0) + 1
    # tile sizes, shallow and deep, by five pairs of formats and scales; 256 x 256: 16 bits only;
    # binary32: also with a scale for each row of W, but not in 128 x 128
    assert count == {("scaled_bf16.hip", "tile"): 30, ("scaled_bf16.hip", "wide"): 5,
                     ("scaled_f32.hip", "tile"): 42}


def test_no_scratch_and_no_flat_or_packed_instructions(texts):
    for src, text in texts.items():
        assert set(re.findall(r"\.private_segment_fixed_size:\s*(\d+)", text)) == {"0"}, src
        assert not re.search(r"^\s+flat_", text, re.M), src
        assert not re.search(r"^\s+v_pk_(add|mul|fma)_f32", text, re.M), src


def test_fragment_reads_wait_for_no_other_stage(texts):
    memory = re.compile(r"(ds_|global_|buffer_|s_barrier|s_endpgm)")
    for _, name, body in products(texts):
        last = max(i for i, x in enumerate(body) if x.startswith("v_mfma"))
        for i, x in enumerate(body[:last]):
            if x.startswith("s_waitcnt") and "vmcnt" in x:
                after = next(y for y in body[i + 1:] if memory.match(y))
                assert not after.startswith("ds_read"), f"{name}: '{x}' before '{after}'"


def test_m0_is_set(texts):
    for _, name, body in products(texts):
        lds = [x for x in body if re.match(r"buffer_load_\w+ .* lds$", x)]
        assert lds and any(re.match(r"s_(mov|add_i|add_u|or_b)\w* m0,", x) for x in body), name


def test_which_matrix_instructions(texts):
    # 16-bit results: a block of 128 in one instruction; binary32: four in bfloat16
    for src, name, body in products(texts):
        used = {x.split()[0] for x in body if x.startswith("v_mfma")}
        if src == "scaled_f32.hip":
            assert used == {"v_mfma_f32_16x16x32_bf16"}, (name, used)
        else:
            assert used <= {"v_mfma_f32_16x16x128_f8f6f4", "v_mfma_scale_f32_16x16x128_f8f6f4"}, (
                name, used)


def test_wide_tiles_take_two_steps_of_16(texts):
    for _, name, body in products(texts):
        if "scaled_wide" not in name:
            continue
        # a loop of two K tiles, each of 2 steps of 16 MFMAs
        marks = [i for i, x in enumerate(body) if x.startswith("s_barrier")]
        per = [sum(y.startswith("v_mfma") for y in body[a:b]) for a, b in zip(marks, marks[1:])]
        assert per.count(16) == 6 and set(per) <= {0, 16}, (name, per)
