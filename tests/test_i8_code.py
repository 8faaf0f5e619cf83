"""Generated code of the 8-bit integer kernels (no GPU), compiled here for gfx950:
no kernel spills to scratch, none holds a packed fp32 instruction, and the large
product's loop meets once for a chunk, with the matrix instructions of a chunk
and nothing that waits for memory in between.
"""
import os
import re
import subprocess

import pytest

from fp32_sgemm_f32_amd import build

SOURCES = ["i8_gemm.hip", "i8_quant.hip", "i8_swiglu.hip", "i8_thin.hip"]


@pytest.fixture(scope="module", params=SOURCES)
def asm(request, tmp_path_factory):
    if not os.path.exists(build.hipcc()):
        pytest.skip("hipcc not found")
    out = str(tmp_path_factory.mktemp("asm") / (request.param + ".s"))
    cmd = [build.hipcc(), *[f for f in build.COMMON if f not in ("-fPIC", "-fvisibility=hidden")],
           "-x", "hip", "--cuda-device-only", "-S", os.path.join(build.CSRC, request.param), "-o", out]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    return request.param, open(out).read()


def test_every_source_is_built():
    assert all(s in build.SOURCES for s in SOURCES)


def test_no_scratch_and_no_packed_fp32(asm):
    _, text = asm
    kernels = re.findall(r"\.name:\s*(_Z\S+)\n.*?\.private_segment_fixed_size:\s*(\d+).*?\.vgpr_spill_count:\s*(\d+)", text, re.S)
    assert kernels and len(kernels) == text.count(".vgpr_spill_count:")
    assert [k for k in kernels if k[1:] != ("0", "0")] == []
    assert not re.search(r"v_pk_(add|mul|fma)_f32", text)


def test_loop_of_the_large_product(asm):
    source, text = asm
    if source != "i8_gemm.hip":
        pytest.skip("the product's")
    found = 0
    # 256 x 256 tiles: four matrix steps of eight products each.
    for m in re.finditer(r"^(_Z\w*i8_gemm_kernel\w*Li256ELi256E\w*):[^\n]*\n(.*?)\n\.Lfunc_end", text, re.S | re.M):
        loops = re.findall(r"^\.LBB\w+:[^\n]*Inner Loop Header.*?s_cbranch_scc\w", m.group(2), re.S | re.M)
        loop = [x for x in loops if "v_mfma_i32" in x]
        assert len(loop) == 1, m.group(1)
        assert loop[0].count("v_mfma_i32_32x32x32_i8") == 32, m.group(1)
        assert loop[0].count("s_barrier") == 1, m.group(1)
        assert len(re.findall(r"vmcnt\((\d+)\)", loop[0])) == 1, m.group(1)          # the one before the barrier
        down = "ELb1ELi" in m.group(1)
        assert (loop[0].count("ds_read_b64_tr_b8") > 0) == down, m.group(1)
        found += 1
    assert found == 7                               # rows and down in three result types each, and pieces in pairs
