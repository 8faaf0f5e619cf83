"""Generated code of the 4-bit product and the quantisation (no GPU), compiled
here for gfx950: no kernel spills to scratch, none holds a packed fp32
instruction, the large product's loop meets once for a chunk and holds the
matrix instructions of a chunk and nothing that waits for memory in between.
"""
import os
import re
import subprocess

import pytest

from fp32_sgemm_f32_amd import build


def assembly(source, folder):
    if not os.path.exists(build.hipcc()):
        pytest.skip("hipcc not found")
    out = str(folder / (source + ".s"))
    cmd = [build.hipcc(), *[f for f in build.COMMON if f not in ("-fPIC", "-fvisibility=hidden")],
           "-x", "hip", "--cuda-device-only", "-S", os.path.join(build.CSRC, source), "-o", out]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    return open(out).read()


@pytest.fixture(scope="module", params=["mx4_gemm.hip", "mx4_quant.hip"])
def asm(request, tmp_path_factory):
    return request.param, assembly(request.param, tmp_path_factory.mktemp("asm"))


def test_no_scratch_and_no_packed_fp32(asm):
    _, text = asm
    sizes = re.findall(r"\.private_segment_fixed_size:\s*(\d+)", text)
    assert sizes and set(sizes) == {"0"}
    assert not re.search(r"v_pk_(add|mul|fma)_f32", text)


def test_loop_of_the_large_product(asm):
    source, text = asm
    if source != "mx4_gemm.hip":
        pytest.skip("the product's")
    found = 0
    # 256 x 256 tiles, chunks of 256 and 128 columns: 4 and 2 matrix steps of 8 products each.
    for m in re.finditer(r"^(_Z\w*mx4_gemm_kernel\w*Li256ELi256ELi(256|128)E\w*):[^\n]*\n(.*?)\n\.Lfunc_end", text, re.S | re.M):
        body, steps = m.group(3), int(m.group(2)) // 64
        loops = re.findall(r"^\.LBB\w+:[^\n]*Inner Loop Header.*?s_cbranch_scc\w", body, re.S | re.M)
        loop = [x for x in loops if "v_mfma_scale" in x]
        assert len(loop) == 1, m.group(1)
        assert loop[0].count("v_mfma_scale_f32_32x32x64_f8f6f4") == 8 * steps, m.group(1)
        assert loop[0].count("s_barrier") == 1, m.group(1)
        waits = re.findall(r"vmcnt\((\d+)\)", loop[0])
        assert len(waits) == 1, m.group(1)          # the one before the barrier
        found += 1
    assert found == 6                               # two chunk lengths, three result types


@pytest.mark.parametrize("source", ["mx4_linear.hip", "mx4_moe.hip"])
def test_streaming_kernels_hold_their_registers(source, tmp_path):
    """The kernels that stream weights past tokens in registers: each bound on the registers of a lane is one that
    the kernel fits without spilling."""
    text = assembly(source, tmp_path)
    kernels = re.findall(r"\.name:\s*(_Z\S+)\n.*?\.private_segment_fixed_size:\s*(\d+).*?\.vgpr_spill_count:\s*(\d+)", text, re.S)
    assert len(kernels) == text.count(".vgpr_spill_count:") and len(kernels) > 20
    assert [k for k in kernels if k[1:] != ("0", "0")] == []
    assert not re.search(r"v_pk_(add|mul|fma)_f32", text)
