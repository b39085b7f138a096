"""Checks on the gfx950 assembly of the orthogonalisation, norm and activation-gradient kernels (CPU only;
hipcc cross-compiles).

The orthogonalisation's product kernels issue their global-to-LDS copies as inline assembly that sets M0
and issues global_load_lds in one statement, which is sound only while nothing else in those kernels reads
M0.  Their accumulators, and the values that the tile kernels hold from their formation to their second
copy, have to stay in registers: no kernel here may use scratch memory.
"""
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")


@pytest.fixture(scope="module")
def asm(tmp_path_factory):
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not available")
    lines = {}
    for stem in ("newton", "fused"):
        out = str(tmp_path_factory.mktemp("isa") / (stem + ".s"))
        r = subprocess.run([HIPCC, "--offload-arch=gfx950", "-O3", "-std=c++17", "-Xclang", "-target-feature",
                            "-Xclang", "-packed-fp32-ops", "--cuda-device-only", "-S", "-o", out,
                            os.path.join(ROOT, "blockwise_fp8_gemm_amd", "csrc", stem + ".hip")],
                           capture_output=True, text=True, timeout=600)
        assert r.returncode == 0, r.stderr[-2000:]
        with open(out) as f:
            lines[stem] = [l.split(";")[0] for l in f]
    return lines


def test_m0_only_feeds_the_copies(asm):
    writes = 0
    code = asm["newton"]
    for i, line in enumerate(code):
        if not re.search(r"\bm0\b", line):
            continue
        assert re.match(r"\s*s_mov_b32 m0, s\d+\s*$", line), ("M0 used outside the LDS copies", i, line)
        assert re.match(r"\s*s_nop 0\s*$", code[i + 1]), ("no wait state between M0 and its copy", i, code[i + 1])
        assert "global_load_lds_dwordx4" in code[i + 2], ("M0 write not followed by its copy", i, code[i + 2])
        writes += 1
    assert writes > 0
    banned = re.compile(r"movrel|set_gpr_idx|s_sendmsg|ds_gws|ds_append|ds_consume|v_interp|lds_direct|ds_ordered")
    assert not any(banned.search(l) for l in code)


@pytest.mark.parametrize("stem,kernels", [("newton", 14), ("fused", 12)])
def test_no_scratch(asm, stem, kernels):
    scratch, name = {}, None
    for line in asm[stem]:
        m = re.match(r"\s*\.amdhsa_kernel (\S+)", line)
        name = m.group(1) if m else name
        m = re.match(r"\s*\.amdhsa_private_segment_fixed_size (\d+)", line)
        if m:
            scratch[name] = int(m.group(1))
    assert len(scratch) == kernels, sorted(scratch)
    assert not any(scratch.values()), {n: b for n, b in scratch.items() if b}
    assert not any(re.search(r"\bv_pk_(add|mul|fma)_f32\b", l) for l in asm[stem])
