"""The wait states between the query tiles' last products and the first read of their results, in the compiled kernel."""
import os
import re
import subprocess

import pytest

from causal_self_exchange_amd import build as B

UNIT = """
#include "paged_scan.h"
#include "paged_tile.h"
namespace rel {
hipError_t unit(const PagedExArgs& a, const HeadParams& hp, hipStream_t s) {
  return launch_tiles<64, 64, __bf16, true>(a, hp, false, s);
}
}
"""


@pytest.mark.skipif(not os.path.exists(B.HIPCC), reason="no hipcc")
def test_results_are_read_behind_the_wait(tmp_path):
    """The check of the results' range, a chain of v_maximum3_f32, is the first to read them; the wait is two s_nop."""
    src, out = tmp_path / "unit.hip", tmp_path / "unit.s"
    src.write_text(UNIT)
    subprocess.run([B.HIPCC, *B.COMMON, "--offload-device-only", "-S", str(src), "-o", str(out)], check=True, capture_output=True)
    kernels = re.split(r"^(?=_ZN\w*tile_kernel\w*:)", out.read_text(), flags=re.M)[1:]
    assert kernels
    for k in kernels:
        lines = [x.strip() for x in k.split("\n")]
        lines = lines[:next(i for i, x in enumerate(lines) if x.startswith(".end_amdhsa_kernel") or x.startswith("s_endpgm"))]
        wait = [i for i, x in enumerate(lines) if x == "s_nop 15"]
        reads = [i for i, x in enumerate(lines) if x.startswith("v_maximum3_f32")]
        assert len(wait) == 2 and reads and wait[0] < reads[0] < wait[1], (wait, reads)
        # Nothing between the products and the wait reads what the wait holds.
        last = max(i for i in range(wait[0]) if lines[i].startswith("v_mfma"))
        held = {(int(a), int(b)) for i in range(wait[0]) for a, b in re.findall(r"^v_mfma_f32_32x32x16_bf16 v\[(\d+):(\d+)\],.*v\[\1:\2\]$", lines[i])}
        held = {r for a, b in held for r in range(a, b + 1)}
        assert held
        for x in lines[last + 1:wait[0]]:
            ops = x.split(";")[0].split(",")[1:] if x.startswith("v_") else []
            used = {int(r) for o in ops for r in re.findall(r"\bv(\d+)\b", o)} | {r for o in ops for a, b in re.findall(r"v\[(\d+):(\d+)\]", o) for r in range(int(a), int(b) + 1)}
            assert not used & held, x
