"""Host-side rules of the paged forward, compiled from the library's header by the host compiler."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CXX = os.environ.get("CXX_HOST", "g++")

PROGRAM = """
#include <cstdio>
#include "rel_internal.h"
int main() {
  long long rows, blocks;
  int groups, bf16;
  while (std::scanf("%lld %lld %d %d", &rows, &blocks, &groups, &bf16) == 4)
    std::printf("%d\\n", (int)rel::paged_whole(rows, blocks, groups, bf16 != 0));
}
"""


@pytest.fixture(scope="module")
def whole(tmp_path_factory):
    if shutil.which(CXX) is None:
        pytest.skip("no host C++ compiler")
    at = tmp_path_factory.mktemp("rules")
    (at / "rules.cpp").write_text(PROGRAM)
    subprocess.run([CXX, "-std=c++17", "-D__HIP_PLATFORM_AMD__", "-I", "/opt/rocm/include", "-I", os.path.join(ROOT, "include"), "-I",
                    os.path.join(ROOT, "causal_self_exchange_amd", "csrc"), str(at / "rules.cpp"), "-o", str(at / "rules")],
                   check=True, capture_output=True, text=True)

    def ask(cases):
        r = subprocess.run([str(at / "rules")], input="\n".join(" ".join(str(int(x)) for x in c) for c in cases),
                           capture_output=True, text=True, check=True)
        return [bool(int(x)) for x in r.stdout.split()]
    return ask


def test_whole_row_blocks_have_few_units(whole):
    """Row blocks stay whole where a table row of that many cached rows gives none of them more than 9 units of 128 keys
    (fp32: 5; a row sees the rows before its own), and each can have a work-group."""
    cases = [(rows, blocks, 512, bf16) for bf16 in (True, False) for rows in (16, 128, 129, 512, 513, 514, 640, 641, 642, 656, 1024, 1025,
                                                                            1136, 1152, 1153, 1154, 1168, 40000, (1 << 31) - 65536)
             for blocks in (1, 512, 513)]
    want = [max(1, -(-(rows - 1) // 128)) <= (9 if bf16 else 5) and blocks <= groups for rows, blocks, groups, bf16 in cases]
    got = whole(cases)
    assert got == want, [c for c, g, w in zip(cases, got, want) if g != w]
