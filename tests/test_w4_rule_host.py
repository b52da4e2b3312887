"""The rule by which the 4-bit expert layer's L2 runs by token or by expert, compiled for the host from the
library's own header: what it launches fits the chip at once, and no batch's weights are read once per token."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

MAIN = """
#include <cstdio>
#include "moe_internal.h"
int main() {
    long T; int H, I;
    while (std::scanf("%ld %d %d", &T, &H, &I) == 3) std::printf("%d\\n", moe::w4_by_token(T, H, I) ? 1 : 0);
}
"""


@pytest.mark.skipif(not (os.path.exists(HIPCC) or shutil.which(HIPCC)), reason="hipcc not found")
def test_l2_by_token_only_while_its_workgroups_are_resident(tmp_path):
    src, exe = tmp_path / "rule.hip", tmp_path / "rule"
    src.write_text(MAIN)
    subprocess.run([HIPCC, "--offload-arch=gfx950", "--offload-host-only", "-std=c++17", "-I", os.path.join(ROOT, "include"),
                    "-I", os.path.join(ROOT, "token_dispatch_grouped_route_amd", "csrc"), "-o", str(exe), str(src)], check=True, capture_output=True)
    cases = [(T, H, I) for T in (1, 2, 3, 4, 5, 16, 32, 33, 100, 128, 4096) for H in (128, 256, 2048, 7168, 32768) for I in (128, 1408, 2048, 2176)]
    out = subprocess.run([str(exe)], input="\n".join("%d %d %d" % c for c in cases), text=True, capture_output=True, check=True).stdout.split()
    by_token = dict(zip(cases, map(int, out)))
    assert len(out) == len(cases)
    cus, per_cu = 256, 2   # workgroups of eight waves
    for (T, H, I), yes in by_token.items():
        assert not yes or T * H // 16 <= cus * per_cu, (T, H, I)
    # one expert of a hundred tokens, and 32 tokens of one slot each: whatever k is, not a read of W2 per token
    assert not by_token[(100, 256, 128)] and not by_token[(32, 2048, 1408)]
    # the decode step of one token, and the longest reduction that one wave takes
    assert by_token[(1, 2048, 1408)] and by_token[(1, 7168, 2048)] and not by_token[(1, 2048, 2176)]
