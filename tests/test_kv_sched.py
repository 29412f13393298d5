"""The whole-number arithmetic that deals the attention's work to workgroups,
compiled for the host (no GPU) and compared with Python's integers."""
import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PROGRAM = r"""
#include <cstdio>
#include "kv_sched.h"
int main() {
  long long off, head;
  while (std::scanf("%lld %lld", &off, &head) == 2) std::printf("%d\n", mlora::sched_head(off, head));
}
"""


def _prompt_line(tokens, group, rows=128, over=3):
    """Line length of one key/value head of a causal prompt."""
    return sum(-(-(min((t + 1) * rows, tokens * group) // group) // 64) + over
               for t in range(-(-tokens * group // rows)))


def test_the_head_of_a_place(tmp_path):
    """Lines of heads on both sides of 2^31 and 2^32, the 3 M token prompt of 8
    query heads to a key/value head among them."""
    hipcc = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(hipcc):
        pytest.skip("hipcc not found")
    src, exe = tmp_path / "head.hip", tmp_path / "head"
    src.write_text(PROGRAM)
    subprocess.run([hipcc, "-O1", "-std=c++17", "--offload-host-only", "-w", "-I",
                    os.path.join(ROOT, "lora_serving_mlora_amd", "csrc"), str(src), "-o", str(exe)], check=True)
    long = _prompt_line(3_000_000, 8)
    assert long > 1 << 32
    rng = random.Random(1)
    heads = [1, 2, 7, 1 << 20, (1 << 31) - 1, 1 << 31, (1 << 32) - 1, 1 << 32, (1 << 32) + 1, 1 << 35, long]
    pairs = [(k * h + d, h) for h in heads for k in (0, 1, 2, 5, 1023) for d in (0, 1, h // 2, h - 1) if d < h]
    pairs += [(rng.randrange(8 * long), long) for _ in range(500)]
    pairs += [((rng.randrange(1024) * h + rng.randrange(h)), h) for h in (rng.randrange(1, 1 << 36) for _ in range(500))]
    out = subprocess.run([str(exe)], input="\n".join(f"{a} {b}" for a, b in pairs), capture_output=True, text=True,
                         check=True).stdout.split()
    assert [int(x) for x in out] == [a // b for a, b in pairs]
