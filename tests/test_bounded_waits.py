"""Warps with roles of their own meet only where a wait has a limit (mbarriers) or the whole block does (__syncthreads, which
every warp reaches after its own waits): no named barriers, at which some warps of a block could stay for others that a
wait which ran out has sent on."""
import glob
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_no_named_barriers():
    sources = [p for end in ("*.cu", "*.cuh", "ops/*.cuh") for p in
               glob.glob(os.path.join(ROOT, "kernelized_linear_attention_gb300", "csrc", end))]
    assert len(sources) > 10
    for path in sources:
        with open(path) as f:
            code = re.sub(r"//.*", "", f.read())
        found = re.findall(r"named_sync\w*|\bbar(?:rier)?(?:\.cta)?\.(?:sync|red|arrive)\b[^;]*", code)
        assert not found, (path, found)
