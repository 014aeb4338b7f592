"""The scope of waits for other CTAs' stores, read from the source: a barrier
on which CTAs of a cluster count their stores into one another's shared memory
is awaited with acquire at cluster scope (the default is the CTA's own).  CPU
only."""

import glob
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "block_scaled_precision_02_gb300", "csrc")
CLUSTER_SCOPE = ("mbar_wait_sleep<true>", "mbar_wait_suspend")


def test_barriers_that_peers_complete_are_awaited_at_cluster_scope():
    counted = 0
    for path in glob.glob(os.path.join(CSRC, "*.cu")):
        text = open(path).read()
        bars = set(re.findall(r"st_async_f2\(smem_u32\([^;]*?\),\s*smem_u32\(&(\w+)\[", text))
        for bar in bars:
            waits = re.findall(r"(mbar_(?:try_)?wait\w*(?:<\w+>)?)\(smem_u32\(&" + bar + r"\[", text)
            assert waits, (path, bar)
            assert set(waits) <= set(CLUSTER_SCOPE), (path, bar, waits)
            counted += 1
    assert counted >= 2              # the norm's statistics, the loss's sums
    common = open(os.path.join(CSRC, "common.cuh")).read()
    body = common[common.index("bool mbar_try_wait_cl_sleep"):]
    assert "try_wait.parity.acquire.cluster" in body[:body.index("return")]
