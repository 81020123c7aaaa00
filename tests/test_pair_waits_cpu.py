"""The waits of the CTA-pair kernels, read from their source: a barrier that threads or copies of the other CTA complete
is waited for with acquire at cluster scope."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "dispatch_ffn_combine_gb300", "csrc")
# completed by the other CTA's copies, commits or arrives
CLUSTER = ("full", "empty", "tmem_full", "tmem_empty", "drain", "slot_full", "slot_empty")
WAIT = re.compile(r"\b(\w*(?:wait|test)\w*)\s*\(\s*smem_u32\(&ctl->(\w+)\[?")


@pytest.mark.parametrize("name", ["gemm8.cu", "gemm_pair.cu", "gemm_wgrad.cu", "fused_pair.cu"])
def test_waits_on_the_pair_s_barriers_are_at_cluster_scope(name):
    with open(os.path.join(CSRC, name)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    found = [(m.group(1), m.group(2)) for m in WAIT.finditer(text) if m.group(2) in CLUSTER]
    assert len(found) >= 6
    assert [w for w in found if not w[0].endswith("_cluster")] == []


def test_cluster_waits_acquire_at_cluster_scope():
    """Every wait of that name holds no barrier instruction but those with .acquire.cluster, itself or in what it calls."""
    text = ""
    for name in ("mk_device.cuh", "pair_ring.cuh", "gemm8.cu"):
        with open(os.path.join(CSRC, name)) as f:
            text += re.sub(r"//[^\n]*", "", f.read())
    defs = dict(re.findall(r"__device__ __forceinline__ bool (\w+_cluster)\([^)]*\) \{(.*?)\n\}", text, re.S))
    assert "mbar_try_wait_cluster" in defs and "mbar_wait_bounded_cluster" in defs
    for name, body in defs.items():
        for inst in re.findall(r"mbarrier\.(?:try|test)_wait[\w.:]*", body):
            assert ".acquire.cluster" in inst, (name, inst)
        for call in re.findall(r"\b(mbar_(?:try_wait|test|wait)\w*)\(", body):
            assert call.endswith("_cluster"), (name, call)
