"""CTA pairs: what the odd CTA's relay hands to the even CTA lies in shared memory,
so its arrival releases at cluster scope.  No run shows the difference (the memory
model asks for it, the hardware may order the stores anyway), so the source is read."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "int4_gemm_gb300", "csrc")


def _source(name):
    with open(os.path.join(CSRC, name)) as f:
        return f.read()


def _releases_at_cluster_scope(helper):
    """The arrival's own release, or one of shared memory by a fence in front of it."""
    body = re.search(r"void %s\(uint32_t \w+\) \{(.*?)\n\}" % helper, _source("common.cuh"), re.S).group(1)
    fence = body.find("fence.release.sync_restrict::shared::cta.cluster;")
    arrive = re.search(r"mbarrier\.arrive\.(\w+)\.cluster\.shared::cluster", body)
    return bool(arrive) and (arrive.group(1) == "release" or 0 <= fence < arrive.start())


@pytest.mark.parametrize("name", ["int8.cu", "w4a8.cu", "fp8.cu"])
def test_relay_releases_at_cluster_scope(name):
    parts = _source(name).split("relay (odd CTA)\n")
    assert len(parts) == 2
    relay = parts[1][:parts[1].index("// ----")]
    arrivals = re.findall(r"\b(mbar_arrive\w*)\(", relay)
    assert len(arrivals) == 1
    assert _releases_at_cluster_scope(arrivals[0])


def test_scale_writers_hand_the_stage_over_at_cluster_scope():
    """The FP4 product has no relay: its scale writers tell the even CTA that the odd
    one's stage, codes in shared memory among it, is there."""
    source = _source("w4a4.cu")
    handing = re.findall(r"if \(lane == 0\) (\w+)\(&sm->sf_full\[stage\]\)", source)
    assert len(handing) == 1
    helper = re.search(r"auto %s = \[&\]\(uint64_t\* bar\) \{\s*if constexpr \(P2\) (\w+)\(" % handing[0], source).group(1)
    assert _releases_at_cluster_scope(helper)
    # and the wait for it acquires at cluster scope
    assert len(re.findall(r"mbar_wait<P2>\(smem_u32\(&sm->sf_full\[stage\]\)", source)) == 1


@pytest.mark.parametrize("name,wait", [("w4a8.cu", r"mbar_wait<true>\(smem_u32\(&sm->pair_full\[stage\]\)"),
                                       ("fp8.cu", r"mbar_wait<true>\(smem_u32\(&sm->pair_full\[stage\]\)"),
                                       ("int8.cu", r"warp_wait<kPair>\(bar0 \+ slot \* 8")])
def test_issuer_acquires_at_cluster_scope(name, wait):
    assert len(re.findall(wait, _source(name))) == 1
