"""Barrier arrivals that hand memory of a cluster from one CTA to another order it at cluster scope: without a
scope, an arrival and a wait order this CTA's memory alone.  (A source check: a missing order is not run.)"""
import glob
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "combine_moe_layout_04_gb300", "csrc")


def _text():
    return {os.path.basename(p): open(p).read() for p in sorted(glob.glob(os.path.join(CSRC, "*.cu*")))}


def test_arrivals_on_other_ctas_release_at_cluster_scope():
    """A release, or a relaxed arrival behind a release fence or (tensor memory alone) the tensor core's own fence."""
    bodies = []
    for name, text in _text().items():
        for m in re.finditer(r"void (\w+)\(uint32_t bar[^{]*\{\n(.*?)\n\}", text, re.S):
            if re.search(r"mbarrier\.arrive[^\"]*shared::cluster", m.group(2)) and "expect_tx" not in m.group(2):
                bodies.append((m.group(1), m.group(2)))
    # (arrivals that only announce bytes of a copy hand nothing over: the copy itself completes the phase)
    assert bodies
    for name, body in bodies:
        assert re.search(r"mbarrier\.arrive\.(release|relaxed)\.cluster\.shared::cluster", body), (name, body)
        if "relaxed" in body and not name.endswith("_tmem"):
            assert "fence.release.sync_restrict::shared::cta.cluster" in body, (name, body)
    text = _text()["moe_experts.cu"]
    kinds = {b: re.findall(r"tc::(arrive_\w+)\(.*%s" % pattern, text) for b, pattern in
             (("seen", r"link\.seen"), ("ready", r"link\.ready"), ("free", r"sh\.free"), ("stage", r"full0 \+ 8 \* at"))}
    # read from other CTAs' shared memory; written in this CTA's; tensor memory; cleared in this CTA's
    assert kinds == {"seen": ["arrive_cluster"], "ready": ["arrive_cluster_smem"], "free": ["arrive_cluster_tmem"],
                     "stage": ["arrive_cluster_smem"]}


def test_waits_for_other_ctas_acquire_at_cluster_scope():
    """The waits that such arrivals end: tensor memory stored (free, over), a stage cleared, a block read (seen) or
    written (ready) by another CTA."""
    text = _text()["moe_experts.cu"]
    for barrier in ("free", "over"):
        waits = re.findall(r"(\w+)\(smem_u32\(&sh\.%s\[" % barrier, text)
        assert [w for w in waits if "wait" in w] == ["warp_wait_cluster"], (barrier, waits)
    for barrier in ("seen", "ready"):
        waits = re.findall(r"(\w+)\(link\.%s, " % barrier, text)
        assert [w for w in waits if "wait" in w] == ["try_wait_cluster"], (barrier, waits)
    assert re.search(r"cleared \? warp_wait_cluster\(full \+ 8 \* ring\.stage", text)
