"""Arrivals that the products' commits send to both CTAs of a pair land before either CTA ends: the last commit arrives
behind all others, and each CTA waits for it before the cluster's last meeting.  (Source checks: a missing wait is not run.)"""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _kernel():
    text = open(os.path.join(ROOT, "combine_moe_layout_04_gb300", "csrc", "moe_experts.cu")).read()
    at = text.index("__global__ void __launch_bounds__(kThreads<OP>, 1)")
    return text[at:text.index("\n}\n", at)]


def test_the_last_commit_is_behind_all_others():
    kernel = _kernel()
    commits = re.findall(r"tc::commit_pair\((.*?), both\)", kernel)
    assert len(commits) >= 6 and commits[-1] == "smem_u32(&sh.last)"
    assert commits.count("smem_u32(&sh.last)") == 1
    assert len(re.findall(r"commit_pair\(", kernel)) == len(commits)     # (all of them reach both CTAs)


def test_both_ctas_wait_for_it_before_they_end():
    kernel = _kernel()
    first = kernel.index("warp_wait(smem_u32(&sh.last), 0)")
    second = kernel.index("warp_wait(smem_u32(&sh.last), 0)", first + 1)
    assert kernel.rindex("if (warp == 1 && cta == 0)", 0, first) > kernel.index("if (warp == 0)")
    ends = kernel.rindex("__syncthreads();")                             # all of this CTA's warps have done their part
    meeting = kernel.rindex("tc::cluster_sync();")
    assert first < ends < kernel.index("if (warp == 1 && cta == 1", ends) < second < meeting
    assert kernel.index("tc::dealloc_pair(") > meeting
