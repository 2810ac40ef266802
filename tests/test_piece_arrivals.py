"""The pieces of widened integers that one CTA of a pair hands to the other: the arrival releases this CTA's shared memory
at cluster scope behind the fences of both other kinds of memory, the wait acquires at cluster scope; and the counts of
stages and pieces keep every widening group on the same barriers.  (Source checks: a missing order is not run.)"""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _text():
    return open(os.path.join(ROOT, "combine_moe_layout_04_gb300", "csrc", "moe_experts.cu")).read()


def test_pieces_are_handed_over_at_cluster_scope():
    text = _text()
    assert re.findall(r"tc::(arrive_\w+)\(made0", text) == ["arrive_cluster_smem"]
    assert re.findall(r"(\w+)\(made \+", text) == ["mbar_init", "warp_wait_cluster"]
    # what comes before the arrival: shared memory to the tensor core's proxy, tensor memory written, then the fence
    before = text[text.index("widen(sa, half"):text.index("tc::arrive_cluster_smem(made0")]
    order = [before.index(s) for s in ("fence_proxy_async_smem()", "tc::wait_st()", "tc::fence_before_sync()", "__syncwarp()")]
    assert order == sorted(order)
    after = text[text.index("warp_wait_cluster(made"):]
    assert after.index("tc::fence_after_sync()") < after.index("tc::mma_tmem_pair")


def test_groups_keep_their_barriers():
    """Two sets of two groups take stages in turn: an even number of stages and two pieces to each in a multiple of
    four give every barrier to one set."""
    text = _text()
    assert "static_assert(kTop<kForward8> + kPieces * kPieceColumns == 512 && kPieces % 4 == 0)" in text
    assert "if (kIntegers<OP> && kInTurn<OP>) cut.stages &= ~1;" in text
    for columns in (128, 256):
        stages = (195 * 1024 - 4 * columns // 2 * 128) // (128 * 128 + columns // 2 * 128) & ~1
        assert stages >= 4
        owner = {}
        for use in range(8 * stages):
            for kind, slot in (("stage", use % stages), ("piece", 2 * use % 4), ("piece", (2 * use + 1) % 4)):
                assert owner.setdefault((kind, slot), use % 2) == use % 2
