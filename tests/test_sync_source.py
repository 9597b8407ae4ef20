"""Ordering between threads that no result shows while the hardware is kind:
the sources are held to the form that the PTX memory model asks for."""

import re
from pathlib import Path

CSRC = Path(__file__).resolve().parent.parent / "sparse_attention_token_03_b200" / "csrc"


def code(name: str) -> str:
    """A source without its line comments."""
    return re.sub(r"//[^\n]*", "", (CSRC / name).read_text())


def test_votes_over_barriers_are_followed_by_a_warp_barrier():
    # a vote is no memory barrier: a lane that learns by __ballot_sync that
    # another lane's mbarrier test passed has acquired nothing itself
    found = 0
    for f in sorted(CSRC.glob("*.cu*")):
        for m in re.finditer(r"__ballot_sync\([^;]*mbar_t\w+\([^;]*;\s*(\w+)", code(f.name)):
            found += 1
            assert m.group(1) == "__syncwarp", f"{f.name}: {m.group(0)}"
    assert found


def test_a_pair_of_blocks_orders_memory_at_cluster_scope():
    # one block's MMAs read the other's shared memory: arrivals on its barriers
    # release and every wait acquires at cluster scope
    src = code("dsa_attend_pair.cu")
    shared = code("dsa_attend.cuh")
    remote = [m.start() for m in re.finditer(r"mbarrier\.arrive[\w.]*\.shared::cluster", src)]
    assert remote
    for at in remote:
        text = src[max(0, at - 120):at + 60]
        assert ".release.cluster.shared::cluster" in text or "fence.release.sync_restrict::shared::cta.cluster" in text, text
    own = {"kBarListed", "kBarTaken", "kBarCF", "kBarCE"}      # only this block's warps arrive on these
    plain = re.findall(r"\bwait_(?:bar|any)\(bar\((\w+)", src)
    assert set(plain) <= own | {"b"}, plain                    # b: the argument of wait_own
    assert set(re.findall(r"\bwait_own\((\w+)", src)) <= own
    assert "wait_bar<true>(" in src and "wait_any<true>(" in src
    assert "fence.acquire.sync_restrict::shared::cluster.cluster" in shared or "try_wait.parity.acquire.cluster" in shared
