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
