"""The recurrence's slots: a block's feeding warp writes a tile into a slot that the tile S before has left.  Every order in
which the block's warps can come, with the arrivals that the source counts: no warp may find a slot two uses on (its wait
for the slot's barrier, by parity, would not end then)."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "packed_sequence_varlen_gb300", "csrc")


def source():
    with open(os.path.join(CSRC, "scan.cu")) as f:
        text = f.read()
    body = text[text.index("void resolve("):]
    body = body[:body.index("\n}\n")]
    count = re.search(r"mbar_init\(smem_u32\(&sh\.empty\[s\]\), ([^)]*)\)", text).group(1)
    resolvers = int(re.search(r"constexpr int kResolvers = (\d+)", text).group(1))
    counted, arrives = "kResolvers" in count, "mbar_arrive(smem_u32(&sh.empty[" in body
    assert counted == arrives                                 # or no slot would ever be given back
    stages = {int(s) for s in re.findall(r"Shape<\d+, \d+, \d+, (\d+),", text)}
    return counted, resolvers, stages


def lapped(counted, resolvers, S, tiles=14):
    """A reachable state in which a resolving warp's next slot has been filled again since, or None.  A state: tiles fed,
    tiles that the working warps have left, and each resolving warp's next tile."""
    todo, seen = [(0, 0, (0,) * resolvers)], set()
    while todo:
        state = todo.pop()
        if state in seen:
            continue
        seen.add(state)
        fed, left, at = state
        if any(n < fed and (fed - 1 - n) // S >= 1 for n in at):
            return state
        # the slot of tile fed - S is given back by the working warps, and by who else is counted
        if fed < tiles and (fed < S or left > fed - S and (not counted or min(at) > fed - S)):
            todo.append((fed + 1, left, at))
        # a tile is left when its state is there (its resolving warp is past it) and the next one's maps are formed
        if left < fed and at[left % resolvers] > left and (left + 1 < fed or fed == tiles):
            todo.append((fed, left + 1, at))
        for r in range(resolvers):
            if at[r] < fed:
                todo.append((fed, left, at[:r] + (at[r] + 1,) + at[r + 1:]))
    assert any(left == tiles for _, left, _ in seen)          # and every tile can be done
    return None


def test_the_model_finds_a_late_warp():
    """With the working warps alone counted, a resolving warp that is held back is lapped."""
    assert lapped(False, 2, 3) is not None


@pytest.mark.parametrize("tiles", [1, 2, 3, 7, 14])
def test_no_warp_is_lapped(tiles):
    counted, resolvers, stages = source()
    assert stages
    for S in stages:
        assert lapped(counted, resolvers, S, tiles) is None
