"""The two softmax warps that share 32 rows of a query tile in the 4-bit prefill meet at a barrier of their own in every key
tile. When a wait has given up, both must leave at the same tile: a warp that left alone would leave the other one at a
barrier for ever. Each tells the other which tile it stopped at, before that tile's barrier, and looks behind it. Every
order of the two warps' steps is walked here, with waits that may give up at any tile. CPU only."""
import pathlib
import re

import pytest

TILES = 4


def leaves(stop, j):
    """The warp leaves behind the barrier of tile j; `stop` is the tile (+ 1) that a warp last stopped at, 0 for none."""
    return stop == j + 1


def leaves_at_any(stop, j):
    return stop != 0


def stuck(rule):
    """Whether some order of steps leaves a warp at a barrier where the other does not come, or comes for another reason."""
    # a warp: (what it does next, tile); at the end both meet twice more, to add their sums up
    seen, todo = set(), [(("wait", 0), ("wait", 0), 0)]
    while todo:
        state = todo.pop()
        if state in seen:
            continue
        seen.add(state)
        *warps, stop = state
        at = [w[0] for w in warps]
        barriers = [w for w in warps if w[0] in ("tile", "end", "end again")]
        if len(barriers) == 2:
            if warps[0] != warps[1]:
                return True
            what, j = warps[0]
            then = {"tile": ("look", j), "end": ("end again", TILES), "end again": ("done", TILES)}[what]
            todo.append((then, then, stop))
            continue
        if barriers and "done" in at:
            return True
        for i in (0, 1):
            what, j = warps[i]
            other = warps[1 - i]

            def step(w, s=stop):
                todo.append((w, other, s) if i == 0 else (other, w, s))

            if what == "wait" and j == TILES:
                step(("end", TILES))
            elif what == "wait":
                if other[1] >= j:  # the scores of tile j come when both have written the weights of tile j - 1
                    step(("tile", j))
                step(("tile", j), j + 1)  # gave up
            elif what == "look":
                step(("end", TILES) if rule(stop, j) else ("wait", j + 1))
    return False


def test_both_warps_leave_at_the_same_tile():
    assert not stuck(leaves)
    assert stuck(leaves_at_any)  # (what the walk finds)


@pytest.mark.parametrize("flag", ["stopped", "grow_at"])
def test_the_kernel_names_the_tile(flag):
    source = (pathlib.Path(__file__).resolve().parent.parent / "paged_kv_cache_238_gb300" / "csrc" / "prefill_fp4.cu").read_text()
    uses = re.findall(rf"&{flag}\[x\]\[quad\]\)\s*(==|!=|=)\s*([^;)]+)", source)
    assert uses and all(value.strip() == "j + 1" for _, value in uses), uses
