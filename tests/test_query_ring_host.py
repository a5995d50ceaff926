"""The ring of query places of the paged attention (csrc/tv_paged_attn.cu), as a protocol on the CPU.

Head blocks of one tile: run r (its tile is tile r) belongs to the four warps with r mod 2; the other four wait for its
queries too, so that no phase of a place's barrier is missed, and go on.  One loading warp issues queries and tiles in
order; copies land in any order.  A wait names a phase by its parity alone.  Every order of events is looked at: a dead
end is a state that is not the last and that nothing leads out of; a wrong one passes a wait before its queries landed."""
import re
from collections import deque
from pathlib import Path

import pytest

SOURCE = Path(__file__).parents[1] / "speculative_tree_verify_gb300" / "csrc" / "tv_paged_attn.cu"
STAGES = int(re.search(r"constexpr int kStages = (\d+);", SOURCE.read_text()).group(1))


def passes(completed, phase):
    """try_wait.parity of phase `phase` (counted from 0) after `completed` phases."""
    return (completed & 1) != (phase & 1)


def search(places, skipper_counts, runs):
    """What goes wrong ('dead end', 'wrong queries') or None.

    State: the loader's step (2 r: queries of run r, 2 r + 1: its tile), which issued queries and tiles have not landed,
    and each group's step in its list: 3 steps for a run of its own (queries, tile, giving the queries' place up at the
    beginning of the join; the join's rest lies before the next step), 1 for one of the other group's."""
    lists = [[(r, k) for r in range(runs) for k in (("q", "t", "f") if r % 2 == g else ("s",))] for g in (0, 1)]
    start = (0, frozenset(), 0, 0)
    seen, todo = {start}, deque([start])
    # steps of each group up to and with its arrivals for run r
    owner_step = {r: lists[r % 2].index((r, "f")) + 1 for r in range(runs)}
    tile_step = {r: lists[r % 2].index((r, "t")) + 1 for r in range(runs)}
    skip_step = {r: lists[1 - r % 2].index((r, "s")) + 1 for r in range(runs)}
    while todo:
        load, flying, *at = todo.popleft()
        at = tuple(at)

        def landed(kind, r):
            return load > 2 * r + (kind == "t") and (kind, r) not in flying

        def given_up(r):   # run r's queries: the place's arrivals are complete
            own = at[r % 2] >= owner_step[r]
            return own and (not skipper_counts or at[1 - r % 2] >= skip_step[r])

        def phases(kind, place, size):
            return sum(landed(kind, r) for r in range(place, runs, size))
        nexts = [(load, flying - {f}) + at for f in flying]
        if load < 2 * runs:
            r, kind = load // 2, "qt"[load % 2]
            old = r - (places if kind == "q" else STAGES)
            if old < 0 or (given_up(old) if kind == "q" else at[old % 2] >= tile_step[old]):
                nexts.append((load + 1, flying | {(kind, r)}) + at)
        for g in (0, 1):
            if at[g] == len(lists[g]):
                continue
            r, kind = lists[g][at[g]]
            if kind in "qs" and not passes(phases("q", r % places, places), r // places):
                continue
            if kind == "t" and not passes(phases("t", r % STAGES, STAGES), r // STAGES):
                continue
            if kind in "qst" and not landed("t" if kind == "t" else "q", r):
                return "wrong queries"
            step = list(at)
            step[g] += 1
            nexts.append((load, flying) + tuple(step))
        if not nexts and not (load == 2 * runs and at == tuple(map(len, lists))):
            return "dead end"
        for s in nexts:
            if s not in seen:
                seen.add(s)
                todo.append(s)
    return None


@pytest.mark.parametrize("places", [2, 3, 4, 5, 6, 8])
def test_every_warp_counts(places):
    assert search(places, True, places + 5) is None


@pytest.mark.parametrize("places", [2, 3, 4, 5, 6])
def test_the_owners_alone_do_not_do(places):
    """What the arrivals of the skipping warps are for."""
    assert search(places, False, places + 5) is not None
