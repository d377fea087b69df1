"""Host model of the second 4-bit product's epilogue (mx4_gemm.cu): two warps take the same tiles, wait
for each one's accumulator with a limit, and meet in two barriers per tile that holds rows.  A
wait may expire for one of them and pass for the other; no interleaving may leave one at a
barrier that the other never reaches."""
import itertools

import pytest

WAIT, FIRST, SECOND, OUT = range(4)


def stuck_states(rows, leave_alone):
    """States in which a warp is not out and nothing can move.  rows[t]: tile t holds rows (else it
    is skipped).  leave_alone: a warp whose wait expired breaks off at once (a planted mistake);
    otherwise it goes on, gives its verdict at the next barrier, and both break there."""
    start = ((0, WAIT, True), (0, WAIT, True))  # tile, place, no wait expired yet
    seen, todo, stuck = {start}, [start], []
    while todo:
        pair = todo.pop()
        moves = []
        for i, (t, place, good) in enumerate(pair):
            if place != WAIT:
                continue
            if t == len(rows):
                to = [(t, OUT, good)]
            else:
                to = []
                for g in ([True, False] if good else [False]):
                    if leave_alone and not g:
                        to.append((t, OUT, g))
                    else:
                        to.append((t, FIRST, g) if rows[t] else (t + 1, WAIT, g))
            moves += [pair[:i] + (s,) + pair[i + 1:] for s in to]
        (ta, pa, ga), (tb, pb, gb) = pair
        if pa == pb == FIRST:
            assert ta == tb
            moves.append(((ta, SECOND, ga), (tb, SECOND, gb)))
        if pa == pb == SECOND:
            moves.append(((ta + 1, WAIT, ga), (tb + 1, WAIT, gb)) if ga and gb else
                         ((ta, OUT, ga), (tb, OUT, gb)))
        if not moves and (pa, pb) != (OUT, OUT):
            stuck.append(pair)
        for m in moves:
            if m not in seen:
                seen.add(m)
                todo.append(m)
    return stuck


@pytest.mark.parametrize("rows", list(itertools.product((True, False), repeat=4)))
def test_pairs_leave_together(rows):
    assert not stuck_states(rows, leave_alone=False)
    if any(rows):  # the model sees the hang where a warp leaves by itself
        assert stuck_states(rows, leave_alone=True)
