"""A CPU model of the softmax warps of the paged attention's tensor-core kernel where a wait for a piece's note
runs out in some of them: every warp must come to its end, since the named barriers that two warps of a quarter
meet at have no limit. The rule that the model runs with is the one that the kernel's source has."""

import itertools
import os
import re

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                      "mtp_speculative_decoding_spec_gb300", "csrc", "trunk", "attn_tc.cuh")
QUADS, PIECES = 2, (1, 2, 3)  # blocks of each piece


def kernel_agrees():
    """Whether a piece is taken by what a barrier of all eight softmax warps says."""
    text = open(SOURCE).read()
    softmax = text[text.index("- softmax\n"):]
    return re.search(r"if constexpr \(kPaged<P>\)\s+more = agreed\(more\);", softmax) is not None \
        and "bar.red.and.pred a, 13, 256, m;" in softmax \
        and len(re.findall(r"next_piece\(\)", softmax)) == len(re.findall(r"more = next_piece\(\);", softmax)) == 2 \
        and softmax.count("more = load_q(a, more);") == 1


def warp(half, quad, notes, agree):
    """What a warp comes to, one thing after another: it yields (barrier, warps it takes, whether it waits) and
    gets what the barrier says of its own words."""
    done = False
    for n, blocks in enumerate(PIECES + (0,)):
        more = blocks > 0 and notes[n]
        if agree:
            more = yield ("all", 2 * QUADS, True, more)
        if done:
            yield ("out", quad), 2, True, True
        if not more:
            return
        for blk in range(blocks):
            if blk % 2 != half:
                continue
            if blk > 0:
                yield ("ref", 1 - half, quad), 2, True, True
            if blk + 1 < blocks:
                yield ("ref", half, quad), 2, False, True
        done = True


def ends(outcomes, agree):
    """outcomes[warp][piece]: whether the warp had the piece's note in time."""
    warps = [warp(h, q, outcomes[h * QUADS + q], agree) for h in range(2) for q in range(QUADS)]
    wants = [next(w, None) for w in warps]
    here = {}  # barrier: its arrivals, of warps that wait (their number) and that do not (None)
    waiting = set()
    while any(x is not None for x in wants):
        moved = False
        for i, x in enumerate(wants):
            if x is None or i in waiting:
                continue
            moved = True
            name, count, waits, word = x
            here.setdefault(name, []).append((i if waits else None, word))
            if waits:
                waiting.add(i)
            else:
                wants[i] = next(warps[i], None)
            if len(here[name]) == count:
                said = all(w for _, w in here[name])
                for j in [j for j, _ in here.pop(name) if j is not None]:
                    waiting.discard(j)
                    try:
                        wants[j] = warps[j].send(said)
                    except StopIteration:
                        wants[j] = None
        if not moved:
            return False
    return True


def outcomes():
    """Each warp has the notes up to some piece and none after the wait that ran out."""
    one = [[n < k for n in range(len(PIECES))] for k in range(len(PIECES) + 1)]
    return itertools.product(one, repeat=2 * QUADS)


def test_the_model_ends_where_all_have_their_notes():
    assert ends([[True] * len(PIECES)] * (2 * QUADS), False)
    assert ends([[True] * len(PIECES)] * (2 * QUADS), True)


def test_the_model_sees_warps_that_part():
    assert any(not ends(o, False) for o in outcomes())


def test_every_softmax_warp_ends_whatever_waits_run_out():
    agree = kernel_agrees()
    assert all(ends(o, agree) for o in outcomes())
