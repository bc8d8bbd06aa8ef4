"""The prompt kernel's barriers in a model (prompt_protocol.py): in no order of its roles does a wait meet a barrier that is two phases
away, and nobody waits forever. Without a GPU."""
import random

import pytest

from tests.prompt_protocol import Lost, run, segments_of


def play(seeds, wide, fp8, boxes, q_box, **how):
    for seed in seeds:
        run(segments_of(random.Random(seed), wide), wide, fp8, boxes, q_box, seed, **how)


@pytest.mark.parametrize("q_box", [False, True])
@pytest.mark.parametrize("fp8", [False, True])
def test_rows_one_by_one(fp8, q_box):
    play(range(200), True, fp8, False, q_box)


def test_the_model_finds_a_loader_that_waits_for_slots_without_filling_them():
    """It may look a page up while the others fill, use and empty its slot, and would wait for the phase after."""
    with pytest.raises(Lost, match="load 0 waits for phase"):
        play(range(200), True, False, False, True, loader_fills=False)


@pytest.mark.parametrize("wide,fp8,boxes,q_box", [(w, f, b, q) for w in (False, True) for f in (False, True) for b in (False, True) for q in (False, True)])
def test_every_form(wide, fp8, boxes, q_box):
    """One and two tiles of rows in turn, values that are looked through, outputs that take one tile's warps longer than the other's."""
    play(range(1000, 1150), wide, fp8, boxes, q_box)


def test_the_model_finds_second_tiles_warps_that_follow_scores():
    with pytest.raises(Lost, match="softmax 1"):
        play(range(200), False, False, True, True, second_waits="scores")
