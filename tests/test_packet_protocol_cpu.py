"""The hand-over of P between the two CTAs of a decode's pair, as a model whose steps are taken in random order: a sender with a few
staging slots, asynchronous copies that land some time after they are sent, a receiver with a few slots, and the forwarder
that tells the sender what has landed and what is free.  The model says which waits keep a slot from being overwritten too early,
and that they never wait for one another.
"""
import random

import pytest


def _run(tiles, staging, receive, wait_for_landing, seed):
    """Takes the steps of all roles in random order; returns the number of slots that were overwritten too early (None: all wait)."""
    rng = random.Random(seed)
    wrote = sent = landed = told = used = freed = 0      # tiles so far: staged, sent, landed, told to the sender, consumed, given back
    forward = 0                                          # the forwarder's next step: 2 T: "T has landed"; 2 T + 1: "T - 1 is free"
    early = 0
    while used < tiles or told < tiles:
        steps = []
        if wrote < tiles and wrote == sent and (not wait_for_landing or told >= wrote - staging + 1):
            steps.append("write")                        # into staging slot `wrote % staging`
        if sent < wrote and freed >= sent - receive + 1:
            steps.append("send")
        if landed < sent:
            steps.append("land")                         # (copies of different tiles land in order: one barrier a slot counts them)
        if used < landed:
            steps.append("use")
        if forward < 2 * tiles:
            tile = forward // 2
            if forward % 2 == 0 and landed > tile or forward % 2 == 1 and used >= tile:
                steps.append("forward")
        if not steps:
            return None
        step = rng.choice(steps)
        if step == "write":
            early += landed < wrote - staging + 1        # the tile that was staged there has not landed
            wrote += 1
        elif step == "send":
            early += used < sent - receive + 1           # the tile that lies there has not been used
            sent += 1
        elif step == "land":
            landed += 1
        elif step == "use":
            used += 1
        else:
            if forward % 2 == 0:
                told = forward // 2 + 1
            else:
                freed = max(freed, forward // 2)
            forward += 1
    return early


@pytest.mark.parametrize("staging,receive", [(1, 2), (2, 4)])      # the 4-bit decode's, the other decodes'
@pytest.mark.parametrize("tiles", [1, 2, 3, 7, 40])
def test_no_slot_is_overwritten_early_and_nothing_waits_for_ever(staging, receive, tiles):
    for seed in range(300):
        assert _run(tiles, staging, receive, True, seed) == 0


@pytest.mark.parametrize("staging,receive", [(1, 2), (2, 4)])
def test_without_the_word_that_a_packet_has_landed_slots_are_overwritten(staging, receive):
    assert sum(_run(40, staging, receive, False, seed) for seed in range(50)) > 0
