"""The meetings at a unit's end in kv_attend_prompt (256 dimensions), on the CPU: every order in which two warps can take
their steps, with barriers that hold one phase at a time."""
import ctypes
import os
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
UNITS = 5


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("meet") / "prompt.so")
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-o", so, os.path.join(HERE, "prompt_host.cpp")])
    return ctypes.CDLL(so)


def explore(barrier, parity):
    """Orders in which both warps get stuck, or in which one goes on although the other has not come as often. barrier(time, slot)
    counts to one, so that an arrival ends its phase; a wait for a parity goes on while a phase of the other parity is open."""
    steps = [[(kind, unit, time) for unit in range(UNITS) for time in range(2) for kind in ("arrive", "wait")] for _ in range(2)]
    seen, todo, faults = set(), [(0, 0)], []
    while todo:
        at = todo.pop()
        if at in seen:
            continue
        seen.add(at)
        ended = {}
        for slot in range(2):
            for kind, unit, time in steps[slot][: at[slot]]:
                if kind == "arrive":
                    ended[barrier(time, slot)] = ended.get(barrier(time, slot), 0) + 1
        moves = []
        for slot in range(2):
            if at[slot] == len(steps[slot]):
                continue
            kind, unit, time = steps[slot][at[slot]]
            if kind == "wait":
                if ended.get(barrier(time, slot ^ 1), 0) % 2 == parity(time, unit):
                    continue
                if ("arrive", unit, time) not in steps[slot ^ 1][: at[slot ^ 1]]:
                    faults.append(("early", at))
            moves.append(tuple(a + (s == slot) for s, a in enumerate(at)))
        if not moves and at != (len(steps[0]), len(steps[1])):
            faults.append(("stuck", at))
        todo += moves
    return faults


def test_no_order_of_steps_keeps_a_warp(host):
    for quarter in range(4):
        assert not explore(lambda time, slot: host.meet_barrier(time, slot, quarter), host.meet_parity)


def test_meetings_have_barriers_of_their_own(host):
    used = [host.meet_barrier(time, slot, quarter) for time in range(2) for slot in range(2) for quarter in range(4)]
    assert sorted(used) == list(range(host.meets()))


def test_the_exploration_finds_an_overrun_phase():
    """Both meetings of a unit on one barrier: a warp may arrive twice before the other has looked once."""
    assert any(kind == "stuck" for kind, _ in explore(lambda time, slot: slot, lambda time, unit: time))
