"""The barriers of a d = 64 Q tile's scores and weights, as a model that takes every order of events.

One Q tile: an MMA warp that issues S(n) = Q K^T, waits for the weights P(n - 1), issues P(n - 1) V; a tensor pipe that finishes
these in order and completes a phase of a barrier for each; softmax warps that wait for S(n), sometimes for the product before the last (to
rescale O), and arrive for P(n).  A wait tells phases apart by one bit; every wait may run out, after which each actor
leaves at its next wait that is not yet satisfied."""
import os
import re

import pytest

WARPS, TILES = 2, 5
CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "attention_forward_07_gb300", "csrc")


def _programs(bars, meet):
    """Steps of the MMA warp and of a softmax warp: ("wait", barrier, parity, phases that must be complete) and others."""
    bar = lambda n: n % bars           # noqa: E731
    nth = lambda n: n // bars          # noqa: E731
    mma = []
    for n in range(TILES + 1):
        if n < TILES:
            mma.append(("issue", ("S", bar(n))))
        if n:
            mma += [("wait", ("P", bar(n - 1)), nth(n - 1)), ("issue", ("OPV", 0))]
    soft = []
    for n in range(TILES):
        soft.append(("wait", ("S", bar(n)), nth(n)))
        if n:
            soft.append(("maybe", ("OPV", 0), n - 1))
        if meet:
            soft.append(("meet", n))
        soft.append(("arrive", ("P", bar(n)), nth(n)))
    return mma, soft


def explore(bars, meet):
    """Runs the model over every order: (wrong phases or arrivals seen, states in which somebody waits for ever)."""
    mma, soft = _programs(bars, meet)
    progs = [mma] + [soft] * WARPS
    start = ((0,) * len(progs), (), (), (0,) * bars, False)  # places, issued, phases complete, arrivals of P's, aborted
    wrong, stuck, seen, todo = set(), 0, {start}, [start]
    while todo:
        pcs, pipe, phases, arrived, aborted = state = todo.pop()
        done = dict(phases)
        count = lambda b: done.get(b, 0)  # noqa: E731
        after = []
        if pipe:  # the tensor pipe finishes its oldest instruction
            after.append((pcs, pipe[1:], tuple(sorted({**done, pipe[0]: count(pipe[0]) + 1}.items())), arrived, aborted))
        for a, prog in enumerate(progs):
            pc = pcs[a]
            if pc >= len(prog):
                continue
            step = prog[pc]
            go = lambda to, ph=phases, ar=arrived, pp=pipe, ab=aborted: after.append((pcs[:a] + (to,) + pcs[a + 1:], pp, ph, ar, ab))  # noqa: E731
            if step[0] == "issue":
                go(pc + 1, pp=pipe + (step[1],))
            elif step[0] == "arrive":
                kind, b = step[1]
                if count(step[1]) != step[2]:
                    wrong.add(("arrival in another phase", step))
                n = arrived[b] + 1
                full = n == WARPS
                go(pc + 1, ar=arrived[:b] + (0 if full else n,) + arrived[b + 1:],
                   ph=tuple(sorted({**done, step[1]: count(step[1]) + 1}.items())) if full else phases)
            elif step[0] == "meet":  # all softmax warps or none: waits without limit
                if all(pcs[w] < len(soft) and (pcs[w] > pc or soft[pcs[w]] == step) for w in range(1, 1 + WARPS)):
                    go(pc + 1)
            else:
                if step[0] == "maybe":
                    go(pc + 1)
                if (count(step[1]) & 1) != (step[2] & 1):  # the phase of that parity is over: what the hardware can tell
                    if count(step[1]) != step[2] + 1:
                        wrong.add(("wait passed", step))
                    go(pc + 1)
                else:  # runs out, or sees that another has
                    go(len(prog), ab=True)
        if not after and any(pc < len(p) for pc, p in zip(pcs, progs)):
            stuck += 1
        for s in after:
            if s not in seen:
                seen.add(s)
                todo.append(s)
    return wrong, stuck


def test_two_barriers_by_turns_need_no_meeting():
    wrong, stuck = explore(bars=2, meet=False)
    assert not wrong and not stuck


def test_a_meeting_without_limit_never_ends_once_a_warp_has_left():
    """Why there is none: a warp that gave up never comes."""
    assert explore(bars=2, meet=True)[1] > 0


def test_the_model_sees_a_shared_barrier():
    """With one barrier for all weights a warp that is ahead would arrive twice in a phase."""
    assert explore(bars=1, meet=False)[0]


@pytest.mark.parametrize("name", ["attn_fwd.cu", "paged_tile.cu", "roles.cuh", "ptx.cuh"])
def test_roles_have_no_barrier_without_a_limit(name):
    """The kernels whose warps may give up: no named barrier, and __syncthreads only in the kernels' own bodies, outside the
    roles, which every thread reaches."""
    with open(os.path.join(CSRC, name), encoding="utf-8") as f:
        text = re.sub(r"//.*", "", f.read())
    assert "bar.sync" not in text and "named_bar" not in text
    for body in re.findall(r"_role\(.*?\n}\n", text, flags=re.S):
        if "template" in body or "__device__" in body:
            body = body.split("\n}\n")[0]
        assert "__syncthreads" not in body.split("__global__")[0]
