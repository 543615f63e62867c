"""The hand-overs of packed_dq_kernel's steps, as a model whose every order of events is tried.

A barrier of several arrivals says that a step is complete only if no arrival for a later
step can be counted for it.  On the GPU a mistake there is one wrong quarter of a dS tile,
now and then, without an error word.  So the roles are written down here as lists of events
(two elementwise warps stand for the sixteen), with the kernel's barriers, and which of
its barriers a step's dS arrives on is read from the source."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "layerwise_weight_offload_slot_gb300", "csrc")
WARPS = 2


def barriers_of_ds():
    """How many barriers the steps' dS arrive on in turn, from the arrival and the wait in packed_dq_kernel."""
    with open(os.path.join(CSRC, "attention_packed_bwd.cu")) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    body = re.search(r"packed_dq_kernel\(const __grid_constant__.*?\n}\n", text, re.S).group()
    turn = r"m\.e0(?: \+ 8 \* \((\w+) & 1\))?"
    arrive = re.findall(r"mbar_arrive\(" + turn + r"\)", body)
    wait = re.findall(r"warp_wait\(" + turn + r", (?:\(\w+ >> 1\)|\w+) & 1, abort_flag\)", body)
    assert len(arrive) == 1 and len(wait) == 1 and bool(arrive[0]) == bool(wait[0])
    return 2 if arrive[0] else 1


def roles(items, turns):
    """Lists of events: ("wait", barrier, phase), ("arrive", barrier), ("write", place, warp, step), ("read", place,
    step) by which dQ takes dS.  Phase n of a barrier is the n-th time that all its arrivals came.  Steps are counted on.
    That a dQ is complete shows on the barrier of its K slot, one of three in turn."""
    issue, grad, warps = [], [], [[] for _ in range(WARPS)]
    s = 0
    for i, n in enumerate(items):
        for j in range(n):
            t = s + j
            # S takes the last one's place, and goes behind dQ two steps before within an item
            if t > 0:
                issue.append(("wait", "s_read", t - 1))
            if j >= 2:
                issue.append(("wait", ("dq", (t - 2) % 3), (t - 2) // 3))
            issue.append(("arrive", "s_full"))
            if t > 0:
                issue.append(("wait", "d_read", t - 1))
            issue.append(("arrive", "d_full"))
            # dQ reads from its issue to its completion
            grad += [("wait", ("e0", t % turns), t // turns), ("read", t % 2, t), ("read", t % 2, t), ("arrive", ("dq", t % 3))]
            for w, events in enumerate(warps):
                events += [("wait", "s_full", t), ("arrive", "s_read"), ("wait", "d_full", t), ("arrive", "d_read"),
                           ("write", t % 2, w, t), ("arrive", ("e0", t % turns))]
        grad.append(("arrive", "done"))
        for events in warps:
            events.append(("wait", "done", i))
        s += n
    return [issue, grad] + warps


def arrivals(barrier):
    return WARPS if barrier in ("s_read", "d_read") or barrier[0] == "e0" else 1


def mistakes(items, turns):
    """What goes wrong in some order of the events: waits see a barrier as the hardware shows it, by the parity of
    its phase."""
    lists = roles(items, turns)
    at = {}
    for e in (e for r in lists for e in r if e[0] == "arrive"):
        at.setdefault(e[1], len(at))
    found = set()
    start = (tuple(0 for _ in lists), tuple(0 for _ in at), tuple((-1,) * WARPS for _ in range(2)))
    seen, todo = {start}, [start]
    while todo:
        pcs, arrived, ds = todo.pop()
        moved = False
        for r, events in enumerate(lists):
            if pcs[r] == len(events):
                continue
            e = events[pcs[r]]
            here, there = list(arrived), ds
            if e[0] == "wait":
                complete = arrived[at[e[1]]] // arrivals(e[1])         # phases so far
                if complete % 2 != (e[2] + 1) % 2:
                    continue
                if complete != e[2] + 1:
                    found.add(f"a wait for {e[1]} two phases behind")
                    continue
            elif e[0] == "arrive":
                here[at[e[1]]] += 1
            elif e[0] == "write":
                rows = list(ds[e[1]])
                rows[e[2]] = e[3]
                there = tuple(tuple(rows) if p == e[1] else ds[p] for p in range(2))
            elif ds[e[1]] != (e[2],) * WARPS:
                found.add("dQ reads another step's dS")
                continue
            moved = True
            state = (tuple(p + (q == r) for q, p in enumerate(pcs)), tuple(here), there)
            if state not in seen:
                seen.add(state)
                todo.append(state)
        if not moved and any(p < len(events) for p, events in zip(pcs, lists)):
            found.add("everyone waits")
    return found


@pytest.mark.parametrize("items", [(5,), (1, 1, 2), (2, 3), (3, 2), (4, 1, 1)], ids=str)
def test_every_order_hands_each_step_over_whole(items):
    assert mistakes(items, barriers_of_ds()) == set()


def test_the_model_finds_the_mistake_of_one_barrier():
    assert "dQ reads another step's dS" in mistakes((3,), 1)


# ------------------------------------------------------------------ slots
#
# The producer, the two issuing warps and the elementwise ones (as one) over the slots of the ring.  An item of more
# than one key tile begins with a step for D, which takes O in the first stream's slot and nothing in the second's.

def lead_waits_for_both_slots():
    """Whether D's product waits for the producer to have had the second slot too, from the source."""
    with open(os.path.join(CSRC, "attention_packed_bwd.cu")) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    lead = re.search(r"if \(ok && lead\) \{\s*const Slot o = first\(t\), v = second\(t\);\s*ok = \(nd == 0.*?if \(ok\) \{", text, re.S).group()
    assert "m.full + 8 * o.s" in lead
    return "m.full + 8 * v.s" in lead


def slot(shared, second, i):
    """Slot and how often it was used before, of tile i of a stream (attention_bwd.cuh: slot_of)."""
    if not shared:
        return i % 3 + (3 if second else 0), i // 3
    if second:                          # slots 2.. begin with this stream: their first tile is number 0
        return (i + 2) % 5, 2 * (i // 5) + (1 if i % 5 >= 3 else 0)
    return i % 5, 2 * (i // 5) + (1 if i % 5 >= 2 else 0)


def ring_roles(items, shared, both):
    """As roles(), for items given by their key tiles, or (1, True) for a single one of several."""
    load, issue, grad, work = [], [], [], []
    uses = {}
    t = s = d = 0                       # steps, S and dP so far
    for i, n in enumerate(items):
        n, lead = n if isinstance(n, tuple) else (n, n > 1)
        for j in range(n + lead):
            (k, ku), (v, vu) = slot(shared, False, t + j), slot(shared, True, t + j)
            for x, u in ((k, ku), (v, vu)):
                uses.setdefault(x, []).append(u)
                if u:
                    load.append(("wait", ("empty", x), u - 1))
                load.append(("arrive", ("full", x)))
        if lead:
            (o, ou), (v, vu) = slot(shared, False, t), slot(shared, True, t)
            issue += [("wait", "d_read", d - 1)] if d else []
            issue += [("wait", ("full", o), ou)] + ([("wait", ("full", v), vu)] if both else [])
            issue += [("arrive", "d_full"), ("arrive", ("empty", o)), ("arrive", ("empty", v))]
            work += [("wait", "d_full", d), ("arrive", "d_read")]
            d += 1
        t += lead
        for j in range(n):
            (k, ku), (v, vu) = slot(shared, False, t + j), slot(shared, True, t + j)
            issue += [("wait", "s_read", s - 1)] if s else []
            issue.append(("wait", ("full", k), ku))
            if j >= 2:
                b, bu = slot(shared, False, t + j - 2)
                issue.append(("wait", ("empty", b), bu))
            issue += [("arrive", "s_full")] + ([("wait", "d_read", d - 1)] if d else [])
            issue += [("wait", ("full", v), vu), ("arrive", "d_full"), ("arrive", ("empty", v))]
            work += [("wait", "s_full", s), ("arrive", "s_read"), ("wait", "d_full", d), ("arrive", "d_read"), ("arrive", ("e0", s % 2))]
            grad += [("wait", ("full", k), ku), ("wait", ("e0", s % 2), s // 2), ("arrive", ("empty", k))]
            s, d = s + 1, d + 1
        grad.append(("arrive", "done"))
        work.append(("wait", "done", i))
        t += n
    assert all(u == list(range(len(u))) for u in uses.values())       # every use of a slot follows the one before
    return [load, issue, grad, work]


def ring_mistakes(items, shared, both, monkeypatch):
    monkeypatch.setitem(globals(), "roles", lambda *_: ring_roles(items, shared, both))
    monkeypatch.setitem(globals(), "arrivals", lambda _: 1)
    return mistakes(items, 2)


RINGS = [(5,), (2, 2, 3), (1, 1, 1, 1, 2, 1), (1, 4, 1, 2), (3, 1, 1, 1, 3), (1, 2, 1, 1, 1, 6), ((1, True), 1, (1, True), (1, True), 2)]


@pytest.mark.parametrize("shared", [False, True], ids=["two rings", "one ring"])
@pytest.mark.parametrize("items", RINGS, ids=str)
def test_every_order_hands_each_slot_over(items, shared, monkeypatch):
    assert ring_mistakes(items, shared, lead_waits_for_both_slots(), monkeypatch) == set()


def test_the_model_finds_the_slot_that_is_given_back_unseen(monkeypatch):
    assert any(ring_mistakes(items, shared, False, monkeypatch) for items in RINGS for shared in (False, True))
