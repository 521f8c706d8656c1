"""The barriers of the attention tiles over the 8-bit cache (csrc/kv8_tile.cu) under every order in which copies can land and
products can end, as a model on the CPU: the product warps' waits are those of csrc/kv8_order.h, which the kernel is made
from; the other roles are restated here.  No product may read keys, values or weights that are not there, and no role
may be left waiting."""
import os
import subprocess

import pytest

from fp4_compressed_sparse_02_gb300 import build

RING = 3                                   # steps of bytes under way
TESTS = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def order(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("order") / "kv8_order")
    r = subprocess.run(["g++", "-O1", "-std=c++17", "-I", build.CSRC, "-o", exe, os.path.join(TESTS, "kv8_order.cpp")],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr

    def ops(by, grp, segments, run=128):
        out = subprocess.run([exe, str(by), str(run), str(grp), *map(str, segments)], capture_output=True, text=True, check=True).stdout
        return [tuple(int(w) if w.isdigit() else w for w in line.split()) for line in out.splitlines()]
    return ops


def passes(done, use):
    """A wait by parity for the barrier's use-th phase, when `done` phases are over."""
    return (done & 1) != (use & 1)


def explore(order, by, segments, run):
    """Every reachable state; raises AssertionError at the first wrong read or at a state in which nothing can go on.

    A state: the program counters of the loader, the converter, the two product warps and the two softmaxes; the copies
    under way; the products issued by each group that have not ended; the phases of each barrier that are over."""
    total = sum(segments)
    begin = [sum(segments[:i]) for i in range(len(segments) + 1)]
    prod = [order(by, g, segments, run) for g in (0, 1)]
    own = [[st for i, n in enumerate(segments) for st in range(begin[i], begin[i] + n) if by == 1 or (st - begin[i]) % 2 == g] for g in (0, 1)]
    # the loader: wait for the stage, copy (keys, then values); the converter: wait, free, wait, done
    load = [x for st in range(total) for x in (("k", st), ("v", st))]
    conv = [x for st in range(total) for x in (("take", st), ("give", st))]
    # a softmax: at a segment's begin it hands out Q (the first group's alone with by = 2), then a step's weights, after a run
    # waits for its sums and reads them, and at the end the two meet
    soft = [[], []]
    for g in (0, 1):
        for i, n in enumerate(segments):
            mine = [st for st in own[g] if begin[i] <= st < begin[i + 1]]
            if by == 1 or g == 0:
                soft[g].append(("query", i))
            for k, st in enumerate(mine):
                soft[g].append(("weigh", st))
                if k % run == run - 1 or k + 1 == len(mine):
                    soft[g].append(("run", (i, k // run)))
            if by == 2:                                      # before and after the first reads the second's sums
                soft[g] += [("meet", i), ("meet again", i)]
    count = lambda g, st: own[g].index(st)           # the how-manieth step of its group
    # sums that group g gives out before a segment
    before = lambda g, i: sum(-(-sum(begin[k] <= st < begin[k + 1] for st in own[g]) // run) for k in range(i))
    empties = {1: 2, 2: 1}[by]                       # arrivals that free a stage of keys (and of fp16 values)
    # state: (load pc, conv pc, prod pcs, soft pcs, copies, queues, bars); bars: phases over, and arrivals of the open phase
    names = ([("k_full", b) for b in range(RING)] + [("k_empty", b) for b in range(RING)] + [("v_full", b) for b in range(RING)]
             + [("v_empty", b) for b in range(RING)] + [("vf_full", b) for b in (0, 1)] + [("vf_empty", b) for b in (0, 1)]
             + [(n, g) for n in ("s_full", "p_full", "o_full", "turn") for g in (0, 1)] + [("q_full", 0)])
    at = {n: i for i, n in enumerate(names)}
    need = {n: 1 for n in names}
    for b in range(RING):
        need["k_empty", b] = empties
    for b in (0, 1):
        need["vf_empty", b] = empties
    need["q_full", 0] = 3 - by

    def arrive(bars, name):
        i = at[name]
        done, n = bars[i]
        n += 1
        new = (done + 1, 0) if n == need[name] else (done, n)
        return bars[:i] + (new,) + bars[i + 1:]

    def done(bars, name):
        return bars[at[name]][0]

    def landed(bars, st):
        return done(bars, ("k_full", st % RING)) == st // RING + 1

    def steps(s):
        """The states after one move."""
        lp, cp, pp, sp, copies, queues, bars = s
        if lp < len(load):
            kind, st = load[lp]
            if passes(done(bars, (kind + "_empty", st % RING)), st // RING + 1):
                yield (lp + 1, cp, pp, sp, copies | {(kind, st)}, queues, bars)
        for c in copies:                                     # copies land in any order
            kind, st = c
            yield (lp, cp, pp, sp, copies - {c}, queues, arrive(bars, (kind + "_full", st % RING)))
        if cp < len(conv):
            kind, st = conv[cp]
            if kind == "take":
                if passes(done(bars, ("v_full", st % RING)), st // RING):
                    assert done(bars, ("v_full", st % RING)) == st // RING + 1, f"values of step {st} are not there"
                    yield (lp, cp + 1, pp, sp, copies, queues, arrive(bars, ("v_empty", st % RING)))
            elif passes(done(bars, ("vf_empty", st & 1)), (st >> 1) + 1):
                assert done(bars, ("vf_empty", st & 1)) >= st >> 1, f"step {st} overwrites fp16 values in use"
                yield (lp, cp + 1, pp, sp, copies, queues, arrive(bars, ("vf_full", st & 1)))
        for g in (0, 1):
            if pp[g] < len(prod[g]):
                op = prod[g][pp[g]]
                name, st = op[0], op[1] if len(op) > 1 else None
                after, go, q = bars, True, queues
                if name == "query":
                    go = passes(done(bars, ("q_full", 0)), st)
                elif name == "keys":
                    go = passes(done(bars, ("k_full", st % RING)), st // RING)
                elif name == "values":
                    go = passes(done(bars, ("vf_full", st & 1)), st >> 1)
                elif name == "turn":
                    had = sum(o[0] == "turn" for o in prod[g][:pp[g]])
                    go = passes(done(bars, ("turn", g)), had + (1 if g == 0 else 0))
                elif name == "weights":
                    had = sum(o[0] == "weights" for o in prod[g][:pp[g]])
                    go = passes(done(bars, ("p_full", g)), had)
                elif name == "scores":
                    assert landed(bars, st), f"group {g} multiplies keys of step {st} that are not there"
                    assert not any(o == ("scores", st) for o in queues[g])
                    q = queues[:g] + (queues[g] + (op,),) + queues[g + 1:]
                elif name == "products":
                    assert done(bars, ("vf_full", st & 1)) == (st >> 1) + 1, f"fp16 values of step {st} are not there"
                    assert done(bars, ("p_full", g)) == count(g, st) + 1, f"weights of step {st} are not there"
                    q = queues[:g] + (queues[g] + (op,),) + queues[g + 1:]
                    k = next(k for k, x in enumerate(soft[g]) if x == ("weigh", st))
                    if not op[2] and k and soft[g][k - 1][0] == "run":
                        assert sp[g] >= k, f"step {st} overwrites sums that are not read"
                elif name == "out":
                    q = queues[:g] + (queues[g] + (op,),) + queues[g + 1:]
                elif name == "pass":
                    after = arrive(bars, ("turn", 1 - g))
                if go:
                    yield (lp, cp, tuple(x + (i == g) for i, x in enumerate(pp)), sp, copies, q, after)
            if queues[g]:                                    # a group's products end in their order
                name, st = (*queues[g][0], None)[:2]
                q = queues[:g] + (queues[g][1:],) + queues[g + 1:]
                if name == "scores":
                    after = arrive(arrive(bars, ("s_full", g)), ("k_empty", st % RING))
                elif name == "out":
                    after = arrive(bars, ("o_full", g))
                else:
                    after = arrive(bars, ("vf_empty", st & 1))
                yield (lp, cp, pp, sp, copies, q, after)
            if sp[g] < len(soft[g]):
                kind, x = soft[g][sp[g]]
                after, go = bars, True
                if kind == "query":
                    after = arrive(bars, ("q_full", 0))
                elif kind == "weigh":
                    go = passes(done(bars, ("s_full", g)), count(g, x))
                    if go:
                        assert done(bars, ("s_full", g)) == count(g, x) + 1, f"scores of step {x} are not there"
                        after = arrive(bars, ("p_full", g))
                elif kind in ("meet", "meet again"):
                    go = sp[1 - g] < len(soft[1 - g]) and soft[1 - g].index((kind, x)) <= sp[1 - g] or sp[1 - g] == len(soft[1 - g])
                else:
                    go = passes(done(bars, ("o_full", g)), before(g, x[0]) + x[1])
                    assert not go or done(bars, ("o_full", g)) == before(g, x[0]) + x[1] + 1, "a run's sums are not there"
                if go:
                    yield (lp, cp, pp, tuple(x + (i == g) for i, x in enumerate(sp)), copies, queues, after)

    first = (0, 0, (0, 0), (0, 0), frozenset(), ((), ()), tuple((0, 0) for _ in names))
    seen, todo = {first}, [first]
    while todo:
        s = todo.pop()
        end = True
        for n in steps(s):
            end = False
            if n not in seen:
                seen.add(n)
                todo.append(n)
        if end:
            assert s[0] == len(load) and s[1] == len(conv) and all(s[2][g] == len(prod[g]) and s[3][g] == len(soft[g]) for g in (0, 1)), \
                f"nothing can go on: {s}"
    return len(seen)


@pytest.mark.parametrize("by,segments", [(2, [1]), (2, [2]), (2, [3]), (2, [4]), (2, [5]), (2, [6]), (2, [7]), (2, [3, 4]), (2, [4, 3]),
                                         (2, [5, 3]), (2, [2, 2, 4]), (2, [1, 5]), (2, [1, 1, 2, 4]), (2, [2, 1, 4]), (2, [1, 1, 1, 3]),
                                         (1, [1]), (1, [4]), (1, [5]), (1, [2, 3])])
def test_no_product_reads_what_is_not_there(order, by, segments):
    explore(order, by, segments, 128)


@pytest.mark.parametrize("by,segments", [(2, [4]), (2, [5]), (2, [6]), (2, [7]), (2, [5, 4]), (2, [1, 5]), (2, [6, 2]), (1, [2]), (1, [3]), (1, [5]), (1, [3, 2])])
def test_sums_of_runs_are_read_before_the_next(order, by, segments):
    """The same with runs of two steps of a group: each run's sums are whole when they are read and stay until then."""
    explore(order, by, segments, 2)
    for g in (0, 1):
        adds = [o[2] for o in order(by, g, segments, 2) if o[0] == "products"]
        mine = [len(range(g if by == 2 else 0, n, by)) for n in segments]
        assert adds == [k % 2 for n in mine for k in range(n)]


@pytest.mark.parametrize("by,segments", [(1, [3, 2]), (2, [3, 1, 4])])
def test_groups_take_turns_through_their_steps(order, by, segments):
    """What each group multiplies: its own steps, once each and in order."""
    total = sum(segments)
    for what in ("scores", "products"):
        got = [[o[1] for o in order(by, g, segments) if o[0] == what] for g in (0, 1)]
        assert all(x == sorted(x) for x in got)
        assert sorted(sum(got, [])) == sorted(list(range(total)) * (3 - by))
