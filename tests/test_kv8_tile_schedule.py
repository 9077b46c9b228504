"""The barrier schedule of the 8-bit cache's many-row attention kernel
(csrc/fa_fwd_kv8_tile.cu), walked on the CPU.

An mbarrier wait names a phase by its parity alone, so it is sound only where
  - the phase before the one it waits for is complete when it is asked (else
    the parity of two phases ago lets it pass at once), and
  - the phase after it cannot complete before the wait has returned (else it
    waits for a phase that may never come).
An arrival likewise has to come after the phase before its own is complete.

The test builds the events of one CTA's run (every role's waits and arrivals in
program order, copies and MMAs as events of their own that may complete late and
in any order) and the edges that order them, and asks for each wait, arrival and
buffer reuse whether the edges alone enforce it: a schedule that passes is sound
for every timing. Ring sizes are read from the kernel's source.
"""

import os
import re

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "exact_softmax_attention_fa_gb300",
                      "csrc", "fa_fwd_kv8_tile.cu")


def config(d):
    """NT, KST, K_BARS, VST, SST, SLOTS of TileCfg<d>, from its source."""
    text = open(SOURCE).read()
    names = {"D": d}

    def value(expr):
        m = re.fullmatch(r"\s*(.+?)\s*\?\s*(.+?)\s*:\s*(.+)\s*", expr)
        if m:
            return value(m[2]) if eval(m[1], {}, names) else value(m[3].strip().removeprefix("(").removesuffix(")"))
        return eval(expr.replace("/", "//"), {}, names)

    for name in ("NT", "KST", "K_BARS", "VST", "SLOTS", "SST"):
        m = re.search(r"static constexpr int %s = ([^;]+);" % name, text)
        if m:
            names[name] = int(value(m[1]))
    names.setdefault("K_BARS", names["KST"])
    return names


class Run:
    """Events and the edges between them."""

    def __init__(self):
        self.edges = []      # predecessors of each event
        self.last = {}       # role -> its latest event
        self.arrivals = {}   # (barrier, phase) -> events
        self.done = {}       # (barrier, phase) -> event of its completion
        self.waits = []      # (event asked, event returned, barrier, phase)
        self.arrived = []    # (event, barrier, phase)
        self.order = []      # (event, event, what): the first has to come first

    def event(self, *after):
        self.edges.append([e for e in after if e is not None])
        return len(self.edges) - 1

    def step(self, role):
        self.last[role] = self.event(self.last.get(role))
        return self.last[role]

    def completion(self, bar, phase):
        if (bar, phase) not in self.done:
            self.done[bar, phase] = self.event()
        return self.done[bar, phase]

    def wait(self, role, bar, phase):
        asked = self.step(role)
        back = self.step(role)
        self.edges[back].append(self.completion(bar, phase))
        self.waits.append((asked, back, bar, phase))

    def arrive(self, role, bar, phase, later=()):
        """An arrival in program order, or with `later` one that only follows those events."""
        e = self.event(*later) if later else self.step(role)
        self.arrivals.setdefault((bar, phase), []).append(e)
        self.arrived.append((e, bar, phase))
        return e

    def sync(self, roles):
        before = [self.last.get(r) for r in roles]
        e = self.event(*before)
        for r in roles:
            self.last[r] = e

    def check(self, count):
        for (bar, phase), e in self.done.items():
            arrivals = self.arrivals.get((bar, phase), [])
            assert len(arrivals) == count(bar), ("arrivals", bar, phase, len(arrivals))
            self.edges[e] += arrivals
        for (bar, phase), events in self.arrivals.items():
            assert len(events) <= count(bar), ("arrivals", bar, phase, len(events))
        # all predecessors of each event, as a bit set, in topological order
        n = len(self.edges)
        left = [len(set(p)) for p in self.edges]
        after = [[] for _ in range(n)]
        for e, p in enumerate(self.edges):
            for x in set(p):
                after[x].append(e)
        seen = [0] * n
        ready = [e for e in range(n) if left[e] == 0]
        walked = 0
        while ready:
            e = ready.pop()
            walked += 1
            for x in after[e]:
                seen[x] |= seen[e] | 1 << e
                left[x] -= 1
                if left[x] == 0:
                    ready.append(x)
        assert walked == n, "the schedule waits for itself"

        def before(a, b):
            return seen[b] >> a & 1

        def complete(bar, phase, by):  # a phase ends with the last of its arrivals
            arrivals = self.arrivals.get((bar, phase), [])
            return len(arrivals) == count(bar) and all(before(a, by) for a in arrivals)

        bad = []
        for asked, back, bar, phase in self.waits:
            if phase > 0 and not complete(bar, phase - 1, asked):
                bad.append(("asked a phase early", bar, phase))
            later = self.arrivals.get((bar, phase + 1), [])
            if len(later) == count(bar) and not any(before(back, a) for a in later):
                bad.append(("can be overtaken", bar, phase))
        for e, bar, phase in self.arrived:
            if phase > 0 and not complete(bar, phase - 1, e):
                bad.append(("arrives a phase early", bar, phase))
        for a, b, what in self.order:
            if not before(a, b):
                bad.append(("reused early",) + what)
        return bad


def walk(d, halves, parts, moves, dead_warps=0):
    """One CTA's run over `parts` = (tiles, tiles that slot 0's rows see, slot 1's); moves: the
    references move at every step; dead_warps: warps of a slot without live rows."""
    c = config(d)
    NT, KST, KB, VST, SST, SLOTS = (c[k] for k in ("NT", "KST", "K_BARS", "VST", "SST", "SLOTS"))
    slots = range(NT)
    r = Run()
    total = sum(p[0] for p in parts)
    seen_by = []  # per tile of the run: the slots that take it
    for n, *lasts in parts:
        for j in range(n):
            seen_by.append([j % 2] if halves else [t for t in slots if j < lasts[t]])

    k_used, v_used, s_done, pv_done_ev = {}, {}, {}, {}
    k_issue, v_write, scale_write, scale_read, stage_issue, stage_read = {}, {}, {}, {}, {}, {}

    # loads
    for i in range(total):
        if i >= KST:
            r.wait("load", ("k_empty", i % KST), i // KST - 1)
        k_issue[i] = r.arrive("load", ("k_full", i % KB), i // KB)        # the expected bytes
        r.arrive(None, ("k_full", i % KB), i // KB, (k_issue[i],))        # the copy lands
        scale_write[i] = r.step("load")
        r.arrive("load", ("scale_full", i % SLOTS), i // SLOTS)
        if i >= SST:
            r.wait("load", ("st_empty", i % SST), i // SST - 1)
        stage_issue[i] = r.arrive("load", ("st_full", i % SST), i // SST)
        r.arrive(None, ("st_full", i % SST), i // SST, (stage_issue[i],))

    # conversion
    for q in range(4):
        role = ("convert", q)
        for i in range(total):
            r.wait(role, ("scale_full", i % SLOTS), i // SLOTS)
            r.wait(role, ("st_full", i % SST), i // SST)
            if i >= VST:
                r.wait(role, ("v_empty", i % VST), i // VST - 1)
            e = r.step(role)
            v_write.setdefault(i, []).append(e)
            scale_read.setdefault(i, []).append(e)
            stage_read.setdefault(i, []).append(e)
            r.arrive(role, ("st_empty", i % SST), i // SST)
            r.arrive(role, ("v_full", i % VST), i // VST)

    # MMA issue
    for t in slots:
        role = ("mma", t)
        issued = []          # MMAs so far: a commit follows all of them
        k = v = 0            # the tiles whose S and PV come next
        use = 0              # uses of each buffer of S by PV so far

        def mma(wait_for_landing):
            e = r.step(role)
            done = r.event(e, *wait_for_landing)
            issued.append(done)
            return done

        def commit(bar, phase):
            r.arrive(None, bar, phase, (r.last[role], *issued))

        def skip_k():
            nonlocal k
            if not halves:
                r.wait(role, ("k_full", k % KB), k // KB)
                r.arrive(role, ("k_empty", k % KST), k // KST)
            k += 1

        def skip_v():
            nonlocal v
            if not halves:
                r.wait(role, ("v_full", v % VST), v // VST)
                r.arrive(role, ("v_empty", v % VST), v // VST)
            v += 1

        def issue_s(b, phase):
            nonlocal k
            if b == 0:
                r.wait(role, ("k_full", k % KB), k // KB)
            if phase >= 0:
                r.wait(role, ("pv_done", t, b), phase)
            e = mma(())
            k_used.setdefault(k, []).append(e)
            commit(("s_full", t, b), phase + 1)
            if b == 1:
                commit(("k_empty", k % KST), k // KST)
                k += 1

        def issue_pv(b):
            nonlocal v
            if b == 0:
                r.wait(role, ("v_full", v % VST), v // VST)
            r.wait(role, ("p_full", t, b), use)
            e = mma(())
            v_used.setdefault(v, []).append(e)
            commit(("pv_done", t, b), use)
            if b == 1:
                commit(("v_empty", v % VST), v // VST)
                v += 1

        for seg, (n, *lasts) in enumerate(parts):
            turns = (n + 1 - t) // 2 if halves else lasts[t]
            r.wait(role, ("q_full", t), seg)
            r.arrive(role, ("q_taken", t), seg)
            if halves and t == 1:
                skip_k(), skip_v()
            if turns > 0:
                issue_s(0, use - 1), issue_s(1, use - 1)
                if seg > 0:
                    r.wait(role, ("o_free", t), seg - 1)
            for j in range(turns):
                more = j + 1 < turns
                if halves and more:
                    skip_k()
                for b in range(2):
                    issue_pv(b)
                    if more:
                        issue_s(b, use)
                if halves and more:
                    skip_v()
                use += 1
            if not halves:
                for _ in range(turns, n):
                    skip_k(), skip_v()
            if halves and turns > 0 and (n - 1) % 2 != t:
                skip_k(), skip_v()
        assert k == v == total, (k, v, total)

    # softmax
    q_write = {}
    roles = {t: [("softmax", t, q) for q in range(4)] for t in slots}
    cnt = {t: 0 for t in slots}
    i0 = 0
    for seg, (n, *lasts) in enumerate(parts):
        for t in slots:
            turns = len(range(t, n, 2)) if halves else lasts[t]
            mine = [i0 + j for j in (range(t, n, 2) if halves else range(lasts[t]))]
            for role in roles[t]:
                if seg > 0:
                    r.wait(role, ("q_taken", t), seg - 1)
            if seg > 0:
                r.sync(roles[t])
            for role in roles[t]:
                q_write.setdefault((seg, t), []).append(r.step(role))
                r.arrive(role, ("q_full", t), seg)
            r.sync(roles[t])
            for role in roles[t]:
                live = role[2] < 4 - dead_warps
                for f in range(2 * turns):
                    i, b = mine[f >> 1], f & 1
                    if b == 0:
                        r.wait(role, ("scale_full", i % SLOTS), i // SLOTS)
                    r.wait(role, ("s_full", t, b), cnt[t] + (f >> 1))
                    if live:
                        scale_read.setdefault(i, []).append(r.step(role))
                        if f > 0 and moves:
                            r.wait(role, ("pv_done", t, b ^ 1), cnt[t] + ((f - 1) >> 1))
                    r.arrive(role, ("p_full", t, b), cnt[t] + (f >> 1))
                if turns:
                    r.wait(role, ("pv_done", t, 1), cnt[t] + turns - 1)
            cnt[t] += turns
        for t in slots:
            for role in roles[t]:
                live = role[2] < 4 - dead_warps
                if halves:
                    r.arrive(role, ("join_ml", role[2]), seg)
                    r.wait(role, ("join_ml", role[2]), seg)
                    r.arrive(role, ("join_o", t, role[2]), seg)
                    if live:
                        r.wait(role, ("join_o", t ^ 1, role[2]), seg)
                r.arrive(role, ("o_free", t), seg)
        i0 += n

    # buffers: what was in them has been used before they are filled again
    for i in range(total):
        for old, uses, fills, name in ((i - KST, k_used, [k_issue[i]], "K"), (i - VST, v_used, v_write[i], "V"),
                                       (i - SST, stage_read, [stage_issue[i]], "staged V"),
                                       (i - SLOTS, scale_read, [scale_write[i]], "scales")):
            if old >= 0:
                r.order += [(a, b, (name, i)) for a in uses.get(old, []) for b in fills]

    both = 1 if halves else NT
    counts = {"k_full": 2, "st_full": 2, "k_empty": both, "v_empty": both, "st_empty": 4, "v_full": 4, "q_full": 4,
              "p_full": 4, "o_free": 4, "join_ml": 2}
    return r.check(lambda bar: counts.get(bar[0], 1))


HALVES = [[(1,)], [(2,)], [(9,)], [(12,)], [(13,)], [(3,), (8,), (1,), (7,)], [(5,), (5,), (5,)], [(2,), (1,), (1,), (12,)]]


@pytest.mark.parametrize("parts", HALVES, ids=str)
@pytest.mark.parametrize("moves", [False, True])
@pytest.mark.parametrize("dead_warps", [0, 3])
@pytest.mark.parametrize("d", [64, 128])
def test_one_tile_of_rows(d, parts, moves, dead_warps):
    assert walk(d, True, parts, moves, dead_warps) == []


@pytest.mark.parametrize("parts", [[(1, 1, 1)], [(12, 12, 12)], [(13, 12, 13)], [(5, 4, 5), (9, 9, 9), (6, 6, 0)],
                                   [(3, 0, 3), (8, 7, 8), (1, 1, 1), (2, 2, 1), (9, 9, 9)]], ids=str)
@pytest.mark.parametrize("moves", [False, True])
@pytest.mark.parametrize("dead_warps", [0, 3])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_two_tiles_of_rows(d, parts, moves, dead_warps):
    assert walk(d, False, parts, moves, dead_warps) == []
