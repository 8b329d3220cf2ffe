"""The order that the mbarriers of the tensor-core recurrence kernels keep, on the CPU.

A kernel's roles (warps) are written down as programs of waits, arrivals and
accesses to shared and tensor memory; the waits themselves, with their
conditions, are read from the kernel's source in the order in which they stand
there.  The programs give a graph of what happens before what: each warp's own
order, the order of one issuer's tensor-core products, and from every arrival
of a barrier's phase to the waits for that phase.  Nothing else may be assumed,
whatever the warps' speed, so

* between a buffer's write and each of its reads, and between those and the
  next write to the same place, there has to be a path;
* a warp that waits for a phase has to have seen it before the next phase can
  complete (a parity tells a phase only from the one before it), and a phase's
  arrivals have to follow the phase before it.
"""
import os
import re

import pytest

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                   "deltanet_sequence_mixing_b200", "csrc", "gated_tc.cu")


def _python(cond):
    """A wait condition of the source as a Python expression."""
    x = re.sub(r"\s+", " ", cond).strip()
    x = re.sub(r"wait_bar\(bar \+ (\w+) \+ 8 \* \(c % 3\), \((.*?)\) & 1, wc\)", r"phase(\1, c % 3, \2)", x)
    x = re.sub(r"GATED \? (done\([^()]*\)) : (\w+\([^()]*\))", r"\1 if GATED else \2", x)
    x = re.sub(r"!(?!=)", " not ", x.replace("&&", " and ").replace("||", " or "))
    return re.sub(r" / ", " // ", x).strip()


def _waits(section, names=("done", "full_v", "have_decays", "wait_bar")):
    """The section's wait conditions in order, without the drains at a role's end."""
    got = []
    for piece in re.sub(r"//[^\n]*", "", section).split(";"):
        if not re.search(r"\b(%s)\(" % "|".join(names), piece) or "(void)" in piece:
            continue
        if "ok = " in piece:
            cond = piece.split("ok = ", 1)[1]
        else:
            cond = re.search(r"if \((.*)\) break$", re.sub(r"\s+", " ", piece).strip()).group(1)
        got.append(_python(cond))
    return got


def _sections(start, end):
    text = open(SRC).read()
    text = text[text.index(start):text.index(end)]
    parts = re.split(r"\n *// -{10,} ([\w ]+?) --\n", text)
    return dict(zip(parts[1::2], parts[2::2]))


class Order:
    """Events and what is known to happen before what."""

    def __init__(self):
        self.before = []  # direct predecessors of every event
        self.name = []
        self.last = {}  # a warp's last event
        self.arrivals = {}  # (barrier, phase) -> events
        self.waits = []  # (barrier, phase, event)
        self.uses = {}  # place -> [(kind, generation, first event, last event)]

    def event(self, name, *preds):
        self.before.append([p for p in preds if p is not None])
        self.name.append(name)
        return len(self.before) - 1

    def step(self, warp, name):
        e = self.event(f"{warp}: {name}", self.last.get(warp))
        self.last[warp] = e
        return e

    def arrive(self, bar, phase, event):
        self.arrivals.setdefault((bar, phase), []).append(event)

    def wait(self, warp, bar, phase):
        self.waits.append((bar, phase, self.step(warp, f"waits for {bar} {phase}")))

    def use(self, place, kind, generation, first, last=None):
        self.uses.setdefault(place, []).append((kind, generation, first, first if last is None else last))

    def ancestors(self):
        for bar, phase, e in self.waits:
            assert (bar, phase) in self.arrivals, f"{self.name[e]}: nobody arrives"
            self.before[e] += self.arrivals[bar, phase]
        n = len(self.before)
        after, left = [[] for _ in range(n)], [len(b) for b in self.before]
        for e, b in enumerate(self.before):
            for p in b:
                after[p].append(e)
        ready, seen, anc = [e for e in range(n) if left[e] == 0], 0, [0] * n
        while ready:
            e = ready.pop()
            seen += 1
            for p in self.before[e]:
                anc[e] |= anc[p] | 1 << p
            for s in after[e]:
                left[s] -= 1
                if left[s] == 0:
                    ready.append(s)
        assert seen == n, "roles wait for one another in a circle"
        return anc

    def faults(self):
        anc = self.ancestors()
        ok = lambda a, b: a == b or anc[b] >> a & 1
        bad = []
        for place, uses in self.uses.items():
            for kind, gen, first, last in uses:
                for kind2, gen2, first2, last2 in uses:
                    if kind == kind2 == "r" or gen > gen2 or (gen == gen2 and not (kind == "w" and kind2 == "r")):
                        continue
                    if (kind, gen, first) != (kind2, gen2, first2) and not ok(last, first2):
                        bad.append(f"{place}: {self.name[first2]} may come before {self.name[last]}")
        for bar, phase, e in self.waits:
            later = self.arrivals.get((bar, phase + 1))
            if later and not any(ok(e, a) for a in later):
                bad.append(f"{bar}: phase {phase + 1} may pass by '{self.name[e]}'")
        for (bar, phase), events in self.arrivals.items():
            for a in self.arrivals.get((bar, phase - 1), []):
                bad += [f"{bar}: '{self.name[e]}' may count for phase {phase - 1}" for e in events if not ok(a, e)]
        return bad


def out_kernel(n, GATED):
    """gated_out_kernel over n chunks; two warps stand for those of a role."""
    sec = _sections("- main kernel --", "- state kernel --")
    src = {r: _waits(sec[r]) for r in ("TMA", "MMA", "decays", "scores", "state", "outputs")}
    assert {r: len(x) for r, x in src.items()} == dict(TMA=3, MMA=4, decays=1, scores=2, state=2, outputs=2)
    od, names = Order(), re.findall(r"\bB_[A-Z]+", " ".join(sum(src.values(), [])))

    def run(warp, cond, c):
        def done(b, i):
            od.wait(warp, (b, i & 1), i >> 1)
            return True

        def phase(b, stage, k):
            od.wait(warp, (b, stage), k)
            return True

        env = dict(done=done, phase=phase, full_v=lambda i: phase("B_FULLV", i % 3, i // 3), all=lambda x: x,
                   have_decays=lambda i: not GATED or phase("B_DECAY", i % 3, i // 3), GATED=GATED, c=c, n=n)
        eval(cond, {**env, **{b: b for b in names}})

    def load(bar, stage, phase, place, c):
        a = od.step("TMA", f"loads {place} {c}")
        b = od.event(f"{place} {c} landed", a)
        od.use(place, "w", c, a, b)
        od.arrive((bar, stage), phase, b)

    for c in range(n):
        run("TMA", src["TMA"][0], c)
        load("B_FULLV", c % 3, c // 3, f"V[{c % 3}]", c)
        run("TMA", src["TMA"][1], c)
        load("B_FULLK", c & 1, c >> 1, f"K[{c & 1}]", c)
        run("TMA", src["TMA"][2], c)
        load("B_FULLQ", c & 1, c >> 1, f"Q[{c & 1}]", c)

    ran = {}  # an issuer's last product

    def product(warp, name, c, reads, writes, bars):
        a = od.step(warp, f"issues {name} {c}")
        b = ran[warp] = od.event(f"{name} {c} ran", a, ran.get(warp))
        for place in reads:
            od.use(place, "r", c, a, b)
        od.use(writes, "w", c, a, b)
        for bar, stage, phase in bars:
            od.arrive((bar, stage), phase, b)

    two = lambda b, c: (b, c & 1, c >> 1)
    v = lambda c: f"V[{c % 3}]"
    for c in range(n + 1):
        if c < n:
            run("MMA", src["MMA"][0], c)
            product("MMA", "scores", c, (f"Q[{c & 1}]", f"K[{c & 1}]"), f"scores[{c & 1}]", [two("B_SC", c)])
        if c >= 1:
            run("MMA", src["MMA"][1], c)
            product("MMA", "P V", c - 1, (f"P[{(c - 1) & 1}]", v(c - 1)), "PV",
                    [two("B_PV", c - 1), ("B_VFREE", (c - 1) % 3, (c - 1) // 3)])
    for c in range(n):
        run("MMA2", src["MMA"][2], c)
        product("MMA2", "increment", c, (f"K[{c & 1}]", "VT" if GATED else v(c)), "dS", [two("B_DS", c)])
        run("MMA2", src["MMA"][3], c)
        product("MMA2", "Q S", c, (f"Q[{c & 1}]", "S"), "QS", [two("B_QS", c)])

    def decays(warp, c):
        if GATED:
            od.use(f"decays[{c % 3}]", "r", c, od.step(warp, f"reads decays {c}"))

    for c in range(n if GATED else 0):
        run("decay", src["decays"][0], c)
        e = od.step("decay", f"decays {c}")
        od.use(f"decays[{c % 3}]", "w", c, e)
        od.arrive(("B_DECAY", c % 3), c // 3, e)
    for w in ("a", "b"):
        s = "scores " + w
        for c in range(n):
            if GATED:
                run(s, src["scores"][0], c)
                decays(s, c)
                od.use(v(c), "r", c, od.step(s, f"reads V {c}"))
                e = od.step(s, f"V~ {c}")
                od.use("VT", "w", c, e)
                od.arrive(("B_VT", c & 1), c >> 1, e)
            run(s, src["scores"][1], c)
            decays(s, c)
            e = od.step(s, f"P {c}")
            od.use(f"scores[{c & 1}]", "r", c, e)
            od.use(f"P[{c & 1}]", "w", c, e)
            od.arrive(("B_P", c & 1), c >> 1, e)
        s = "state " + w
        put = lambda c: (od.use("S", "w", c, od.step(s, f"S {c}")), od.arrive(("B_S", c & 1), c >> 1, od.last[s]))
        put(0)
        for c in range(n):
            run(s, src["state"][0], c)
            decays(s, c)
            e = od.step(s, f"reads the increment {c}")
            od.use("dS", "r", c, e)
            od.arrive(("B_DSFREE", c & 1), c >> 1, e)
            if c + 1 < n:
                run(s, src["state"][1], c)
                put(c + 1)
        s = "outputs " + w
        for c in range(n + 1):
            if GATED and c < n:
                run(s, src["outputs"][0], c)
                decays(s, c)
            if c >= 1:
                run(s, src["outputs"][1], c)
                e = od.step(s, f"reads O {c - 1}")
                od.use("QS", "r", c - 1, e)
                od.use("PV", "r", c - 1, e)
                od.arrive(("B_OFREE", (c - 1) & 1), (c - 1) >> 1, e)
    # the P of a chunk lies over its scores
    for i in range(2):
        for kind, gen, first, last in od.uses.get(f"P[{i}]", []):
            if kind == "r":  # the next scores have to wait for it
                od.use(f"scores[{i}]", "r", gen, first, last)
    return od


@pytest.mark.parametrize("n", [1, 2, 3, 4, 5, 9])
@pytest.mark.parametrize("gated", [True, False])
def test_main_kernel(n, gated):
    assert out_kernel(n, gated).faults() == []


@pytest.mark.parametrize("drop,place", [("done(B_PV, c - 2)", "scores"), ("done(B_DSFREE, c - 1)", "dS"),
                                        ("done(B_DS, c - 1)", "VT"), ("done(B_OFREE, c - 1)", "QS"),
                                        ("done(B_OFREE, 0)", "decays")])
def test_the_model_sees_a_missing_wait(monkeypatch, drop, place):
    """The same programs with one of the waits left out of what was read."""
    waits, drop = _waits, _python(drop)
    monkeypatch.setitem(globals(), "_waits", lambda s: [w.replace(drop, "True") for w in waits(s)])
    assert any(f.startswith(place) for f in out_kernel(9, True).faults())
