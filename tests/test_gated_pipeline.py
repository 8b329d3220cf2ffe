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
    x = re.sub(r"STORE \? (named_bar_and\(.*\)) : (all\(.*\))$", r"\1 if STORE else \2", x)
    x = re.sub(r"(\w+) \? (\w+) : (\w+)", r"\2 if \1 else \3", x).replace("0xffffffffu", "0")
    x = re.sub(r"!(?!=)", " not ", x.replace("&&", " and ").replace("||", " or "))
    return re.sub(r" / ", " // ", x).strip()


def _waits(section, names=("done", "full_v", "have_decays", "wait_bar", "wait", "wait_all", "wait_before")):
    """The section's wait conditions in order, without the drains at a role's end."""
    got = []
    for piece in re.sub(r"//[^\n]*", "", section).split(";"):
        if not re.search(r"\b(%s)\(" % "|".join(names), piece) or "(void)" in piece:
            continue
        if re.search(r"\b(ok|room) = ", piece):
            cond = re.split(r"\b(?:ok|room) = ", piece, maxsplit=1)[1]
        else:
            cond = re.search(r"if \((.*)\) break$", re.sub(r"\s+", " ", piece).strip()).group(1)
        got.append(_python(cond))
    return got


def _sections(start, end, *cuts):
    """The source between two marks, at its comments' rules or at the cuts."""
    text = open(SRC).read()
    text = text[text.index(start):text.index(end)]
    if not cuts:
        parts = re.split(r"\n *// -{10,} ([\w ]+?) --\n", text)
        return dict(zip(parts[1::2], parts[2::2]))
    at = [text.index(c) for c in cuts] + [len(text)]
    return [text[a:b] for a, b in zip(at, at[1:])]


class Order:
    """Events and what is known to happen before what."""

    def __init__(self):
        self.before = []  # direct predecessors of every event
        self.name = []
        self.last = {}  # a warp's last event
        self.arrivals = {}  # (barrier, phase) -> events
        self.waits = []  # (barrier, phase, event)
        self.uses = {}  # place -> [(kind, generation, first event, last event)]
        self.ran = {}  # an issuer's last product

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

    def meet(self, warps, name):
        """A named barrier of all the warps given."""
        e = self.event(name, *(self.last.get(w) for w in warps))
        for w in warps:
            self.last[w] = e

    def load(self, warp, place, generation, bar, phase):
        """A copy into the place, which arrives when it has landed."""
        a = self.step(warp, f"loads {place} {generation}")
        b = self.event(f"{place} {generation} landed", a)
        self.use(place, "w", generation, a, b)
        self.arrive(bar, phase, b)

    def product(self, warp, name, generation, reads, writes, fresh=True):
        """A tensor-core product; an issuer's run one after another."""
        a = self.step(warp, f"issues {name} {generation}")
        b = self.ran[warp] = self.event(f"{name} {generation} ran", a, self.ran.get(warp))
        for place, gen in reads:
            self.use(place, "r", gen, a, b)
        if fresh:  # else it adds to what the issuer's last product left
            self.use(writes, "w", generation, a, b)
        return b

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

    for c in range(n):
        run("TMA", src["TMA"][0], c)
        od.load("TMA", f"V[{c % 3}]", c, ("B_FULLV", c % 3), c // 3)
        run("TMA", src["TMA"][1], c)
        od.load("TMA", f"K[{c & 1}]", c, ("B_FULLK", c & 1), c >> 1)
        run("TMA", src["TMA"][2], c)
        od.load("TMA", f"Q[{c & 1}]", c, ("B_FULLQ", c & 1), c >> 1)

    def product(warp, name, c, reads, writes, bars):
        b = od.product(warp, name, c, [(r, c) for r in reads], writes)
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


def state_kernel(n, GATED, STORE):
    """gated_state_kernel over n chunks."""
    tma, mma, state, scale = (_waits(x) for x in _sections(
        "- state kernel --", "- gradient kernel --", "if (warp == kWarpTma)", "} else if (warp == kWarpMma)",
        "} else if (warp >= 4 && warp < 12)", "} else if (GATED && warp >= 12)"))
    assert [len(x) for x in (tma, mma, state, scale)] == [1, 1, 1, 1]
    od = Order()
    bar = lambda b, i: ((b, i & 1), i >> 1)

    def run(warp, cond, i):
        def done(b, k):
            od.wait(warp, *bar(b, k))
            return True

        eval(cond, dict(done=done, all=lambda x: x, named_bar_and=lambda b, n, x: x, kBarS=0, GATED=GATED,
                        STORE=STORE, i=i, **{b: b for b in ("C_FULL", "C_FREE", "C_VT", "C_DS", "C_DSFREE")}))

    for i in range(n):
        run("TMA", tma[0], i)
        a = od.step("TMA", f"loads chunk {i}")
        b = od.event(f"chunk {i} landed", a)
        for place in "XZ":
            od.use(f"{place}[{i & 1}]", "w", i, a, b)
        od.arrive(*bar("C_FULL", i), b)
        run("MMA", mma[0], i)
        b = od.product("MMA", "increment", i, [(f"X[{i & 1}]", i), (f"{'VT' if GATED else 'Z'}[{i & 1}]", i)],
                       f"dS[{i & 1}]")
        od.arrive(*bar("C_FREE", i), b)
        od.arrive(*bar("C_DS", i), b)
    for w in ("scale a", "scale b") if GATED else ():
        for i in range(n):
            run(w, scale[0], i)
            e = od.step(w, f"scales chunk {i}")
            od.use(f"Z[{i & 1}]", "r", i, e)
            od.use(f"VT[{i & 1}]", "w", i, e)
            od.arrive(*bar("C_VT", i), e)
    warps, copied = ("state a", "state b"), None
    for i in range(n):
        if STORE:
            od.last[warps[0]] = od.event("the leader's copy has read", od.last.get(warps[0]), copied)
            od.meet(warps, f"staging free {i}")
            for w in warps:
                od.use("staging", "w", i, od.step(w, f"stages {i}"))
            od.meet(warps, f"staged {i}")
            a = od.step(warps[0], f"copies the state {i}")
            copied = od.event(f"state {i} copied", a)
            od.use("staging", "r", i, a, copied)
        for w in warps:
            run(w, state[0], i)
        if STORE:
            od.meet(warps, f"increment {i}")
        for w in warps:
            e = od.step(w, f"reads the increment {i}")
            od.use(f"dS[{i & 1}]", "r", i, e)
            od.arrive(*bar("C_DSFREE", i), e)
    return od


def grad_kernel(n, GATED):
    """gated_grad_kernel, a CTA with n chunks."""
    tma, mma, epi, dots = (_waits(x) for x in _sections(
        "- gradient kernel --", "template <int DK, bool GATED>\ncudaError_t launch_out(", "  if (warp == kWarpTma)",
        "} else if (warp == kWarpMma)", "} else if (warp >= 4 && warp < 12)", "} else if (GATED && warp >= 12)"))
    assert [len(x) for x in (tma, mma, epi, dots)] == [5, 7, 5, 4]
    od, names = Order(), set(re.findall(r"\bG_[A-Z]+", " ".join(tma + mma + epi + dots)))
    warps, dwarps = ("epilogue a", "epilogue b"), ("dots a", "dots b")

    def run(warp, cond, it, **more):
        def wait(b, k=it):
            od.wait(warp, b, k)
            return True

        env = dict(wait=wait, wait_all=wait, wait_before=lambda b: it == 0 or wait(b, it - 1), ok=True, room=False,
                   __all_sync=lambda m, x: x, named_bar_and=lambda b, n, x: x, GATED=GATED, kBarE=0, kBarT=0)
        eval(cond, {**env, **more, **{b: b for b in names}})

    def loads(it, bar, *places):
        a = od.step("TMA", f"loads {' '.join(places)} {it}")
        b = od.event(f"{' '.join(places)} {it} landed", a)
        for place in places:
            od.use(place.split()[0], "w", 2 * it + ("S" in place[1:]), a, b)
        od.arrive(bar, it, b)

    def mm(it, name, reads, writes, fresh=True):
        return od.product("MMA", name, it, reads, writes, fresh)

    # a place's generations: two to a chunk, what is loaded or made first and what follows it there
    stores = {}
    for it in range(n):
        a, b = 2 * it, 2 * it + 1
        run("TMA", tma[0], it)
        loads(it, "G_VO", "O", "V")
        loads(it, "G_RH", "X")
        if GATED:
            run("TMA", tma[1], it)
            loads(it, "G_RL", "PA")
        run("TMA", tma[2], it)
        loads(it, "G_QK", "K", "Q")
        run("TMA", tma[3], it)
        if GATED:
            loads(it, "G_SL", "V S")
        run("TMA", tma[4], it)
        loads(it, "G_SH", "X S")

        run("MMA", mma[0], it)
        mm(it, "V R hi", [("V", a), ("X", a)], "C")
        if GATED:
            run("MMA", mma[1], it)
            mm(it, "V R lo", [("V", a), ("PA", a)], "C", False)
        run("MMA", mma[2], it)
        mm(it, "Q K", [("Q", a), ("K", a)], "A")
        od.arrive("G_SC", it, mm(it, "dO V", [("O", a), ("V", a)], "B"))
        od.arrive("G_XR", it, mm(it, "K R", [("K", a), ("X", a)], "D"))
        run("MMA", mma[3], it)
        e = od.product("MMA", "A dO", b, [("PA", b), ("O", a)], "A'")
        od.arrive("G_DV", it, e)
        od.product("MMA", "B Q", b, [("PB", b), ("Q", a)], "B'")
        run("MMA", mma[4], it)
        od.arrive("G_DK", it, od.product("MMA", "B K", b, [("PB", b), ("K", a)], "A''"))
        run("MMA", mma[5], it)
        e = od.product("MMA", "dO S hi", b, [("O", a), ("X", b)], "D'")
        if GATED:
            run("MMA", mma[6], it)
            e = od.product("MMA", "dO S lo", b, [("O", a), ("V", b)], "D'", False)
        od.arrive("G_DQ", it, e)

        def each(name, cond=None, read=(), write=(), arrive=None, **more):
            for w in warps:
                if cond is not None:
                    run(w, cond, it, **more)
                e = od.step(w, f"{name} {it}")
                for place, gen in read:
                    od.use(place, "r", gen, e)
                for place, gen in write:
                    od.use(place, "w", gen, e)
                if arrive:
                    od.arrive(arrive, it, e)

        def store(place, gen):
            od.meet(warps, f"{place} {gen} staged")
            s = od.step(warps[0], f"stores {place} {gen}")
            stores[place] = od.event(f"{place} {gen} stored", s)
            od.use(place, "r", gen, s, stores[place])

        def read_by_store(place, arrive):
            od.last[warps[0]] = od.event(f"the leader sees {place} {it} stored", od.last[warps[0]], stores[place])
            od.arrive(arrive, it, od.last[warps[0]])

        each("decays", write=[("suf", it)])
        for w in warps:
            run(w, epi[0], it)
        od.meet(warps, f"scores {it}")
        each("reads the scores", read=[("A", it), ("B", it), ("suf", it)])
        each("A and B", epi[1] if GATED else None, write=[("PA", b), ("PB", b)], arrive="G_P")
        for w in warps:
            run(w, epi[2], it)
        od.meet(warps, f"dV {it}")
        each("dV", read=[("D", it), ("A'", b)], write=[("PA", b + 0.5)], arrive="G_ACCFREE")
        store("PA", b + 0.5)
        for w in warps:
            run(w, epi[3], it)
        od.meet(warps, f"dK {it}")
        # dK over K, dQ over Q: a thread reads the pieces of K and Q that it writes over
        each("dK", read=[("C", it), ("B'", b)], write=[("K", b)])
        store("K", b)
        read_by_store("PA", "G_PAFREE")
        for w in warps:
            run(w, epi[4], it)
        od.meet(warps, f"dQ {it}")
        each("dQ", read=[("D'", b), ("A''", b)], write=[("Q", b)], arrive="G_ENDFREE")
        if GATED:
            each("sums", write=[("PB", b + 0.5)], arrive="G_DOTS")
        store("Q", b)
        read_by_store("K", "G_KFREE")
        read_by_store("Q", "G_QFREE")

        for w in dwarps if GATED else ():
            for cond, more, reads, arrive in ((0, {}, ("X", a), "G_RHREAD"), (1, {}, ("PA", a), "G_RLREAD"),
                                              (2, dict(part=0), ("X", b), None), (2, dict(part=1), ("V", b), "G_SREAD")):
                run(w, dots[cond], it, **more)
                e = od.step(w, f"reads {reads} {it}")
                od.use(*reads[:1], "r", reads[1], e)
                if arrive:
                    od.arrive(arrive, it, e)
            od.use(f"dots[{it & 1}]", "w", it, od.step(w, f"dot {it}"))
        if GATED:
            for w in dwarps:
                run(w, dots[3], it)
            od.meet(dwarps, f"dots {it}")
            e = od.step(dwarps[0], f"the gate's gradient {it}")
            od.use(f"dots[{it & 1}]", "r", it, e)
            od.use("PB", "r", b + 0.5, e)

    # the accumulators share columns: A, A' and A'' are one, as are B and B', D and D'
    for base, others in (("A", ("A'", "A''")), ("B", ("B'",)), ("D", ("D'",))):
        order = {base: 0.0, others[0]: 0.3, others[-1]: 0.6 if len(others) > 1 else 0.3}
        merged = []
        for place, shift in order.items():
            for kind, gen, first, last in od.uses.pop(place):
                merged.append((kind, (gen if place == base else (gen - 1) // 2) + shift, first, last))
        od.uses[base] = merged
    return od


@pytest.mark.parametrize("n", [1, 2, 3, 4, 7])
@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("store", [True, False])
def test_state_kernel(n, gated, store):
    assert state_kernel(n, gated, store).faults() == []


@pytest.mark.parametrize("n", [1, 2, 3, 5])
@pytest.mark.parametrize("gated", [True, False])
def test_gradient_kernel(n, gated):
    assert grad_kernel(n, gated).faults() == []


@pytest.mark.parametrize("n", [1, 2, 3, 4, 5, 9])
@pytest.mark.parametrize("gated", [True, False])
def test_main_kernel(n, gated):
    assert out_kernel(n, gated).faults() == []


@pytest.mark.parametrize("drop,place,kernel", [
    ("done(C_FREE, i - 2)", "X", lambda: state_kernel(5, True, True)),
    ("done(C_DSFREE, i - 2)", "dS", lambda: state_kernel(5, True, True)),
    ("wait_before(G_ENDFREE)", "C", lambda: grad_kernel(3, True)),
    ("wait(G_RLREAD)", "PA", lambda: grad_kernel(3, True)),
    ("wait(G_RHREAD)", "X", lambda: grad_kernel(3, True)),
    ("wait_before(G_SREAD)", "X", lambda: grad_kernel(3, True)),
    ("wait_before(G_PAFREE)", "PA", lambda: grad_kernel(3, True)),
    ("wait_before(G_QFREE)", "Q", lambda: grad_kernel(3, False)),
    ("wait_all(G_ACCFREE)", "A", lambda: grad_kernel(3, False))])
def test_the_models_see_a_missing_wait(monkeypatch, drop, place, kernel):
    waits = _waits
    monkeypatch.setitem(globals(), "_waits", lambda s: [w.replace(drop, "True") for w in waits(s)])
    assert any(f.startswith(place) for f in kernel().faults())


@pytest.mark.parametrize("drop,place", [("done(B_PV, c - 2)", "scores"), ("done(B_DSFREE, c - 1)", "dS"),
                                        ("done(B_DS, c - 1)", "VT"), ("done(B_OFREE, c - 1)", "QS"),
                                        ("done(B_OFREE, 0)", "decays")])
def test_the_model_sees_a_missing_wait(monkeypatch, drop, place):
    """The same programs with one of the waits left out of what was read."""
    waits, drop = _waits, _python(drop)
    monkeypatch.setitem(globals(), "_waits", lambda s: [w.replace(drop, "True") for w in waits(s)])
    assert any(f.startswith(place) for f in out_kernel(9, True).faults())
