"""A model of the expert product's barriers, for one CTA pair: every mbarrier,
every warp that waits or arrives, and the asynchronous copies and products, with
random delays.  It reports a deadlock, an arrival too many, an operand written
before the products that read it are done, a product that reads another stage's
operands, an accumulator or tile batch used by two at once, and an arrival that
reaches a CTA after it has left.

Its numbers come from the kernel's source (constants()), so a change of a
constant there is a change of the model.
"""
import heapq
import os
import random
import re

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                      "combine_moonep_plan_gb300", "csrc", "product.cu")


def constants():
    """The kernel's integer constants, by name; which barrier its scale warps wait
    at for a stage (scales_wait), and whether its load warps wait for the last
    stages to be released before they leave (drain)."""
    c, text = {}, open(SOURCE).read()
    for name, value in re.findall(r"^constexpr int (k\w+) = ([^;]+);", text, re.M):
        c[name] = eval(value.replace("/", "//"), {}, c)
    loads = text[text.index("if (warp == 0) {"):text.index("} else if (warp < 7) {")]
    c["drain"] = "wait(sh, &sh->empty[q]" in loads
    scales = text[text.index("auto fill = "):text.index("auto pass = ")]
    c["scales_wait"], = re.findall(r"wait\(sh, &sh->(\w+)\[s\]", scales)
    assert ("arrive(&sh->passed[s])" in loads) == (c["scales_wait"] == "passed")
    return c


class Fault(Exception):
    pass


class Bar:
    def __init__(self, name, count):
        self.name, self.count, self.left, self.tx, self.phase = name, count, count, 0, 0
        self.gone = False

    def _settle(self):
        if self.left == 0 and self.tx == 0:
            self.phase += 1
            self.left = self.count

    def arrive(self, tx=0):
        if self.gone:
            raise Fault("late arrival at " + self.name)
        self.tx += tx
        self.left -= 1
        if self.left < 0:
            raise Fault("too many arrivals at " + self.name)
        self._settle()

    def copied(self):
        self.tx -= 1
        self._settle()

    def passes(self, parity):
        return (self.phase & 1) != parity


def run(c, tiles, stages, seed, ring=0):
    """`tiles` tiles of `stages` stages on one pair; raises Fault.  ring: the two
    sets of scale warps take their chunks from one shared ring of that many
    boxes, copied there asynchronously, instead of loading them themselves (a
    form that the kernel does not use)."""
    rnd = random.Random(seed)
    S, sets, wide = c["kStages"], c["kScaleSets"], c["kChunkStages"]
    roles, chunks = c["kScaleWarps"], -(-stages // wide)
    readers = (c["kTileReaders"] + 1, c["kTileReaders"])
    per = c["kTileBatch"]
    now, order, events = [0.0], [0], []

    def at(t, f):
        order[0] += 1
        heapq.heappush(events, (t, order[0], f))

    def bars(r, name, count, n):
        return [Bar("%s[%d] of CTA %d" % (name, i, r), count) for i in range(n)]

    cta = [dict(full=bars(r, "full", c["kFullArrivals"], S), empty=bars(r, "empty", 1, S),
                passed=bars(r, "passed", 1, S),
                acc_full=bars(r, "acc_full", 1, 2),
                acc_empty=bars(r, "acc_empty", c["kAccReaders"], 2),
                tile_full=bars(r, "tile_full", 1, 2),
                tile_empty=bars(r, "tile_empty", readers[r], 2),
                box_full=bars(r, "box_full", 1, ring), box_empty=bars(r, "box_empty", roles, ring))
           for r in range(2)]
    lead = cta[0]
    held = [[{} for _ in range(S)] for _ in range(2)]  # operand -> the stage it belongs to
    box = [[None] * max(ring, 1) for _ in range(2)]
    batch, read = [[None, None] for _ in range(2)], [{} for _ in range(2)]
    acc, acc_read = [None, None], [[0, 0] for _ in range(2)]
    done, pipe = [0], [0.0]  # products of stages finished; when the pipe is free

    def put(r, s, what, g):
        if done[0] < g - S + 1:
            raise Fault("operand overwritten")
        held[r][s][what] = g

    def take_tile(r, i):
        if i % per == 0:
            yield cta[r]["tile_full"][i // per % 2], i // per // 2 % 2
        if batch[r][i // per % 2] != i // per:
            raise Fault("tile of another batch")
        if i % per == per - 1:
            read[r][i // per] = read[r].get(i // per, 0) + 1
            cta[r]["tile_empty"][i // per % 2].arrive()

    def schedule(r):
        for b in range(-(-tiles // per)):
            yield cta[r]["tile_empty"][b % 2], (b // 2 % 2) ^ 1
            if b >= 2 and read[r].get(b - 2) != readers[r]:
                raise Fault("tiles overwritten")
            yield rnd.random() * 5
            batch[r][b % 2] = b
            cta[r]["tile_full"][b % 2].arrive()

    def loads(r):
        s = phase = g = 0
        for i in range(tiles):
            yield from take_tile(r, i)
            for _ in range(stages):
                yield cta[r]["empty"][s], phase ^ 1
                cta[r]["passed"][s].arrive()
                yield rnd.random()
                if r == 0:
                    lead["full"][s].arrive(tx=2)

                def landed(s=s, g=g, r=r):
                    put(r, s, "codes", g)
                    lead["full"][s].copied()
                if done[0] < g - S + 1:
                    raise Fault("operand overwritten")
                at(now[0] + rnd.uniform(2, 30), landed)
                g += 1
                s, phase = (0, phase ^ 1) if s == S - 1 else (s + 1, phase)
        for q in range(S if c["drain"] else 0):
            yield cta[r]["empty"][q], phase if q < s else phase ^ 1

    def boxes(r):
        for q in range(tiles * chunks):
            yield cta[r]["box_empty"][q % ring], (q // ring % 2) ^ 1
            yield rnd.random()
            cta[r]["box_full"][q % ring].arrive(tx=1)

            def landed(q=q, r=r):
                box[r][q % ring] = q
                cta[r]["box_full"][q % ring].copied()
            at(now[0] + rnd.uniform(2, 30), landed)

    def scales(r, turn, role):
        pos = [0, 0, 0]  # stage, phase, stages so far

        def skip(n):
            pos[0] += n
            pos[2] += n
            if pos[0] >= S:
                pos[0] -= S
                pos[1] ^= 1
        seen = -1
        nxt = turn  # chunk of the sequence to load next

        def load():
            nonlocal seen, nxt
            while seen < min(nxt // chunks, tiles - 1):
                yield from take_tile(r, seen + 1)
                seen += 1
            nxt += sets
        yield from load()
        yield from load()
        for q in range(tiles * chunks):
            here = min(wide, stages - q % chunks * wide)
            if q % sets != turn:
                skip(here)
                continue
            if ring:
                yield cta[r]["box_full"][q % ring], q // ring % 2
                if box[r][q % ring] != q:
                    raise Fault("scales of another chunk")
                yield rnd.random() * 3
                cta[r]["box_empty"][q % ring].arrive()
            for _ in range(here):
                if c["scales_wait"] == "passed":
                    yield cta[r]["passed"][pos[0]], pos[1]
                else:
                    yield cta[r]["empty"][pos[0]], pos[1] ^ 1
                yield rnd.random() * rnd.choice((1, 1, 20))
                put(r, pos[0], "scales%d" % role, pos[2])
                lead["full"][pos[0]].arrive()
                skip(1)
            yield from load()

    def products():
        s = phase = g = 0
        for i in range(tiles):
            yield from take_tile(0, i)
            yield lead["acc_empty"][i & 1], (i >> 1 & 1) ^ 1
            if i >= 2 and acc_read[0][i & 1] + acc_read[1][i & 1] != (i >> 1) * c["kAccReaders"]:
                raise Fault("accumulator overwritten")
            acc[i & 1] = None
            for k in range(stages):
                yield lead["full"][s], phase
                for h in held:
                    if [h[s].get(w) for w in ["codes"] + ["scales%d" % j for j in range(roles)]] \
                            != [g] * (roles + 1):
                        raise Fault("operand of another stage")
                yield rnd.random()
                pipe[0] = max(pipe[0], now[0]) + rnd.uniform(1, 4)

                def finish(s=s, i=i, last=k == stages - 1):
                    done[0] += 1
                    if last:
                        acc[i & 1] = i
                    # the CTAs hear of it at any time after
                    for t in cta:
                        for bar in [t["empty"][s]] + [t["acc_full"][i & 1]] * last:
                            at(now[0] + rnd.random() * rnd.choice((3, 3, 3, 60)), bar.arrive)
                at(pipe[0], finish)
                g += 1
                s, phase = (0, phase ^ 1) if s == S - 1 else (s + 1, phase)

    def epilogue(r):
        for i in range(tiles):
            yield from take_tile(r, i)
            yield cta[r]["acc_full"][i & 1], i >> 1 & 1
            if acc[i & 1] != i:
                raise Fault("accumulator of another tile")
            yield rnd.uniform(0, 12)
            if acc[i & 1] != i:
                raise Fault("accumulator overwritten")
            acc_read[r][i & 1] += 1
            lead["acc_empty"][i & 1].arrive()

    live = [(products(), "products")]
    for r in range(2):
        live += [(schedule(r), "schedule"), (loads(r), "loads")]
        live += [(epilogue(r), "epilogue") for _ in range(readers[1] - 1 - sets * roles)]
        live += [(scales(r, t, j), "scales") for t in range(sets) for j in range(roles)]
        if ring:
            live.append((boxes(r), "boxes"))
    live = [[g, name, None, 0.0] for g, name in live]
    while live:
        moved = False
        for p in list(live):
            if now[0] < p[3] or p[2] is not None and not p[2][0].passes(p[2][1]):
                continue
            moved = True
            try:
                step = next(p[0])
            except StopIteration:
                live.remove(p)
                continue
            if isinstance(step, tuple):  # a wait, that any warp may come late to
                p[2], p[3] = step, now[0] + rnd.choice((0, 0, 0, 0, 0, 0, 0, 60)) * rnd.random()
            else:
                p[2], p[3] = None, now[0] + step
            at(p[3], lambda: None)
        if not moved:
            if not events:
                raise Fault("deadlock of " + ", ".join(sorted({p[1] for p in live})))
            t, _, f = heapq.heappop(events)
            now[0] = max(now[0], t)
            f()
    # both CTAs have left
    for t in cta:
        for group in t.values():
            for bar in group:
                bar.gone = True
    for _, _, f in events:
        f()
