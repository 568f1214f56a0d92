"""A model of the weight gradients' barriers, for one CTA pair, in the manner of
product_model.py: every mbarrier, every warp that waits or arrives, and the
asynchronous copies and products, with random delays, warps that come late and
releases that arrive in any order.  Tiles are given by their rows: none (zeros are
written, no product), whole steps of 16, or ragged ends that pass through the
CTA's own barrier and the warp that clears rows.

Its numbers come from the kernel's source, so a change there is a change of the
model.
"""
import heapq
import os
import random
import re

from tests.product_model import Bar, Fault

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                      "combine_moonep_plan_gb300", "csrc", "wgrad.cu")


def constants():
    """The kernel's integer constants and its barriers' arrival counts, by name."""
    c, text = {}, open(SOURCE).read()
    for name, value in re.findall(r"^constexpr int (k\w+) = ([^;]+);", text, re.M):
        c[name] = eval(value.replace("/", "//"), {}, c)
    for name, value in re.findall(r"init\(&sh->(\w+)\[\w\], ([^;]+)\);", text):
        if name != "tile_empty":
            c[name] = eval(value, {}, c)
    loads = text[text.index("if (warp == 0) {"):text.index("} else if (warp == 1) {")]
    c["drain"] = "wait(sh, &sh->empty[q]" in loads
    return c


def run(c, tiles, seed, clear=True):
    """Tiles of so many rows on one pair; raises Fault.  clear=False: ragged stages
    arrive like others and the clearing warp only looks at them (a form that the
    kernel does not use)."""
    rnd = random.Random(seed)
    S, deep, part = c["kStages"], c["kDeep"], c["kPart"]
    warps = c["kEpilogueWarps"]
    readers = (c["kTileReaders"] + 1, c["kTileReaders"])
    now, order, events = [0.0], [0], []

    def at(t, f):
        order[0] += 1
        heapq.heappush(events, (t, order[0], f))

    def bars(r, name, count, n):
        return [Bar("%s[%d] of CTA %d" % (name, i, r), count) for i in range(n)]

    cta = [dict(full=bars(r, "full", c["full"], S), empty=bars(r, "empty", c["empty"], S),
                tail=bars(r, "tail", c["tail"], S),
                acc_full=bars(r, "acc_full", c["acc_full"], 2),
                acc_empty=bars(r, "acc_empty", c["acc_empty"], 2),
                tile_full=bars(r, "tile_full", c["tile_full"], 2),
                tile_empty=bars(r, "tile_empty", readers[r], 2))
           for r in range(2)]
    lead = cta[0]
    held = [[None] * S for _ in range(2)]      # the stage whose rows lie there,
    cleared = [[None] * S for _ in range(2)]   # and the ragged one that was cleared
    batch, read = [[None, None] for _ in range(2)], [{} for _ in range(2)]
    acc, acc_read = [None, None], [[0, 0] for _ in range(2)]
    done, pipe = [0], [0.0]  # products of stages finished; when the pipe is free

    def stages_of(rows):
        return -(-rows // deep)

    def take_tile(r, i):
        if i % 32 == 0:
            yield cta[r]["tile_full"][i // 32 % 2], i // 64 % 2
        if batch[r][i // 32 % 2] != i // 32:
            raise Fault("tile of another batch")
        if i % 32 == 31:
            read[r][i // 32] = read[r].get(i // 32, 0) + 1
            cta[r]["tile_empty"][i // 32 % 2].arrive()

    def schedule(r):
        for b in range(-(-len(tiles) // 32)):
            yield cta[r]["tile_empty"][b % 2], (b // 2 % 2) ^ 1
            if b >= 2 and read[r].get(b - 2) != readers[r]:
                raise Fault("tiles overwritten")
            yield rnd.random() * 5
            batch[r][b % 2] = b
            cta[r]["tile_full"][b % 2].arrive()

    def loads(r):
        s = phase = g = 0
        for i, rows in enumerate(tiles):
            yield from take_tile(r, i)
            n = stages_of(rows)
            for k in range(n):
                yield cta[r]["empty"][s], phase ^ 1
                yield rnd.random()
                ragged = clear and k == n - 1 and rows % 16
                bar = cta[r]["tail"][s] if ragged else lead["full"][s]
                # the leader expects both CTAs' bytes, the other CTA only arrives
                bar.arrive(tx=1 if ragged else 2 if r == 0 else 0)

                def landed(s=s, g=g, r=r, bar=bar):
                    if done[0] < g - S + 1:
                        raise Fault("rows overwritten")
                    held[r][s] = g
                    bar.copied()
                at(now[0] + rnd.uniform(2, 30), landed)
                g += 1
                s, phase = (0, phase ^ 1) if s == S - 1 else (s + 1, phase)
        for q in range(S if c["drain"] else 0):
            yield cta[r]["empty"][q], phase if q < s else phase ^ 1

    def clears(r):
        s, g, use = 0, 0, 0
        for i, rows in enumerate(tiles):
            yield from take_tile(r, i)
            n = stages_of(rows)
            s, g = (s + n) % S, g + n
            if not rows % 16 or not clear:
                continue
            q = (s + S - 1) % S
            yield cta[r]["tail"][q], use >> q & 1
            use ^= 1 << q
            if held[r][q] != g - 1:
                raise Fault("rows of another stage cleared")
            yield rnd.random() * rnd.choice((1, 1, 20))
            if held[r][q] != g - 1:
                raise Fault("rows of another stage cleared")
            cleared[r][q] = g - 1
            lead["full"][q].arrive()

    def products():
        s = phase = g = used = 0
        for i, rows in enumerate(tiles):
            yield from take_tile(0, i)
            n = stages_of(rows)
            for k in range(n):
                if k % part == 0:
                    yield lead["acc_empty"][used & 1], (used >> 1 & 1) ^ 1
                    if used >= 2 and acc_read[0][used & 1] + acc_read[1][used & 1] != \
                            (used >> 1) * 2 * warps:
                        raise Fault("accumulator overwritten")
                    acc[used & 1] = None
                yield lead["full"][s], phase
                for r in range(2):
                    if held[r][s] != g:
                        raise Fault("rows of another stage")
                    if k == n - 1 and rows % 16 and cleared[r][s] != g:
                        raise Fault("rows not cleared")
                yield rnd.random()
                pipe[0] = max(pipe[0], now[0]) + rnd.uniform(1, 4)
                last = k % part == part - 1 or k == n - 1

                def finish(s=s, used=used, last=last):
                    done[0] += 1
                    if last:
                        acc[used & 1] = used
                    # the CTAs hear of it at any time after
                    for t in cta:
                        for bar in [t["empty"][s]] + [t["acc_full"][used & 1]] * last:
                            at(now[0] + rnd.random() * rnd.choice((3, 3, 3, 60)), bar.arrive)
                at(pipe[0], finish)
                used += last
                g += 1
                s, phase = (0, phase ^ 1) if s == S - 1 else (s + 1, phase)

    def epilogue(r):
        used = 0
        for i, rows in enumerate(tiles):
            yield from take_tile(r, i)
            for _ in range(-(-rows // (part * deep))):
                yield cta[r]["acc_full"][used & 1], used >> 1 & 1
                if acc[used & 1] != used:
                    raise Fault("accumulator of another part")
                yield rnd.uniform(0, 12)
                if acc[used & 1] != used:
                    raise Fault("accumulator overwritten")
                acc_read[r][used & 1] += 1
                lead["acc_empty"][used & 1].arrive()
                used += 1
            yield rnd.uniform(0, 6)  # the stores

    live = [[products(), "products", None, 0.0]]
    for r in range(2):
        live += [[f(r), f.__name__, None, 0.0] for f in (schedule, loads, clears)]
        live += [[epilogue(r), "epilogue", None, 0.0] for _ in range(warps)]
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
