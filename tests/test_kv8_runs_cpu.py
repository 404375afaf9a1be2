"""The 8-bit document pass's plan and barriers, host side.

The kernel's roles (loaders, converters, MMA issuer, softmax warps of two streams)
are walked as programs of waits and arrivals over the library's own list of runs,
with a vector clock each.  A wait tells a barrier's phase from the next one only by
parity, so a phase must not complete before every waiter has seen the one before
it, whatever the timing: the arrivals that complete phase k + 1 have to come after
every wait for phase k, and a role's arrival k + 1 after phase k is complete.
Memory that is used again (queries, page scales, accumulators) is checked alike.
"""
import itertools

import pytest

from shared_context_decode_b200 import build as ppbuild


@pytest.fixture(scope="module")
def pp():
    ppbuild.build()
    from shared_context_decode_b200 import ppattn
    return ppattn


class Fault(Exception):
    pass


class Walk:
    """Runs role programs; a program yields
    ("wait", barrier, k)  return once phase k of the barrier is complete
    ("arrive", barrier)   its next arrival, the k-th one belonging to phase k
    ("mark", name)        remember this moment
    ("after", name)       this moment must come after the marked one, if there is one
    """

    def __init__(self, programs, arrivals):
        self.names = list(programs)
        self.prog = [programs[n] for n in self.names]
        self.arrivals = arrivals            # barrier -> arrivals a phase takes
        n = len(self.names)
        self.vc = [[0] * n for _ in range(n)]
        self.phases = {}                    # barrier -> [(arrivals, clock)]
        self.sent = {}                      # (role, barrier) -> arrivals made
        self.waits = {}                     # (barrier, k) -> [(role, time)]
        self.marks = {}

    def join(self, a, b):
        for i, x in enumerate(b):
            if x > a[i]:
                a[i] = x

    def done(self, bar, k):
        ph = self.phases.get(bar, [])
        return k < len(ph) and ph[k][0] == self.arrivals(bar)

    def step(self, i, op):
        vc = self.vc[i]
        if op[0] == "wait":
            if not self.done(op[1], op[2]):
                return False
            self.join(vc, self.phases[op[1]][op[2]][1])
            vc[i] += 1
            self.waits.setdefault((op[1], op[2]), []).append((i, vc[i]))
            return True
        vc[i] += 1
        if op[0] == "mark":
            self.marks.setdefault(op[1], []).append((i, vc[i]))
        elif op[0] == "after":
            for j, t in self.marks.get(op[1], []):
                if vc[j] < t:
                    raise Fault(f"{self.names[i]} is not behind {op[1]} of {self.names[j]}")
        else:
            bar = op[1]
            k = self.sent.get((i, bar), 0)
            self.sent[i, bar] = k + 1
            ph = self.phases.setdefault(bar, [])
            while len(ph) <= k:
                ph.append([0, [0] * len(vc)])
            if k and not (self.done(bar, k - 1) and
                          all(x >= y for x, y in zip(vc, ph[k - 1][1]))):
                raise Fault(f"{self.names[i]} arrives at {bar} before its phase {k - 1} is complete")
            ph[k][0] += 1
            self.join(ph[k][1], vc)
        return True

    def run(self):
        cur = [next(p, None) for p in self.prog]
        moved = True
        while moved:
            moved = False
            for i, p in enumerate(self.prog):
                while cur[i] is not None and self.step(i, cur[i]):
                    cur[i] = next(p, None)
                    moved = True
        if any(c is not None for c in cur):
            raise Fault(f"stuck: {[(n, c) for n, c in zip(self.names, cur) if c]}")
        for (bar, k), ws in self.waits.items():
            if self.done(bar, k + 1):
                clock = self.phases[bar][k + 1][1]
                for i, t in ws:
                    if clock[i] < t:
                        raise Fault(f"{bar} may complete phase {k + 1} before {self.names[i]} has "
                                    f"seen phase {k}")


NF, INFO = 4, 8


def walk_cta(runs, d):
    """runs: (tiles, two M tiles, bits of the streams with a tile)."""
    apart = d == 64
    NR = 2 if apart else 1

    def loader(kinds):
        kt = 0
        for n, _, _ in runs:
            for _ in range(n):
                for kv in kinds:
                    sl, f = kt % NR, kt // NR
                    if f:
                        yield "wait", f"raw_empty{kv}.{sl}", f - 1
                    if apart or kv == 0:
                        yield "after", f"scales read {kt - INFO}"
                    yield "arrive", f"raw_full{kv}.{sl}"
                kt += 1

    def converter(kinds):
        kt = 0
        for n, _, _ in runs:
            for _ in range(n):
                for kv in kinds:
                    ft = 2 * kt + kv
                    yield "wait", f"raw_full{kv}.{kt % NR}", kt // NR
                    if ft >= NF:
                        yield "wait", f"f_empty{ft % NF}", ft // NF - 1
                    yield "mark", f"scales read {kt}"
                    yield "arrive", f"raw_empty{kv}.{kt % NR}"
                    yield "arrive", f"f_full{ft % NF}"
                kt += 1

    def mma():
        t0, nq, np_ = 0, [0, 0], [0, 0]

        def wait_f(half):
            return "wait", f"f_full{half % NF}", half // NF

        def scores(r, st, half, two):
            yield wait_f(half)
            yield "mark", f"queries read {r}.{st}"
            yield "arrive", f"s_full{st}"
            if not two or st == 1:
                yield "arrive", f"f_empty{half % NF}"

        for r, (n, two, has) in enumerate(runs):
            step = 1 if two else 2
            for st in range(2):
                if not has >> st & 1:
                    continue
                yield "wait", f"q_full{st}", nq[st]
                nq[st] += 1
                tile = 0 if two else st
                if tile < n:
                    yield from scores(r, st, 2 * (t0 + tile), two)
            for i in range(2 * n if two else n):
                st, tile = i & 1, i >> 1 if two else i
                hv = 2 * (t0 + tile) + 1
                yield wait_f(hv)
                yield "wait", f"p_full{st}", np_[st]
                np_[st] += 1
                if tile < step:                     # overwrites the accumulator
                    yield "after", f"result read {st}"
                if not two or st == 1:
                    yield "arrive", f"f_empty{hv % NF}"
                if tile + step < n:
                    yield from scores(r, st, 2 * (t0 + tile + step), two)
                else:
                    yield "arrive", f"o_done{st}"
            t0 += n

    def softmax(st):
        t0 = ns = no = 0
        for r, (n, two, has) in enumerate(runs):
            first, step = (0, 1) if two else (st, 2)
            if has >> st & 1:
                for b in range(r):
                    yield "after", f"queries read {b}.{st}"
                yield "arrive", f"q_full{st}"
            for tile in range(first, n, step):
                yield "wait", f"s_full{st}", ns
                ns += 1
                yield "mark", f"scales read {t0 + tile}"
                yield "arrive", f"p_full{st}"
            if first < n:
                yield "wait", f"o_done{st}", no
                no += 1
                yield "mark", f"result read {st}"
            t0 += n

    W = 2        # warps a role
    programs = {"mma": mma()}
    for kinds in ([(0,), (1,)] if apart else [(0, 1)]):
        programs[f"loader{kinds}"] = loader(kinds)
        for w in range(W):
            programs[f"converter{kinds}.{w}"] = converter(kinds)
    for st, w in itertools.product(range(2), range(W)):
        programs[f"softmax{st}.{w}"] = softmax(st)
    many = ("raw_empty", "f_full", "q_full", "p_full")
    Walk(programs, lambda bar: W if bar.startswith(many) else 1).run()


def by_cta(plan):
    out = {}
    for cta, _, _, n, two, has in plan["runs"]:
        out.setdefault(cta, []).append((n, two, has))
    return out


def short(runs):
    """A long run cut where the barriers' parities repeat (every eight tiles)."""
    return tuple((n if n < 16 else 8 + n % 8, two, has) for n, two, has in runs)


# rows a key head: one M tile, two, a further group of one, a further group of two
ROWS = (64, 256, 300, 400)


def test_the_runs_cover_every_tile_once(pp):
    for H, rows, N, splits in ((32, 64, 4096, 0), (3, 300, 2100, 7), (1, 1, 5000, 1000),
                               (5, 513, 129, 11), (64, 128, 2000, 0), (2, 8192, 12000, 4000)):
        p = pp.kv8_runs(rows, H, H, N, splits=splits)
        tiles = -(-N // 128)
        assert p["C"] > 0 and p["units"] == H * -(-rows // 256)
        seen = {}
        for cta, u, j0, n, two, has in p["runs"]:
            assert n > 0 and 0 <= j0 and j0 + n <= tiles and 0 <= cta < p["C"]
            assert two == (rows - u % (p["units"] // H) * 256 > 128)
            seen.setdefault(u, []).append((cta, j0, n))
        assert sorted(seen) == list(range(p["units"]))
        for u, x in seen.items():
            assert [c for c, _, _ in x] == sorted({c for c, _, _ in x})
            assert len(x) <= p["max_chunks"]
            at = 0
            for _, j0, n in x:
                assert j0 == at
                at += n
            assert at == tiles


@pytest.mark.parametrize("splits", [46340, 46341, 60000, 100351, 2 ** 31 - 1])
def test_more_splits_than_32_bit_products_hold(pp, splits):
    """256 questions of 32 rows, 32 heads, behind 12000 tokens: 100352 steps."""
    p = pp.kv8_runs(8192, 32, 32, 12000, decode=False, splits=splits)
    assert 0 < p["C"] and p["C"] * (p["W"] % p["C"]) < 2 ** 31
    at = {}
    for cta, u, j0, n, _, _ in p["runs"]:
        assert 0 <= u < p["units"] and 0 <= cta < p["C"] and j0 == at.get(u, 0)
        at[u] = j0 + n
    assert at == dict.fromkeys(range(p["units"]), -(-12000 // 128))
    # the workspace is that of the same plan
    slots = p["units"] * p["max_chunks"] * 256
    size = pp.kv8_prefill_workspace_bytes(8192, 32, 32, 128, 12000, pp.Options(splits=splits))
    assert 0 <= size - slots * (128 + 2) * 4 < 1024


def test_a_stream_takes_part_in_a_run_only_with_a_tile(pp):
    """Every head count to 64, documents to 8192 tokens."""
    lone = 0
    for H, rows, tiles in itertools.product(range(1, 65), (64, 300), range(1, 65)):
        for _, _, _, n, two, has in pp.kv8_runs(rows, H, H, tiles * 128 - 5, splits=0)["runs"]:
            assert has == (3 if two or n > 1 else 1), (H, rows, tiles, n, two)
            lone += has == 1
    assert lone > 1000      # runs of one tile are ordinary


@pytest.mark.parametrize("d", [64, 128])
def test_no_barrier_passes_its_waiter(pp, d):
    seqs = set()
    for H, rows in itertools.product(range(1, 65), ROWS):
        for tiles in sorted({1, 2, 3, 5, 8, 13, 16, 21, 24, 27, 30, 33, 40, 47, 55, 64}):
            for splits in (0, 37):
                p = pp.kv8_runs(rows, H, H, tiles * 128, splits=splits)
                seqs.update(short(r)[:6] for r in by_cta(p).values())
    assert len(seqs) > 500
    # every sequence of up to four runs that has a lone tile, the others sampled
    seqs = sorted(seqs)
    pick = [s for i, s in enumerate(seqs) if i % 7 == 0 or any(h == 1 for _, _, h in s)]
    for s in pick:
        walk_cta(s, d)


@pytest.mark.parametrize("d", [64, 128])
def test_the_walk_sees_an_arrival_without_a_tile(pp, d):
    """The rule broken on purpose, in the list: both streams arrive in every run."""
    p = pp.kv8_runs(64, 32, 32, 4096)
    bad = [r for r in by_cta(p).values() if any(h == 1 for _, _, h in r[:-1])]
    assert bad
    for r in bad:
        walk_cta(short(r), d)
        with pytest.raises(Fault, match="q_full1"):
            walk_cta(tuple((n, two, 3) for n, two, _ in short(r)), d)
