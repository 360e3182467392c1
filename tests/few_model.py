"""A model of the few-token kernel's barrier protocol, run as random
interleavings of its roles on the CPU.

Every role is a generator that yields where it may be overtaken.  Waits on
barriers look at the parity only, as the hardware does, and the model checks
that the phase behind the parity is the one that was meant; that no scale slot
is overwritten before every promotion warp has read it; that the stuck roles of
a launch with a withheld tile all come to an end; that each thread waits for
each phase of the cluster's barrier exactly once; and that every tile copy has
been waited for by the time its CTA may exit.
"""
import random


class Bar:
    """An mbarrier: `count` arrivals complete a phase."""

    def __init__(self, count):
        self.count, self.left, self.phase = count, count, 0

    def arrive(self):
        self.left -= 1
        if self.left == 0:
            self.phase += 1
            self.left = self.count

    def passes(self, want):
        """Parity wait for phase `want`."""
        ok = ((self.phase - 1) & 1) == (want & 1)
        assert not ok or self.phase - 1 == want, f"parity of phase {want} passed in phase {self.phase - 1}"
        return ok


class Cluster:
    """barrier.cluster: every thread arrives and waits in turn."""

    def __init__(self, threads):
        self.arrived = dict.fromkeys(threads, 0)
        self.waited = dict.fromkeys(threads, 0)

    def arrive(self, t):
        assert self.arrived[t] == self.waited[t], "a second arrive before the wait for the first"
        self.arrived[t] += 1

    def wait(self, t):
        assert self.waited[t] < self.arrived[t], "a wait for the cluster without an arrive"
        phase = self.waited[t]
        while any(a <= phase for a in self.arrived.values()):
            yield
        self.waited[t] += 1


class Rank:
    def __init__(self, c, S, work):
        self.work = work
        self.full = [Bar(2) for _ in range(c["stages"])]
        self.empty = [Bar(1) for _ in range(c["stages"])]
        self.sc = [Bar(1) for _ in range(c["slots"])]
        self.tfull = [Bar(1) for _ in range(c["buffers"])]
        self.tempty = [Bar(c["epi_warps"]) for _ in range(c["buffers"])]
        warps = c["epi_warps"] if c["ring"] else 4
        self.red_full = [Bar(warps * S) for _ in range(2)]
        self.red_empty = [Bar(warps * S) for _ in range(2)]
        self.values = [None] * c["slots"]             # the block whose scales a slot holds
        self.queue = [[] for _ in range(c["mma_warps"])]
        self.copies, self.seen = set(), set()         # (block, role) requested; waited for at the end
        self.expired = 0
        self.left = 0                                 # roles that have not reached the CTA's last barrier


def run(c, work, S=1, meetings=0, withhold=None, seed=0, patience=None, count_first=True, wait_copies=True):
    """One launch of a cluster of S ranks.  work[r]: K blocks of rank r's
    segments.  After the last segment the promotion warps meet `meetings` times.
    withhold: rank 0's weight tile that is never requested.  count_first,
    wait_copies: False plants the form without that care.  Returns how many
    waits expired."""
    rng = random.Random(seed)
    ranks = [Rank(c, S, work[r]) for r in range(S)]
    stages, slots, buffers = c["stages"], c["slots"], c["buffers"]
    tok_warps, mma_warps, epi_warps = c["token_warps"], c["mma_warps"], c["epi_warps"]
    names = (["tma"] + [f"tok{w}" for w in range(tok_warps)] + [f"mma{w}" for w in range(mma_warps)]
             + [f"epi{q}" for q in range(epi_warps)])
    cluster = Cluster([(r, n) for r in range(S) for n in names])
    for t in cluster.arrived:
        if S > 1:
            cluster.arrive(t)                         # before the roles part

    def bounded(bar, want, k):
        """A bounded wait: False when it expires."""
        tries = 0
        while not bar.passes(want):
            tries += 1
            if patience is not None and tries > patience * rng.uniform(0.7, 1.3):
                k.expired += 1
                return False
            yield
        return True

    def stage_free(k, u):
        return (yield from bounded(k.empty[u % stages], u // stages - 1, k)) if u >= stages else True

    def leave(r, name, waited):
        """The CTA's last barrier and the cluster's second phase."""
        k = ranks[r]
        k.left -= 1
        while k.left:
            yield
        if S > 1:
            if not waited:
                yield from cluster.wait((r, name))
            cluster.arrive((r, name))
            yield from cluster.wait((r, name))
        missing = k.copies - k.seen
        assert not missing, f"copies {sorted(missing)[:3]} may land after the CTA's exit"

    def tma(r):
        k, total, it = ranks[r], sum(work[r]), 0
        while it < total:
            if not (yield from stage_free(k, it)):
                break
            if not (r == 0 and it == withhold):
                k.copies.add((it, "tma"))
                k.full[it % stages].arrive()
            it += 1
            yield
        for u in range(max(0, it - stages), it):
            yield from bounded(k.full[u % stages], u // stages, k)
        # the wait for a block's barrier is one for both its copies; blocks before the last ring were consumed
        k.seen |= {(u, n) for u in range(it) for n in ("tma", "tok")}
        yield from leave(r, "tma", False)

    def tok(r, w):
        k, total = ranks[r], sum(work[r])
        own = [u for u in range(total) if (u % stages) % tok_warps == w]
        done = []
        for u in own:
            if not (yield from stage_free(k, u)):
                break
            k.values[u % slots] = u
            if c["copies"]:
                k.copies.add((u, "tok"))
            yield
            k.full[u % stages].arrive()
            k.sc[u % slots].arrive()
            done.append(u)
            yield
        if wait_copies and c["copies"]:
            end = own[len(done)] if len(done) < len(own) else total
            for u in done:
                if u >= end - stages:
                    yield from bounded(k.full[u % stages], u // stages, k)
            k.seen |= {(u, "tok") for u in done}
        yield from leave(r, f"tok{w}", False)

    def pairs_of(r):
        """(pair number, first block, blocks) over all segments."""
        pair = it = 0
        for n in work[r]:
            for kb in range(0, n, 2):
                yield pair, it, min(2, n - kb)
                it += min(2, n - kb)
                pair += 1

    def mma(r, me):
        k, ok = ranks[r], True
        for pair, it, blocks in pairs_of(r):
            if pair % mma_warps != me:
                continue
            b = pair % buffers
            got = pair < buffers or (yield from bounded(k.tempty[b], pair // buffers - 1, k))
            for h in range(blocks):
                s = (it + h) % stages
                got = got and (yield from bounded(k.full[s], (it + h) // stages, k))
                if not got:
                    ok = False
                    break
                k.queue[me].append((s, b if h + 1 == blocks else None))
                yield
            if not ok:
                break
        while k.queue[me]:                            # its own MMAs, which complete without anyone's help
            yield
        yield from leave(r, f"mma{me}", False)

    def pipe(r, me):
        """The tensor core: the MMAs of an issuer complete in order."""
        k = ranks[r]
        while True:
            if k.queue[me]:
                s, b = k.queue[me][0]
                k.empty[s].arrive()
                if b is not None:
                    k.tfull[b].arrive()
                k.queue[me].pop(0)
            yield

    def epi(r, q):
        k, name, ok = ranks[r], f"epi{q}", True
        grp = 0 if c["groups"] == 1 else q // 4
        for pair, it, blocks in pairs_of(r):
            b = pair % buffers
            ok = yield from bounded(k.tfull[b], pair // buffers, k)
            for h in range(blocks):
                ok = ok and (yield from bounded(k.sc[(it + h) % slots], (it + h) // slots, k))
            if not ok:
                break
            for _ in range(2):                        # at the start and at the end of its reads
                for h in range(blocks):
                    assert k.values[(it + h) % slots] == it + h, "scales overwritten"
                yield
            k.tempty[b].arrive()
            yield
        meets = 0
        if c["ring"]:
            if S > 1:
                yield from cluster.wait((r, name))
                if ok:
                    for o in ranks:
                        o.red_empty[0].arrive()
                    ok = yield from bounded(k.red_empty[0], 0, k)
                if ok:
                    for o in ranks:
                        o.red_full[0].arrive()
                    ok = yield from bounded(k.red_full[0], 0, k)
                meets = 1
        else:
            for m in range(meetings if S > 1 else 0):
                if not ok:
                    break
                if meets == 0:
                    yield from cluster.wait((r, name))
                if count_first:
                    meets += 1
                if m > 0:
                    ok = yield from bounded(k.red_empty[grp], m - 1, k)
                if not ok:
                    break
                for o in ranks:
                    o.red_full[grp].arrive()
                    yield
                ok = yield from bounded(k.red_full[grp], m, k)
                if not ok:
                    break
                for o in ranks:
                    o.red_empty[grp].arrive()
                if not count_first:
                    meets += 1
        if S > 1 and meets == 0:
            yield from cluster.wait((r, name))
        yield from leave(r, name, True)

    live, engines = [], []
    for r in range(S):
        roles = ([tma(r)] + [tok(r, w) for w in range(tok_warps)] + [mma(r, i) for i in range(mma_warps)]
                 + [epi(r, q) for q in range(epi_warps)])
        ranks[r].left = len(roles)
        live += roles
        engines += [pipe(r, i) for i in range(mma_warps)]
    speed = [rng.choice([1, 1, 3, 10]) for _ in live]
    steps = 0
    while live:
        for e in engines:
            if rng.random() < 0.3:
                next(e)
        for i in rng.choices(range(len(live)), speed, k=min(8, len(live))):
            if i < len(live):
                try:
                    next(live[i])
                except StopIteration:
                    live.pop(i), speed.pop(i)
        steps += 1
        assert steps < 400_000, "a role waits for good"
    return sum(k.expired for k in ranks)
