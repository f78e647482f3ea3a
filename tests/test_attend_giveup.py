"""How attend_tc_kernel (csrc/sfa_paged_attend_tc.cu) ends when a bounded wait
runs out, modelled on the CPU.

The roles and barriers are those of test_attend_protocol, but a wait may fail at
any time, and copies and products complete late.  Whatever fails, every role has
to end, nothing may still be on its way into shared or tensor memory when the
CTA leaves, no barrier may get more arrivals than its phase takes, and no buffer
may be filled while it is being filled.
"""
import random

import pytest

WARPS = 4  # of a stream


class Bar:
    def __init__(self, name, count):
        self.name, self.count, self.pending, self.done, self.flying = name, count, 0, 0, 0

    def arrive(self, flying=0):
        assert self.pending < self.count, f"{self.name}: more arrivals than its phase takes"
        self.pending += 1
        self.flying += flying
        self._close()

    def land(self):
        self.flying -= 1
        self._close()

    def _close(self):
        if self.pending == self.count and self.flying == 0:
            self.pending, self.done = 0, self.done + 1


class Model:
    def __init__(self, pieces, pair, ns, few, rng, fail, old_exit=False):
        self.pieces, self.pair, self.ns, self.few, self.rng, self.fail, self.old = pieces, pair, ns, few, rng, fail, old_exit
        self.q_bufs = 2 if few else 1
        self.steps = 1 if pair else 2
        self.bars, self.flight, self.tensor = {}, [], []
        self.fills = [0] * ns       # of every ring buffer
        self.q_fills = [0] * self.q_bufs
        self.ended = 0
        self.bad = False

    def bar(self, *key, count=1):
        if key[0] == "p_full":
            count = WARPS
        elif key[0] == "softmax":
            count = 2 * WARPS
        elif key[0] == "end":
            count = 3 + 2 * WARPS
        return self.bars.setdefault(key, Bar(str(key), count))

    def wait(self, key, phase, sure=False):
        """Yields until the wait passes (True) or runs out (False)."""
        return (yield (self.bar(*key), phase, sure))

    def barrier(self, name, n):
        """A CTA barrier, which has no limit."""
        b = self.bar(name)
        b.arrive()
        yield (b, n, True)

    def k_pos(self, i, n):
        return 2 * i if self.pair else (i if i < 2 else 2 * i - 1)

    def v_pos(self, i, n):
        return 2 * i + 1 if self.pair else (1 if n == 1 else min(2 * i + 2, n + i))

    def copy(self, bar):
        bar.arrive(flying=1)
        self.flight.append(bar)

    def loads(self, keys):
        ok, base, n_q, last, filled = True, 0, 0, 0, 0
        for n, _ in self.pieces:
            for i in range(n):
                at = base + (self.k_pos(i, n) if keys else self.v_pos(i, n))
                if at >= self.ns:
                    ok = yield from self.wait(("kv_empty", at % self.ns), at // self.ns - 1)
                if not ok:
                    break
                full = self.bar("kv_full", at % self.ns)
                assert full.flying == 0, "filled while it is being filled"
                self.copy(full)
                self.fills[at % self.ns] += 1
                last, filled = at, filled + 1
                if keys and i == (0 if self.pair else min(n, 2) - 1):
                    qb = n_q % self.q_bufs
                    if n_q >= self.q_bufs:
                        ok = yield from self.wait(("q_empty", qb), n_q // self.q_bufs - 1)
                    if not ok:
                        break
                    self.copy(self.bar("q_full", qb))
                    self.q_fills[qb] += 1
                    n_q += 1
            if not ok:
                break
            base += 2 * n
        if self.old and not ok:  # the exit as it was: each role for itself
            for at in range(0 if last < self.ns else last - self.ns + 1, last + 1 if filled else 0):
                yield from self.wait(("kv_full", at % self.ns), at // self.ns)
            for i in range(max(0, n_q - self.q_bufs), n_q):
                yield from self.wait(("q_full", i % self.q_bufs), i // self.q_bufs)
        yield from self.leave(ok)

    def mma(self):
        ok = yield from self.products()
        if self.old and not ok:
            self.tensor.append(self.bar("drain"))
            yield from self.wait(("drain",), 0)
        yield from self.leave(ok)
        if not self.old and self.bad:  # nothing in flight outlives the CTA
            self.tensor.append(self.bar("drain"))
            yield from self.wait(("drain",), 0, sure=True)
            for st in range(self.ns):
                if self.fills[st]:
                    yield from self.wait(("kv_full", st), self.fills[st] - 1, sure=True)
            for qb in range(self.q_bufs):
                if self.q_fills[qb]:
                    yield from self.wait(("q_full", qb), self.q_fills[qb] - 1, sure=True)

    def products(self):
        at = n_q = 0
        n_p = [[0, 0], [0, 0]]
        commit = lambda *key: self.tensor.append(self.bar(*key))  # noqa: E731
        pair, ns, steps, few = self.pair, self.ns, self.steps, self.few

        def pv(s):
            if steps > 1:
                commit("o_step", s)

        for n, _ in self.pieces:
            qb = n_q % self.q_bufs
            if not (yield from self.wait(("q_full", qb), n_q // self.q_bufs)):
                return False
            n_q += 1
            if pair:
                if not (yield from self.wait(("kv_full", at % ns), at // ns)):
                    return False
                st_k, at = at % ns, at + 1
                commit("s_full", 0, 0)
                commit("s_full", 1, 0)
                commit("kv_empty", st_k)
                if n == 1:
                    commit("q_empty", qb)
                for i in range(n):
                    more = i + 1 < n
                    if not (yield from self.wait(("kv_full", at % ns), at // ns)):
                        return False
                    st_v, at = at % ns, at + 1
                    for s in range(2):
                        if not (yield from self.wait(("p_full", s, 0), n_p[s][0])):
                            return False
                        n_p[s][0] += 1
                        pv(s)
                        if more and s == 0:
                            if not (yield from self.wait(("kv_full", at % ns), at // ns)):
                                return False
                            st_k, at = at % ns, at + 1
                        if more:
                            commit("s_full", s, 0)
                    if more:
                        commit("kv_empty", st_v)
                        commit("kv_empty", st_k)
                    if i + 2 == n:
                        commit("q_empty", qb)
                    if not more:
                        commit("o_done", 0)
                        commit("o_done", 1)
            elif n == 1:
                if not (yield from self.wait(("kv_full", at % ns), at // ns)):
                    return False
                st_k, at = at % ns, at + 1
                commit("s_full", 0, 0)
                commit("s_full", 1, 1)
                commit("kv_empty", st_k)
                commit("q_empty", qb)
                if not (yield from self.wait(("kv_full", at % ns), at // ns)):
                    return False
                st_v, at = at % ns, at + 1
                for s in range(2):
                    if not (yield from self.wait(("p_full", s, s), n_p[s][s])):
                        return False
                    n_p[s][s] += 1
                    pv(s)
                if few:
                    commit("kv_empty", st_v)
                commit("o_done", 0)
            else:
                for i in range(2):
                    if not (yield from self.wait(("kv_full", at % ns), at // ns)):
                        return False
                    st_k, at = at % ns, at + 1
                    for h in range(steps):
                        commit("s_full", i, h)
                    commit("kv_empty", st_k)
                if n == 2:
                    commit("q_empty", qb)
                for i in range(n):
                    s, more = i & 1, i + 2 < n
                    if not (yield from self.wait(("kv_full", at % ns), at // ns)):
                        return False
                    st_v, at = at % ns, at + 1
                    for h in range(steps):
                        if not (yield from self.wait(("p_full", s, h), n_p[s][h])):
                            return False
                        n_p[s][h] += 1
                        pv(s)
                        if more and h == 0:
                            if not (yield from self.wait(("kv_full", at % ns), at // ns)):
                                return False
                            st_k, at = at % ns, at + 1
                        if more:
                            commit("s_full", s, h)
                    if i + 1 < n or few:
                        commit("kv_empty", st_v)
                    if more:
                        commit("kv_empty", st_k)
                    if i + 3 == n:
                        commit("q_empty", qb)
                commit("o_done", 0)
        return True

    def softmax(self, s, warp):
        ok, n_o, n_piece, base, n_bar = True, 0, 0, 0, 0
        n_s = [0, 0]
        pair, ns, few = self.pair, self.ns, self.few
        for n, masked in self.pieces:
            halves = not pair and n == 1
            for i in range(0 if pair or halves else s, n, 1 if pair else 2):
                if not ok:
                    break
                at = base + self.v_pos(i, n)
                for h in range(self.steps):
                    if halves and h != s:
                        continue
                    ok = yield from self.wait(("s_full", s, h), n_s[h])
                    n_s[h] += 1
                    if ok and masked and h == 0 and (not pair or s == 0):
                        ok = yield from self.wait(("kv_full", at % ns), at // ns)
                    first = halves or (h == 0 and (i == 0 if pair else i < 2))
                    if ok and self.steps > 1 and not first and self.rng.random() < 0.3:
                        ok = yield from self.wait(("o_step", s), n_o - 1)
                    if not ok:
                        break
                    self.bar("p_full", s, h).arrive()
                    n_o += 1
            base += 2 * n
            if ok:
                ok = yield from self.wait(("o_done", s if pair else 0), n_piece)
            if not pair:
                yield from self.barrier("softmax", n_bar)
                n_bar += 1
            yield from self.barrier("softmax", n_bar)
            n_bar += 1
            if s == 0 and warp == 0 and not few and (ok or self.old):
                self.bar("kv_empty", (base - 1) % ns).arrive()
            n_piece += 1
        yield from self.leave(ok)

    def leave(self, ok):
        self.bad = self.bad or not ok
        yield from self.barrier("end", 0)

    def run(self):
        rng = self.rng
        roles = [self.loads(True), self.loads(False), self.mma()] + [self.softmax(s, w) for s in range(2) for w in range(WARPS)]
        want = [None] * len(roles)
        alive = dict.fromkeys(range(len(roles)))
        speed = [rng.choice((0.1, 0.5, 1.0)) for _ in roles]
        lag = rng.choice((0.02, 0.2, 0.7))
        failed = idle = 0

        def step(r, value):
            try:
                want[r] = roles[r].send(value)
            except StopIteration:
                del alive[r]

        for r in list(alive):
            step(r, None)
        while alive:
            moved = False
            if self.flight and rng.random() < lag:
                self.flight.pop(rng.randrange(len(self.flight))).land()
                moved = True
            if self.tensor and rng.random() < lag:   # in the order of issue
                self.tensor.pop(0).arrive()
                moved = True
            for r in list(alive):
                if rng.random() > speed[r]:
                    continue
                bar, phase, sure = want[r]
                if (bar.done & 1) != (phase & 1):
                    # (a barrier of the whole CTA may be a phase ahead when the last of it looks)
                    assert failed or sure or bar.done == phase + 1, f"{bar.name}: passed on another phase than {phase}"
                    step(r, True)
                    moved = True
                elif not sure and rng.random() < self.fail(r, failed, idle):
                    failed += 1
                    step(r, False)
                    moved = True
            idle = 0 if moved else idle + 1
            if idle > 400 and not self.flight and not self.tensor:
                raise AssertionError("a role does not end")
        assert not self.flight, "a copy is on its way into shared memory of a CTA that has left"
        assert not self.tensor, "a product is on its way when tensor memory is given back"
        return failed


def _pieces(rng):
    return [(rng.choice((1, 1, 2, 3, 4, 9)), rng.random() < 0.7) for _ in range(rng.randint(1, 6))]


def _first(role, when):
    """Role `role` gives up after some polls, the others once nothing moves."""
    def fail(r, failed, idle):
        if failed == 0:
            return when if r == role else 0.0
        return 0.3 if idle > 30 else 0.0
    return fail


def _any(p):
    return lambda r, failed, idle: p if idle <= 30 or failed == 0 else 0.3


KINDS = [(True, 5, False), (True, 11, False), (False, 6, False), (False, 6, True), (False, 12, False), (False, 12, True)]


@pytest.mark.parametrize("pair,ns,few", KINDS)
def test_no_wait_runs_out_in_a_good_run(pair, ns, few):
    for seed in range(60):
        rng = random.Random(seed)
        assert Model(_pieces(rng), pair, ns, few, rng, lambda *_: 0.0).run() == 0


@pytest.mark.parametrize("pair,ns,few", KINDS)
@pytest.mark.parametrize("role", ["keys", "values", "products", "softmax 0", "softmax 1", "any"])
def test_every_role_may_give_up(pair, ns, few, role):
    r = {"keys": 0, "values": 1, "products": 2, "softmax 0": 3, "softmax 1": 3 + WARPS}.get(role)
    ran_out = 0
    for seed in range(150):
        rng = random.Random(seed)
        when = rng.choice((0.02, 0.3, 1.0))
        fail = _any(when * 0.1) if r is None else _first(r, when)
        ran_out += Model(_pieces(rng), pair, ns, few, rng, fail).run() > 0
    assert ran_out > 20


def test_an_exit_of_each_role_for_itself_is_caught():
    """The roles' own exits, and a softmax that returns a buffer after a wait
    that ran out."""
    caught = set()
    for pair, ns, few in KINDS:
        for seed in range(600):
            rng = random.Random(seed)
            fail = _first(rng.choice((2, 3, 7)), 0.3) if seed % 2 else _any(rng.choice((0.002, 0.03)))
            try:
                Model(_pieces(rng), pair, ns, few, rng, fail, old_exit=True).run()
            except AssertionError as e:
                caught.add(str(e).split("\n")[0])
    assert {c[:10] for c in caught} >= {"a copy is ", "a product ", "filled whi"}, caught
