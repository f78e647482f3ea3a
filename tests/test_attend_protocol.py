"""The mbarrier protocol of the paged attention's tensor-core kernel
(attend_tc_kernel in csrc/sfa_paged_attend_tc.cu), modelled on the CPU.

A CTA walks pieces of 1 .. n key tiles.  Its roles: a warp that loads keys and
q, a warp that loads values, a warp that issues the products, and four warps
per stream for the softmax.  With PAIR both streams take every tile in one
step; without, they take the tiles in turn, in two steps each, or a step each of
an only tile.

Each role is a generator that waits and arrives in the kernel's order.  A wait
passes as the hardware's parity wait does.  Random interleavings must finish,
and every wait must pass on exactly the phase it means.  Copies and products
complete at once, or late: a late product's commit is an extra role that may
run at any time but keeps the order in which products were issued.
"""
import random

import pytest

WARPS = 4  # of a stream


class _Bar:
    def __init__(self, name, count):
        self.name, self.count, self.pending, self.done = name, count, 0, 0

    def arrive(self):
        self.pending += 1
        assert self.pending <= self.count, f"{self.name}: more arrivals than its count"
        if self.pending == self.count:
            self.pending, self.done = 0, self.done + 1


def _roles(pieces, pair, ns, q_bufs, rng, epilogue="o_done", clean_first=False):
    steps = 1 if pair else 2
    few = not pair and q_bufs == 2  # up to 64 rows: results leave from registers
    B = {}

    def bar(*key, count=1):
        return B.setdefault(key, _Bar(str(key), count))

    for s in range(2):
        for h in range(steps):
            bar("p_full", s, h, count=WARPS)
    bar("cta", count=2 * WARPS)
    wait = lambda key, phase: ("wait", bar(*key), phase)
    tensor = []  # commits in the order of issue

    def k_pos(i, n):
        return 2 * i if pair else (i if i < 2 else 2 * i - 1)

    def v_pos(i, n):
        return 2 * i + 1 if pair else (1 if n == 1 else min(2 * i + 2, n + i))

    def loads(keys):
        base = n_q = 0
        for n, _ in pieces:
            for i in range(n):
                at = base + (k_pos(i, n) if keys else v_pos(i, n))
                if at >= ns:
                    yield wait(("kv_empty", at % ns), at // ns - 1)
                bar("kv_full", at % ns).arrive()
                if keys and i == (0 if pair else min(n, 2) - 1):
                    if n_q >= q_bufs:
                        yield wait(("q_empty", n_q % q_bufs), n_q // q_bufs - 1)
                    bar("q_full", n_q % q_bufs).arrive()
                    n_q += 1
            base += 2 * n

    def mma():
        at = n_q = 0
        n_p = [[0, 0], [0, 0]]
        commit = lambda *key: tensor.append(bar(*key))

        def qk(s, h):
            commit("s_full", s, h)

        def pv(s, h):
            if steps > 1:
                commit("o_step", s)

        for n, _ in pieces:
            qb = n_q % q_bufs
            yield wait(("q_full", qb), n_q // q_bufs)
            n_q += 1
            if pair:
                yield wait(("kv_full", at % ns), at // ns)
                st_k, at = at % ns, at + 1
                for s in range(2):
                    qk(s, 0)
                commit("kv_empty", st_k)
                if n == 1:
                    commit("q_empty", qb)
                for i in range(n):
                    more = i + 1 < n
                    yield wait(("kv_full", at % ns), at // ns)
                    st_v, at = at % ns, at + 1
                    for s in range(2):
                        yield wait(("p_full", s, 0), n_p[s][0])
                        n_p[s][0] += 1
                        pv(s, 0)
                        if more and s == 0:
                            yield wait(("kv_full", at % ns), at // ns)
                            st_k, at = at % ns, at + 1
                        if more:
                            qk(s, 0)
                    if more:  # the last values' buffer is the softmax's, for its result
                        commit("kv_empty", st_v)
                        commit("kv_empty", st_k)
                    if i + 2 == n:
                        commit("q_empty", qb)
                    if not more:
                        commit("o_done", 0)
                        commit("o_done", 1)
            elif n == 1:  # one tile: a half for each stream
                yield wait(("kv_full", at % ns), at // ns)
                st_k, at = at % ns, at + 1
                qk(0, 0)
                qk(1, 1)
                commit("kv_empty", st_k)
                commit("q_empty", qb)
                yield wait(("kv_full", at % ns), at // ns)
                st_v, at = at % ns, at + 1
                for s in range(2):
                    yield wait(("p_full", s, s), n_p[s][s])
                    n_p[s][s] += 1
                    pv(s, s)
                if few:
                    commit("kv_empty", st_v)
                commit("o_done", 0)
            else:
                for i in range(2):
                    yield wait(("kv_full", at % ns), at // ns)
                    st_k, at = at % ns, at + 1
                    for h in range(steps):
                        qk(i, h)
                    commit("kv_empty", st_k)
                if n == 2:
                    commit("q_empty", qb)
                for i in range(n):
                    s, more = i & 1, i + 2 < n
                    yield wait(("kv_full", at % ns), at // ns)
                    st_v, at = at % ns, at + 1
                    for h in range(steps):
                        yield wait(("p_full", s, h), n_p[s][h])
                        n_p[s][h] += 1
                        pv(s, h)
                        if more and h == 0:
                            yield wait(("kv_full", at % ns), at // ns)
                            st_k, at = at % ns, at + 1
                        if more:
                            qk(s, h)
                    if i + 1 < n or few:
                        commit("kv_empty", st_v)
                    if more:
                        commit("kv_empty", st_k)
                    if i + 3 == n:
                        commit("q_empty", qb)
                commit("o_done", 0)
        tensor.append(None)  # no more

    def completions():
        while True:
            while not tensor:
                yield ("poll", None, None)
            b = tensor.pop(0)
            if b is None:
                return
            b.arrive()
            yield ("poll", None, None)

    def softmax(s, warp):
        n_o = n_piece = base = n_bar = 0
        n_s = [0, 0]

        def cta():
            nonlocal n_bar
            bar("cta").arrive()
            n_bar += 1
            return wait(("cta",), n_bar - 1)

        for n, masked in pieces:
            halves = not pair and n == 1
            for i in range(0 if pair or halves else s, n, 1 if pair else 2):
                at = base + v_pos(i, n)
                clean = masked and i >= n - 2 and (not pair or s == 0)
                if clean and clean_first:  # planted: before the scores
                    yield wait(("kv_full", at % ns), at // ns)
                for h in range(steps):
                    if halves and h != s:
                        continue
                    yield wait(("s_full", s, h), n_s[h])
                    n_s[h] += 1
                    if clean and h == 0:
                        yield wait(("kv_full", at % ns), at // ns)
                    first = halves or (h == 0 and (i == 0 if pair else i < 2))
                    if steps > 1 and not first and rng.random() < 0.3:  # the maximum moved
                        yield wait(("o_step", s), n_o - 1)
                    bar("p_full", s, h).arrive()
                    n_o += 1
            base += 2 * n
            if epilogue == "o_done":
                yield wait(("o_done", s if pair else 0), n_piece)
            else:  # planted: the last two steps by their own barrier
                for k in range(max(0, n_o - 2), n_o):
                    yield wait(("o_step", s), k)
            n_piece += 1
            if not pair:
                yield cta()
            yield cta()
            if s == 0 and warp == 0 and not few:
                bar("kv_empty", (base - 1) % ns).arrive()

    return [loads(True), loads(False), mma(), completions()] + [softmax(s, w) for s in range(2) for w in range(WARPS)]


def _run(pieces, pair, ns, q_bufs, seed, epilogue="o_done", clean_first=False):
    rng = random.Random(seed)
    roles = _roles(pieces, pair, ns, q_bufs, rng, epilogue, clean_first)
    pending = [None] * len(roles)
    alive = set(range(len(roles)))
    pause = [rng.choice((0.05, 0.3, 0.9)) for _ in roles]
    skip = [rng.choice((0.0, 0.0, 0.5, 0.9)) for _ in roles]
    all_in, idle = False, 0
    while alive:
        progress = 0
        for r in sorted(alive, key=lambda _: rng.random()):
            if not all_in and rng.random() < skip[r]:
                continue
            while True:
                if pending[r] is not None and pending[r][0] == "wait":
                    _, b, phase = pending[r]
                    if (b.done & 1) != (phase & 1):  # the hardware's parity wait passes
                        assert b.done == phase + 1, f"{b.name}: wait for phase {phase} passed at {b.done}"
                        progress += 1
                    else:
                        assert b.done == phase, f"{b.name}: waiting for phase {phase} with {b.done} done"
                        break
                    pending[r] = None
                polled = pending[r] is not None
                try:
                    pending[r] = next(roles[r])
                    progress += not polled
                except StopIteration:
                    alive.discard(r)
                    progress += 1
                    break
                if pending[r][0] == "poll" or rng.random() < pause[r]:
                    break
        idle = 0 if progress else idle + 1
        all_in = idle > 0
        assert idle < 50, "deadlock"


def _pieces(rng):
    return [(rng.choice((1, 1, 2, 3, 4, 9)), rng.random() < 0.7) for _ in range(rng.randint(1, 8))]


@pytest.mark.parametrize("pair,ns,q_bufs", [(True, 5, 1), (True, 11, 1), (False, 6, 1), (False, 6, 2), (False, 12, 1),
                                            (False, 12, 2)])
def test_attend_pipeline_finishes_on_the_phases_it_means(pair, ns, q_bufs):
    for seed in range(250):
        _run(_pieces(random.Random(seed)), pair, ns, q_bufs, seed)


def _caught(**planted):
    n = 0
    for seed in range(250):
        try:
            _run(_pieces(random.Random(seed)), False, 6, 1, seed, **planted)
        except AssertionError:
            n += 1
    return n


def test_waiting_for_the_last_steps_by_their_own_barrier_is_caught():
    """A wait for the last but one step may come after the last one: a parity
    wait cannot tell that phase from the next, and runs out."""
    assert _caught(epilogue="o_step") > 0


def test_waiting_for_values_before_their_scores_is_caught():
    """The buffer may then be two fills behind: a parity wait passes on the old
    one, and the clean-up would meet the copy."""
    assert _caught(clean_first=True) > 0
