"""The 4-bit prefill's barrier protocol in the host-side model (no GPU).

q4_prefill_kernel differs from prefill_tc_kernel in how operands reach the tensor cores: packed keys
land in a 2-stage ring and packed values in a single stage; one role turns the keys, another the
values into operand rings of 2 stages each.  With one live Q tile in every CTA (key halves) the softmax and
MMA roles are the model's own; otherwise a tile's keys are taken in halves, with a score buffer for each Q
tile and half.  Random interleavings must show no deadlock, no wait ahead of or two phases
behind a barrier, and no stage or metadata slot reused too early; planted mistakes must be caught.
"""
import random

import pytest

from tests import prefill_protocol_model as pm


class Q4Sim(pm.Sim):
    def __init__(self, n, nq, seed=0, slots=6, kh=False):
        super().__init__(n, nq, seed=seed, slots=slots, kst=2, kh=kh)
        self.PK_FULL = [pm.Bar(f"PK_FULL{s}", 1) for s in range(2)]
        self.PK_FREE = [pm.Bar(f"PK_FREE{s}", 1) for s in range(2)]
        self.PV_FULL, self.PV_FREE = pm.Bar("PV_FULL", 1), pm.Bar("PV_FREE", 1)
        self.V_READY = [pm.Bar(f"V_READY{s}", 1) for s in range(2)]
        self.half_qk, self.half_pv = set(), set()
        self.S_HALF = [pm.Bar(f"S_HALF{i}", 1) for i in range(4)]
        self.P_HALF = [pm.Bar(f"P_HALF{i}", 1) for i in range(4)]
        self.PV_HALF = [pm.Bar(f"PV_HALF{i}", 1) for i in range(2)]
        self.packed = {"K": [None, None], "V": [None]}   # landed tile of each packed stage
        self.pending = {"K": [False, False], "V": [False]}  # landed and not read yet

    # packed copies
    def issue_tma(self, kind, j, bar):
        st = j % len(self.packed[kind])
        if self.pending[kind][st]:
            raise pm.ProtocolError(f"packed {kind}({j}) issued into stage {st} before it was read")
        self.pending[kind][st] = True
        self.tma.append((kind, st, j, bar, self.now + self.rng.randint(0, self.max_latency)))

    def step_tma(self):
        i = self.rng.choice(self.tma_ready())
        kind, st, j, bar, _ = self.tma.pop(i)
        self.packed[kind][st] = j
        bar.complete_tx(1)

    def producer(self):
        def issue_k(j):
            s = j % 2
            if j >= 2:
                yield ("wait", self.PK_FREE[s], j // 2 - 1)
            self.publish(j)
            self.PK_FULL[s].arrive(expect_tx=1)
            self.issue_tma("K", j, self.PK_FULL[s])
            yield ("step",)

        yield from issue_k(0)
        for j in range(self.n):
            if j + 1 < self.n:
                yield from issue_k(j + 1)
            if j >= 1:
                yield ("wait", self.PV_FREE, j - 1)
            self.PV_FULL.arrive(expect_tx=1)
            self.issue_tma("V", j, self.PV_FULL)
            yield ("step",)

    def wait_free(self, bars, j):
        if j >= 2:
            yield ("wait", bars[j % 2], j // 2 - 1)

    def dequantise(self, kind, j, users, stages, holder):
        ring, st = self.packed[kind], j % len(self.packed[kind])
        if ring[st] != j:
            raise pm.ProtocolError(f"dequantisation of {kind}({j}) finds packed {ring[st]}")
        self.read_slot(j, f"dequantise {kind}")
        if users[j % 2]:
            raise pm.ProtocolError(f"{kind}({j}) written into stage {j % 2} while {sorted(users[j % 2])} still use it")
        holder[j % 2] = j
        users[j % 2] = {stages + "0"} | ({stages + "1"} if self.nq == 2 else set())
        self.pending[kind][st] = False

    def rotation(self):  # the keys' role
        for j in range(self.n):
            yield ("wait", self.PK_FULL[j % 2], j // 2)
            yield from self.wait_free(self.K_FREE, j)
            self.dequantise("K", j, self.kstage_users, "qk", self.kstage)
            yield ("step",)
            self.PK_FREE[j % 2].arrive()
            self.K_READY[j % 2].arrive()

    def values(self):
        for j in range(self.n):
            yield ("wait", self.PV_FULL, j)
            yield from self.wait_free(self.V_FREE, j)
            self.dequantise("V", j, self.vstage_users, "pv", self.vstage)
            yield ("step",)
            self.PV_FREE.arrive()
            self.V_READY[j % 2].arrive()

    def actors(self):
        return super().actors() | {"values": self.values()}

    def mma_wait_v(self, jj):
        yield ("wait", self.V_READY[jj % 2], jj // 2)

    # ---- halves of tiles: step x = 2 j + h
    def qk_half(self, q, x):
        j, h = x >> 1, x & 1
        buf, st = 2 * q + h, (x >> 1) % 2

        def run():
            if self.kstage[st] != j:
                raise pm.ProtocolError(f"QK{q}({x}) reads K stage {st} holding {self.kstage[st]}")
            prev = self.s_buf.get(buf)
            if prev is not None and (prev[0] != "P" or (q, prev[1]) not in self.half_pv):
                raise pm.ProtocolError(f"QK{q}({x}) overwrites {prev} in S{buf}")
            self.s_buf[buf] = ("S", x)
            self.half_qk.add((q, x))
            if h == 1:
                self.done_qk.add((q, j))
                self.kstage_users[st].discard(f"qk{q}")
        self.pipe.append(("mma", run))
        self.commit(self.S_HALF[buf])

    def pv_half(self, q, x):
        j, h = x >> 1, x & 1
        buf, st = 2 * q + h, j % 2

        def run():
            if self.vstage[st] != j:
                raise pm.ProtocolError(f"PV{q}({x}) reads V stage {st} holding {self.vstage[st]}")
            if self.s_buf.get(buf) != ("P", x):
                raise pm.ProtocolError(f"PV{q}({x}) reads S{buf} holding {self.s_buf.get(buf)}")
            self.half_pv.add((q, x))
            if h == 1:
                self.done_pv.add((q, j))
                self.vstage_users[st].discard(f"pv{q}")
        self.pipe.append(("mma", run))
        self.commit(self.PV_HALF[q])

    def softmax(self, i):
        if self.kh:
            yield from super().softmax(i)
            return
        self.Q_READY.arrive()
        if i >= self.nq:
            return
        yield ("step",)
        for x in range(2 * self.n):
            j, buf = x >> 1, 2 * i + (x & 1)
            yield ("wait", self.S_HALF[buf], j)
            if self.s_buf.get(buf) != ("S", x):
                raise pm.ProtocolError(f"softmax{i} reads S{buf} for step {x}, holds {self.s_buf.get(buf)}")
            self.read_slot(j, f"softmax{i}")
            yield ("step",)
            if x > 0 and self.rng.random() < 0.3:  # a rescale of O; the other steps leave the phase unwaited
                yield from self.wait_pv(i, x)
                if (i, x - 1) not in self.half_pv:
                    raise pm.ProtocolError(f"softmax{i} rescales O before PV({x - 1})")
            self.read_slot(j, f"softmax{i}")
            self.s_buf[buf] = ("P", x)
            self.P_HALF[buf].arrive()
        yield ("wait", self.FINAL, 0)

    def wait_pv(self, i, x):
        yield ("wait", self.PV_HALF[i], x - 1)

    def mma(self):
        if self.kh:
            yield from super().mma()
            return
        yield ("wait", self.Q_READY, 0)
        yield ("wait", self.K_READY[0], 0)
        for h in range(2):
            for q in range(self.nq):
                self.qk_half(q, h)
        self.commit(self.K_FREE[0])
        for x in range(2 * self.n):
            j, more = x >> 1, (x >> 1) + 1 < self.n
            for q in range(self.nq):
                yield ("wait", self.P_HALF[2 * q + (x & 1)], j)
                if q == 0 and not x & 1:
                    yield ("wait", self.V_READY[j % 2], j // 2)
                self.pv_half(q, x)
                if more:
                    if q == 0 and not x & 1:
                        yield ("wait", self.K_READY[(j + 1) % 2], (j + 1) // 2)
                    self.qk_half(q, x + 2)
            if x & 1:
                self.commit(self.V_FREE[j % 2])
                if more:
                    self.commit(self.K_FREE[(j + 1) % 2])
        self.commit(self.FINAL)
        yield ("wait", self.FINAL, 0)

    def run(self, *a):
        if self.kh:
            return super().run(*a)
        steps = super().run(*a)
        want = {(q, x) for q in range(self.nq) for x in range(2 * self.n)}
        if self.half_qk != want or self.half_pv != want:
            raise pm.ProtocolError("not every half ran")
        return steps

    def read_slot(self, j, who):
        if not who.startswith("mma"):  # this kernel's MMA thread reads no metadata
            super().read_slot(j, who)


def _schedules(n_runs, seed0=0):
    for seed in range(seed0, seed0 + n_runs):
        rng = random.Random(seed)
        yield seed, rng.choice([1, 2, 3, 4, 5, 8, 9, 16, 17]), rng.choice([1, 2])


@pytest.mark.parametrize("part", range(4))
def test_protocol_is_safe_under_random_interleavings(part):
    for seed, n, nq in _schedules(400, seed0=400 * part):
        for kh in (False, True):
            try:
                Q4Sim(n, nq, seed=seed, kh=kh).run()
            except pm.ProtocolError as e:
                pytest.fail(f"seed {seed}, {n} tiles, {nq} live Q tiles, key halves {kh}: {e}")


def _caught(cls, **kw):
    caught = 0
    for seed, n, nq in _schedules(200):
        try:
            cls(n, nq, seed=seed, **kw).run()
        except pm.ProtocolError:
            caught += 1
    return caught


def test_model_catches_too_few_metadata_slots():
    assert _caught(Q4Sim, slots=3) > 0


def test_model_catches_operands_written_before_their_products_are_done():
    class NoWait(Q4Sim):
        def wait_free(self, bars, j):
            yield ("step",)
    assert _caught(NoWait) > 0


def test_model_catches_a_rescale_that_does_not_wait():
    class NoWait(Q4Sim):
        def wait_pv(self, i, x):
            yield ("step",)
    assert _caught(NoWait) > 0


def test_model_catches_packed_values_overwritten():
    class Early(Q4Sim):
        def producer(self):
            for x in super().producer():
                if x[0] == "wait" and x[1] is self.PV_FREE:
                    continue
                yield x
    assert _caught(Early) > 0
