"""The 4-bit prefill's barrier protocol in the host-side model (no GPU).

q4_prefill_kernel differs from prefill_tc_kernel in how operands reach the tensor cores: packed keys
land in a 2-stage ring, packed values in a single stage (4 and 2 where the softmax warpgroups share one
Q tile by halves of its keys); one role turns the keys, another the values into operand rings of 2 stages
each.  Softmax and MMA roles are the model's own.  Random interleavings must show no deadlock, no wait
ahead of or two phases behind a barrier, and no stage or metadata slot reused too early; planted mistakes
must be caught.
"""
import random

import pytest

from tests import prefill_protocol_model as pm


class Q4Sim(pm.Sim):
    def __init__(self, n, nq, seed=0, slots=8, kh=False):
        super().__init__(n, nq, seed=seed, slots=slots, kst=2, kh=kh)
        self.pkst, self.vst = pk, pv = (4, 2) if self.kh else (2, 1)
        self.PK_FULL = [pm.Bar(f"PK_FULL{s}", 1) for s in range(pk)]
        self.PK_FREE = [pm.Bar(f"PK_FREE{s}", 1) for s in range(pk)]
        self.PV_FULL = [pm.Bar(f"PV_FULL{s}", 1) for s in range(pv)]
        self.PV_FREE = [pm.Bar(f"PV_FREE{s}", 1) for s in range(pv)]
        self.V_READY = [pm.Bar(f"V_READY{s}", 1) for s in range(2)]
        self.packed = {"K": [None] * pk, "V": [None] * pv}   # landed tile of each packed stage
        self.pending = {"K": [False] * pk, "V": [False] * pv}  # landed and not read yet

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
            s, n = j % self.pkst, j // self.pkst
            if n >= 1:
                yield ("wait", self.PK_FREE[s], n - 1)
            self.publish(j)
            self.PK_FULL[s].arrive(expect_tx=1)
            self.issue_tma("K", j, self.PK_FULL[s])
            yield ("step",)

        def issue_v(j):
            s, n = j % self.vst, j // self.vst
            if n >= 1:
                yield ("wait", self.PV_FREE[s], n - 1)
            self.PV_FULL[s].arrive(expect_tx=1)
            self.issue_tma("V", j, self.PV_FULL[s])
            yield ("step",)

        lead = self.pkst - 1
        for i in range(lead + self.n):
            if self.kh and i >= lead:
                yield from issue_v(i - lead)
            if i < self.n:
                yield from issue_k(i)
            if not self.kh and i >= lead:
                yield from issue_v(i - lead)

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
            yield ("wait", self.PK_FULL[j % self.pkst], j // self.pkst)
            yield from self.wait_free(self.K_FREE, j)
            self.dequantise("K", j, self.kstage_users, "qk", self.kstage)
            yield ("step",)
            self.PK_FREE[j % self.pkst].arrive()
            self.K_READY[j % 2].arrive()

    def values(self):
        for j in range(self.n):
            yield ("wait", self.PV_FULL[j % self.vst], j // self.vst)
            yield from self.wait_free(self.V_FREE, j)
            self.dequantise("V", j, self.vstage_users, "pv", self.vstage)
            yield ("step",)
            self.PV_FREE[j % self.vst].arrive()
            self.V_READY[j % 2].arrive()

    def actors(self):
        return super().actors() | {"values": self.values()}

    def mma_wait_v(self, jj):
        yield ("wait", self.V_READY[jj % 2], jj // 2)

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


def test_model_catches_packed_values_overwritten():
    class Early(Q4Sim):
        def producer(self):
            for x in super().producer():
                if x[0] == "wait" and x[1] in self.PV_FREE:
                    continue
                yield x
    assert _caught(Early) > 0
    assert _caught(Early, kh=True) > 0
