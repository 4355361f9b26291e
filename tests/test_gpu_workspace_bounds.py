"""GPU tests of the workspaces of key weights and shared decode: they lie inside a larger buffer, and what is before and
behind them stays as it was.  Tolerances are those of the calls' own tests."""
import pytest

from tests import share_reference as ref
from tests import test_gpu_evict as ev
from tests import test_gpu_shared as sh
from tests.gpu_common import lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lk():
    return lib()


class Fenced:
    """``n`` bytes of workspace with ``room`` bytes of a pattern on either side."""

    def __init__(self, n, room):
        import torch
        room = max(room, 256) + 255 & ~255
        self.all = torch.full((2 * room + n,), 0xA5, dtype=torch.uint8, device="cuda")
        self.ws, self.lo, self.hi = self.all[room:room + n], room, room + n

    def check(self):
        assert (self.all[:self.lo] == 0xA5).all() and (self.all[self.hi:] == 0xA5).all()


def votes(lk, name, case=None):
    if case is None:
        return ev.Votes(lk, name)
    ev.WEIGHTS[name] = case
    try:
        return ev.Votes(lk, name)
    finally:
        del ev.WEIGHTS[name]


def run(lk, v):
    x = v.x
    # behind the workspace: room for every sum that any call could write
    f = Fenced(v.ws.numel(), 16 * x.Hkv * x.B * x.max_blocks * 16 * 4)
    f.ws.fill_(0xFF)
    v.ws = f.ws
    v.check(v.run())
    f.check()
    assert lk.device_status() == 0


@pytest.mark.parametrize("name", ev.WEIGHTS)
def test_key_weights_stay_inside(lk, name):
    run(lk, votes(lk, name))


@pytest.mark.parametrize("kind", ["alibi", "rope"])
@pytest.mark.parametrize("tokens,G", [(65, 1), (17, 4), (33, 4), (128, 4), (200, 4), (300, 4)])
def test_one_request_of_several_groups(lk, tokens, G, kind):
    """One short list, so that every 64 (ALiBi) or 128 query rows of a KV head become a group of their own."""
    run(lk, votes(lk, "one", ([[70, 233]], [tokens], [tokens], 0, 2 * G, 2, 128, sh.pos_of(kind))))


@pytest.mark.parametrize("kind", ["alibi", "rope"])
def test_one_long_request_among_short_ones(lk, kind):
    run(lk, votes(lk, "uneven", ([[70, 233], [9], [40]], [90, 3, 1], [90, 3, 1], 0, 8, 2, 64, sh.pos_of(kind, 64))))


@pytest.mark.parametrize("name", sh.CASES)
def test_shared_decode_stays_inside(lk, name):
    x = sh.lists(name)
    g = sh.OnGpu(lk, x)
    f = Fenced(g.ws.numel(), 1 << 20)
    f.ws.fill_(0xFF)
    g.ws = f.ws
    sh.check(*g.decode(), ref.decode(x))
    f.check()
    assert lk.device_status() == 0
