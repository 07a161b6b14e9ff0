"""Host-side checks of the layer norm's test helpers, and of how its kernels' warps wait for one
another, that need no GPU."""
import random

import pytest

from test_train_host import AT, nsp, refused  # noqa: F401


def probe(nsp, back=False, fed=4, **kw):
    v = dict(x=AT, x_row=8, weight=AT, bias=None, doc=None, N=6, D=8, dtype=nsp.NS_BF16,
             weight_dtype=nsp.NS_F32, eps=1e-5)
    call = dict(mean=AT, rstd=AT, dy=AT, dy_row=8, dx=AT, dweight=AT, dbias=AT, workspace=AT)
    if not back:
        call = dict(y=AT, mean=None, rstd=None)
    for k, x in kw.items():
        (v if k in v else call)[k] = x
    s = nsp._lib.ns_norm_inputs(*v.values())
    f = nsp._lib.ns_norm_probe_backward if back else nsp._lib.ns_norm_probe_forward
    return lambda: f(s, fed, *call.values(), None)


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("kw", [dict(fed=1), dict(fed=5), dict(x=None), dict(x_row=7), dict(dtype=5)])
def test_norm_probe_refuses(nsp, kw, back):
    refused(nsp, probe(nsp, back=back, **kw))


def test_norm_probe_of_nothing_is_ok(nsp):
    probe(nsp, N=0, x=None, y=None)()


# ---- the ring's protocol (csrc/ring.cuh, norm.cuh), step by step ----------------------------
class Barrier:
    """A shared-memory barrier: a phase ends with `count` arrivals and all announced bytes."""

    def __init__(self, count):
        self.count = self.pending = count
        self.bytes = self.phase = 0

    def change(self, arrivals, bytes_):
        assert arrivals <= self.pending, "arrival past the count"
        self.pending -= arrivals
        self.bytes += bytes_
        if self.pending == 0 and self.bytes == 0:
            self.phase += 1
            self.pending = self.count

    def passed(self, parity):
        return (self.phase & 1) != parity


OVER = object()


def run_ring(seed, lost_leave, drain):
    """One block under a random schedule: the warp that copies, copies that arrive in any order,
    warps that compute; waits run out at random.  `lost_leave`: a warp that lost a batch leaves
    its stage all the same; `drain`: the copying warp waits for its last copies."""
    r = random.Random(seed)
    stages, warps, batches = r.randint(2, 4), r.randint(1, 4), r.randint(1, 14)
    full = [Barrier(1) for _ in range(stages)]
    empty = [Barrier(warps) for _ in range(stages)]
    flight, synced, over = [], [0] * warps, [False] * (warps + 1)
    copier_loses, warp_loses = r.choice([0, 0, 0.02]), r.choice([0, 0.02, 0.3])

    def copier():
        stage = turn = 0
        for _ in range(batches):
            gave_up = False
            while turn and not empty[stage].passed((turn - 1) & 1) and not gave_up:
                gave_up = r.random() < copier_loses or all(over[1:])
                yield
            if gave_up:
                break
            assert stage not in flight, "a stage is filled again before its copies have arrived"
            full[stage].change(1, 1)
            flight.append(stage)
            yield
            stage += 1
            if stage == stages:
                stage, turn = 0, turn + 1
        for i in range((stages if turn else stage) if drain else 0):
            while not full[i].passed((turn if i < stage else turn - 1) & 1):
                yield

    def warp(w):
        stage = turn = 0
        lost = False
        for n in range(batches):
            while not lost and not full[stage].passed(turn & 1):
                lost = r.random() < warp_loses or over[0]
                yield
            synced[w] = n + 1
            while min(synced) <= n:  # the exchange of sums
                yield
            if lost_leave or not lost:
                empty[stage].change(1, 0)
            stage += 1
            if stage == stages:
                stage, turn = 0, turn + 1
            yield

    threads = [copier(), *(warp(w) for w in range(warps))]
    while not all(over):
        if flight and r.random() < 0.15:
            full[flight.pop(r.randrange(len(flight)))].change(0, -1)
        i = r.randrange(warps + 1)
        if not over[i]:
            over[i] = next(threads[i], OVER) is OVER
    assert not flight, "the block ended before its copies"


def test_ring_ends_after_its_copies_whichever_wait_runs_out():
    for seed in range(3000):
        run_ring(seed, lost_leave=False, drain=True)


@pytest.mark.parametrize("kw,what", [
    (dict(lost_leave=True, drain=True), "filled again"),
    (dict(lost_leave=False, drain=False), "ended before its copies")])
def test_ring_needs_both_rules(kw, what):
    with pytest.raises(AssertionError, match=what):
        for seed in range(3000):
            run_ring(seed, **kw)
