"""Evictions while another stream records errors or clears them: a call goes by what its own check found, so
it moves all rows and weights or none."""
import time

import pytest
import torch

from tests.test_gpu_evict import Cache, pa  # noqa: F401
from tests.test_gpu_spec_bounds import Clearing

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Call:
    """An eviction that can be made again over the same start."""

    def __init__(self, pa, lens, new, Hkv, D, tables=None):
        c = Cache(lens, Hkv, D, seed=len(lens))
        self.arrays = [c.kb.view(torch.uint8), c.vb.view(torch.uint8), c.w]
        self.start = [t.clone() for t in self.arrays]
        self.ws = torch.zeros(pa.pa_evict_keys_workspace_size(len(lens), Hkv, c.tables.shape[1], 16),
                              dtype=torch.uint8, device="cuda")
        args = (c.kb, c.vb, c.tables if tables is None else tables(c), i32(lens), i32(new), c.w, 4, 32)
        self.run = lambda stream=None: pa.pa_evict_keys(*args, workspace=self.ws, stream=stream)
        self.run()
        self.status = pa.pa_device_status()
        self.done = [t.clone() for t in self.arrays]

    def restore(self):
        for t, s in zip(self.arrays, self.start):
            t.copy_(s)

    def holds(self, what):
        return all(torch.equal(t, w) for t, w in zip(self.arrays, what))


CASES = {"many waves": ([900 - i % 50 for i in range(220)], 8, 128),
         "longest first": ([2000 + 40 * i for i in range(64)], 8, 64),
         "clusters": ([3000, 2900], 2, 128),
         "long": ([30000 - 100 * i for i in range(40)], 2, 64)}


@pytest.mark.parametrize("case", CASES)
def test_errors_of_another_stream(pa, case):
    lens, Hkv, D = CASES[case]
    call = Call(pa, lens, [n // 2 for n in lens], Hkv, D)
    assert call.status == pa.PA_OK and not call.holds(call.start)
    bad = Cache([20], 1, 16)
    wrong = (bad.kb, bad.vb, bad.tables, i32([20]), i32([-1]), bad.w)  # refused
    ws = torch.zeros(pa.pa_evict_keys_workspace_size(1, 1, bad.tables.shape[1], 16), dtype=torch.uint8,
                     device="cuda")
    ours, other = torch.cuda.Stream(), torch.cuda.Stream(priority=-1)
    found = [0, 0]
    for trial in range(60):
        call.restore()
        torch.cuda.synchronize()
        call.run(ours)
        until = time.perf_counter() + 4e-6 * (trial % 30)  # (at any time within the call, or after it)
        while time.perf_counter() < until:
            pass
        pa.pa_evict_keys(*wrong, workspace=ws, stream=other)
        torch.cuda.synchronize()
        assert pa.pa_device_status() == pa.PA_EINVAL
        done = call.holds(call.done)
        assert done or call.holds(call.start), f"half an eviction (trial {trial})"
        found[done] += 1
    assert found[True] > 0


def test_a_recorded_error_stops_the_whole_call(pa):
    lens = [900] * 10
    call = Call(pa, lens, [400] * 10, 4, 64)
    bad = Cache([20], 1, 16)
    call.restore()
    pa.pa_evict_keys(bad.kb, bad.vb, bad.tables, i32([20]), i32([-1]), bad.w)
    call.run()
    assert pa.pa_device_status() == pa.PA_EINVAL
    assert call.holds(call.start)
    call.run()
    assert pa.pa_device_status() == pa.PA_OK
    assert call.holds(call.done)


@pytest.mark.parametrize("what", ["table", "new"])
def test_a_bad_batch_moves_nothing_though_its_error_is_cleared(pa, what):
    """The error is found by one check; whoever reads the status word in between, nothing moves."""
    lens = [900 - i % 50 for i in range(220)]
    new = [n // 2 for n in lens]

    def tables(c):
        t = c.tables.clone()
        t[219, 5] = -1
        return t

    if what == "new":
        new[219] = -1
    call = Call(pa, lens, new, 8, 128, tables if what == "table" else None)
    assert call.status == pa.PA_EINVAL and call.holds(call.start)
    with Clearing(pa):
        for _ in range(300):
            call.run()
    assert call.holds(call.start)
