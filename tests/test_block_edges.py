"""Calls of layer norm, the linear layer and AdamW at the edges of what they take, as
far as the C ABI decides them before any HIP call (the fake addresses are never
dereferenced)."""

import pytest
import torch

from momentum_compression_amd import onebit as ob
from tests.test_block_refusals import P, _linear_args


@pytest.fixture(scope="module")
def lib():
    return ob.load()


def test_round_dz_is_a_truth_value(lib):
    for bad in (-1, 2):
        assert lib.linear_backward(_linear_args(round_dz=bad), 9 * P, 1 << 30,
                                   None) == ob.ONEBIT_E_ARG
    # the workspace, which is checked last, stops these calls
    for good in (0, 1):
        assert lib.linear_backward(_linear_args(round_dz=good), None, 0,
                                   None) == ob.ONEBIT_E_WORKSPACE


def test_a_plan_is_known_on_the_streams_of_its_steps(monkeypatch):
    """The allocator is told of each stream but the plan's own, once, before the step
    is enqueued."""
    said = []

    class Memory:
        def record_stream(self, stream):
            said.append(("record", stream))

        def data_ptr(self):
            return P

    class Lib:
        @staticmethod
        def adamw_step(*args):
            said.append(("step", args[-1]))
            return ob.ONEBIT_OK

    plan = object.__new__(ob.AdamWPlan)
    plan.plan, plan.device, plan._streams = Memory(), 0, {7}
    plan.n_tensors = plan.tiles = 1
    plan.state_bits, plan.g_dtype, plan.copy_dtype = 32, 0, 0
    monkeypatch.setattr(ob, "load", lambda: Lib)
    monkeypatch.setattr(ob, "_stream_of", lambda stream, *tensors: stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda raw, device: (raw, device))
    for on in (7, 9, 9, 8, 7):
        ob.adamw_step(plan, 1e-3, 0.9, 0.99, 1e-8, 1, stream=on)
    assert said == [("step", 7), ("record", (9, 0)), ("step", 9), ("step", 9),
                    ("record", (8, 0)), ("step", 8), ("step", 7)]


def test_linear_backward_takes_anything_for_what_it_does_not_read(lib):
    """x without dw and w without dx, and their strides, are not looked at (the
    workspace, which is checked last, stops these calls)."""
    for kw in (dict(dw=None, ld_x=0), dict(dx=None, ld_w=0), dict(dx=None, dw=None, ld_x=0, ld_w=0),
               dict(dw=None, ld_x=-24), dict(dx=None, w=7 * P - 64, ld_w=1),
               dict(dw=None, x=5 * P + 2), dict(dx=None, w=6 * P + 1), dict(dx=None, w=7 * P)):
        assert lib.linear_backward(_linear_args(**kw), None, 0, None) == ob.ONEBIT_E_WORKSPACE, kw
    # what is read is looked at
    for kw in (dict(x=5 * P + 2), dict(w=6 * P + 2), dict(dw=None, w=5 * P), dict(dx=None, x=6 * P)):
        assert lib.linear_backward(_linear_args(**kw), None, 0, None) == ob.ONEBIT_E_ARG, kw
