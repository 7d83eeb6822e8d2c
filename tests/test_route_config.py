"""RouteConfig is a plain value: it is copied, compared, replaced and sent between processes as Config is (CPU)."""
import copy
import ctypes
import dataclasses
import pickle

import pytest

import moe_expert_dispatch_online_gb300 as bep

RC = bep.RouteConfig(bep.BEP_SCORE_SIGMOID, groups=8, top_groups=4, group_top=2, renorm=False, scale=2.5)


def passed(rc):
    """What a call hands to the library."""
    c = ctypes.cast(rc._ref, ctypes.POINTER(bep._RouteConfig)).contents
    return tuple(getattr(c, n) for n, _ in c._fields_)


@pytest.mark.parametrize("again", (copy.copy, copy.deepcopy, lambda rc: pickle.loads(pickle.dumps(rc)),
                                   dataclasses.replace))
def test_copies_are_equal_and_stand_alone(again):
    rc = again(RC)
    assert rc == RC and hash(rc) == hash(RC) and rc is not RC
    assert passed(rc) == passed(RC) == (1, 8, 4, 2, 0, 2.5)
    assert ctypes.addressof(rc._ref._obj) != ctypes.addressof(RC._ref._obj)


def test_a_layer_that_holds_one_can_be_copied():
    layer = copy.deepcopy({"route": RC, "sizes": bep.Config(1, 8, 8, 2, 4, 64, 64)})
    assert layer["route"] == RC and pickle.loads(pickle.dumps(layer)) == layer
