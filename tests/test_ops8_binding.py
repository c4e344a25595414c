"""CPU checks of the binding's HOST arrays: one that is shorter than the call
reads is refused before the call."""
import ctypes

import numpy as np
import pytest

from speculative_tree_verify_mla_b200 import build, kdv
from tests.test_ops8_host import attn_params, rope_params, write_params


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return kdv.load()


@pytest.mark.parametrize("call,params", [
    (kdv.kdv_rope, lambda: rope_params(h_inv_freq=np.ones(31))),
    (kdv.kdv_rope, lambda: rope_params(h_inv_freq=[])),
    (kdv.kdv_latent8_write, lambda: write_params(h_inv_freq=np.ones(31))),
    (kdv.kdv_verify_attn8, lambda: attn_params(batch=2)),
    (kdv.kdv_verify_attn8, lambda: attn_params(batch=2, h_prefix_len=[5, 6])),
    (kdv.kdv_verify_attn8_workspace, lambda: attn_params(batch=2, h_tree_T=[1, 1])),
    (kdv.kdv_verify_attn8_plan, lambda: attn_params(batch=2)),
])
def test_short_host_arrays_are_refused(call, params):
    with pytest.raises(ValueError, match="values are wanted"):
        call(params())


def test_arrays_that_are_long_enough_or_the_callers_own():
    p = attn_params(batch=1, h_prefix_len=[50, 60], h_tree_T=[4, 4])
    assert kdv.kdv_verify_attn8_plan(p)[0]
    p.batch = 2
    assert len(kdv.kdv_verify_attn8_plan(p)[0]) == 2
    p.batch = 3
    with pytest.raises(ValueError):
        kdv.kdv_verify_attn8_plan(p)
    own = [(ctypes.c_int32 * 3)(*v) for v in ([1, 2, 3], [4, 5, 6])]
    p.h_prefix_len, p.h_tree_T = (ctypes.cast(a, ctypes.POINTER(ctypes.c_int32)) for a in own)
    assert len(kdv.kdv_verify_attn8_plan(p)[0]) == 3


def test_lengths_change_in_place():
    """The copied lengths are the struct's: a step writes the new ones there."""
    p = attn_params(num_splits=1)
    short = kdv.kdv_verify_attn8_plan(attn_params(h_prefix_len=[200000]))
    p.num_splits, p.h_prefix_len[0] = 0, 200000
    assert kdv.kdv_verify_attn8_plan(p) == short
