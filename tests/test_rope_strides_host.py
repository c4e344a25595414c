"""CPU checks of kdv_rope's output strides: what would write an element twice is
refused, everything else is not. Calls that pass this check end at a later one (a
batch above the limit), so nothing is launched."""
import ctypes
import itertools

import numpy as np
import pytest

from speculative_tree_verify_mla_b200 import build, kdv

P = 0x10000                      # a 16-byte aligned address that no refused call reads


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return kdv.load()


def status(tokens, heads, dim, ts, hs):
    p = kdv.make_rope_params(tokens=tokens, heads=heads, dim=dim, rot_dim=2, layout=0, inverse=0, x_dtype=0, y_dtype=1, x=P, x_token_stride=0,
                             x_head_stride=1 << 20, y=2 * P, y_token_stride=ts, y_head_stride=hs, h_inv_freq=np.ones(1), pos=None, batch=129,
                             tree_off=P, prefix_len=P, depth=P)
    return kdv.load().kdv_rope(ctypes.byref(p), None)


def twice(tokens, heads, dim, ts, hs):
    at = [i * ts + h * hs + d for i, h, d in itertools.product(range(tokens), range(heads), range(dim))]
    return len(set(at)) < len(at)


def check(*a):
    assert status(*a) == (kdv.KDV_ERR_INVALID_ARG if twice(*a) else kdv.KDV_ERR_UNSUPPORTED), a


@pytest.mark.parametrize("tokens,heads", list(itertools.product(range(1, 5), range(1, 5))))
def test_small_strides(tokens, heads):
    for dim in (2, 3, 5):
        for ts, hs in itertools.product(range(-16, 17), repeat=2):
            check(tokens, heads, dim, ts, hs)


def test_layouts_in_use():
    rng = np.random.default_rng(0)
    for _ in range(300):
        n, h, dim = (int(rng.integers(1, 40)) for _ in range(3))
        dim += 1
        gap = int(rng.integers(0, 4))
        for ts, hs in [(h * dim, dim), (h * dim + gap, dim), (dim, n * dim), (dim + gap, n * (dim + gap)), (dim, dim), (2 * dim, dim),
                       (dim, 2 * dim), (h * dim - 1, dim), (2 * dim, (2 * n + 1) * dim), (3 * dim, 2 * dim)]:
            check(n, h, dim, ts, hs)


def test_strides_near_the_ends_of_their_type():
    big = 2 ** 62
    assert status(3, 4, 8, big, 8) == kdv.KDV_ERR_UNSUPPORTED
    assert status(3, 4, 8, 8, big) == kdv.KDV_ERR_UNSUPPORTED
    assert status(2 ** 31 - 1, 2, 8, 16, -8) == kdv.KDV_ERR_UNSUPPORTED
    assert status(3, 4, 8, big, big) == kdv.KDV_ERR_INVALID_ARG
    assert status(3, 4, 8, -2 ** 63, 8) == kdv.KDV_ERR_INVALID_ARG
    assert status(3, 4, 8, 64, -2 ** 63) == kdv.KDV_ERR_INVALID_ARG
