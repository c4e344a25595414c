"""The 8-bit cache write with given slots and positions from the tree."""
import numpy as np
import pytest

from speculative_tree_verify_mla_b200 import kdv
from tests.test_gpu_latent8 import Pool, check, i32, rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dims", [(512, 64), (96, 16)])
@pytest.mark.parametrize("first,last,err", [(0, 8, 0), (0, 6, kdv.KDV_DERR_BAD_LENGTH), (2, 8, kdv.KDV_DERR_BAD_LENGTH)])
def test_rows_outside_the_tree(first, last, err, dims):
    """Rows in front of the first request's nodes or behind the last one's have no position: reported, not written."""
    c, k = rows(8, *dims, "bf16", 40)
    freq = kdv.kdv_rope_freqs(dims[1], 10000.0)[0]
    slot, depth, prefix = np.array([9, 3, 0, 7, 5, 11, 2, 14]), np.array([0, 1, 2, 0, 1, 1, 0, 1]), [30, 500]
    pool = Pool(20, *dims)
    pool.write(c, k, "bf16", slot=i32(slot), batch=2, tree_off=i32([first, 3, last]), prefix_len=i32(prefix), depth=i32(depth), h_inv_freq=freq,
               rot_dim=dims[1], layout=0)
    inside = (np.arange(8) >= first) & (np.arange(8) < last)
    pos = np.where(np.arange(8) < 3, prefix[0], prefix[1]) + depth
    assert pool.err.item() == err
    check(pool, c, k, np.where(inside, slot, -1), freq, 0, pos)


def test_rows_outside_the_tree_that_need_no_position():
    """Without a rotation, or with positions given, given slots are all that counts."""
    c, k = rows(5, 512, 64, "bf16", 41)
    freq = kdv.kdv_rope_freqs(64, 10000.0)[0]
    slot, pos = np.array([4, 2, 0, 3, 1]), np.array([5, 6, 7, 8, 9])
    for rot in (False, True):
        pool = Pool(6)
        kw = dict(h_inv_freq=freq, rot_dim=64, layout=0, pos=i32(pos)) if rot else {}
        pool.write(c, k, "bf16", slot=i32(slot), batch=1, tree_off=i32([0, 2]), prefix_len=i32([0]), **kw)
        assert pool.err.item() == 0
        check(pool, c, k, slot, freq if rot else None, 0, pos)
