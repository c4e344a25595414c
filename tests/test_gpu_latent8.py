"""The quantising cache write against its 64-bit form: scales and codes exactly
(dividing by a power of two is exact; other scales divide in fp32, IEEE), the
rope part to bf16's half step plus fp32's 2^-21 (|u| + |v|) / scale."""
import numpy as np
import pytest
import torch

from speculative_tree_verify_mla_b200 import kdv
from tests import plain8

pytestmark = pytest.mark.gpu
DT = {"bf16": (torch.bfloat16, kdv.KDV_BF16), "f32": (torch.float32, kdv.KDV_F32)}
i32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")  # noqa: E731


class Pool:
    def __init__(self, slots, D_c=512, D_r=64, block=1, scale=None):
        self.c8 = torch.full((slots, D_c), 0x11, dtype=torch.uint8, device="cuda")
        self.kr = torch.full((slots, max(1, D_r)), 5.0, dtype=torch.bfloat16, device="cuda")
        n = (slots + block - 1) // block
        self.scale = torch.full((n,), -3.0, device="cuda") if scale is None else scale.clone()
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.slots, self.D_c, self.D_r, self.block = slots, D_c, D_r, block

    def write(self, c, k, dtype, stream=None, **kw):
        p = kdv.make_latent8_params(rows=c.shape[0], d_latent=self.D_c, d_rope=self.D_r, dtype=DT[dtype][1], c=c, c_stride=c.stride(0),
                                    k_rope=k, k_stride=0 if k is None else k.stride(0), c8=self.c8, kr=self.kr, kv_scale=self.scale,
                                    num_slots=self.slots, scale_block=self.block, d_err=self.err, **kw)
        kdv.kdv_latent8_write(p, stream)
        return p


def rows(n, D_c, D_r, dtype, seed, spread=2.0):
    g = torch.Generator().manual_seed(seed)
    c = (torch.randn(n, D_c, generator=g) * torch.exp(spread * torch.randn(n, 1, generator=g))).to(DT[dtype][0]).cuda()
    return c, torch.randn(n, max(1, D_r), generator=g).to(DT[dtype][0]).cuda()


def check(pool, c, k, slot, freq, half, pos, mscale=1.0, static=None):
    n = c.shape[0]
    live = np.asarray(slot) >= 0
    at = torch.tensor(np.asarray(slot)[live], dtype=torch.long, device="cuda")
    cs = c.float().cpu().numpy()[live]
    s = plain8.row_scale(cs) if static is None else static[(at // pool.block).cpu().numpy()].astype(np.float64)
    if static is None:
        np.testing.assert_array_equal(pool.scale[at].double().cpu().numpy(), s)
    np.testing.assert_array_equal(pool.c8[at].cpu().numpy(), plain8.codes(cs, s))
    if pool.D_r:
        kk = k.double().cpu().numpy()[live]
        want, size = kk.copy(), np.zeros_like(kk)
        if freq is not None:
            rot = 2 * len(freq)
            want = plain8.rope(kk[:, None], np.asarray(pos)[live], freq, rot, half, mscale)[:, 0]
            i, j = (slice(0, rot // 2), slice(rot // 2, rot)) if half else (slice(0, rot, 2), slice(1, rot, 2))
            size[:, i] = size[:, j] = np.abs(kk[:, i]) + np.abs(kk[:, j])
        want, size = want / s[:, None], size / s[:, None]
        err = np.abs(pool.kr[at].double().cpu().numpy()[:, :pool.D_r] - want)
        # bf16 keeps 8 significant bits: steps of at most 2^-7 of the value, half of one is 2^-8; the
        # division by the scale rounds once more in fp32 (2^-24)
        tol = plain8.half_step(torch.bfloat16) * np.abs(want) * (1 + 2.0 ** -7) + 2.0 ** -21 * size * mscale + 2.0 ** -24 * np.abs(want)
        assert np.all(err <= tol), float((err - tol).max())
    # every other slot is as it was
    rest = torch.ones(pool.slots, dtype=torch.bool, device="cuda")
    rest[at] = False
    assert torch.all(pool.c8[rest] == 0x11) and torch.all(pool.kr[rest] == 5.0)
    if static is None and pool.block == 1:
        assert torch.all(pool.scale[rest] == -3.0)
    assert n == len(slot)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("half", [0, 1])
@pytest.mark.parametrize("n,D_c,D_r,rot", [(1, 512, 64, 64), (104, 512, 64, 64), (9, 512, 64, 32), (7, 512, 0, 0), (33, 96, 16, 8), (5, 1, 1, 0), (3, 509, 63, 62), (1030, 512, 64, 64)])
def test_rows(n, D_c, D_r, rot, half, dtype):
    c, k = rows(n, D_c, D_r, dtype, n + D_c)
    rng = np.random.default_rng(n)
    slot, pos = rng.permutation(n + 50)[:n], rng.integers(0, 300000, n)
    pool = Pool(n + 50, D_c, D_r)
    freq = kdv.kdv_rope_freqs(rot, 10000.0)[0] if rot else None
    pool.write(c, k if D_r else None, dtype, slot=i32(slot), h_inv_freq=freq, rot_dim=rot, layout=half, pos=i32(pos) if rot else None)
    check(pool, c, k, slot, freq, half, pos)
    assert pool.err.item() == 0


def test_scale_borders_and_rounding_ties():
    """amax at, just above and just below 448 2^e; zeros; subnormals; the largest values; ties to even."""
    c = torch.zeros(12, 512)
    for i, top in enumerate([448.0, 450.0, 446.0, 7.0, 7.0625, 0.0, 2.0 ** -130, 3e38, 2.0 ** -100, 1.0, 224.0, 2.0 ** -92 * 448]):
        c[i, 17] = -top
        c[i, 100:108] = torch.tensor([17.0, 19.0, 1.0625, 1.1875, 2.0 ** -10, 3 * 2.0 ** -10, 5 * 2.0 ** -10, 2.0 ** -11]) * top / 448
    for dtype in ("bf16", "f32"):
        cc = c.to(DT[dtype][0]).cuda()
        k = torch.ones(12, 64, device="cuda", dtype=DT[dtype][0])
        pool = Pool(20)
        pool.write(cc, k * 0, dtype, slot=i32(range(12)))
        check(pool, cc, k * 0, list(range(12)), None, 0, None)


def test_values_not_finite():
    c, k = rows(6, 512, 64, "bf16", 3, spread=0.0)
    c[1, 5], c[2, 511], c[3, 0] = float("nan"), float("inf"), -float("inf")
    c[4] = float("nan")
    k[5, 3] = float("nan")
    pool = Pool(8)
    pool.write(c, k, "bf16", slot=i32([0, 1, 2, 3, 4, 5]))
    assert pool.err.item() == kdv.KDV_DERR_RANGE
    got = pool.c8.cpu().numpy()
    np.testing.assert_array_equal(got[:6], plain8.codes(c.float().cpu().numpy(), plain8.row_scale(c.float().cpu().numpy())))
    assert torch.isnan(pool.kr[5, 3]) and torch.isfinite(pool.kr[:5]).all() and pool.scale[4].item() == 1.0


@pytest.mark.parametrize("block", [1, 16, 4096])
def test_static_scales(block):
    n, slots = 200, 333
    c, k = rows(n, 512, 64, "f32", 8, spread=1.0)
    nb = (slots + block - 1) // block
    scale = torch.exp(torch.randn(nb, generator=torch.Generator().manual_seed(2)) - 5).cuda()       # saturates some, any mantissa
    slot = np.random.default_rng(1).permutation(slots)[:n]
    pool = Pool(slots, block=block, scale=scale)
    pool.write(c, k, "f32", slot=i32(slot), static_scale=1)
    check(pool, c, k, slot, None, 0, None, static=scale.cpu().numpy())
    assert torch.equal(pool.scale, scale) and pool.err.item() == 0


@pytest.mark.parametrize("bad", [0.0, -1.0, float("nan"), float("inf")])
def test_bad_static_scale(bad):
    c, k = rows(2, 512, 64, "bf16", 8)
    pool = Pool(32, block=16, scale=torch.tensor([bad, 0.5], device="cuda"))
    pool.write(c, k, "bf16", slot=i32([3, 20]), static_scale=1)
    assert pool.err.item() == kdv.KDV_DERR_RANGE
    assert torch.all(pool.c8[3] == 0x11) and not torch.all(pool.c8[20] == 0x11)


def test_slots_skipped_and_outside():
    c, k = rows(6, 512, 64, "bf16", 4)
    pool = Pool(10)
    pool.write(c, k, "bf16", slot=i32([2, -1, 9, 4, -1, 0]))
    check(pool, c, k, [2, -1, 9, 4, -1, 0], None, 0, None)
    assert pool.err.item() == 0
    for slot in (10, -2, 2 ** 31 - 1):
        pool = Pool(10)
        pool.write(c, k, "bf16", slot=i32([2, slot, 9, 4, -1, 0]))
        assert pool.err.item() == kdv.KDV_DERR_BAD_SLOT
        check(pool, c, k, [2, -1, 9, 4, -1, 0], None, 0, None)


@pytest.mark.parametrize("paged", [False, True])
def test_tree_nodes(paged):
    prefix, sizes = [5, 0, 130], [3, 1, 4]
    kv_off, tree_off = np.cumsum([0, 8, 1, 140]), np.cumsum([0] + sizes)       # the last range has room behind its nodes
    depth = [0, 1, 1, 0, 0, 1, 2, 1]
    pos = [5, 6, 6, 0, 130, 131, 132, 131]
    logical = [5, 6, 7, 8, 9 + 130, 9 + 131, 9 + 132, 9 + 133]
    table = np.random.default_rng(0).permutation(200)[:149]
    slot = table[logical] if paged else np.array(logical)
    c, k = rows(8, 512, 64, "bf16", 6)
    freq = kdv.kdv_rope_freqs(64, 10000.0)[0]
    pool = Pool(200)
    pool.write(c, k, "bf16", batch=3, tree_off=i32(tree_off), prefix_len=i32(prefix), depth=i32(depth), kv_off=i32(kv_off),
               page_table=i32(table) if paged else None, h_inv_freq=freq, rot_dim=64, layout=0)
    check(pool, c, k, slot, freq, 0, pos)
    assert pool.err.item() == 0
    # a range that is too short: that request's nodes are left out
    pool = Pool(200)
    pool.write(c, k, "bf16", batch=3, tree_off=i32(tree_off), prefix_len=i32([5, 1, 130]), depth=i32(depth), kv_off=i32(kv_off),
               page_table=i32(table) if paged else None, h_inv_freq=freq, rot_dim=64, layout=0)
    assert pool.err.item() == kdv.KDV_DERR_BAD_LENGTH
    check(pool, c, k, np.where(np.arange(8) == 3, -1, slot), freq, 0, pos)


def test_strides_offsets_and_far_slots():
    """Row strides, unaligned bases, and a pool whose byte offsets pass 32 bits."""
    n, slots = 16, 9_000_000
    wide = torch.randn(n, 700, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    c, k = wide[:, 3:515], wide[:, 601:665]
    c8 = torch.zeros(slots, 512, dtype=torch.uint8, device="cuda")
    kr = torch.zeros(slots, 64, dtype=torch.bfloat16, device="cuda")
    scale = torch.zeros(slots, device="cuda")
    slot = np.concatenate([[slots - 1, 8_388_608, 4_194_304], np.arange(13)])
    p = kdv.make_latent8_params(rows=n, d_latent=512, d_rope=64, dtype=0, c=c, c_stride=700, k_rope=k, k_stride=700, slot=i32(slot),
                                c8=c8, kr=kr, kv_scale=scale, num_slots=slots)
    kdv.kdv_latent8_write(p)
    at = torch.tensor(slot, device="cuda")
    s = plain8.row_scale(c.float().cpu().numpy())
    np.testing.assert_array_equal(c8[at].cpu().numpy(), plain8.codes(c.float().cpu().numpy(), s))
    assert int((scale != 0).sum()) == n


def test_stream_and_graph():
    c, k = rows(50, 512, 64, "bf16", 7)
    slot = np.arange(50) * 2
    pool = Pool(100)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    p = pool.write(c, k, "bf16", stream=side, slot=i32(slot))
    torch.cuda.current_stream().wait_stream(side)
    check(pool, c, k, slot, None, 0, None)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kdv.kdv_latent8_write(p)
    c.copy_(torch.randn_like(c))
    graph.replay()
    check(pool, c, k, slot, None, 0, None)
