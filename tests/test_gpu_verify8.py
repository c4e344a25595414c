"""Attention over the 8-bit latent cache against its 64-bit form. Every bound is
plain8.Attn.answer's, counted before the first run: a logit's fp32 rounding, the
numerators' (2^-9 where they are split into 8-bit terms), the stored partials'
and the output type's."""
import numpy as np
import pytest
import torch

from speculative_tree_verify_mla_b200 import kdv
from tests import plain8

pytestmark = pytest.mark.gpu
i32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")  # noqa: E731
CODE = {torch.bfloat16: kdv.KDV_BF16, torch.float32: kdv.KDV_F32}
SIMT, TC, AUTO = kdv.KDV_IMPL_SIMT, kdv.KDV_IMPL_TC, kdv.KDV_IMPL_AUTO


class Run:
    def __init__(self, case, impl=AUTO, out=torch.float32, splits=0, chain=False, **kw):
        self.case, c = case, case
        rows = int(c.tree_off[-1]) * c.H
        self.q = c.q.cuda()
        self.c8, self.kr, self.scale = torch.from_numpy(c.c8).cuda(), c.kr.cuda(), torch.from_numpy(c.scale).cuda()
        self.o = torch.full((rows, c.D_c), 5.0, dtype=out, device="cuda")
        self.lse = torch.full((rows,), 5.0, device="cuda")
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        m = np.array([x if x < 2 ** 63 else x - 2 ** 64 for x in c.masks], dtype=np.int64)
        self.mask = None if chain else torch.from_numpy(m).cuda()
        base = dict(batch=c.B, num_heads=c.H, d_latent=c.D_c, d_rope=c.D_r, scale=c.sm_scale, dtype=CODE[self.q.dtype], out_dtype=CODE[out],
                    impl=impl, q=self.q, q_row_stride=0, c8=self.c8, kr=self.kr if c.D_r else None, kv_scale=self.scale, scale_block=c.block,
                    num_slots=c.slots, page_table=i32(c.table) if c.table is not None else None, kv_off=i32(c.kv_off), tree_off=i32(c.tree_off),
                    prefix_len=i32(c.prefix), h_prefix_len=c.prefix, h_tree_T=c.T, mask=self.mask, num_splits=splits, o=self.o, lse=self.lse,
                    d_err=self.err)
        self.p = kdv.make_verify8_params(**{**base, **kw})
        n = kdv.kdv_verify_attn8_workspace(self.p)
        self.ws = torch.full((max(16, n),), 0xA5, dtype=torch.uint8, device="cuda")
        self.p.workspace, self.p.workspace_bytes = self.ws.data_ptr(), n

    def go(self, stream=None):
        kdv.kdv_verify_attn8(self.p, stream)
        return self

    def check(self, err=0, drop=None, rows=None):
        o, lse, ob, lb = self.case.answer(drop=drop)
        got, gl = self.o.double().cpu().numpy(), self.lse.double().cpu().numpy()
        assert self.err.item() == err
        rows = np.arange(len(o)) if rows is None else rows
        got, gl, o, lse, ob, lb = got[rows], gl[rows], o[rows], lse[rows], ob[rows], lb[rows]
        none = np.isneginf(lse)
        assert np.array_equal(np.isneginf(gl), none)
        assert np.all(got[none] == 0.0)
        tol = ob + plain8.half_step(self.o.dtype) * (np.abs(o) + ob)
        e = np.abs(got - o)
        assert np.all(e <= tol), (float((e / np.maximum(tol, 1e-30)).max()), float(e.max()))
        el = np.abs(gl[~none] - lse[~none])
        assert np.all(el <= lb[~none]), float((el / lb[~none]).max())
        return self


def tree(T, seed=0, reach=3):
    return plain8.random_tree(np.random.default_rng(seed), T, reach)


@pytest.mark.parametrize("q_dtype,D_c,D_r", [("bf16", 512, 64), ("f32", 512, 64), ("f32", 32, 8), ("bf16", 7, 0), ("f32", 509, 63), ("bf16", 1, 1)])
@pytest.mark.parametrize("paged", [False, True])
def test_simt_types_and_dims(q_dtype, D_c, D_r, paged):
    c = plain8.Attn(D_c, [40, 0, 3], [tree(5), tree(1), tree(9, 2)], H=3, D_c=D_c, D_r=D_r, block=4, paged=paged, q_dtype=q_dtype)
    Run(c, SIMT).go().check()
    Run(c, SIMT, splits=3, out=torch.bfloat16).go().check()


SHAPES = [
    ([0], [1], 64), ([1], [1], 16), ([127], [1], 64), ([128], [1], 1), ([126, 127, 128, 129], [1, 1, 1, 1], 8),
    ([300], [13], 64), ([5], [64], 5), ([700, 0, 33], [3, 64, 7], 16), ([1000], [2], 128), ([255], [16], 17),
    ([95], [1], 64), ([96], [1], 33), ([94, 95, 96, 97], [1, 2, 1, 3], 8), ([191, 192], [64, 1], 3), ([190], [4], 64),
]


@pytest.mark.parametrize("prefix,sizes,H", SHAPES)
@pytest.mark.parametrize("paged,block", [(False, 1), (True, 1), (True, 16)])
def test_shapes(prefix, sizes, H, paged, block):
    c = plain8.Attn(sum(prefix) + H, prefix, [tree(T, i) for i, T in enumerate(sizes)], H, block=block, paged=paged)
    Run(c).go().check()
    Run(c, splits=1, out=torch.bfloat16).go().check()
    Run(c, splits=3).go().check()


def test_more_splits_than_tiles_and_repeats():
    c = plain8.Attn(3, [200, 10], [tree(4), tree(2)], 32)
    a = Run(c, splits=7).go().check()
    first = a.o.clone()
    a.o.zero_()
    a.go()
    assert torch.equal(a.o, first)                                    # the same bits again


def test_chain_is_causal_and_single_tokens():
    c = plain8.Attn(4, [77, 500], [list(range(-1, 5)), [-1]], 64)
    a, b = Run(c, chain=True).go().check(), Run(c).go()
    assert torch.equal(a.o, b.o)
    c = plain8.Attn(5, [10], [list(range(-1, 63))], 4)
    Run(c, chain=True).go().check()


def test_rows_that_see_nothing():
    """Empty masks: with a prefix the node sees it alone; without one its rows are empty."""
    masks = [0, 0b10, 0, 0b1]
    c = plain8.Attn(6, [0, 9], [[-1, 0], [-1, 0]], 64, masks=masks)
    Run(c).go().check()
    Run(c, splits=2).go().check()
    c = plain8.Attn(7, [0], [tree(40)], 16, masks=[0] * 40)
    r = Run(c).go().check()
    assert torch.all(r.o == 0) and torch.all(torch.isneginf(r.lse))


@pytest.mark.parametrize("impl", [AUTO, SIMT])
def test_unseen_keys_never_reach_an_output(impl):
    """NaN codes, NaN rope parts, NaN and infinite scales in slots that a row does not see change no bit of it."""
    sizes, prefix, H = [6, 3], [130, 0], 64
    trees = [[-1, 0, 0, 1, 1, 2], [-1, 0, 0]]
    for what in ("codes", "rope", "scale_nan", "scale_inf"):
        c = plain8.Attn(8, prefix, trees, H)
        clean = Run(c, impl).go().check()
        # node 3 of request 0 (seen by itself alone), and every slot that no request owns
        node = int(c.table[c.kv_off[0] + prefix[0] + 3])
        free = np.setdiff1d(np.arange(c.slots), c.table)
        dirty = np.append(free, node)
        if what == "codes":
            c.c8[dirty] = 0x7F
        elif what == "rope":
            c.kr[torch.from_numpy(dirty)] = float("nan")
        else:
            c.scale[dirty] = np.nan if what == "scale_nan" else np.inf
        r = Run(c, impl).go()
        own = np.arange(3 * H, 4 * H)
        rest = np.setdiff1d(np.arange(sum(sizes) * H), own)
        assert torch.equal(r.o[rest], clean.o[rest]) and torch.equal(r.lse[rest], clean.lse[rest]), what
        assert torch.isnan(r.o[own]).any(1).all() and torch.isnan(r.lse[own]).all(), what


@pytest.mark.parametrize("impl", [AUTO, SIMT])
@pytest.mark.parametrize("what", ["codes", "rope_nan", "rope_inf", "scale_nan", "scale_inf"])
def test_neighbours_in_a_contiguous_pool_never_reach_an_output(impl, what):
    """A tile behind a request's last key holds the next request's rows: whatever they are, the first one keeps its bits."""
    c = plain8.Attn(30, [100, 40, 5], [tree(3), tree(2), tree(1)], 64, paged=False)
    clean = Run(c, impl).go().check()
    lo, hi = int(c.kv_off[1]), int(c.kv_off[2])
    if what == "codes":
        c.c8[lo:hi] = 0x7F
    elif what.startswith("rope"):
        c.kr[lo:hi] = float("nan") if what == "rope_nan" else float("inf")
    else:
        c.scale[lo:hi] = np.nan if what == "scale_nan" else np.inf
    r = Run(c, impl).go()
    rest = np.setdiff1d(np.arange(6 * 64), np.arange(3 * 64, 5 * 64))
    assert torch.equal(r.o[rest], clean.o[rest]) and torch.equal(r.lse[rest], clean.lse[rest])
    assert torch.isnan(r.lse[3 * 64:5 * 64]).all()


@pytest.mark.parametrize("impl", [AUTO, SIMT])
def test_contiguous_keys_beyond_the_pool(impl):
    """Keys of a contiguous request that lie behind the pool's end are left out and reported."""
    c = plain8.Attn(31, [250], [tree(2)], 64, paged=False)
    Run(c, impl, num_slots=200).go().check(err=kdv.KDV_DERR_BAD_SLOT, drop=np.arange(200, 252))
    r = Run(c, impl, num_slots=0).go()
    assert r.err.item() == kdv.KDV_DERR_BAD_SLOT and torch.all(r.o == 0) and torch.all(torch.isneginf(r.lse))


def test_query_that_is_not_finite_stays_in_its_row():
    c = plain8.Attn(9, [200], [tree(3)], 64)
    clean = Run(c).go().check()
    for bad in (float("nan"), float("inf")):
        r = Run(c)
        r.q[70, 5] = bad
        r.q[10, 550] = bad
        r.go()
        rest = [i for i in range(192) if i not in (70, 10)]
        assert torch.equal(r.o[rest], clean.o[rest]) and torch.equal(r.lse[rest], clean.lse[rest])
        assert torch.isnan(r.lse[[70, 10]]).all()


@pytest.mark.parametrize("impl", [AUTO, SIMT])
def test_half_of_the_heads_not_finite(impl):
    """Queries that are NaN for whole groups of 32 rows leave the other rows' bits alone."""
    c = plain8.Attn(22, [200], [tree(2)], 64)
    clean = Run(c, impl).go().check()
    for lo in (0, 32):
        r = Run(c, impl)
        r.q[lo:lo + 32] = float("nan")
        r.go()
        rest = [i for i in range(128) if not lo <= i < lo + 32]
        assert torch.equal(r.o[rest], clean.o[rest]) and torch.equal(r.lse[rest], clean.lse[rest])
        assert torch.isnan(r.o[lo:lo + 32]).all() and torch.isnan(r.lse[lo:lo + 32]).all()


def test_queries_over_the_whole_exponent_range():
    """Rows of 2^100 and 2^-100 under scales that bring the logits back."""
    for e in (100, -40):
        c = plain8.Attn(23, [150], [tree(2)], 64)
        c.q = c.q * 2.0 ** e
        c.scale = (c.scale * 2.0 ** -e).astype(np.float32)
        Run(c).go().check()


@pytest.mark.parametrize("splits", [1, 3])
def test_growing_logits_and_scales(splits):
    """The reference maximum and the scale's unit move in every tile; then they fall again."""
    c = plain8.Attn(10, [900], [tree(2)], 64, sharp=2.0)
    order = np.arange(900)
    at = c.table[order]
    c.scale[at] = (2.0 ** -12 * 1.013 ** np.minimum(order, 900 - order)).astype(np.float32)
    Run(c, splits=splits).go().check()
    c.scale[at] = (2.0 ** -3 * 0.99 ** order).astype(np.float32)
    Run(c, splits=splits).go().check()


def test_a_sink_and_a_long_flat_tail():
    """One key holds half of the weight; thousands of keys far below it hold the rest."""
    c = plain8.Attn(11, [6000], [[-1]], 64)
    c.q = c.q * 0.02
    q = c.q.double().mean(0).numpy()
    sink = int(c.table[0])
    c.c8[sink] = plain8.codes((np.sign(q[:512]) * 400)[None], np.ones(1))[0]
    c.q[:, :512] = torch.from_numpy(np.sign(q[:512]) * 0.09).to(c.q.dtype)
    Run(c, splits=1).go().check()
    Run(c).go().check()


def test_zero_and_negative_scales():
    """A scale of 0 makes a row of zeros; a negative one its mirror."""
    c = plain8.Attn(12, [300], [tree(2)], 64)
    c.scale[c.table[:100]] = 0.0
    c.scale[c.table[100:200]] *= -1.0
    Run(c).go().check()
    c.scale[:] = 0.0
    r = Run(c).go().check()
    assert torch.all(r.o == 0)


def test_zero_queries_and_tiny_and_huge_values():
    c = plain8.Attn(13, [200], [tree(3)], 64)
    c.q[:64] = 0.0
    c.q[64:128] *= 2.0 ** -40
    c.q[100] *= 2.0 ** 30
    c.scale *= 2.0 ** -20
    Run(c).go().check()


def test_bad_slots_and_lengths():
    c = plain8.Attn(14, [150, 40], [tree(3), tree(2)], 64)
    good = Run(c).go().check()
    table = c.table.copy()
    lost = [int(table[5]), int(table[149])]
    table[5], table[149] = c.slots, -7
    Run(c, page_table=i32(table)).go().check(err=kdv.KDV_DERR_BAD_SLOT, drop=lost)
    Run(c, page_table=i32(table), impl=SIMT).go().check(err=kdv.KDV_DERR_BAD_SLOT, drop=lost)
    # a request whose range is too short has no keys; the other is whole
    off = c.kv_off.copy()
    off[1] -= 1
    r = Run(c, kv_off=i32(np.array([off[0], off[1], off[1] + 200])), page_table=None, num_slots=c.slots)
    r.go()
    assert r.err.item() == kdv.KDV_DERR_BAD_LENGTH
    assert torch.all(r.o[:192] == 0) and torch.all(torch.isneginf(r.lse[:192])) and torch.isfinite(r.lse[192:]).all()
    r = Run(c, prefix_len=i32([150, 41])).go()
    assert r.err.item() == kdv.KDV_DERR_BAD_LENGTH and torch.equal(r.o, good.o)


def test_query_strides_and_nullable_outputs():
    c = plain8.Attn(15, [100], [tree(2)], 64)
    base = Run(c).go().check()
    wide = torch.zeros(128, 640, dtype=torch.bfloat16, device="cuda")
    wide[:, :576] = base.q
    r = Run(c, q=wide, q_row_stride=640, lse=None, d_err=None).go()
    assert torch.equal(r.o, base.o)
    odd = torch.zeros(128, 577, dtype=torch.bfloat16, device="cuda")       # rows that are not 16-byte aligned
    odd[:, :576] = base.q
    Run(c, q=odd, q_row_stride=577).go().check()


def test_rows_behind_the_last_request_stay():
    c = plain8.Attn(16, [64], [tree(3)], 20)
    rows = 60
    o = torch.full((rows + 100, 512), 5.0, device="cuda")
    lse = torch.full((rows + 100,), 5.0, device="cuda")
    r = Run(c, o=o, lse=lse).go()
    assert torch.all(o[rows:] == 5.0) and torch.all(lse[rows:] == 5.0)
    r.o, r.lse = o[:rows], lse[:rows]
    r.check()


def test_slots_beyond_32_bit_offsets():
    slots = 9_000_000
    c = plain8.Attn(17, [300], [tree(2)], 16)
    far = np.concatenate([np.arange(8_388_600, 8_388_600 + 150), np.arange(slots - 152, slots)])
    c8 = torch.zeros(slots, 512, dtype=torch.uint8, device="cuda")
    kr, scale = torch.zeros(slots, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(slots, device="cuda")
    old = torch.from_numpy(c.table.astype(np.int64))
    c8[far], kr[far], scale[far] = torch.from_numpy(c.c8)[old].cuda(), c.kr[old].cuda(), torch.from_numpy(c.scale)[old].cuda()
    Run(c, c8=c8, kr=kr, kv_scale=scale, num_slots=slots, page_table=i32(far)).go().check()


def test_streams_and_graphs_with_their_own_workspaces():
    a, b = Run(plain8.Attn(18, [700], [tree(5)], 64)), Run(plain8.Attn(19, [500, 20], [tree(2), tree(9)], 32))
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (sa, sb):
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):                                                # two calls at once
        a.go(sa)
        b.go(sb)
    for s in (sa, sb):
        torch.cuda.current_stream().wait_stream(s)
    a.check()
    b.check()
    want = a.o.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.go()
        b.go()
    a.o.zero_()
    b.o.zero_()
    a.ws.fill_(0xFF)
    for _ in range(2):
        graph.replay()
    a.check()
    b.check()
    assert torch.equal(a.o, want)


def test_writes_just_before_are_seen():
    c = plain8.Attn(20, [400], [tree(4)], 64)
    r = Run(c)
    q, c8 = r.q.clone(), r.c8.clone()
    for _ in range(3):
        r.q.zero_()
        r.c8.zero_()
        r.go()
        r.q.copy_(q)
        r.c8.copy_(c8)
        r.go()
    r.check()


def test_long_context():
    c = plain8.Attn(21, [40000], [[-1]], 16, paged=False)
    Run(c).go().check()


def test_many_short_requests():
    """The largest batch, lengths around a tile's, single tokens."""
    c = plain8.Attn(24, [i % 5 * 48 for i in range(128)], [[-1]] * 128, 16)
    Run(c).go().check()
    Run(c, chain=True, out=torch.bfloat16).go().check()


def test_a_wait_that_runs_out_is_reported():
    """Waits limited to 1 ns end the call with an error; the next call is right. The same without splits."""
    for splits, paged in ((0, True), (1, True), (0, False), (1, False)):
        c = plain8.Attn(25, [3000], [tree(4)], 64, paged=paged)
        good = Run(c, TC, splits=splits).go().check()
        r = Run(c, TC, splits=splits, wait_limit_ns=1).go()
        torch.cuda.synchronize()
        assert r.err.item() == kdv.KDV_DERR_TIMEOUT
        again = Run(c, TC, splits=splits).go()
        assert torch.equal(again.o, good.o) and torch.equal(again.lse, good.lse)


def test_calls_back_to_back_share_a_workspace():
    """A call's launch overlaps the end of the call before it: the same workspace and outputs, other inputs."""
    cases = [plain8.Attn(26 + k, [1500 + 300 * k], [tree(3)], 64, paged=False) for k in range(3)]
    runs = [Run(c) for c in cases]
    size = max(r.ws.numel() for r in runs)
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    for r in runs:
        r.p.workspace, r.p.workspace_bytes = ws.data_ptr(), size
    for _ in range(5):
        for r in runs:
            r.go()
    for r in runs:
        r.check()


def test_millions_of_keys_through_shared_slots():
    """A page table that names the same 1000 slots 3000 times over: every weight repeats, so o is theirs and lse grows by ln 3000."""
    c = plain8.Attn(32, [1000], [[-1]], 16, masks=[0])
    o, lse, ob, lb = c.answer()
    many = 3000
    table = i32(np.concatenate([np.tile(c.table[:1000], many), c.table[1000:]]))
    n = 1000 * many
    r = Run(c, page_table=table, kv_off=i32([0, n + 1]), prefix_len=i32([n]), h_prefix_len=[n])
    size = kdv.kdv_verify_attn8_workspace(r.p)
    r.ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    r.p.workspace, r.p.workspace_bytes = r.ws.data_ptr(), size
    r.go()
    assert r.err.item() == 0
    # sums of 3e6 / 148 items' equal terms round in fp32: 2^-24 for each of at most 2^15 additions in a chain, 2^-9 in all
    e = np.abs(r.o.double().cpu().numpy() - o)
    assert np.all(e <= ob + 2.0 ** -9 * (np.abs(o) + ob) + 2.0 ** -24 * np.abs(o))
    assert np.all(np.abs(r.lse.double().cpu().numpy() - (lse + np.log(many))) <= lb + 2.0 ** -9)


@pytest.mark.parametrize("impl", [AUTO, SIMT])
@pytest.mark.parametrize("H", [64, 5])
@pytest.mark.parametrize("scale", [1e30, 1e8, 2.0 ** -110])
def test_unseen_scales_of_any_size_never_reach_an_output(impl, H, scale):
    """Scales far from the others' in slots that a row does not see leave it as it was: with 64 heads, where
    its 16 rows share no reference with the node that sees it, to the last bit; else within the bounds."""
    c = plain8.Attn(34, [130, 0], [[-1, 0, 0, 1, 1, 2], [-1, 0, 0]], H)
    clean = Run(c, impl).go().check()
    node = int(c.table[c.kv_off[0] + 130 + 3])                        # seen by node 3 of request 0 alone
    c.scale[np.append(np.setdiff1d(np.arange(c.slots), c.table), node)] = scale
    r = Run(c, impl).go()
    own = np.arange(3 * H, 4 * H)
    rest = np.setdiff1d(np.arange(9 * H), own)
    if H == 64:
        assert torch.equal(r.o[rest], clean.o[rest]) and torch.equal(r.lse[rest], clean.lse[rest])
    r.check(rows=rest)


@pytest.mark.parametrize("splits", [1, 4])
@pytest.mark.parametrize("impl", [AUTO, SIMT])
def test_seen_key_of_a_large_scale_and_no_weight(impl, splits):
    """One key of scale 2^14 (the others' are about 2^-6) whose logit is far below the rest takes no precision from them."""
    c = plain8.Attn(35, [300], [[-1]], 64, paged=False)
    c.scale[:] = 2.0 ** -6
    # queries and the large key point away from one another; the other keys are as they were
    c.q = (0.01 * c.q.float() + 1.0).bfloat16()
    c.c8[150] = plain8.codes(np.full((1, c.D_c), -1.0), np.ones(1))
    c.scale[150] = 2.0 ** 14
    Run(c, impl, splits=splits).go().check()


@pytest.mark.parametrize("impl", [AUTO, SIMT])
def test_scales_that_differ_between_tiles(impl):
    """Scales rise by 2^20 and fall by 2^40 from one part of the keys to the next, the logits staying moderate:
    o is the large ones'; a request that holds small ones alone keeps its precision."""
    c = plain8.Attn(36, [400, 200], [tree(2), tree(3)], 64, paged=False)
    c.q = (2.0 ** -30 * c.q.float()).bfloat16()
    e = np.full(c.slots, -6.0)
    e[130:260] += 20
    e[260:] -= 20
    e[int(c.kv_off[1]):] = -60
    c.scale[:] = np.exp2(e)
    Run(c, impl).go().check()
    Run(c, impl, splits=5).go().check()


@pytest.mark.parametrize("impl", [AUTO, SIMT])
@pytest.mark.parametrize("power", [27, 40, 90])
def test_logits_beyond_the_exponents_precision(impl, power):
    """Logits so large that neighbouring fp32 numbers are far apart: each row gives its largest key's values."""
    c = plain8.Attn(37, [250], [tree(2)], 64, paged=False)
    c.scale[:] = 2.0 ** -6
    c.q = (2.0 ** power * c.q.float()).bfloat16()
    o, lse, _, _ = c.answer()
    r = Run(c, impl).go()
    # A logit's products round by 80 2^-24 of their magnitudes, whose sums are below 8 times the row's largest logit here:
    # a gap of 2^-9 of it leaves one key, off by the numerators' and the parts' steps.
    vals = np.concatenate([plain8.code_values(c.c8), c.kr.to(torch.float64).numpy()], 1) * 2.0 ** -6
    x = c.sm_scale * (c.q.to(torch.float64).numpy() @ vals.T)
    for node in range(c.T[0]):
        x[node * 64:(node + 1) * 64, [k for k in range(c.n[0]) if k not in set(c.node_keys(0, node))]] = -np.inf
    y = np.sort(x, 1)
    sure = y[:, -1] - y[:, -2] > 2.0 ** -9 * np.abs(y[:, -1])
    assert sure.mean() > 0.5
    got = r.o.double().cpu().numpy()
    assert r.err.item() == 0 and np.isfinite(got).all() and torch.isfinite(r.lse).all()
    assert np.all(np.abs(got - o)[sure] <= (2.0 ** -9 + 2.0 ** -11) * np.abs(o)[sure] + 2.0 ** -20)
    assert np.all(np.abs(r.lse.double().cpu().numpy() - lse)[sure] <= 2.0 ** -9 * np.abs(lse)[sure])
