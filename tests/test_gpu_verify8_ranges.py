"""Attention over the 8-bit cache on the tensor cores at the ends of its ranges,
against the 64-bit form with bounds of its own, counted before the first run.

A logit: the split of q is exact for elements down to 2^-13 of the row's largest
latent one and off by 2^-21 of that largest one below. 16 matrix instructions add 32
products of codes each and 4 add 16 of the rope part; each may round its sum by
2^-23 of the magnitudes that it adds up, 40 2^-24 in all, and joining the two
terms, the key's factor (two roundings) and the product with it are 4 2^-24 more.
The exponent's argument rounds at 2^-24 of its terms, twice.

A numerator is rounded to 2^-9 of itself, and to half of e5m2's least step, 2^-17,
where a row's largest is at least 2^8 by then: 2^-25 of the largest one so far. A
stored part is fp16 (2^-11) in a unit that leaves at most keys 2^-24 of its largest
weight times scale as an absolute step."""
import numpy as np
import pytest
import torch

from speculative_tree_verify_mla_b200 import kdv
from tests import plain8
from tests.test_gpu_verify8 import Run, i32

pytestmark = pytest.mark.gpu
TILE = 96
TC = kdv.KDV_IMPL_TC


def form(q, codes, rope, s, sm, times=None, part_keys=0, running=True):
    """(o, lse, bound of o, bound of lse, weights times multiplicity) of rows that see all n keys, in the kernel's
    key order. times: how often each key occurs. part_keys: keys of a stored part, 0 where o is written directly.
    running: a numerator's least step follows the largest one so far, else the largest one of all."""
    times = np.ones(len(s)) if times is None else times
    k = np.concatenate([codes, rope], 1) * s[:, None]
    aq, ak = np.abs(q), np.abs(k)
    x, size = sm * (q @ k.T), sm * (aq @ ak.T)
    big = aq[:, :512].max(1, keepdims=True)
    lost = sm * 2.0 ** -21 * big * ((aq[:, :512] < 2.0 ** -13 * big) @ ak[:, :512].T)
    top = x.max(1, keepdims=True)
    e = np.exp(x - top)
    l = (e * times).sum(1, keepdims=True)
    w = e * times / l
    eps = 44 * 2.0 ** -24 * size + lost + 2.0 ** -22 * np.maximum(np.abs(x), np.abs(top)) + 2.0 ** -20
    ws = e * np.abs(s) / l
    if running:
        tops = np.stack([ws[:, i:i + TILE].max(1) for i in range(0, len(s), TILE)], 1)
        most = np.repeat(np.maximum.accumulate(tops, 1), TILE, 1)[:, :len(s)]
    else:
        most = ws.max(1, keepdims=True)
    step = 2.0 ** -9 + (2.0 ** -11 if part_keys else 0.0) + 2 * eps
    o = w @ k[:, :512]
    ob = (w * step) @ ak[:, :512] + (2.0 ** -25 * most * times) @ np.abs(codes)
    if part_keys:
        ob = ob + 2.0 ** -24 * part_keys * ws.max(1, keepdims=True)
    lse = (top + np.log(l))[:, 0]
    return o, lse, ob + 2.0 ** -20 * np.abs(o), (w * eps).sum(1) + 2.0 ** -22 * np.abs(lse) + 2.0 ** -20, w


def of(c, b=0):
    """q, codes, rope parts and scales of request b's keys in their order, 64 bits."""
    keys = np.arange(c.kv_off[b], c.kv_off[b + 1])
    slot = c.table[keys] if c.table is not None else keys
    s = np.repeat(c.scale.astype(np.float64), c.block)[slot]
    r = slice(int(c.tree_off[b]) * c.H, int(c.tree_off[b + 1]) * c.H)
    return c.q.to(torch.float64).numpy()[r], plain8.code_values(c.c8[slot]), c.kr.to(torch.float64).numpy()[slot], s


def compare(run, o, lse, ob, lb):
    assert run.err.item() == 0
    got, gl = run.o.double().cpu().numpy(), run.lse.double().cpu().numpy()
    e, el = np.abs(got - o), np.abs(gl - lse)
    assert np.all(el <= lb), float((el / lb).max())
    assert np.all(e <= ob), float((e / np.maximum(ob, 1e-300)).max())


def one_token(seed, n, H=64):
    """One token of H heads over n keys (itself the last one), keys where they lie."""
    return plain8.Attn(seed, [n - 1], [[-1]], H, paged=False)


@pytest.mark.parametrize("how,e", [("keys", e) for e in (100, 60, -40, -60, -72, -98)]
                         + [("scale", e) for e in (100, 40, -60, -72, -100, -118, -130)])
def test_queries_of_any_magnitude(how, e):
    """Queries of 2^e, with the keys' scales or the softmax scale of 2^-e: the same logits, the same accuracy.
    (At 2^-130 they are subnormal and hold two or three bits each, which then count.)"""
    c = one_token(60, 300)
    c.q = (c.q.double() * 2.0 ** e).bfloat16()
    if how == "keys":
        c.scale = (c.scale * 2.0 ** -e).astype(np.float32)
    else:
        c.sm_scale = float(np.float32(c.sm_scale * 2.0 ** -e))
    for splits in (1, 2):
        f = form(*of(c), c.sm_scale, part_keys=192 if splits == 2 else 0, running=splits == 1)
        assert np.ptp(f[4], 1).min() > 2.0 ** -12                     # the logits differ
        compare(Run(c, TC, splits=splits).go(), *f[:4])


def test_queries_of_many_magnitudes_in_a_tile():
    """Rows of 2^0 to 2^-132 beside one another: the small ones weigh all keys alike."""
    c = one_token(61, 200)
    c.q = (c.q.double() * torch.tensor([2.0 ** -(12 * (r % 12)) for r in range(64)], dtype=torch.float64)[:, None]).bfloat16()
    compare(Run(c, TC, splits=1).go(), *form(*of(c), c.sm_scale)[:4])
    c.sm_scale = 2.0 ** 60                                            # rows of 2^-60 have moderate logits, those above one key
    q, codes, rope, s = of(c)
    r = np.flatnonzero(np.array([12 * (r % 12) for r in range(64)]) >= 60)
    o, lse, ob, lb, _ = form(q[r], codes, rope, s, c.sm_scale)
    run = Run(c, TC, splits=1).go()
    run.o, run.lse = run.o[r.tolist()], run.lse[r.tolist()]
    compare(run, o, lse, ob, lb)


@pytest.mark.parametrize("lat,rope,rope_keys", [(-45, 0, False), (-100, -60, False), (-100, -100, True), (None, -100, True), (None, 0, True),
                                                (38, 40, True), (None, -126, True), (-60, 10, True), (-110, 5, True)])
def test_latent_and_rope_parts_of_different_magnitudes(lat, rope, rope_keys):
    """q_lat of 2^lat (None: zeros) beside q_rope of 2^rope, the softmax scale bringing the part that counts back: the latent
    one where the keys' rope parts are zeros (rope_keys False), else the larger one."""
    c = one_token(62, 250)
    q = c.q.double()
    q[:, :512] *= 0.0 if lat is None else 2.0 ** lat
    q[:, 512:] *= 2.0 ** rope
    c.q = q.bfloat16()
    if not rope_keys:
        c.kr = torch.zeros_like(c.kr)
    c.sm_scale = float(np.float32(c.sm_scale * 2.0 ** -(rope if lat is None or rope_keys and rope > lat else lat)))
    f = form(*of(c), c.sm_scale)
    assert np.ptp(f[4], 1).min() > 2.0 ** -12
    compare(Run(c, TC, splits=1).go(), *f[:4])


@pytest.mark.parametrize("others", [0, -124])
def test_rows_of_zeros_at_any_softmax_scale(others):
    """Queries of zeros weigh all keys alike, also beside rows of 2^-124 that a softmax scale of 2^120 brings back."""
    c = one_token(66, 250)
    c.q = (c.q.double() * (2.0 ** others if others else 0.0)).bfloat16()
    c.q[::3] = 0.0
    c.sm_scale = float(np.float32(c.sm_scale * 2.0 ** 124))
    compare(Run(c, TC, splits=1).go(), *form(*of(c), c.sm_scale)[:4])


def moves(ws):
    """How often a row's reference moves behind its first tile: ws log2 of the weights times scales, rows x keys."""
    n = np.zeros(len(ws), dtype=int)
    m = ws[:, :TILE].max(1) - 8.0
    for i in range(TILE, ws.shape[1], TILE):
        top = ws[:, i:i + TILE].max(1)
        go = top - m > 15.0
        m, n = np.where(go, top - 8.0, m), n + go
    return n


def steps(seed, level, flat=False):
    """One token over tiles whose largest weight times scale is about 2^(8 level): by their logits, or (flat) by their scales
    alone. Tile i's keys have 44 dims to themselves, so a tile's share of the output is seen whatever the others weigh."""
    n = len(level) * TILE
    c = one_token(seed, n)
    rng = np.random.default_rng(seed)
    t = np.repeat(np.arange(len(level)), TILE)
    lv = np.repeat(np.array(level), TILE)
    v = np.zeros((n, 512))
    for i in range(len(level)):
        v[t == i, 44 * i:44 * i + 44] = 100 + 20 * rng.standard_normal((TILE, 44))
    q = np.zeros((64, 576))
    if flat:
        c.scale = np.exp2(-40.0 + 8 * lv).astype(np.float32)
        q[:, 512:] = rng.standard_normal((64, 64)) * 2.0 ** (36 - 8 * max(level))
    else:
        c.scale = np.full(n, 2.0 ** -6, np.float32)
        v[:, 448:] = 32 * lv[:, None]
        q[:, 448:512] = (1 + np.arange(64) / 2000)[:, None] * 5.5 / (c.sm_scale * 32)
        q[:, 512:] = rng.standard_normal((64, 64)) * 0.3
    c.c8 = plain8.codes(v, np.ones(n))
    c.q = torch.from_numpy(q.astype(np.float32)).bfloat16()
    return c


def log2_ws(c):
    q, codes, rope, s = of(c)
    return c.sm_scale * (q @ (np.concatenate([codes, rope], 1) * s[:, None]).T) / np.log(2) + np.log2(s)


@pytest.mark.parametrize("flat", [False, True])
def test_references_that_move_in_every_tile(flat):
    """Ten tiles, each 2^8 above the one before, by logits or by scales: each one's share of o and lse comes through
    all the moves behind it."""
    c = steps(63, list(range(10)), flat)
    n = moves(log2_ws(c))
    assert n.min() >= 8, n
    compare(Run(c, TC, splits=1).go(), *form(*of(c), c.sm_scale)[:4])
    compare(Run(c, TC, splits=3).go(), *form(*of(c), c.sm_scale, part_keys=384, running=False)[:4])


@pytest.mark.parametrize("flat", [False, True])
def test_references_that_rise_and_stay(flat):
    """The same up to the middle and down again: five moves, none behind the middle."""
    c = steps(64, [0, 1, 2, 3, 4, 5, 4, 3, 2, 1], flat)
    n = moves(log2_ws(c))
    assert np.all(n == 5), n
    compare(Run(c, TC, splits=1).go(), *form(*of(c), c.sm_scale)[:4])


@pytest.mark.parametrize("many", [6, 128])
@pytest.mark.parametrize("splits", [1, 0])
def test_a_sink_that_holds_half_and_a_tail_that_holds_the_rest(many, splits):
    """One key with half of the weight, then 1000 slots that the page table names `many` times over: 2^-12.5 and 2^-17 of the
    sink each. The tail's codes have a mean in 64 dims, so an answer without it is far off."""
    c = plain8.Attn(65, [1000], [[-1]], 16, paged=False)
    rng = np.random.default_rng(65)
    v = np.zeros((1001, 512))
    v[1:, :64] = 100 + 60 * rng.standard_normal((1000, 64))
    v[1:, 64:256] = 60 * rng.standard_normal((1000, 192))
    v[0, :64], v[0, 64:256], v[0, 256:] = -200.0, 60 * rng.standard_normal(192), 256.0
    c.c8 = plain8.codes(v, np.ones(1001))
    c.scale = np.full(1001, 2.0 ** -6, np.float32)
    q = np.zeros((16, 576))
    q[:, :256] = 0.02 * rng.standard_normal((16, 256))
    q[:, 512:] = 0.02 * rng.standard_normal((16, 64))
    _, codes, rope, s = of(c)
    k = np.concatenate([codes, rope], 1) * s[:, None]
    # the sink's logit: ln of the tail's sum of weights, by the dims that it has to itself
    x = c.sm_scale * (q @ k.T)
    q[:, 256:512] = ((np.log(many * np.exp(x[:, 1:]).sum(1)) - x[:, 0]) / (c.sm_scale * 256 * 4.0))[:, None]
    c.q = torch.from_numpy(q.astype(np.float32)).bfloat16()
    times = np.concatenate([[1.0], np.full(1000, float(many))])
    n = 1000 * many + 1                                               # keys: the sink, then the slots over and over
    table = i32(np.concatenate([[0], np.tile(np.arange(1, 1001), many)]))
    f = form(*of(c), c.sm_scale, times=times, part_keys=0 if splits == 1 else n, running=False)
    assert np.all((f[4][:, 0] > 0.4) & (f[4][:, 0] < 0.6))
    alone = np.abs(k[0, :512] - f[0])
    assert np.all(alone[:, :64] > 8 * f[2][:, :64])                   # the sink's row alone does not pass
    r = Run(c, TC, splits=splits, page_table=table, kv_off=i32([0, n]), prefix_len=i32([n - 1]), h_prefix_len=[n - 1])
    size = kdv.kdv_verify_attn8_workspace(r.p)
    r.ws = torch.zeros(max(16, size), dtype=torch.uint8, device="cuda")
    r.p.workspace, r.p.workspace_bytes = r.ws.data_ptr(), size
    # sums of n / 32 equal terms a lane round by 2^-24 of themselves each time, to one side at worst
    compare(r.go(), f[0], f[1], f[2] + 2.0 ** -24 * (n / 32) * np.abs(f[0]), f[3] + 2.0 ** -24 * (n / 32))
