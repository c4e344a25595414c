"""Rotary positions on the GPU against the 64-bit form.

Tolerance of one element: the output type's half step of the value, plus the
fp32 arithmetic: cos and sin (2 ulp of sincospi and one rounding of the angle's
fraction, 2^-22 each relative to 1), two products and their sum: 2^-21 mscale
(|u| + |v|) in all."""
import numpy as np
import pytest
import torch

from speculative_tree_verify_mla_b200 import kdv
from tests import plain8

pytestmark = pytest.mark.gpu
DT = {"bf16": (torch.bfloat16, kdv.KDV_BF16), "f32": (torch.float32, kdv.KDV_F32)}


def make(n, heads, dim, rot, half, seed, xt="bf16", yt="bf16", gap=0, far=5000, mscale=1.0, inverse=0, freq=None):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, heads, dim + gap, generator=g).to(DT[xt][0]).cuda()[:, :, gap:]
    pos = torch.randint(0, far, (n,), generator=g, dtype=torch.int32).cuda()
    if freq is None:
        freq, _ = kdv.kdv_rope_freqs(rot, 10000.0)
    y = torch.full((n, heads, dim + gap), 7.0, dtype=DT[yt][0], device="cuda")
    p = kdv.make_rope_params(tokens=n, heads=heads, dim=dim, rot_dim=rot, layout=half, inverse=inverse, x_dtype=DT[xt][1], y_dtype=DT[yt][1],
                             x=x, x_token_stride=x.stride(0), x_head_stride=x.stride(1), y=y[:, :, gap:], y_token_stride=y.stride(0),
                             y_head_stride=y.stride(1), pos=pos, h_inv_freq=freq, mscale=mscale)
    return x, pos, freq, y, p


def check(x, pos, freq, got, rot, half, mscale=1.0, inverse=False):
    want = plain8.rope(x.double().cpu().numpy(), pos.cpu().numpy(), freq, rot, half, mscale, inverse)
    ax = x.double().abs().cpu().numpy()
    size = np.zeros_like(want)
    i, j = (slice(0, rot // 2), slice(rot // 2, rot)) if half else (slice(0, rot, 2), slice(1, rot, 2))
    size[..., i] = size[..., j] = abs(mscale) * (ax[..., i] + ax[..., j])
    tol = plain8.half_step(got.dtype) * np.abs(want) * (1 + 2.0 ** -7) + 2.0 ** -21 * size
    err = np.abs(got.double().cpu().numpy() - want)
    assert np.all(err <= tol), float((err - tol).max())
    rest = got[..., rot:]
    assert torch.equal(rest, x[..., rot:].to(got.dtype))


@pytest.mark.parametrize("half", [0, 1])
@pytest.mark.parametrize("n,heads,dim,rot,gap", [
    (1, 1, 2, 2, 0), (13, 64, 64, 64, 512), (1, 128, 64, 64, 0), (7, 3, 96, 32, 1), (5, 2, 130, 66, 3), (300, 1, 64, 64, 0),
    (33, 17, 192, 128, 64), (3, 700, 256, 256, 0), (4099, 1, 8, 8, 0), (2, 5000, 16, 16, 0)])
def test_shapes(n, heads, dim, rot, gap, half):
    x, pos, freq, y, p = make(n, heads, dim, rot, half, seed=n + heads, gap=gap)
    kdv.kdv_rope(p)
    check(x, pos, freq, y[:, :, gap:], rot, half)
    assert torch.all(y[:, :, :gap] == 7.0)                  # nothing outside the head vectors


@pytest.mark.parametrize("xt,yt", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("n,heads,dim,rot", [(19, 5, 128, 64), (3, 3, 192, 64), (2, 1, 64, 32), (1, 3, 64, 16), (70, 9, 256, 256), (11, 2, 192, 128), (5, 1, 96, 48)])
def test_halves_at_all_distances(n, heads, dim, rot, xt, yt):
    """Partners 1 to 16 units of eight elements away, and distances and widths that do not divide."""
    x, pos, freq, y, p = make(n, heads, dim, rot, 1, n + rot, xt, yt)
    kdv.kdv_rope(p)
    check(x, pos, freq, y, rot, 1)


@pytest.mark.parametrize("xt,yt", [("bf16", "f32"), ("f32", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("half", [0, 1])
def test_types_and_far_positions(xt, yt, half):
    freq, m = kdv.kdv_rope_freqs(64, 50000.0, kdv.KDV_ROPE_SCALE_YARN, factor=32.0)
    x, pos, freq, y, p = make(50, 4, 80, 64, half, 3, xt, yt, far=2 ** 31 - 1, mscale=m, freq=freq)
    kdv.kdv_rope(p)
    # positions up to 2^31: the 64-bit reference itself rounds the angle at 2^31 * 2^-53 rad = 2^-22
    check(x, pos, freq, y, 64, half, mscale=float(np.float32(m)))


@pytest.mark.parametrize("half", [0, 1])
def test_in_place_inverse_and_gradient(half):
    x, pos, freq, y, p = make(40, 6, 96, 64, half, 9, "f32", "f32", mscale=1.25)
    kdv.kdv_rope(p)
    # in place gives the same bits
    z = x.clone()
    kw = dict(tokens=40, heads=6, dim=96, rot_dim=64, layout=half, x_dtype=1, y_dtype=1, pos=pos, h_inv_freq=freq)
    st = dict(x_token_stride=z.stride(0), x_head_stride=z.stride(1), y_token_stride=z.stride(0), y_head_stride=z.stride(1))
    kdv.kdv_rope(kdv.make_rope_params(x=z, y=z, mscale=1.25, **kw, **st))
    assert torch.equal(z, y)
    # inverse = transpose: <R x, g> = <x, R^T g>, and a pure rotation is undone
    g = torch.randn_like(x)
    back = torch.empty_like(x)
    kdv.kdv_rope(kdv.make_rope_params(x=g, y=back, inverse=1, mscale=1.25, **kw, **st))
    check(g, pos, freq, back, 64, half, mscale=1.25, inverse=True)
    lhs, rhs = (y.double() * g.double()).sum(), (x.double() * back.double()).sum()
    assert abs(lhs - rhs) <= 2.0 ** -20 * (y.double() * g.double()).abs().sum()
    # the gradient against differences of the plain form in 64 bits
    xs = x.double().cpu().numpy()
    d = np.random.default_rng(0).standard_normal(xs.shape)
    f = lambda v: float((plain8.rope(v, pos.cpu().numpy(), freq, 64, half, 1.25) * g.double().cpu().numpy()).sum())  # noqa: E731
    h = 1e-4
    diff = (f(xs + h * d) - f(xs - h * d)) / (2 * h)
    assert abs(diff - float((back.double().cpu().numpy() * d).sum())) <= 1e-5 * np.abs(back.double().cpu().numpy() * d).sum()
    kdv.kdv_rope(kdv.make_rope_params(x=z, y=z, inverse=1, mscale=1 / 1.25, **kw, **st))
    assert (z - x).abs().max() <= 2.0 ** -19 * x.abs().max()


def test_tree_positions():
    prefix, sizes, depth = [17, 0, 5553], [3, 5, 2], [0, 1, 2, 0, 1, 1, 2, 3, 0, 1]
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    pos = i32([17, 18, 19, 0, 1, 1, 2, 3, 5553, 5554])
    x, _, freq, y, _ = make(10, 16, 64, 64, 0, 4)
    kw = dict(tokens=10, heads=16, dim=64, rot_dim=64, layout=0, x_dtype=0, y_dtype=0, x=x, x_token_stride=x.stride(0), x_head_stride=64,
              y=y, y_token_stride=y.stride(0), y_head_stride=64, h_inv_freq=freq)
    kdv.kdv_rope(kdv.make_rope_params(batch=3, tree_off=i32(np.cumsum([0] + sizes)), prefix_len=i32(prefix), depth=i32(depth), **kw))
    check(x, pos, freq, y, 64, 0)
    a = y.clone()
    kdv.kdv_rope(kdv.make_rope_params(pos=pos, **kw))
    assert torch.equal(a, y)


def test_broadcast_input_and_negative_positions():
    x, pos, freq, y, _ = make(20, 1, 64, 64, 1, 5, "f32", "f32")
    neg = -pos
    wide = torch.empty(20, 4, 64, device="cuda")
    # one row turned by 20 positions: x with token stride 0
    p = kdv.make_rope_params(tokens=20, heads=1, dim=64, rot_dim=64, layout=1, x_dtype=1, y_dtype=1, x=x, x_token_stride=0, x_head_stride=64,
                             y=wide, y_token_stride=256, y_head_stride=64, pos=neg, h_inv_freq=freq)
    wide.fill_(3.0)
    kdv.kdv_rope(p)
    check(x[:1].expand(20, 1, 64), neg, freq, wide[:, :1], 64, 1)
    assert torch.all(wide[:, 1:] == 3.0)


def test_streams_and_graph():
    x, pos, freq, y, p = make(64, 8, 64, 64, 0, 6)
    kdv.kdv_rope(p)
    want = y.clone()
    side = torch.cuda.Stream()
    y.zero_()
    side.wait_stream(torch.cuda.current_stream())
    kdv.kdv_rope(p, side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kdv.kdv_rope(p)
    y.zero_()
    x2 = torch.randn_like(x)
    x.copy_(x2)
    graph.replay()
    check(x2, pos, freq, y, 64, 0)
