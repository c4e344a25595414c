"""Logits processing against its 64-bit form. Tolerance: the output type's half
step plus fp32's rounding of up to six operations, 2^-22 of the magnitudes."""
import numpy as np
import pytest
import torch

from speculative_tree_verify_mla_b200 import kdv
from tests import plain8

pytestmark = pytest.mark.gpu
DT = {"bf16": (torch.bfloat16, kdv.KDV_BF16), "f32": (torch.float32, kdv.KDV_F32)}
i32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")  # noqa: E731
f32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.float32, device="cuda")  # noqa: E731


class Problem:
    def __init__(self, seed, sizes, V, hist, xt="bf16", yt="bf16", pool=None, nbias=20, gap=0, penal=True, allow=True):
        rng = np.random.default_rng(seed)
        self.rng, self.sizes, self.V, self.xt, self.yt = rng, sizes, V, xt, yt
        B, n = len(sizes), sum(sizes)
        pool = pool or max(1, V // 30)                    # tokens repeat
        self.x = torch.from_numpy(rng.standard_normal((n, V + gap)) * 3).to(DT[xt][0]).cuda()[:, :V]
        self.y = torch.full((n, V + gap), 9.0, dtype=DT[yt][0], device="cuda")
        self.gap = gap
        self.tree_off = np.cumsum([0] + list(sizes))
        self.parent = np.concatenate([plain8.random_tree(rng, T) for T in sizes if T > 0]) if n else np.zeros(0)
        self.token = rng.integers(0, pool, n)
        self.hist_len = np.array(hist)
        self.ld = max(1, int(self.hist_len.max(initial=0)))
        self.hist = rng.integers(0, pool, (B, self.ld))
        self.prompt_len = np.array([int(rng.integers(0, h + 1)) for h in hist])
        self.rep, self.pres, self.freq = (np.float32(rng.uniform(0.7, 1.6, B)), np.float32(rng.uniform(-1, 1, B)), np.float32(rng.uniform(-0.3, 0.5, B))) \
            if penal else (np.ones(B, np.float32), np.zeros(B, np.float32), np.zeros(B, np.float32))
        counts = [min(V, int(rng.integers(0, nbias + 1))) for _ in range(B)]
        self.bias_off = np.cumsum([0] + counts)
        self.bias_tok = np.concatenate([np.sort(rng.permutation(V)[:c]) for c in counts]).astype(np.int32)
        self.bias_val = np.float32(rng.standard_normal(len(self.bias_tok)) * 4)
        words = (V + 31) // 32
        self.allow = rng.integers(-2 ** 31, 2 ** 31, (n + 2, words)).astype(np.int32) if allow else None
        self.allow_row = np.where(rng.random(n) < 0.3, -1, rng.integers(0, n + 2, n)) if allow else None
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def params(self, **kw):
        has = self.allow is not None
        base = dict(batch=len(self.sizes), max_T=max(1, max(self.sizes)), total_nodes=sum(self.sizes), vocab=self.V, dtype=DT[self.xt][1],
                    out_dtype=DT[self.yt][1], logits=self.x, logits_ld=self.x.stride(0), out=self.y, out_ld=self.y.stride(0),
                    tree_off=i32(self.tree_off), parent=i32(self.parent), token=i32(self.token), hist=i32(self.hist), hist_ld=self.ld,
                    hist_len=i32(self.hist_len), prompt_len=i32(self.prompt_len), repetition=f32(self.rep), presence=f32(self.pres),
                    frequency=f32(self.freq), bias_off=i32(self.bias_off), bias_token=i32(self.bias_tok) if len(self.bias_tok) else i32([0]),
                    bias_value=f32(self.bias_val) if len(self.bias_tok) else f32([0]), allow=i32(self.allow) if has else None,
                    allow_ld=(self.V + 31) // 32, allow_rows=0 if not has else self.allow.shape[0], allow_row=i32(self.allow_row) if has else None,
                    d_err=self.err)
        return kdv.make_logits_params(**{**base, **kw})

    def check(self, y=None, x=None, skip=(), no_path=(), rep=None):
        y = (self.y if y is None else y)[:, :self.V].double().cpu().numpy()
        x = (self.x if x is None else x).double().cpu().numpy()
        for b, T in enumerate(self.sizes):
            bias = np.zeros(self.V)
            for i in range(self.bias_off[b], self.bias_off[b + 1]):
                bias[self.bias_tok[i]] = self.bias_val[i]
            for t in range(T):
                i = self.tree_off[b] + t
                if i in skip:
                    continue
                path, u = [], t
                while b not in no_path and self.parent[self.tree_off[b] + u] >= 0:
                    path.append(int(self.token[self.tree_off[b] + u]))
                    u = int(self.parent[self.tree_off[b] + u])
                bits = None
                if self.allow is not None and self.allow_row[i] >= 0:
                    w = self.allow[self.allow_row[i]].astype(np.int64) & 0xFFFFFFFF
                    bits = ((w[:, None] >> np.arange(32)) & 1).reshape(-1)[:self.V] == 1
                n, p = int(self.hist_len[b]), int(min(self.prompt_len[b], self.hist_len[b]))
                want, size = plain8.penalised(x[i], self.hist[b, :n], p, path, float(self.rep[b] if rep is None else rep), float(self.pres[b]),
                                              float(self.freq[b]), bias, bits)
                inf = np.isneginf(want)
                assert np.array_equal(np.isneginf(y[i]), inf)
                ok = np.isfinite(want)
                tol = plain8.half_step(DT[self.yt][0]) * np.abs(want[ok]) * (1 + 2.0 ** -7) + 2.0 ** -22 * size[ok]
                err = np.abs(y[i][ok] - want[ok])
                assert np.all(err <= tol), (b, t, float((err - tol).max()))
                assert np.array_equal(np.isnan(y[i]), np.isnan(want))


@pytest.mark.parametrize("xt,yt", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("sizes,V,hist,gap", [([1], 1, [0], 0), ([13], 5000, [300], 0), ([1, 5, 64], 2048, [0, 1, 700], 0), ([3, 2], 2049, [50, 4000], 7),
                                              ([4], 33, [10], 1), ([2, 0, 3], 8191, [9, 9, 9], 1), ([16], 50000, [20000], 0)])
def test_shapes(sizes, V, hist, gap, xt, yt):
    p = Problem(V + len(sizes), sizes, V, hist, xt, yt, gap=gap)
    kdv.kdv_logits_process(p.params())
    p.check()
    assert p.err.item() == 0
    assert torch.all(p.y[:, V:] == 9.0)


def test_each_part_alone():
    for kw, off in [(dict(hist=None, parent=None, token=None, bias_off=None, allow=None), "none"), (dict(parent=None, token=None), "path"),
                    (dict(hist=None), "hist"), (dict(bias_off=None), "bias"), (dict(allow=None), "allow"), (dict(repetition=None), "rep"),
                    (dict(presence=None), "pres"), (dict(frequency=None), "freq"), (dict(prompt_len=None), "prompt")]:
        p = Problem(5, [6, 3], 3000, [400, 90])
        kdv.kdv_logits_process(p.params(**kw))
        if off in ("none", "hist"):
            p.hist_len[:] = 0
            p.prompt_len[:] = 0
        if off in ("none", "path"):
            p.parent[:] = -1
        if off in ("none", "bias"):
            p.bias_off[:] = 0
        if off in ("none", "allow"):
            p.allow = None
        if off == "rep":
            p.rep[:] = 1
        if off == "pres":
            p.pres[:] = 0
        if off == "freq":
            p.freq[:] = 0
        if off == "prompt":
            p.prompt_len[:] = 0
        p.check()
        if off == "none":
            assert torch.equal(p.y, p.x)


def test_in_place_equals_out_of_place():
    p = Problem(6, [13, 4], 4096, [500, 60], "f32", "f32")
    kdv.kdv_logits_process(p.params())
    z = p.x.clone()
    kdv.kdv_logits_process(p.params(logits=z, out=z, out_ld=z.stride(0)))
    assert torch.equal(z, p.y)


def test_same_token_along_a_path():
    """A chain whose nodes all hold one token: node t counts it t times; forests and several roots."""
    p = Problem(7, [64], 300, [12], "f32", "f32", allow=False)
    p.parent[:] = np.arange(-1, 63)
    p.token[:] = 17
    kdv.kdv_logits_process(p.params())
    p.check()
    p.parent[:] = -1                                          # all roots: no path counts
    kdv.kdv_logits_process(p.params())
    p.check()


def test_values_not_finite():
    p = Problem(8, [3], 1000, [100], "f32", "f32")
    p.x[0, 5], p.x[1, 6], p.x[2, 7] = float("nan"), float("inf"), -float("inf")
    p.allow_row[:] = -1
    p.allow_row[2] = 0
    p.allow[0, 0] = 0                                         # tokens 0..31 of node 2 forbidden
    p.x[2, 9] = float("nan")
    kdv.kdv_logits_process(p.params())
    y = p.y.cpu()
    assert torch.isnan(y[0, 5]) and y[1, 6] == float("inf") and torch.all(torch.isneginf(y[2, :32]))
    p.x[torch.isinf(p.x)] = 0.0
    p.check(skip=(1,))


def test_no_token_allowed():
    p = Problem(9, [2], 777, [10])
    p.allow[:] = 0
    p.allow_row[:] = 1
    kdv.kdv_logits_process(p.params())
    assert torch.all(torch.isneginf(p.y))


def test_bad_data_is_reported():
    p = Problem(10, [4, 3], 2000, [50, 60])
    p.hist[0, 3], p.hist[1, 5] = 2000, -1
    kdv.kdv_logits_process(p.params())
    assert p.err.item() == kdv.KDV_DERR_BAD_TOKEN
    keep = [np.delete(p.hist[0, :50], 3), np.delete(p.hist[1, :60], 5)]
    p.prompt_len -= np.array([int(p.prompt_len[0] > 3), int(p.prompt_len[1] > 5)])
    p.hist_len -= 1
    p.hist[0, :49], p.hist[1, :59] = keep
    p.check()

    p = Problem(11, [4, 3], 2000, [50, 60])
    p.parent[2] = 3
    kdv.kdv_logits_process(p.params())
    assert p.err.item() == kdv.KDV_DERR_BAD_PARENT
    p.check(no_path=(0,))

    p = Problem(12, [4, 3], 2000, [50, 60])
    p.rep[0] = float("nan")
    kdv.kdv_logits_process(p.params())
    assert p.err.item() == kdv.KDV_DERR_BAD_SCORE
    p.rep[0] = 1.0
    p.check()

    p = Problem(13, [4, 3], 2000, [50, 60])
    p.allow_row[1] = p.allow.shape[0]
    kdv.kdv_logits_process(p.params())
    assert p.err.item() == kdv.KDV_DERR_BAD_TOKEN
    p.allow_row[1] = -1
    p.check()

    p = Problem(14, [4, 3], 2000, [50, 60])
    kdv.kdv_logits_process(p.params(max_T=3))                 # the first request is longer: left alone
    assert p.err.item() == kdv.KDV_DERR_BAD_LENGTH and torch.all(p.y[:4] == 9.0)
    p.check(skip=(0, 1, 2, 3))

    p = Problem(15, [4], 2000, [50])
    kdv.kdv_logits_process(p.params(hist_len=i32([51])))
    assert p.err.item() == kdv.KDV_DERR_BAD_LENGTH
    p.check()

    p = Problem(16, [4], 2000, [50])
    p.bias_off, p.bias_tok, p.bias_val = np.array([0, 3]), np.array([-4, 7, 2000], np.int32), np.array([1, 2, 3], np.float32)
    kdv.kdv_logits_process(p.params())
    assert p.err.item() == kdv.KDV_DERR_BAD_TOKEN
    p.bias_off, p.bias_tok, p.bias_val = np.array([0, 1]), np.array([7], np.int32), np.array([2], np.float32)
    p.check()


def test_stream_and_graph():
    p = Problem(17, [5, 2], 3333, [50, 60])
    q = p.params()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    kdv.kdv_logits_process(q, side)
    torch.cuda.current_stream().wait_stream(side)
    p.check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kdv.kdv_logits_process(q)
    p.x.copy_(torch.randn_like(p.x))
    p.y.zero_()
    graph.replay()
    p.check()
