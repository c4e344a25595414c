"""CPU checks of the rotary, 8-bit cache and logits entry points: frequencies
against their formulas, and refusals made on the host before any launch."""
import ctypes
import math
import os
import subprocess

import numpy as np
import pytest
import torch

from speculative_tree_verify_mla_b200 import build, kdv

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, UNSUPPORTED, WORKSPACE = kdv.KDV_ERR_INVALID_ARG, kdv.KDV_ERR_UNSUPPORTED, kdv.KDV_ERR_WORKSPACE
P = 0x10000                      # a 16-byte aligned address that no refused call reads


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return kdv.load()


def status(fn, params):
    return getattr(kdv.load(), fn)(ctypes.byref(params), None)


@pytest.mark.parametrize("cls,cname", [(kdv.RopeParams, "kdv_rope_params"), (kdv.Latent8Params, "kdv_latent8_params"),
                                       (kdv.Verify8Params, "kdv_verify8_params"), (kdv.LogitsParams, "kdv_logits_params")])
def test_struct_layout(tmp_path, cls, cname):
    fields = [f[0] for f in cls._fields_]
    src = tmp_path / "probe.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "kdv.h"\nint main(void){'
                   + "".join(f'printf("%zu\\n", offsetof({cname}, {f}));' for f in fields)
                   + f'printf("%zu\\n", sizeof({cname})); return 0;}}')
    exe = tmp_path / "probe"
    subprocess.check_call(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)])
    got = [int(x) for x in subprocess.check_output([str(exe)]).split()]
    assert got == [getattr(cls, f).offset for f in fields] + [ctypes.sizeof(cls)]


# ---------------------------------------------------------------- frequencies
@pytest.mark.parametrize("rot,base", [(2, 10000.0), (64, 50000.0), (128, 1e6), (256, 10000.0)])
def test_freqs_plain_and_scaled(rot, base):
    k = np.arange(rot // 2)
    plain = np.array([math.pow(base, -2.0 * i / rot) for i in k])
    f, m = kdv.kdv_rope_freqs(rot, base)
    np.testing.assert_allclose(f, plain, rtol=1e-14)
    assert m == 1.0
    f, m = kdv.kdv_rope_freqs(rot, base, kdv.KDV_ROPE_SCALE_LINEAR, factor=8.0)
    np.testing.assert_allclose(f, plain / 8, rtol=1e-14)
    assert m == 1.0
    if rot > 2:
        f, m = kdv.kdv_rope_freqs(rot, base, kdv.KDV_ROPE_SCALE_NTK, factor=8.0)
        # the lowest frequency is divided by the factor, the highest is kept
        np.testing.assert_allclose(f[-1], plain[-1] / 8, rtol=1e-12)
        assert f[0] == 1.0 and m == 1.0


@pytest.mark.parametrize("rot,base,factor,trained", [(64, 50000.0, 32.0, 4096.0), (128, 10000.0, 4.0, 8192.0), (64, 10000.0, 1.0, 2048.0)])
def test_freqs_yarn(rot, base, factor, trained):
    f, m = kdv.kdv_rope_freqs(rot, base, kdv.KDV_ROPE_SCALE_YARN, factor=factor, trained_len=trained)
    assert m == pytest.approx(0.1 * math.log(factor) + 1.0, rel=1e-15)
    plain = np.array([math.pow(base, -2.0 * i / rot) for i in range(rot // 2)])
    turns = trained * plain / (2 * math.pi)
    # pairs beyond either border by a whole index are one rule's; all lie between the two
    up, down = np.roll(turns, -1), np.roll(turns, 1)
    up[-1], down[0] = 0.0, np.inf
    np.testing.assert_allclose(f[up > 32.0], plain[up > 32.0], rtol=1e-14)
    np.testing.assert_allclose(f[down < 1.0], plain[down < 1.0] / factor, rtol=1e-14)
    assert np.all(f <= plain * (1 + 1e-15)) and np.all(f >= plain / factor * (1 - 1e-15))
    assert np.all(np.diff(f) < 0)


def test_freqs_refusals():
    for kw in [dict(rot_dim=0), dict(rot_dim=7), dict(rot_dim=258), dict(base=1.0), dict(base=float("nan")), dict(rule=4),
               dict(rule=-1), dict(rule=1, factor=0.5), dict(rule=1, factor=float("inf")), dict(rule=2, rot_dim=2),
               dict(rule=3, trained_len=0.0), dict(rule=3, beta_slow=0.0), dict(rule=3, beta_fast=1.0, beta_slow=1.0)]:
        with pytest.raises(kdv.KdvError) as e:
            kdv.kdv_rope_freqs(**{"rot_dim": 64, "base": 10000.0, "factor": 2.0, **kw})
        assert e.value.status == INVALID, kw


# ------------------------------------------------------------------- refusals
def rope_params(**kw):
    base = dict(tokens=4, heads=2, dim=64, rot_dim=64, layout=0, inverse=0, x_dtype=0, y_dtype=0, x=P, x_token_stride=128,
                x_head_stride=64, y=P, y_token_stride=128, y_head_stride=64, pos=P, h_inv_freq=np.ones(32))
    return kdv.make_rope_params(**{**base, **kw})


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(tokens=-1)), (INVALID, dict(heads=0)), (INVALID, dict(dim=0)), (INVALID, dict(rot_dim=0)),
    (INVALID, dict(rot_dim=63)), (INVALID, dict(rot_dim=66)), (UNSUPPORTED, dict(dim=300, rot_dim=258, x_head_stride=300, y_head_stride=300, h_inv_freq=np.ones(129))),
    (INVALID, dict(layout=2)), (INVALID, dict(inverse=2)), (INVALID, dict(x_dtype=2)), (INVALID, dict(y_dtype=-1)),
    (INVALID, dict(h_inv_freq=None)), (INVALID, dict(mscale=float("nan"))), (INVALID, dict(h_inv_freq=np.full(32, np.inf))),
    (INVALID, dict(x_head_stride=63)), (INVALID, dict(y_head_stride=32)), (INVALID, dict(x=None)), (INVALID, dict(y=None)),
    (INVALID, dict(x=P + 1)), (INVALID, dict(y_token_stride=0, y=2 * P)), (INVALID, dict(y_dtype=1)),       # in place with another type
    (INVALID, dict(x_token_stride=256)), (INVALID, dict(pos=None)), (INVALID, dict(pos=None, batch=1, tree_off=P, prefix_len=P)),
    (UNSUPPORTED, dict(pos=None, batch=129, tree_off=P, prefix_len=P, depth=P)),
])
def test_rope_refusals(want, kw):
    assert status("kdv_rope", rope_params(**kw)) == want


def write_params(**kw):
    base = dict(rows=3, d_latent=512, d_rope=64, dtype=0, c=P, c_stride=512, k_rope=P, k_stride=64, slot=P, h_inv_freq=np.ones(32),
                rot_dim=64, layout=0, pos=P, c8=P, kr=P, kv_scale=P, num_slots=10)
    return kdv.make_latent8_params(**{**base, **kw})


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(rows=-1)), (INVALID, dict(d_latent=0)), (INVALID, dict(d_rope=-1)), (UNSUPPORTED, dict(d_latent=513, c_stride=513)),
    (UNSUPPORTED, dict(d_rope=65, k_stride=65)), (INVALID, dict(dtype=3)), (INVALID, dict(c_stride=511)), (INVALID, dict(k_stride=63)),
    (INVALID, dict(scale_block=0)), (INVALID, dict(scale_block=3, static_scale=1)), (INVALID, dict(scale_block=8192, static_scale=1)),
    (UNSUPPORTED, dict(scale_block=2)), (INVALID, dict(static_scale=2)), (INVALID, dict(num_slots=-1)), (INVALID, dict(rot_dim=66)),
    (INVALID, dict(rot_dim=3)), (INVALID, dict(layout=5)), (INVALID, dict(mscale=float("inf"))), (INVALID, dict(slot=None)),
    (INVALID, dict(slot=None, batch=1, tree_off=P, prefix_len=P)), (UNSUPPORTED, dict(slot=None, batch=200, tree_off=P, prefix_len=P, kv_off=P)),
    (INVALID, dict(pos=None)), (INVALID, dict(pos=None, batch=1, tree_off=P, prefix_len=P)), (INVALID, dict(c=None)), (INVALID, dict(c8=None)),
    (INVALID, dict(kr=None)), (INVALID, dict(k_rope=None)), (INVALID, dict(kv_scale=None)), (INVALID, dict(c=P + 1)), (INVALID, dict(kv_scale=P + 2)),
])
def test_write_refusals(want, kw):
    assert status("kdv_latent8_write", write_params(**kw)) == want


def attn_params(**kw):
    base = dict(batch=1, num_heads=64, d_latent=512, d_rope=64, scale=0.1, dtype=0, out_dtype=0, impl=0, q=P, c8=P, kr=P, kv_scale=P,
                num_slots=100, kv_off=P, tree_off=P, h_prefix_len=[50], h_tree_T=[4], mask=P, o=P, lse=P)
    return kdv.make_verify8_params(**{**base, **kw})


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(batch=0)), (UNSUPPORTED, dict(batch=129)), (INVALID, dict(num_heads=0)), (INVALID, dict(d_latent=0)),
    (UNSUPPORTED, dict(d_latent=513)), (UNSUPPORTED, dict(d_rope=65)), (INVALID, dict(dtype=2)), (INVALID, dict(out_dtype=7)),
    (INVALID, dict(impl=9)), (INVALID, dict(impl=-1)), (UNSUPPORTED, dict(impl=kdv.KDV_IMPL_TC_STAGED)), (UNSUPPORTED, dict(impl=kdv.KDV_IMPL_TC_1SM)),
    (INVALID, dict(scale=float("nan"))), (INVALID, dict(num_splits=-1)), (INVALID, dict(scale_block=0)), (INVALID, dict(scale_block=48)),
    (INVALID, dict(h_prefix_len=[-1])), (INVALID, dict(h_tree_T=[0])), (UNSUPPORTED, dict(h_tree_T=[65])), (INVALID, dict(q_row_stride=575)),
    (UNSUPPORTED, dict(impl=kdv.KDV_IMPL_TC, dtype=1)), (UNSUPPORTED, dict(impl=kdv.KDV_IMPL_TC, d_latent=256)),
    (UNSUPPORTED, dict(impl=kdv.KDV_IMPL_TC, scale=0.0)), (UNSUPPORTED, dict(num_splits=5000)),
    (INVALID, dict(q=None)), (INVALID, dict(c8=None)), (INVALID, dict(kr=None)), (INVALID, dict(kv_scale=None)), (INVALID, dict(kv_off=None)),
    (INVALID, dict(tree_off=None)), (INVALID, dict(o=None)), (INVALID, dict(q=P + 1)), (INVALID, dict(mask=P + 4)), (INVALID, dict(num_slots=-1)),
    (INVALID, dict(impl=kdv.KDV_IMPL_TC, q=P + 8)), (INVALID, dict(impl=kdv.KDV_IMPL_TC, q_row_stride=577)), (INVALID, dict(impl=kdv.KDV_IMPL_TC, c8=P + 8)),
    (INVALID, dict(impl=kdv.KDV_IMPL_TC, kr=P + 2)), (INVALID, dict(impl=kdv.KDV_IMPL_TC, o=P + 4)), (WORKSPACE, dict(num_splits=2)), (WORKSPACE, dict(num_splits=2, workspace=P, workspace_bytes=100)),
])
def test_attn_refusals(want, kw):
    assert status("kdv_verify_attn8", attn_params(**kw)) == want


def test_attn_workspace_and_plan():
    assert kdv.kdv_verify_attn8_workspace(attn_params(num_splits=1)) == 0
    n = kdv.kdv_verify_attn8_workspace(attn_params(num_splits=3))
    assert n >= 3 * 4 * 64 * (512 * 2 + 8)
    splits, items = kdv.kdv_verify_attn8_plan(attn_params(num_splits=3))
    assert splits == [3] and items >= 3
    splits, items = kdv.kdv_verify_attn8_plan(attn_params(batch=3, h_prefix_len=[0, 5000, 200000], h_tree_T=[1, 2, 64]))
    assert all(s >= 1 for s in splits) and splits[2] > splits[0]


def logits_params(**kw):
    base = dict(batch=1, max_T=4, total_nodes=4, vocab=100, dtype=0, out_dtype=0, logits=P, logits_ld=100, out=2 * P, out_ld=100, tree_off=P)
    return kdv.make_logits_params(**{**base, **kw})


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(batch=0)), (INVALID, dict(max_T=0)), (INVALID, dict(total_nodes=-1)), (INVALID, dict(vocab=0)), (UNSUPPORTED, dict(batch=129)),
    (UNSUPPORTED, dict(max_T=65)), (INVALID, dict(dtype=2)), (INVALID, dict(out_dtype=2)), (INVALID, dict(logits_ld=99)), (INVALID, dict(out_ld=99)),
    (INVALID, dict(logits=None)), (INVALID, dict(out=None)), (INVALID, dict(tree_off=None)), (INVALID, dict(parent=P)), (INVALID, dict(token=P)),
    (INVALID, dict(hist=P)), (INVALID, dict(hist=P, hist_len=P, hist_ld=-1)), (INVALID, dict(bias_off=P, bias_token=P)),
    (INVALID, dict(allow=P, allow_ld=3, allow_rows=4)), (INVALID, dict(allow=P, allow_ld=4, allow_rows=3)), (INVALID, dict(allow=P, allow_ld=4, allow_rows=-1, allow_row=P)),
    (INVALID, dict(logits=P + 1)), (INVALID, dict(out=P, out_dtype=1)), (INVALID, dict(out=P, out_ld=104)),
])
def test_logits_refusals(want, kw):
    assert status("kdv_logits_process", logits_params(**kw)) == want


def test_empty_calls_launch_nothing():
    assert status("kdv_rope", rope_params(tokens=0, x=None, y=None, pos=None)) == kdv.KDV_OK
    assert status("kdv_latent8_write", write_params(rows=0, c=None, c8=None)) == kdv.KDV_OK
    assert status("kdv_logits_process", logits_params(total_nodes=0, logits=None, out=None)) == kdv.KDV_OK
    for fn in ("kdv_rope", "kdv_latent8_write", "kdv_verify_attn8", "kdv_logits_process"):
        assert getattr(kdv.load(), fn)(None, None) == INVALID


def test_binding_refuses_host_tensors():
    with pytest.raises(ValueError):
        rope_params(x=torch.zeros(4, 2, 64))
    with pytest.raises(ValueError):
        attn_params(q=torch.zeros(256, 576))
