"""One verify step over the 8-bit cache as a program makes it: tree masks and
depths, rotated queries, the draft rows' quantising write, attention, processed
logits, acceptance with the page commit. On one stream, captured in a graph and
replayed; every stage against its 64-bit form on the stage before's values."""
import numpy as np
import pytest
import torch

from speculative_tree_verify_mla_b200 import kdv
from tests import plain8

pytestmark = pytest.mark.gpu
i32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")  # noqa: E731


@pytest.mark.parametrize("half", [0, 1])
def test_verify_step(half):
    rng = np.random.default_rng(31 + half)
    g = torch.Generator(device="cuda").manual_seed(5)
    prefix, T, H, V = [300, 97], [9, 5], 64, 3000
    B, n = len(T), sum(T)
    trees = [plain8.random_tree(rng, t) for t in T]
    parent = np.concatenate(trees)
    case = plain8.Attn(40, prefix, trees, H)                       # lengths, offsets, page table, masks
    freq, mscale = kdv.kdv_rope_freqs(64, 50000.0, kdv.KDV_ROPE_SCALE_YARN, factor=8.0)
    layout = kdv.KDV_ROPE_HALF if half else kdv.KDV_ROPE_INTERLEAVED
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    parent_d, tree_off, kv_off, prefix_d = i32(parent), i32(case.tree_off), i32(case.kv_off), i32(prefix)
    table0 = i32(case.table)
    table = table0.clone()
    mask, depth = torch.zeros(n, dtype=torch.int64, device="cuda"), torch.zeros(n, dtype=torch.int32, device="cuda")
    # the cache holds the prefixes already, written as a prompt is
    c8 = torch.zeros(case.slots, 512, dtype=torch.uint8, device="cuda")
    kr, scale = torch.zeros(case.slots, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(case.slots, device="cuda")
    old_slot = np.concatenate([case.table[case.kv_off[b]:case.kv_off[b] + prefix[b]] for b in range(B)])
    old_pos = np.concatenate([np.arange(L) for L in prefix])
    normal = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    common = dict(d_latent=512, d_rope=64, dtype=kdv.KDV_BF16, c_stride=512, k_stride=64, h_inv_freq=freq, rot_dim=64, layout=layout,
                  mscale=mscale, c8=c8, kr=kr, kv_scale=scale, num_slots=case.slots, d_err=err)
    old_c, old_k = normal(len(old_slot), 512), normal(len(old_slot), 64)
    kdv.kdv_latent8_write(kdv.make_latent8_params(rows=len(old_slot), c=old_c, k_rope=old_k, slot=i32(old_slot), pos=i32(old_pos), **common))
    # this step's inputs
    q0, new_c, new_k = normal(n * H, 576), normal(n, 512), normal(n, 64)
    q = q0.clone()
    logits0 = normal(n, V) * 3
    logits = logits0.clone()
    token = rng.integers(0, 40, n)
    for i in range(n):                                             # the target agrees with most drafted tokens
        if parent[i] >= 0 and i % 4:
            b = int(np.searchsorted(case.tree_off, i, side="right")) - 1
            logits0[int(case.tree_off[b]) + parent[i], token[i]] = 40.0
    hist = rng.integers(0, 40, (B, 60))
    hist_len, prompt_len, rep, pres, fq = [60, 33], [20, 0], [1.3, 0.9], [0.5, -0.25], [0.125, 0.25]
    allow = torch.full((B, (V + 31) // 32), -1, dtype=torch.int32, device="cuda")
    allow[1, 3:] = 0                                               # request 1 may only make tokens below 96
    allow_row = i32([-1] * T[0] + [1] * T[1])
    f32 = lambda a: torch.tensor(a, dtype=torch.float32, device="cuda")  # noqa: E731
    o, lse = torch.zeros(n * H, 512, dtype=torch.bfloat16, device="cuda"), torch.zeros(n * H, device="cuda")

    rope = kdv.make_rope_params(tokens=n, heads=H, dim=64, rot_dim=64, layout=layout, inverse=0, x_dtype=kdv.KDV_BF16, y_dtype=kdv.KDV_BF16,
                                x=q[:, 512:], x_token_stride=H * 576, x_head_stride=576, y=q[:, 512:], y_token_stride=H * 576, y_head_stride=576,
                                batch=B, tree_off=tree_off, prefix_len=prefix_d, depth=depth, h_inv_freq=freq, mscale=mscale)
    write = kdv.make_latent8_params(rows=n, c=new_c, k_rope=new_k, batch=B, tree_off=tree_off, prefix_len=prefix_d, depth=depth, kv_off=kv_off,
                                    page_table=table, **common)
    attn = kdv.make_verify8_params(batch=B, num_heads=H, d_latent=512, d_rope=64, scale=case.sm_scale, dtype=kdv.KDV_BF16, out_dtype=kdv.KDV_BF16,
                                   impl=kdv.KDV_IMPL_AUTO, q=q, q_row_stride=576, c8=c8, kr=kr, kv_scale=scale, num_slots=case.slots, page_table=table,
                                   kv_off=kv_off, tree_off=tree_off, prefix_len=prefix_d, h_prefix_len=prefix, h_tree_T=T, mask=mask, o=o, lse=lse,
                                   d_err=err)
    ws = torch.empty(max(16, kdv.kdv_verify_attn8_workspace(attn)), dtype=torch.uint8, device="cuda")
    attn.workspace, attn.workspace_bytes = ws.data_ptr(), ws.numel()
    token_d = i32(token)
    proc = kdv.make_logits_params(batch=B, max_T=max(T), total_nodes=n, vocab=V, dtype=kdv.KDV_BF16, out_dtype=kdv.KDV_BF16, logits=logits,
                                  logits_ld=V, out=logits, out_ld=V, tree_off=tree_off, parent=parent_d, token=token_d, hist=i32(hist), hist_ld=60,
                                  hist_len=i32(hist_len), prompt_len=i32(prompt_len), repetition=f32(rep), presence=f32(pres), frequency=f32(fq),
                                  allow=allow, allow_ld=allow.stride(0), allow_rows=B, allow_row=allow_row, d_err=err)
    target, path = torch.zeros(n, dtype=torch.int32, device="cuda"), torch.zeros(B, max(T), dtype=torch.int32, device="cuda")
    length, bonus = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
    acc = kdv.make_accept_params(batch=B, max_T=max(T), total_nodes=n, vocab=V, dtype=kdv.KDV_BF16, logits=logits, logits_ld=V, target_in=None,
                                 token=token_d, parent=parent_d, tree_off=tree_off, target_out=target, accept_len=length, accept_path=path,
                                 bonus=bonus, page_table=table, kv_off=kv_off, prefix_len=prefix_d, prefix_len_out=None, workspace=None,
                                 workspace_bytes=0, d_err=err)
    aws = torch.empty(max(16, kdv.kdv_tree_accept_workspace(acc)), dtype=torch.uint8, device="cuda")
    acc.workspace, acc.workspace_bytes = aws.data_ptr(), aws.numel()

    def step():
        q.copy_(q0)
        logits.copy_(logits0)
        table.copy_(table0)
        kdv.kdv_tree_mask_build(parent_d, tree_off, B, max(T), mask, depth, err)
        kdv.kdv_rope(rope)
        kdv.kdv_latent8_write(write)
        kdv.kdv_verify_attn8(attn)
        kdv.kdv_logits_process(proc)
        kdv.kdv_tree_accept(acc)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    eager = [t.clone() for t in (o, lse, logits, target, path, length, bonus, table)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t in (o, lse, mask, depth, target, path, length, bonus):
        t.zero_()
    ws.fill_(0xA5)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert err.item() == 0
    for a, b in zip(eager, (o, lse, logits, target, path, length, bonus, table)):
        assert torch.equal(a, b)

    # ---- rotated queries: bf16's half step and fp32's arithmetic
    pos = np.array([prefix[b] + int(depth[int(case.tree_off[b]) + t]) for b in range(B) for t in range(T[b])])
    x = q0[:, 512:].double().cpu().numpy().reshape(n, H, 64)
    want = plain8.rope(x, pos, freq, 64, half, mscale)
    got = q[:, 512:].double().cpu().numpy().reshape(n, H, 64)
    assert np.all(np.abs(got - want) <= 2.0 ** -8 * np.abs(want) * (1 + 2.0 ** -7) + 2.0 ** -21 * 2 * mscale * np.abs(x).max(-1, keepdims=True))
    assert torch.equal(q[:, :512], q0[:, :512])
    # ---- the draft rows in the cache
    slot = np.concatenate([case.table[case.kv_off[b] + prefix[b]:case.kv_off[b + 1]] for b in range(B)])
    rows = new_c.float().cpu().numpy()
    sc = plain8.row_scale(rows)
    np.testing.assert_array_equal(scale.cpu().numpy()[slot], sc.astype(np.float32))
    np.testing.assert_array_equal(c8.cpu().numpy()[slot], plain8.codes(rows, sc))
    # ---- attention on those queries and that cache
    case.c8, case.kr, case.scale, case.q = c8.cpu().numpy(), kr.cpu(), scale.cpu().numpy(), q.cpu()
    ref, ref_lse, ob, lb = case.answer()
    assert np.all(np.abs(o.double().cpu().numpy() - ref) <= ob + 2.0 ** -8 * (np.abs(ref) + ob))
    assert np.all(np.abs(lse.double().cpu().numpy() - ref_lse) <= lb)
    # ---- logits, and what acceptance makes of them
    y = logits.float().cpu().numpy()
    want_len = []
    for b in range(B):
        t0 = int(case.tree_off[b])
        for t in range(T[b]):
            walk, u = [], t
            while trees[b][u] >= 0:
                walk.append(int(token[t0 + u]))
                u = trees[b][u]
            bits = np.arange(V) < 96 if b == 1 else None
            ref, size = plain8.penalised(logits0[t0 + t].double().cpu().numpy(), hist[b, :hist_len[b]], prompt_len[b], walk, np.float32(rep[b]),
                                         np.float32(pres[b]), np.float32(fq[b]), np.zeros(V), bits)
            ok = np.isfinite(ref)
            assert np.array_equal(np.isneginf(y[t0 + t]), ~ok)
            assert np.all(np.abs(y[t0 + t][ok] - ref[ok]) <= 2.0 ** -8 * np.abs(ref[ok]) * (1 + 2.0 ** -7) + 2.0 ** -22 * size[ok])
        best = y[t0:t0 + T[b]].argmax(1)
        np.testing.assert_array_equal(target.cpu().numpy()[t0:t0 + T[b]], best)
        accepted = [False] * T[b]
        deep = []
        for t in range(T[b]):
            p = trees[b][t]
            accepted[t] = p < 0 or (accepted[p] and best[p] == token[t0 + t])
            if accepted[t]:
                deep.append(int(depth[t0 + t]))
        want_len.append(max(deep) + 1)
    np.testing.assert_array_equal(length.cpu().numpy(), want_len)
    assert max(want_len) >= 2
