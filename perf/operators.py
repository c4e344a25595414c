"""What is measured of the operators around an 8-bit latent cache: rotary
positions, the cache's quantising write, tree-verify attention over it, and
the processing of the target model's logits before acceptance.

``run`` computes each operator in its plain form (elementary torch operations
in 32 bits, angles in 64) or, where ``own`` is true, through the library's
entry points. ``exact`` computes the same from the definitions in 64 bits.

Shared definitions: a request b has L committed tokens and a draft tree of T
nodes; node t sits at position L + depth(t) and sees keys 0..L-1 and its own
ancestors (itself included). A cache row is scale x (c8[512] || kr[64]), c8 in
e4m3, kr in bf16, one scale for each block of consecutive slots.
"""
import math
import random

import torch

own = False

D_C, D_R, D_Q = 512, 64, 576       # latent dims, rope dims, query row
VOCAB = 163840                     # vocabulary of the acceptance workloads
E4M3_MAX = 448.0


# --------------------------------------------------------------------- cases
def listed():
    return [
        # the rope part of a verify step's query rows: one request, 13 nodes, 64 heads, in rows of 576
        dict(name="rope_step", op="rope", tokens=13, heads=64, dim=64, rot=64, row=576, layout="interleaved",
             yarn=True, far=5600, dtype="bf16"),
        # queries of a prompt chunk: half layout on part of each head, the rest passed through
        dict(name="rope_prompt", op="rope", tokens=8192, heads=64, dim=128, rot=64, row=128, layout="half",
             yarn=False, far=1000000, dtype="bf16"),
        # a verify step of eight requests writes its draft nodes' rows (rotated keys, a scale for each row)
        dict(name="write_step", op="write", rows=104, slots=32768, block=1, dtype="bf16", layout="interleaved", far=30000),
        # a long prompt goes into the cache
        dict(name="write_prompt", op="write", rows=65536, slots=81920, block=1, dtype="bf16", layout="half", far=200000),
        # the same with calibrated scales for blocks of 64 slots, from 32-bit rows, an odd count
        dict(name="write_blocks", op="write", rows=9001, slots=16384, block=64, dtype="f32", layout="interleaved", far=9001),
        # one token of one request with few heads: the smallest call
        dict(name="attn_one", op="attn", batch=1, heads=16, tree=1, lo=700, hi=700, paged=False, block=1),
        # the verify layer of the default benchmark (one request, 13 nodes, 64 heads)
        dict(name="attn_layer", op="attn", batch=1, heads=64, tree=13, lo=5553, hi=5553, paged=True, block=1),
        # single tokens of a ragged serving batch, paged
        dict(name="attn_decode", op="attn", batch=32, heads=64, tree=1, lo=1024, hi=16384, paged=True, block=1),
        # a tree over a very long context, scales for blocks of 64 slots
        dict(name="attn_long", op="attn", batch=1, heads=64, tree=16, lo=200000, hi=200000, paged=False, block=64),
        # one node of a small vocabulary: the smallest call
        dict(name="logits_one", op="logits", batch=1, tree=1, vocab=32000, hist=700, dtype="bf16"),
        # the target logits of a verify step
        dict(name="logits_step", op="logits", batch=1, tree=13, vocab=VOCAB, hist=5553, dtype="bf16"),
        # a serving batch in 32 bits
        dict(name="logits_batch", op="logits", batch=32, tree=5, vocab=VOCAB, hist=8192, dtype="f32"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["rope", "write", "attn", "attn", "logits"])
    if op == "rope":
        dim = rng.choice([64, 128, 192])
        rot = rng.choice([32, 64]) if dim == 64 else rng.choice([64, 96, 128])
        heads = _log(rng, 1, 128)
        return dict(op=op, tokens=_log(rng, 1, 8192 * 64 * 128 // (heads * dim * 2)), heads=heads, dim=dim, rot=min(rot, dim),
                    row=dim + rng.choice([0, 64, 512]), layout=rng.choice(["interleaved", "half"]),
                    yarn=rng.random() < 0.5, far=_log(rng, 100, 2000000), dtype=rng.choice(["bf16", "f32"]))
    if op == "write":
        rows, block = _log(rng, 1, 40000), rng.choice([1, 1, 16, 64])
        return dict(op=op, rows=rows, slots=rows + _log(rng, 1, 20000), block=block, dtype=rng.choice(["bf16", "f32"]),
                    layout=rng.choice(["interleaved", "half"]), far=_log(rng, 100, 1000000))
    if op == "attn":
        batch, heads, tree = _log(rng, 1, 32), rng.choice([8, 16, 32, 64, 128]), rng.choice([1, 1, 2, _log(rng, 2, 64)])
        most = min(200000, 250000 // batch, 150000000 // (batch * heads * tree))
        hi = _log(rng, 1, max(2, most))
        return dict(op=op, batch=batch, heads=heads, tree=tree, lo=rng.randint(0, hi), hi=hi, paged=rng.random() < 0.7,
                    block=rng.choice([1, 1, 64]))
    tree = _log(rng, 1, 32)
    return dict(op=op, batch=_log(rng, 1, max(1, 128 // tree)), tree=tree, vocab=_log(rng, 1000, VOCAB), hist=_log(rng, 1, 16384),
                dtype=rng.choice(["bf16", "f32"]))


# -------------------------------------------------------------------- inputs
def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _inv_freq(rot, yarn):
    """The inverse frequencies of base 50000 (64 bits), unscaled or scaled for
    32 times the trained context by the YaRN rule; and the magnitude factor."""
    base, factor, trained, fast, slow = 50000.0, 32.0, 4096.0, 32.0, 1.0
    plain = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    if not yarn:
        return torch.tensor(plain, dtype=torch.float64), 1.0
    where = lambda turns: rot * math.log(trained / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
    low, high = max(math.floor(where(fast)), 0), min(math.ceil(where(slow)), rot - 1)
    ramp = [min(max((i - low) / max(high - low, 0.001), 0.0), 1.0) for i in range(rot // 2)]
    return (torch.tensor([f / factor * r + f * (1 - r) for f, r in zip(plain, ramp)], dtype=torch.float64),
            0.1 * math.log(factor) + 1.0)


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _tree(rng, T, reach):
    """parent[] of a random tree in discovery order."""
    return [-1] + [rng.randint(max(0, i - reach), i - 1) for i in range(1, T)]


def _signed64(m):
    return m - (1 << 64) if m >> 63 else m


def _lengths(case, rng):
    """Ragged prefix lengths between lo and hi; the first is hi."""
    return [case["hi"]] + [rng.randint(case["lo"], case["hi"]) for _ in range(case["batch"] - 1)]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = random.Random(seed)
    normal = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    s = {"case": case}
    if case["op"] == "rope":
        n, h, d = case["tokens"], case["heads"], case["dim"]
        # rows of `row` elements a head; the rotated head sits at the end of the row, as q_rope does in a query row
        s["x"] = normal(n, h, case["row"]).to(_dtype(case))[:, :, case["row"] - d:]
        s["pos"] = torch.randint(0, case["far"], (n,), generator=g, device="cuda", dtype=torch.int32)
        s["inv_freq"], s["mscale"] = _inv_freq(case["rot"], case["yarn"])
        s["inv_dev"] = s["inv_freq"].cuda()
    elif case["op"] == "write":
        n, slots, block = case["rows"], case["slots"], case["block"]
        # tokens differ in magnitude
        s["c"] = (normal(n, D_C) * torch.exp(0.5 * normal(n, 1))).to(_dtype(case))
        s["k"] = normal(n, D_R).to(_dtype(case))
        s["slot"] = torch.randperm(slots, generator=g, device="cuda")[:n].to(torch.int32)
        s["pos"] = torch.randint(0, case["far"], (n,), generator=g, device="cuda", dtype=torch.int32)
        s["inv_freq"], s["mscale"] = _inv_freq(D_R, False)
        s["inv_dev"] = s["inv_freq"].cuda()
        s["c8"] = torch.zeros(slots, D_C, dtype=torch.uint8, device="cuda")
        s["kr"] = torch.zeros(slots, D_R, dtype=torch.bfloat16, device="cuda")
        blocks = (slots + block - 1) // block
        # blocks of several slots have calibrated scales (powers of two here), single rows get theirs in the write
        s["scale"] = (torch.exp2(torch.randint(-6, -3, (blocks,), generator=g, device="cuda").float()) if block > 1
                      else torch.zeros(blocks, device="cuda"))
    elif case["op"] == "attn":
        B, H, T = case["batch"], case["heads"], case["tree"]
        lens = _lengths(case, rng)
        ns = [L + T for L in lens]
        off = [0]
        for n in ns:
            off.append(off[-1] + n)
        masks = []
        for _ in range(B):
            parent, m = _tree(rng, T, 3), []
            for t in range(T):
                m.append((m[parent[t]] if parent[t] >= 0 else 0) | (1 << t))
            masks += m
        slots, block = off[-1] + (97 if case["paged"] else 0), case["block"]
        s.update(lens=lens, ns=ns, slots=slots)
        s["kv_off"], s["tree_off"], s["prefix"] = _i32(off), _i32([b * T for b in range(B + 1)]), _i32(lens)
        s["mask"] = torch.tensor([_signed64(m) for m in masks], dtype=torch.int64, device="cuda")
        s["table"] = torch.randperm(slots, generator=g, device="cuda")[:off[-1]].to(torch.int32) if case["paged"] else None
        s["q"] = torch.cat([normal(B * T * H, D_C) * 0.5, normal(B * T * H, D_R)], 1).bfloat16()
        # rows of N(0, 1) latents with magnitudes that differ from token to token, each under its block's scale
        amp = torch.exp(0.3 * normal((slots + block - 1) // block))
        s["scale"] = torch.exp2(torch.ceil(torch.log2(amp * 4.5 / E4M3_MAX)))
        unit = (1.0 / s["scale"]).repeat_interleave(block)[:slots, None]
        size = (amp.repeat_interleave(block)[:slots, None] * unit)
        s["c8"] = (normal(slots, D_C) * size).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
        s["kr"] = (normal(slots, D_R) * unit).bfloat16()
    else:
        B, T, V = case["batch"], case["tree"], case["vocab"]
        sumT = B * T
        s["logits"] = (normal(sumT, V) * 3).to(_dtype(case))
        s["parent"] = _i32([p for _ in range(B) for p in _tree(rng, T, 3)])
        # tokens come from a small part of the vocabulary, so that they repeat
        s["token"] = torch.randint(0, max(1, V // 50), (sumT,), generator=g, device="cuda", dtype=torch.int32)
        s["hist"] = torch.randint(0, max(1, V // 50), (B, case["hist"]), generator=g, device="cuda", dtype=torch.int32)
        lens = [case["hist"]] + [rng.randint(0, case["hist"]) for _ in range(B - 1)]
        s["hist_len"], s["prompt_len"] = _i32(lens), _i32([rng.randint(0, n) for n in lens])
        s["repeat"] = 1.0 + 0.5 * torch.rand(B, generator=g, device="cuda")
        s["presence"] = torch.rand(B, generator=g, device="cuda")
        s["frequency"] = 0.5 * torch.rand(B, generator=g, device="cuda")
        nb = min(V, 200)                       # biased tokens of a request, in ascending order
        s["bias_tok"] = torch.stack([torch.sort(torch.randperm(V, generator=g, device="cuda")[:nb])[0] for _ in range(B)]).to(torch.int32).reshape(-1)
        s["bias_val"] = 5 * normal(B * nb)
        s["bias_off"] = _i32([b * nb for b in range(B + 1)])
        words = (V + 31) // 32
        s["allow"] = torch.randint(-2 ** 31, 2 ** 31, (sumT, words), generator=g, device="cuda", dtype=torch.int64).to(torch.int32)
        s["allow_row"] = _i32([t if rng.random() < 0.6 else -1 for t in range(sumT)])   # the others are unconstrained
        s["tree_off"] = _i32([b * T for b in range(B + 1)])
    if own:
        s["call"] = _handle(s)                 # the filled parameter block and the output buffers that a program keeps
    return s


# ----------------------------------------------------------------- the calls
def _handle(s):
    from speculative_tree_verify_mla_b200 import kdv

    case = s["case"]
    code = {torch.bfloat16: kdv.KDV_BF16, torch.float32: kdv.KDV_F32}
    layout = {"interleaved": kdv.KDV_ROPE_INTERLEAVED, "half": kdv.KDV_ROPE_HALF}
    if case["op"] == "rope":
        x = s["x"]
        y = torch.empty(x.shape, dtype=x.dtype, device="cuda")
        p = kdv.make_rope_params(tokens=x.shape[0], heads=x.shape[1], dim=x.shape[2], rot_dim=case["rot"], layout=layout[case["layout"]],
                                 x_dtype=code[x.dtype], y_dtype=code[y.dtype], x=x, x_token_stride=x.stride(0), x_head_stride=x.stride(1),
                                 y=y, y_token_stride=y.stride(0), y_head_stride=y.stride(1), pos=s["pos"],
                                 h_inv_freq=s["inv_freq"], mscale=s["mscale"])
        return lambda: (kdv.kdv_rope(p), y)[1]
    if case["op"] == "write":
        p = kdv.make_latent8_params(rows=case["rows"], d_latent=D_C, d_rope=D_R, dtype=code[s["c"].dtype], c=s["c"], c_stride=D_C,
                                    k_rope=s["k"], k_stride=D_R, slot=s["slot"], pos=s["pos"], rot_dim=D_R, layout=layout[case["layout"]],
                                    h_inv_freq=s["inv_freq"], mscale=s["mscale"], c8=s["c8"], kr=s["kr"], kv_scale=s["scale"],
                                    num_slots=case["slots"], scale_block=case["block"], static_scale=int(case["block"] > 1))
        return lambda: (kdv.kdv_latent8_write(p), (s["c8"].view(torch.float8_e4m3fn), s["kr"], s["scale"]))[1]
    if case["op"] == "attn":
        rows = s["q"].shape[0]
        o, lse = torch.empty(rows, D_C, dtype=torch.bfloat16, device="cuda"), torch.empty(rows, device="cuda")
        p = kdv.make_verify8_params(batch=case["batch"], num_heads=case["heads"], d_latent=D_C, d_rope=D_R, scale=192 ** -0.5,
                                    dtype=kdv.KDV_BF16, out_dtype=kdv.KDV_BF16, impl=kdv.KDV_IMPL_AUTO, q=s["q"], q_row_stride=D_Q,
                                    c8=s["c8"], kr=s["kr"], kv_scale=s["scale"], scale_block=case["block"], num_slots=s["slots"],
                                    page_table=s["table"], kv_off=s["kv_off"], tree_off=s["tree_off"], prefix_len=s["prefix"],
                                    h_prefix_len=s["lens"], h_tree_T=[case["tree"]] * case["batch"], mask=s["mask"], o=o, lse=lse)
        ws = torch.empty(max(16, kdv.kdv_verify_attn8_workspace(p)), dtype=torch.uint8, device="cuda")
        p.workspace, p.workspace_bytes = ws.data_ptr(), ws.numel()
        s["workspace"] = ws
        return lambda: (kdv.kdv_verify_attn8(p), (o, lse))[1]
    x = s["logits"]
    out = torch.empty_like(x)
    p = kdv.make_logits_params(batch=case["batch"], max_T=case["tree"], total_nodes=x.shape[0], vocab=case["vocab"], dtype=code[x.dtype],
                               out_dtype=code[x.dtype], logits=x, logits_ld=x.stride(0), out=out, out_ld=out.stride(0), tree_off=s["tree_off"],
                               parent=s["parent"], token=s["token"], hist=s["hist"], hist_ld=case["hist"], hist_len=s["hist_len"],
                               prompt_len=s["prompt_len"], repetition=s["repeat"], presence=s["presence"], frequency=s["frequency"],
                               bias_off=s["bias_off"], bias_token=s["bias_tok"], bias_value=s["bias_val"], allow=s["allow"],
                               allow_ld=s["allow"].stride(0), allow_rows=s["allow"].shape[0], allow_row=s["allow_row"])
    return lambda: (kdv.kdv_logits_process(p), out)[1]


# ----------------------------------------------------------- the plain forms
def _rotate(x, pos, inv_freq, mscale, rot, layout):
    """x [tokens, heads, dim] in 32 bits; the first `rot` dims are turned."""
    a = pos.double()[:, None] * inv_freq[None, :]
    cos, sin = (torch.cos(a) * mscale).float()[:, None, :], (torch.sin(a) * mscale).float()[:, None, :]
    x = x.float()
    r, rest = x[..., :rot], x[..., rot:]
    if layout == "interleaved":
        u, v = r[..., 0::2], r[..., 1::2]
        turned = torch.stack([u * cos - v * sin, u * sin + v * cos], -1).flatten(-2)
    else:
        u, v = r[..., :rot // 2], r[..., rot // 2:]
        turned = torch.cat([u * cos - v * sin, u * sin + v * cos], -1)
    return torch.cat([turned, rest], -1)


def _rope_plain(s):
    c = s["case"]
    return _rotate(s["x"], s["pos"], s["inv_dev"], s["mscale"], c["rot"], c["layout"]).to(_dtype(c))


def _write_plain(s):
    c = s["case"]
    rows, slot = s["c"].float(), s["slot"].long()
    if c["block"] == 1:
        # the least power of two that brings the row's largest value to 448 or below
        m, e = torch.frexp(rows.abs().amax(1))
        scale = torch.where(m == 0, torch.ones_like(m), torch.ldexp(torch.ones_like(m), torch.where(m <= 0.875, e - 9, e - 8)))
        s["scale"][slot] = scale
    else:
        scale = s["scale"][slot // c["block"]]
    s["c8"][slot] = (rows / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
    k = _rotate(s["k"][:, None, :], s["pos"], s["inv_dev"], s["mscale"], D_R, c["layout"])[:, 0]
    s["kr"][slot] = (k / scale[:, None]).bfloat16()
    return s["c8"].view(torch.float8_e4m3fn), s["kr"], s["scale"]


def _attn_plain(s):
    c = s["case"]
    B, H, T = c["batch"], c["heads"], c["tree"]
    j = torch.arange(max(s["ns"]), device="cuda")
    n = s["prefix"].long()[:, None] + T
    key = s["kv_off"][:-1].long()[:, None] + torch.minimum(j[None, :], n - 1)
    slot = s["table"].long()[key] if s["table"] is not None else key
    rows = torch.cat([s["c8"].view(torch.float8_e4m3fn)[slot].float(), s["kr"][slot].float()], 2) * s["scale"][slot // c["block"]][..., None]
    u = j[None, :] - s["prefix"].long()[:, None]                       # which node a key is, below 0 for the prefix
    bit = (s["mask"].view(B, T, 1) >> u.clamp(0, 63)[:, None, :]) & 1
    seen = ((u < 0)[:, None, :] | (bit == 1)) & (u < T)[:, None, :]    # [B, T, keys]
    x = torch.bmm(s["q"].float().view(B, T * H, D_Q), rows.transpose(1, 2)) * 192 ** -0.5
    x = x.view(B, T, H, -1).masked_fill_(~seen[:, :, None, :], -math.inf)
    top = x.amax(-1, keepdim=True)
    x = torch.exp(x - top)
    total = x.sum(-1, keepdim=True)
    o = torch.bmm(x.view(B, T * H, -1), rows[..., :D_C]) / total.view(B, T * H, 1)
    return o.view(-1, D_C).bfloat16(), (top + torch.log(total)).view(-1)


def _path(s):
    """[nodes, T] truth: node w of the same request lies on node t's path, itself included, roots left out."""
    c = s["case"]
    B, T = c["batch"], c["tree"]
    step = torch.zeros(B, T, T + 1, device="cuda")
    step.scatter_(2, torch.where(s["parent"] < 0, T, s["parent"]).long().view(B, T, 1), 1.0)
    up = step[:, :, :T] + torch.eye(T, device="cuda")
    reach = torch.matrix_power(up, max(1, T)) > 0
    return (reach & (s["parent"].view(B, 1, T) >= 0)).view(B * T, T)


def _logits_plain(s):
    c = s["case"]
    B, T, V = c["batch"], c["tree"], c["vocab"]
    at = torch.arange(c["hist"], device="cuda")[None, :]
    live, out = at < s["hist_len"][:, None], at >= s["prompt_len"][:, None]
    hist = s["hist"].long()
    prompt = torch.zeros(B, V, device="cuda").scatter_add_(1, hist, (live & ~out).float())
    made = torch.zeros(B, V, device="cuda").scatter_add_(1, hist, (live & out).float())
    drafted = torch.zeros(B * T, V, device="cuda").scatter_add_(
        1, s["token"].long().view(B, 1, T).expand(B, T, T).reshape(B * T, T), _path(s).float())
    made = (made[:, None, :] + drafted.view(B, T, V)).view(B * T, V)
    each = lambda v: v.repeat_interleave(T)[:, None]  # noqa: E731
    seen = (made > 0) | (prompt[:, None, :].expand(B, T, V).reshape(B * T, V) > 0)
    x = s["logits"].float()
    x = torch.where(seen, torch.where(x > 0, x / each(s["repeat"]), x * each(s["repeat"])), x)
    x = x - each(s["frequency"]) * made - each(s["presence"]) * (made > 0).float()
    per = s["bias_val"].numel() // B
    bias = torch.zeros(B, V, device="cuda").scatter_add_(1, s["bias_tok"].long().view(B, per), s["bias_val"].view(B, per))
    x = (x.view(B, T, V) + bias[:, None, :]).view(B * T, V)
    v = torch.arange(V, device="cuda")
    bits = (s["allow"][s["allow_row"].clamp(min=0).long()][:, v // 32] >> (v % 32)) & 1
    banned = (bits == 0) & (s["allow_row"] >= 0)[:, None]
    return x.masked_fill(banned, -math.inf).to(_dtype(c))


def run(state):
    if own:
        return state["call"]()
    return {"rope": _rope_plain, "write": _write_plain, "attn": _attn_plain, "logits": _logits_plain}[state["case"]["op"]](state)


# ---------------------------------------------------------- 64-bit definition
def exact(case, seed):
    s = prepare(case, seed)
    turn = lambda pos: torch.polar(torch.full((pos.numel(), s["inv_dev"].numel()), float(s["mscale"]), dtype=torch.float64, device="cuda"),  # noqa: E731
                                   pos.double()[:, None] * s["inv_dev"])
    if case["op"] in ("rope", "write"):
        x, rot = (s["x"].double(), case["rot"]) if case["op"] == "rope" else (s["k"].double()[:, None, :], D_R)
        y = x.clone()
        first, second = (slice(0, rot, 2), slice(1, rot, 2)) if case["layout"] == "interleaved" else (slice(0, rot // 2), slice(rot // 2, rot))
        z = torch.complex(x[..., first], x[..., second]) * turn(s["pos"])[:, None, :]
        y[..., first], y[..., second] = z.real, z.imag
        if case["op"] == "rope":
            return y
        c8, kr, scale = s["c8"].double(), s["kr"].double(), s["scale"].double()
        at = s["slot"].long()
        if case["block"] == 1:
            top = s["c"].double().abs().amax(1)
            e = torch.ceil(torch.log2(top / E4M3_MAX))
            e = e + (top > E4M3_MAX * torch.exp2(e)).double() - (top <= E4M3_MAX * torch.exp2(e - 1)).double()
            scale[at] = torch.exp2(e)
        by = scale[at // case["block"]][:, None]
        v = s["c"].double() / by
        grid = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)    # e4m3's step at each value
        c8[at] = (torch.round(v / grid) * grid).clamp(-E4M3_MAX, E4M3_MAX)
        kr[at] = y[:, 0] / by
        return c8, kr, scale
    if case["op"] == "attn":
        B, H, T, o, lse = case["batch"], case["heads"], case["tree"], [], []
        off = 0
        for b in range(B):
            L, n = s["lens"][b], s["ns"][b]
            slot = s["table"][off:off + n].long() if s["table"] is not None else torch.arange(off, off + n, device="cuda")
            off += n
            by = s["scale"].double()[slot // case["block"]]
            c, k = s["c8"].view(torch.float8_e4m3fn)[slot].double() * by[:, None], s["kr"][slot].double() * by[:, None]
            for t in range(T):                       # a node at a time: all heads share its keys
                m = int(s["mask"][b * T + t])
                keys = torch.tensor([L + u for u in range(T) if m >> u & 1], device="cuda", dtype=torch.long)
                q = s["q"][(b * T + t) * H:(b * T + t + 1) * H].double()
                take = lambda a: torch.cat([a[:L], a[keys]])  # noqa: E731
                x = (q[:, :D_C] @ take(c).T + q[:, D_C:] @ take(k).T) / math.sqrt(192)
                lse.append(torch.logsumexp(x, 1))
                o.append(torch.softmax(x, 1) @ take(c))
        return torch.cat(o), torch.cat(lse)
    B, T, V = case["batch"], case["tree"], case["vocab"]
    x = s["logits"].double()
    parent, token = s["parent"].tolist(), s["token"].tolist()
    allow_row = s["allow_row"].tolist()
    per = s["bias_val"].numel() // B
    for b in range(B):
        n, p = int(s["hist_len"][b]), int(s["prompt_len"][b])
        old = torch.bincount(s["hist"][b, :p].long(), minlength=V)
        new = torch.bincount(s["hist"][b, p:n].long(), minlength=V)
        bias = torch.zeros(V, dtype=torch.float64, device="cuda")
        bias[s["bias_tok"][b * per:(b + 1) * per].long()] = s["bias_val"][b * per:(b + 1) * per].double()
        for t in range(T):
            i, w, path = b * T + t, t, []
            while parent[b * T + w] >= 0:
                path.append(token[b * T + w])
                w = parent[b * T + w]
            made = new + torch.bincount(torch.tensor(path, dtype=torch.long, device="cuda"), minlength=V)
            r, row = s["repeat"][b].double(), x[i]
            row = torch.where(old + made > 0, torch.where(row > 0, row / r, row * r), row)
            row = row - s["frequency"][b].double() * made - s["presence"][b].double() * (made > 0) + bias
            if allow_row[i] >= 0:
                words = s["allow"][allow_row[i]].long() & 0xFFFFFFFF
                bits = (words[:, None] >> torch.arange(32, device="cuda")[None, :]) & 1
                row = torch.where(bits.reshape(-1)[:V] == 1, row, -math.inf)
            x[i] = row
    return x


# -------------------------------------------------------------- what it takes
def work(case):
    esz = 2 if case.get("dtype") == "bf16" else 4
    if case["op"] == "rope":
        n = case["tokens"] * case["heads"]
        return {"bytes": 2 * n * case["dim"] * esz + 4 * case["tokens"], "flops": 3 * n * case["rot"]}
    if case["op"] == "write":
        n = case["rows"]
        return {"bytes": n * (D_Q * esz + D_C + 2 * D_R + 4 + 4 + 4), "flops": n * (3 * D_C + 4 * D_R)}
    if case["op"] == "attn":
        # lengths between lo and hi: their mean for all but the first request
        keys = case["hi"] + (case["batch"] - 1) * (case["lo"] + case["hi"]) / 2
        T, rows = case["tree"], case["batch"] * case["tree"] * case["heads"]
        kv = (keys + case["batch"] * T) * (D_C + 2 * D_R + 4 / case["block"] + (4 if case["paged"] else 0))
        return {"bytes": kv + rows * (D_Q * 2 + D_C * 2 + 4), "flops": 2 * (D_Q + D_C) * case["heads"] * T * (keys + case["batch"])}
    rows, V = case["batch"] * case["tree"], case["vocab"]
    return {"bytes": rows * V * (2 * esz + 1 / 8) + 4 * case["batch"] * case["hist"], "flops": 4 * rows * V}
