"""Plain 64-bit forms of rotary positions, the 8-bit latent cache and logits
processing, and the input makers that their tests share. Test infrastructure;
none of the library's arithmetic."""
import numpy as np
import torch

E4M3_MAX = 448.0


def rope(x, pos, inv_freq, rot, half, mscale=1.0, inverse=False):
    """x [n, heads, dim] -> float64, the first `rot` dims turned."""
    y = np.array(x, dtype=np.float64)
    a = np.asarray(pos, dtype=np.float64)[:, None] * np.asarray(inv_freq, dtype=np.float64)[None, :]
    if inverse:
        a = -a
    c, s = np.cos(a)[:, None, :], np.sin(a)[:, None, :]
    i, j = (slice(0, rot // 2), slice(rot // 2, rot)) if half else (slice(0, rot, 2), slice(1, rot, 2))
    u, v = y[..., i].copy(), y[..., j].copy()
    y[..., i], y[..., j] = mscale * (u * c - v * s), mscale * (u * s + v * c)
    return y


def row_scale(c):
    """Least power of two (>= 2^-100) that brings each row's largest finite magnitude to 448 or below."""
    out = []
    for row in np.asarray(c, dtype=np.float64):
        top = np.max(np.abs(row[np.isfinite(row)]), initial=0.0)
        e = -100
        while top > E4M3_MAX * 2.0 ** e:
            e += 1
        out.append(1.0 if top == 0 else 2.0 ** e)
    return np.array(out)


def codes(c, scale):
    """e4m3 codes (uint8) of c / scale: nearest even, saturating, NaN where c is not finite."""
    c = np.asarray(c, dtype=np.float32)
    v = np.nan_to_num(c / np.asarray(scale, dtype=np.float32)[:, None], nan=0.0, posinf=0.0, neginf=0.0)
    t = torch.from_numpy(np.clip(v, -E4M3_MAX, E4M3_MAX)).to(torch.float8_e4m3fn).view(torch.uint8).numpy().copy()
    t[~np.isfinite(c)] = 0x7F
    return t


def code_values(c8):
    return torch.from_numpy(np.ascontiguousarray(c8)).view(torch.float8_e4m3fn).to(torch.float64).numpy()


def random_tree(rng, T, reach=3):
    return [-1] + [int(rng.integers(max(0, i - reach), i)) for i in range(1, T)]


def tree_masks(parent):
    m = []
    for t, p in enumerate(parent):
        m.append((m[p] if p >= 0 else 0) | (1 << t))
    return m


class Attn:
    """A random problem over an 8-bit cache, and its 64-bit answer with error bounds."""

    def __init__(self, seed, prefix, trees, H, D_c=512, D_r=64, block=1, paged=True, spread=0.5, q_dtype="bf16",
                 masks=None, sharp=1.0):
        rng = np.random.default_rng(seed)
        self.H, self.D_c, self.D_r, self.block = H, D_c, D_r, block
        self.prefix, self.T = list(prefix), [len(t) for t in trees]
        self.B = len(prefix)
        self.n = [L + T for L, T in zip(self.prefix, self.T)]
        self.kv_off = np.concatenate([[0], np.cumsum(self.n)]).astype(np.int32)
        self.tree_off = np.concatenate([[0], np.cumsum(self.T)]).astype(np.int32)
        self.parent = np.concatenate([np.array(t) for t in trees]).astype(np.int32)
        self.masks = masks if masks is not None else [m for t in trees for m in tree_masks(t)]
        total = int(self.kv_off[-1])
        self.slots = total + (37 if paged else 0)
        self.table = rng.permutation(self.slots)[:total].astype(np.int32) if paged else None
        blocks = (self.slots + block - 1) // block
        # powers of two and other scales both occur
        self.scale = (np.exp2(rng.normal(-6, spread, blocks)) * np.where(rng.random(blocks) < 0.5, 1.0, 1.37)).astype(np.float32)
        self.c8 = codes(rng.standard_normal((self.slots, D_c)) * 60, np.ones(self.slots))
        self.kr = torch.from_numpy((rng.standard_normal((self.slots, D_r)) * 60).astype(np.float32)).bfloat16()
        rows = int(self.tree_off[-1]) * H
        q = rng.standard_normal((rows, D_c + D_r)) * sharp
        q[:, :D_c] *= 0.5
        self.q = torch.from_numpy(q.astype(np.float32))
        if q_dtype == "bf16":
            self.q = self.q.bfloat16()
        self.sm_scale = float(np.float32((D_c / 4 + D_r) ** -0.5))

    def node_keys(self, b, t):
        """Logical keys that node t of request b sees."""
        L = self.prefix[b]
        m = self.masks[int(self.tree_off[b]) + t]
        return np.array(list(range(L)) + [L + u for u in range(self.T[b]) if m >> u & 1], dtype=np.int64)

    def answer(self, p_step=2.0 ** -9, part_step=2.0 ** -11, drop=None):
        """(o, lse, bound of |o error|, bound of |lse error|), 64 bits. Bounds count the
        fp32 rounding of a logit, the rounding of each numerator before P.V (p_step,
        relative), and of the stored split partials (part_step). drop: slots left out.

        A logit's products are summed in fp32 chains. A chain of m additions rounds m
        times, each by at most 2^-24 of a partial sum that the products' magnitudes bound:
        m 2^-24 of their sum. The CUDA-core kernel has chains of 576 / 8 = 72, joined in 3
        more; with the factors' own roundings 80 2^-24 covers it (a first version of this
        bound, 2^-20 = 16 2^-24, was short of that: a logit of 576 products of one sign went
        past it). The exponent's argument rounds at 2^-24 of its terms, twice."""
        rows = int(self.tree_off[-1]) * self.H
        o, lse = np.zeros((rows, self.D_c)), np.full(rows, -np.inf)
        ob, lb = np.zeros((rows, self.D_c)), np.zeros(rows)
        vals = np.concatenate([code_values(self.c8), self.kr.to(torch.float64).numpy()], 1)
        vals = vals * np.repeat(self.scale.astype(np.float64), self.block)[:self.slots, None]
        q = self.q.to(torch.float64).numpy()
        for b in range(self.B):
            for t in range(self.T[b]):
                keys = self.kv_off[b] + self.node_keys(b, t)
                slot = self.table[keys] if self.table is not None else keys
                if drop is not None:
                    slot = slot[~np.isin(slot, drop)]
                r = slice((int(self.tree_off[b]) + t) * self.H, (int(self.tree_off[b]) + t + 1) * self.H)
                if len(slot) == 0:
                    continue
                k = vals[slot]
                x = self.sm_scale * (q[r] @ k.T)
                size = self.sm_scale * (np.abs(q[r]) @ np.abs(k).T)
                top = x.max(1, keepdims=True)
                e = np.exp(x - top)
                l = e.sum(1, keepdims=True)
                w = e / l
                o[r] = w @ k[:, :self.D_c]
                lse[r] = (top + np.log(l))[:, 0]
                eps = 80 * 2.0 ** -24 * size + 2.0 ** -22 * np.abs(x) + 2.0 ** -20
                ob[r] = (w * (p_step + part_step + 2 * eps)) @ np.abs(k[:, :self.D_c])
                lb[r] = (w * eps).sum(1) + 2.0 ** -22 * np.abs(lse[r]) + 2.0 ** -20
        return o, lse, ob, lb


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def penalised(x, hist, prompt_len, path, rep, pres, freq, bias, bits):
    """One node's processed logits in 64 bits, and the magnitude its fp32 arithmetic rounds at."""
    V = x.shape[0]
    x = x.astype(np.float64)
    old = np.bincount(hist[:prompt_len], minlength=V)
    made = np.bincount(np.concatenate([hist[prompt_len:], np.array(path, dtype=np.int64)]).astype(np.int64), minlength=V)
    seen = (old + made) > 0
    with np.errstate(invalid="ignore"):
        y = np.where(seen, np.where(x > 0, x / rep, x * rep), x)
    size = np.abs(y) + np.abs(freq) * made + np.abs(pres) * (made > 0) + np.abs(bias)
    y = y - freq * made - pres * (made > 0) + bias
    return (y if bits is None else np.where(bits, y, -np.inf)), size
