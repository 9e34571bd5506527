"""Cases of the paged-cache tests: seeded inputs on the CPU, the library's handles on the
GPU, and the error bounds of fp_tree_attention."""
from __future__ import annotations

import numpy as np
import torch

from block_sparse_long_blocks_b200 import binding as fb
from oracle import paged_cache as pc

E4M3_MAX = 448.0


def bits8(x):
    return x.view(torch.uint8) if x.dtype is torch.float8_e4m3fn else x


def quantise(x, scale):
    """float32 x / scale -> e4m3 by the definition (IEEE division, clamp, nearest even)."""
    return (x / scale).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


class Case:
    """A cache with `kv` cached tokens per request of which the last `n` are new.

    poison: every slot that belongs to no cached token (and its token scale) holds NaN."""

    def __init__(self, kv, n, hkv=2, G=4, d=128, page=16, fmt="bf16", seed=0, poison=True, extra_pages=2, spare_cols=1):
        g = torch.Generator().manual_seed(seed)
        self.rng = np.random.default_rng(seed)
        self.kv, self.n, self.hkv, self.G, self.hq, self.d, self.page, self.fmt = kv, n, hkv, G, hkv * G, d, page, fmt
        self.R, self.total = len(kv), sum(n)
        self.cu = torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32)
        need = [-(-x // page) for x in kv]
        pages = sum(need) + extra_pages
        order = self.rng.permutation(pages)
        self.table = torch.full((self.R, max(max(need), 1) + spare_cols), -7, dtype=torch.int32)
        at = 0
        for r in range(self.R):
            self.table[r, :need[r]] = torch.from_numpy(order[at:at + need[r]].astype(np.int32))
            at += need[r]
        self.kv_lens = torch.tensor(kv, dtype=torch.int32)
        # a shared direction in a few keys and in every query: scores as peaked as a model's
        u = torch.randn(d, generator=g)
        self.u = 4 * u / u.norm()
        x = {name: torch.randn(pages, page, hkv, d, generator=g) for name in "kv"}
        x["k"] += self.u * (torch.rand(pages, page, 1, 1, generator=g) < 0.03)
        x["v"] *= torch.exp2(torch.randint(-3, 3, (pages, page, 1, 1), generator=g).float())  # uneven token scales
        self.pool, self.scale = {}, {}
        for name, y in x.items():
            if fmt == "bf16":
                self.pool[name], self.scale[name] = y.bfloat16(), None
            elif fmt == "e4m3_head":
                self.scale[name] = y.abs().amax((0, 1, 3)) / E4M3_MAX
                self.pool[name] = quantise(y, self.scale[name][:, None])
            else:
                sc = y.abs().amax(-1) / E4M3_MAX
                self.scale[name] = sc.transpose(1, 2).contiguous()
                self.pool[name] = quantise(y, sc[..., None])
        if poison:
            free = torch.ones(pages * page, dtype=torch.bool)
            for r in range(self.R):
                free[self.flat(r, np.arange(kv[r]))] = False
            for name in "kv":
                self.fill(name, free.nonzero()[:, 0], float("nan"), scale=float("nan"))
        self.q = (torch.randn(self.total, self.hq, d, generator=g) + self.u).bfloat16()
        self.mask = None

    # ---- layout
    def flat(self, r, pos):
        pos = np.asarray(pos)
        return torch.from_numpy(self.table[r].numpy()[pos // self.page].astype(np.int64) * self.page + pos % self.page)

    def new_slots(self, r):
        return self.flat(r, np.arange(self.kv[r] - self.n[r], self.kv[r]))

    def fill(self, name, flat, value, scale=None):
        v = torch.tensor(value).to(self.pool[name].dtype)
        bits8(self.pool[name]).flatten(0, 1)[flat] = bits8(v)
        if scale is not None and self.fmt == "e4m3_token":
            s = self.scale[name]
            s[flat // self.page, :, flat % self.page] = scale

    def trees(self, empty_rows=False, self_bit=True):
        """Random trees (ancestors and self); with empty_rows, some rows see no new token."""
        self.see = np.zeros((self.total, max(self.n)), dtype=bool)
        for r in range(self.R):
            a = int(self.cu[r])
            for j in range(self.n[r]):
                if j:
                    parent = int(self.rng.integers(max(0, j - 4), j))
                    self.see[a + j] |= self.see[a + parent]
                if self_bit:
                    self.see[a + j, j] = True
                elif j:
                    self.see[a + j, parent] = True
            if empty_rows:
                self.see[a:a + self.n[r]][self.rng.random(self.n[r]) < 0.4] = False
        words = -(-max(self.n) // 32) + 1  # one word more than needed, and stray bits behind n_r
        bits = self.rng.integers(0, 2, (self.total, words * 32), dtype=np.uint8)
        for r in range(self.R):
            a, b = int(self.cu[r]), int(self.cu[r + 1])
            bits[a:b, :self.n[r]] = self.see[a:b, :self.n[r]]
        packed = np.packbits(bits.reshape(self.total, words, 32), axis=-1, bitorder="little").view(np.int32)
        self.mask = torch.from_numpy(packed.reshape(self.total, words).copy())
        return self

    # ---- reference
    def oracle(self):
        c = dict(fmt=self.fmt, table=self.table.numpy(), kv_lens=self.kv_lens.numpy())
        for name in "kv":
            c[name] = self.pool[name].double().numpy()
            c[name + "_scale"] = None if self.scale[name] is None else self.scale[name].double().numpy()
        return c

    # ---- GPU
    def cuda(self):
        up = lambda t: None if t is None else t.cuda()  # noqa: E731
        self.gpu = {k: up(v) for k, v in dict(k=self.pool["k"], v=self.pool["v"], ks=self.scale["k"],
                                              vs=self.scale["v"], table=self.table, kv_lens=self.kv_lens, cu=self.cu,
                                              q=self.q, mask=self.mask).items()}
        self.cache = fb.Cache(self.gpu["k"], self.gpu["v"], self.gpu["table"], self.gpu["kv_lens"], self.gpu["ks"],
                              self.gpu["vs"])
        return self

    def plan(self, **kw):
        return fb.Tree(self.cache, hq=self.hq, total_tokens=self.total, max_tokens=max(max(self.n), 1), **kw)

    def attend(self, plan=None, q=None):
        o = torch.full((self.total, self.hq, self.d), float("nan"), dtype=torch.bfloat16, device="cuda")
        lse = torch.full((self.hq, self.total), float("nan"), device="cuda")
        fb.fp_tree_attention(plan or self.plan(), self.gpu["cu"], self.gpu["q"] if q is None else q, o,
                             mask=self.gpu["mask"], lse=lse)
        return o, lse


def check_tree(case, o, lse, scale=None):
    """O and lse of the kernel against float64, within what its roundings can add up to.

    Per key, with A = scale * sum |q_i k_i| (natural-log units): the float32 dot product of d
    terms, the scalings and the subtraction of the maximum put the exponent off by at most
    (d + 8) 2^-23 A, the maximum's own error included by doubling; ex2.approx and its argument's
    rounding add 2^-21. So a weight is off by delta = 2 (d + 8) 2^-23 A + 2^-21 relative, before
    it is rounded for the product with V: f16 (2^-11) for e4m3 caches, two bf16 (2^-16) otherwise up
    to 16 rows, and below f16's normal range by 2^-38 of the largest v. Above 16 rows bf16 caches round
    the weights to bf16, p (1 + e) with |e| <= 2^-8, and divide by the sum of the rounded ones:
    O' - O = sum p e (v - O') / sum p, at most 2^-8 (W + |O'|) <= 2^-7 W. Sums over kv keys run in float32, in
    16-key products whose accumulation may truncate: (kv / 16 + 16) 2^-23. lse sees the weights'
    errors through their sum; O, a quotient, sees them twice, relative to W = sum p |v| / sum p;
    its own rounding to bf16 is 2^-8 |O|."""
    c = case.oracle()
    see = case.see if case.mask is not None else None
    O, L, W, A = pc.tree_attention(c, case.cu.numpy(), case.q.double().numpy(), see,
                                   scale or 1 / np.sqrt(case.d))
    o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    kv = max(case.kv)
    delta = 2 * (case.d + 8) * 2.0 ** -23 * A + 2.0 ** -21 + (kv / 16 + 16) * 2.0 ** -23
    wide = max(case.n) * case.G > 16
    p_round = 2.0 ** -11 if case.fmt != "bf16" else 2.0 ** -7 if wide else 2.0 ** -16
    vmax = np.nanmax(np.where(np.isfinite(W), W, 0)) if W.size else 0.0
    tol = 2.0 ** -8 * np.abs(O) + (2 * delta + p_round)[..., None] * W * 1.01 + kv * 2.0 ** -38 * vmax * 64
    finite = np.isfinite(O)
    assert np.array_equal(np.isnan(O), np.isnan(o)), "NaN in other places"
    assert np.array_equal(O[~finite & ~np.isnan(O)], o[~finite & ~np.isnan(O)])
    err = np.abs(o[finite] - O[finite])
    worst = (err / np.maximum(np.where(finite, tol, 1)[finite], 1e-300)).max() if err.size else 0.0
    assert worst <= 1.0, f"O off by {worst:.2f} of its bound (max abs {err.max():.3e})"
    fin = np.isfinite(L)
    assert np.array_equal(np.isneginf(L), np.isneginf(lse)) and np.array_equal(np.isnan(L), np.isnan(lse))
    lerr, ltol = np.abs(lse[fin] - L[fin]), (delta.T + 2.0 ** -22 * (np.abs(L) + 4))[fin]
    lworst = (lerr / ltol).max() if lerr.size else 0.0
    assert lworst <= 1.0, f"lse off by {lworst:.2f} of its bound (max abs {lerr.max():.3e})"
    return worst, lworst
