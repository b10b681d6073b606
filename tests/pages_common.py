"""Inputs and the 64-bit definition for the tests of the paged cache: the reference works on
numpy copies of the same bytes, token by token, and shares nothing with the kernels."""
import math

import numpy as np
import torch

H, D = 16, 512


def e4m3_table():
    return torch.arange(256, dtype=torch.int16).to(torch.uint8).view(torch.float8_e4m3fn).double().numpy()


E4M3 = e4m3_table()


class Cache:
    """CPU copy of a paged cache with random pages: pool uint8, scales, table, n_tokens."""

    def __init__(self, seed, lens, page=64, pos0=0, spare=2, max_pages=None, n_pages=None, latent=1.0):
        rng = np.random.default_rng(seed)
        self.page, self.pos0, self.B = page, pos0, len(lens)
        need = [-(-n // page) for n in lens]
        width = max(1, max(need)) if max_pages is None else max_pages
        total = max(1, sum(need)) + spare if n_pages is None else n_pages
        order = rng.permutation(total)
        self.table = np.full((self.B, width), -1, np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        x = rng.standard_normal((total * page, D)).astype(np.float32) * latent
        sc = np.abs(x).max(1) / 448
        codes = torch.from_numpy(x / np.maximum(sc, 1e-30)[:, None]).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
        self.kv = codes.reshape(total, page, D).copy()
        self.kv_sc = sc.reshape(total, page).astype(np.float32)
        self.n_tokens = np.array(lens, np.int32)

    def row(self, b, pos):
        """(page, slot) of a token position, or None where the table names no page."""
        t = pos - self.pos0
        if t < 0 or t >= self.table.shape[1] * self.page:
            return None
        p = self.table[b, t // self.page]
        return (p, t % self.page) if 0 <= p < self.kv.shape[0] else None

    def poison_dead(self, seen):
        """NaN bytes and scales in every slot that is not in `seen` (a set of (page, slot))."""
        live = np.zeros(self.kv.shape[:2], bool)
        for p, s in seen:
            live[p, s] = True
        self.kv[~live] = 0x7F
        self.kv_sc[~live] = np.nan

    def gpu(self):
        import sparse_attention_fp4_quant_b200 as csa
        t = [torch.from_numpy(a.copy()).cuda() for a in (self.kv, self.kv_sc, self.table, self.n_tokens)]
        return csa.Pages.of(*t, pos0=self.pos0)


def visible(cache, b, i, window=None, sink=0, start=None):
    """Token positions that the query at token i of sequence b sees, in order."""
    if i < 0:
        return []
    end = min(i + 1, cache.pos0 + int(np.clip(cache.n_tokens[b], 0, cache.table.shape[1] * cache.page)))
    low = -1 if window is None else i - window + 1
    if start is not None:
        low = max(low, start)
    return [j for j in range(cache.pos0, end) if (j >= low or j < sink) and cache.row(b, j) is not None]


def attend(q, parts, scale):
    """q [16, 512] float64; parts: [(cache, b, positions)].  -> out, lse, and each output's error bound.

    The bound counts, in relative terms of the value it stands on: the output's bf16 rounding 2^-8;
    each probability's rounding 2^-9 (three E5M2 terms, or one f16); and the logits: the query held
    to 2^-18 of the head's largest value, products summed in fp32 with at most 2^-18 of the sum of
    their magnitudes, an error dz that changes a weight by at most 2 dz; the exponential 2^-20.

    One absolute term beside them: a weight enters the product times its token's scale, with the row's
    largest such value at 2^12 or above, and E5M2's step is never finer than 2^-16, so the last term's
    rounding (half a step) is up to 2^-17 / 2^12 = 2^-29 of the largest, times the key's E4M3 code."""
    keys = [cache.kv[cache.row(b, j)] for cache, b, pos in parts for j in pos]
    if not keys:
        return np.zeros((H, D)), np.full(H, -np.inf), np.zeros((H, D)), np.zeros(H)
    sc = np.array([cache.kv_sc[cache.row(b, j)] for cache, b, pos in parts for j in pos], np.float64)
    codes = E4M3[np.array(keys)]
    k = codes * sc[:, None]
    z = q @ k.T * scale
    m = z.max(1, keepdims=True)
    p = np.exp(z - m)
    total = p.sum(1, keepdims=True)
    w = p / total
    out, lse = w @ k, (m + np.log(total))[:, 0]
    dz = scale * 2.0 ** -18 * (np.abs(q).max(1)[:, None] * np.abs(k).sum(1) + np.abs(q) @ np.abs(k).T)
    mean_dz = (w * dz).sum(1)
    tol = 2.0 ** -8 * np.abs(out) + (w * (2.0 ** -9 + 2.0 ** -20 + 2 * dz)) @ np.abs(k) + (2 * mean_dz)[:, None] * np.abs(out)
    tol = tol + 2.0 ** -29 * (w * sc).max(1)[:, None] * np.abs(codes).sum(0)
    return out, lse, tol + 1e-30, mean_dz + dz.max(1) * 2.0 ** -8 + 2.0 ** -20 * (1 + np.abs(lse))


def reference(q, q_pos, caches, window=None, sink=0, start=None, scale=1 / math.sqrt(D)):
    """caches: [(cache, per_row)]: a shared cache has per_row False (its row 0 for every sequence)."""
    B, Q = q_pos.shape
    got = [np.zeros((B, Q, H, D)), np.full((B, Q, H), -np.inf), np.zeros((B, Q, H, D)), np.zeros((B, Q, H))]
    qd = q.detach().cpu().double().numpy()
    for b in range(B):
        for c in range(Q):
            i = int(q_pos[b, c])
            parts = [(cache, b if per_row else 0,
                      visible(cache, b if per_row else 0, i, window, sink, None if start is None else int(start[b])))
                     for cache, per_row in caches]
            for a, v in zip(got, attend(qd[b, c], parts, scale)):
                a[b, c] = v
    return got


def check(out, lse, ref):
    o, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
    ro, rl, to, tl = ref
    assert np.isfinite(o).all()
    worst = (np.abs(o - ro) / np.maximum(to, 1e-30)).max() if o.size else 0.0
    assert worst <= 1.0, f"output off by {worst:.3g} of its bound"
    dead = np.isneginf(rl)
    assert np.array_equal(dead, np.isneginf(l))
    assert not o[dead].any()
    off = (np.abs(l[~dead] - rl[~dead]) / tl[~dead]).max() if (~dead).any() else 0.0
    assert off <= 1.0, f"lse off by {off:.3g} of its bound"


def queries(seed, B, Q, factor=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((B, Q, H, D), generator=g) * factor).to(torch.bfloat16)
