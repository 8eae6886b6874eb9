"""The 4-bit block cache in plain 64-bit arithmetic on the CPU, token by token from its definition
(include/spec_verify.h), for the tests of spec_cache_*."""
import numpy as np
import torch

MAG = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=np.float64)


def e4m3_table():
    """Value of each of the 256 bytes (NaN for 0x7f, 0xff)."""
    b = np.arange(256)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e == 0, m * 2.0 ** -9, (1 + m / 8.0) * 2.0 ** (e - 7.0))
    v = np.where((b & 127) == 127, np.nan, v)
    return np.where(b >= 128, -v, v)


E4M3 = e4m3_table()


def nearest_even(x, grid):
    """Index of the value of the ascending `grid` nearest to each x, ties to the even index."""
    hi = np.clip(np.searchsorted(grid, x), 1, len(grid) - 1)
    lo = hi - 1
    dl, dh = x - grid[lo], grid[hi] - x
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    return np.where(up, hi, lo)


def quantise(x, g):
    """x [..., d] (any float dtype), g a float32 scalar -> (codes uint8 [..., d], scale bytes
    [..., d/16])."""
    x = np.asarray(x, dtype=np.float32)
    rg = np.float32(1.0) / np.float32(g)
    with np.errstate(all="ignore"):
        y = (x * rg).astype(np.float32).reshape(x.shape[:-1] + (x.shape[-1] // 16, 16))
        bad = ~np.isfinite(y).all(-1)
        top = np.where(bad, 0, np.abs(y).max(-1)).astype(np.float32)
        q = np.minimum((top / np.float32(6.0)).astype(np.float32).astype(np.float64), 448.0)
        sb = np.maximum(nearest_even(q, E4M3[:127]), 1).astype(np.uint8)
        s = E4M3[sb]
        z = np.where(bad[..., None], 0, y).astype(np.float64)
        r = np.minimum(np.abs(z) / s[..., None], 6.0)  # exact ties survive: s has four bits
        c = nearest_even(r, MAG).astype(np.uint8) | (np.signbit(z).astype(np.uint8) << 3)
    c[bad] = 0
    sb[bad] = 0x7f
    return c.reshape(x.shape), sb


class Pool:
    """Pages [num, heads, page/16, 18 d] as the library lays them out, on the CPU."""

    def __init__(self, raw, page):
        self.raw, self.page = raw, page  # uint8 numpy
        self.d = raw.shape[-1] // 18
        self.heads = raw.shape[1]

    def where(self, table_row, pos):
        p = int(table_row[pos // self.page])
        if p < 0 or p >= self.raw.shape[0]:
            return None
        return self.raw[p, :, (pos % self.page) // 16], pos % 16

    def put(self, table_row, pos, kc, ks, vc, vs):
        """One token: codes [heads, d], scales [heads, d/16]."""
        at = self.where(table_row, pos)
        if at is None:
            return
        run, t = at
        d = self.d
        for h in range(self.heads):
            r = run[h]
            k = r[:8 * d].reshape(d // 32, 16, 16)
            k[:, t] = (kc[h, 0::2] | (kc[h, 1::2] << 4)).reshape(d // 32, 16)
            r[8 * d:9 * d].reshape(16, d // 16)[t] = ks[h]
            v = r[9 * d:17 * d].reshape(d, 8)
            sh = 4 * (t % 2)
            v[:, t // 2] = (v[:, t // 2] & (0xF0 >> sh)) | (vc[h] << sh)
            r[17 * d:].reshape(d // 16, 16)[:, t] = vs[h]

    def get(self, table_row, pos):
        """(k, v) [heads, d] in fp64 without the heads' scales, or None."""
        at = self.where(table_row, pos)
        if at is None:
            return None
        run, t = at
        d = self.d
        k, v = np.empty((self.heads, d)), np.empty((self.heads, d))
        for h in range(self.heads):
            r = run[h]
            b = r[:8 * d].reshape(d // 32, 16, 16)[:, t].reshape(d // 2)
            c = np.stack([b & 15, b >> 4], -1).reshape(d)
            val = np.where(c & 8, -MAG[c & 7], MAG[c & 7])
            k[h] = val * np.repeat(E4M3[r[8 * d:9 * d].reshape(16, d // 16)[t]], 16)
            c = (r[9 * d:17 * d].reshape(d, 8)[:, t // 2] >> (4 * (t % 2))) & 15
            val = np.where(c & 8, -MAG[c & 7], MAG[c & 7])
            v[h] = val * np.repeat(E4M3[r[17 * d:].reshape(d // 16, 16)[:, t]], 16)
        return k, v


def to_np(t):
    return t.detach().cpu().double().numpy()


def write(raw, page, table, cache_len, k, v, block_len=None, k_scale=None, v_scale=None):
    """The pool's bytes after a spec_cache_write (a copy)."""
    pool = Pool(raw.copy(), page)
    B, T, H = k.shape[:3]
    kf, vf = k.detach().float().cpu().numpy(), v.detach().float().cpu().numpy()
    for i in range(B):
        L = T if block_len is None else min(max(int(block_len[i]), 0), T)
        n = int(cache_len[i])
        if n < 0 or n + L > table.shape[1] * page:
            continue
        for j in range(L):
            rows = []
            for x, g in ((kf, k_scale), (vf, v_scale)):
                per = [quantise(x[i, j, h], 1.0 if g is None else g[h]) for h in range(H)]
                rows += [np.stack([a for a, _ in per]), np.stack([b for _, b in per])]
            pool.put(table[i], n + j, *rows)
    return pool.raw


def attend(raw, page, table, cache_len, q, block_len=None, scale=1.0, causal=True, window=0, k_scale=None,
           v_scale=None):
    """(out, lse, a, s) in fp64: a = sum_t p_t |v_t|, s = the largest scale * sum_c |q_c k_c| of a row's
    visible tokens (what rounding errors are measured against).  Rows that are not computed are None
    in `done`."""
    pool = Pool(raw, page)
    B, T, HQ, d = q.shape
    H = pool.heads
    G = HQ // H
    qd = to_np(q)
    out, a = np.zeros((B, T, HQ, d)), np.zeros((B, T, HQ, d))
    lse, size = np.full((B, T, HQ), -np.inf), np.zeros((B, T, HQ))
    done = np.zeros((B, T), dtype=bool)
    with np.errstate(all="ignore"):
        for i in range(B):
            L = T if block_len is None else min(max(int(block_len[i]), 0), T)
            n = int(cache_len[i])
            if n < 0 or n + L > table.shape[1] * page:
                continue
            tokens = {}
            for j in range(L):
                done[i, j] = True
                end = n + j + 1 if causal else n + L
                first = max(0, n + j + 1 - window) if window else 0
                see = []
                for t in range(first, end):
                    if t not in tokens:
                        tokens[t] = pool.get(table[i], t)
                    if tokens[t] is not None:
                        see.append(tokens[t])
                if not see:
                    continue
                k = np.stack([x for x, _ in see])  # [t, H, d]
                v = np.stack([x for _, x in see])
                for h in range(HQ):
                    g = h // G
                    kg = 1.0 if k_scale is None else float(np.float32(k_scale[g]))
                    vg = 1.0 if v_scale is None else float(np.float32(v_scale[g]))
                    x = (k[:, g] @ qd[i, j, h]) * kg * scale
                    size[i, j, h] = np.max(np.abs(k[:, g]) @ np.abs(qd[i, j, h])) * abs(kg * scale)
                    m = np.max(x)
                    p = np.exp(x - m)
                    z = p.sum()
                    p /= z
                    out[i, j, h] = (p[:, None] * v[:, g]).sum(0) * vg
                    a[i, j, h] = (p[:, None] * np.abs(v[:, g])).sum(0) * vg
                    lse[i, j, h] = m + np.log(z)
    return out, lse, a, size, done


def attend_bounds(out, lse, a, size, tokens, d, dtype):
    """How far spec_cache_attend may be from the fp64 values.

    Scores: products are exact in fp32 and their d-term sum rounds at most once a term, each time by
    2^-23 (a truncating adder) of the terms' magnitudes; the product with the row's factor (itself the
    product of three rounded numbers) and the difference to the maximum add four roundings of the score:
    es = (d + 8) 2^-23 size absolute, so a relative error of p of es, and as much of its sum's.  ex2 is
    good to 2^-22.  Each p is rounded to fp16 (2^-11; below 2^-14 by 2^-25 absolute where the row's
    maximum is at least 2^1), sums of `tokens` terms round by 2^-23 a term, and the result once to its
    type."""
    es = (d + 8) * 2.0 ** -23 * size
    rel = 2 * es + 2.0 ** -11 + tokens * 2.0 ** -22 + 2.0 ** -20
    half = torch.finfo(dtype).eps / 2
    flush = tokens * 2.0 ** -26 * np.max(np.nan_to_num(a), axis=-1, keepdims=True)
    tol = a * rel[..., None] + flush + np.abs(out) * half + float(torch.finfo(dtype).smallest_normal)
    tol_lse = es + tokens * 2.0 ** -23 + 2.0 ** -21 + np.abs(np.where(np.isfinite(lse), lse, 0)) * 2.0 ** -22
    return tol, tol_lse
