"""Quantized, paged KV cache.  TEST INFRASTRUCTURE.

Rows (one token of one KV head) by the round-to-nearest of rtn.py with the
whole row as its group, at 4 or 8 bits, the layout of include/qcache.h, and
attention over ragged sequences; everything in fp64.
"""
from __future__ import annotations

import numpy as np

from .rtn import fp16_round_down, fp16_round_up

VMAX = 65280.0


def quantize_rows(X: np.ndarray, bits: int):
    """(q uint8 [..., D], s, o float16 [...]); a row with a non-finite value gets s = o = NaN, q = 0."""
    L = (1 << bits) - 1
    X = np.asarray(X, dtype=np.float64)
    bad = ~np.isfinite(X).all(-1)
    x = np.where(bad[..., None], 0.0, np.clip(X, -VMAX, VMAX))
    o = fp16_round_down(x.min(-1))
    o64 = o.astype(np.float64)
    s = fp16_round_up((x.max(-1) - o64) / L)
    s64 = s.astype(np.float64)[..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.rint((x - o64[..., None]) / s64)
    q = np.clip(np.where(s64 == 0, 0, q), 0, L).astype(np.uint8)
    q = np.where(bad[..., None], 0, q).astype(np.uint8)
    nan = np.float16(np.nan)
    return q, np.where(bad, nan, s).astype(np.float16), np.where(bad, nan, o).astype(np.float16)


def row_values(q, s, o):
    return q.astype(np.float64) * s.astype(np.float64)[..., None] + o.astype(np.float64)[..., None]


def pack_codes(q: np.ndarray, bits: int) -> np.ndarray:
    return q if bits == 8 else (q[..., 0::2] | (q[..., 1::2] << 4)).astype(np.uint8)


def unpack_codes(c: np.ndarray, bits: int) -> np.ndarray:
    return c if bits == 8 else np.stack([c & 15, c >> 4], -1).reshape(c.shape[:-1] + (-1,))


def pack_meta(s, o) -> np.ndarray:
    return s.view(np.uint16).astype(np.uint32) | (o.view(np.uint16).astype(np.uint32) << 16)


def unpack_meta(m: np.ndarray):
    return (m & 0xFFFF).astype(np.uint16).view(np.float16), (m >> 16).astype(np.uint16).view(np.float16)


class Cache:
    """The same buffers as the library's, on the host: codes [page][head][slot][.] and meta [page][head][slot]."""

    def __init__(self, n_pages, page_size, heads, head_dim, bits):
        self.n_pages, self.page_size, self.heads, self.D, self.bits = n_pages, page_size, heads, head_dim, bits
        shape = (n_pages, heads, page_size)
        self.codes = [np.zeros(shape + (head_dim * bits // 8,), np.uint8) for _ in range(2)]
        self.meta = [np.zeros(shape, np.uint32) for _ in range(2)]

    def place(self, pages, lens, b, pos):
        """(page, slot) of position pos of sequence b, or None."""
        if pos < 0 or pos // self.page_size >= pages.shape[1]:
            return None
        page = int(pages[b, pos // self.page_size])
        return (page, pos % self.page_size) if 0 <= page < self.n_pages else None

    @staticmethod
    def rows(lens, starts):
        """(row, sequence, position) of every owned row."""
        for b in range(len(lens)):
            s0, s1 = (b, b + 1) if starts is None else (int(starts[b]), int(starts[b + 1]))
            for t in range(s0, s1):
                yield t, b, int(lens[b]) - (s1 - t)

    def write(self, K, V, pages, lens, starts=None):
        for x, c, m in zip((K, V), self.codes, self.meta):
            q, s, o = quantize_rows(x, self.bits)
            q, w = pack_codes(q, self.bits), pack_meta(s, o)
            for t, b, pos in self.rows(lens, starts):
                at = self.place(pages, lens, b, pos)
                if at:
                    c[at[0], :, at[1]] = q[t]
                    m[at[0], :, at[1]] = w[t]

    def values(self, which):
        """Every row of the cache, fp64 [page][head][slot][D]."""
        return row_values(unpack_codes(self.codes[which], self.bits), *unpack_meta(self.meta[which]))

    def read(self, T, pages, lens, starts=None):
        """[K, V] fp64 [T][heads][D]; unowned rows None-like (NaN mask returned as third)."""
        out = [np.zeros((T, self.heads, self.D)) for _ in range(2)]
        owned = np.zeros(T, bool)
        vals = [self.values(0), self.values(1)]
        for t, b, pos in self.rows(lens, starts):
            owned[t] = True
            at = self.place(pages, lens, b, pos)
            if at:
                for i in range(2):
                    out[i][t] = vals[i][at[0], :, at[1]]
        return out[0], out[1], owned

    def attend(self, Q, pages, lens, starts=None, scale=None, prefix_pages=None, prefix_len=0):
        """(out fp64 [T][Hq][D], M [2][T][Hq][D], owned): M[0] = sum_j p_j |v_jd| is what relative roundings of p and v
        act on, M[1] = sum_j p_j (s_j q_jd + |o_j|) what roundings of the two parts of v = s q + o do."""
        T, Hq, D = Q.shape
        G = Hq // self.heads
        scale = D ** -0.5 if scale is None else scale
        kv, vv = self.values(0), self.values(1)
        out, mag, owned = np.zeros((T, Hq, D)), np.zeros((2, T, Hq, D)), np.zeros(T, bool)
        vo = np.abs(unpack_meta(self.meta[1])[1].astype(np.float64))

        def slots(table, n):
            return [a for a in (self.place(table[None], None, 0, j) for j in range(n)) if a]

        pre = slots(np.asarray(prefix_pages), prefix_len) if prefix_len else []
        for t, b, pos in self.rows(lens, starts):
            owned[t] = True
            cap = pages.shape[1] * self.page_size
            at = pre + slots(pages[b], max(0, min(pos + 1, cap)))
            if not at:
                continue
            p_, s_ = np.array([a[0] for a in at]), np.array([a[1] for a in at])
            for h in range(self.heads):
                k, v = kv[p_, h, s_], vv[p_, h, s_]
                z = scale * (Q[t, h * G:(h + 1) * G].astype(np.float64) @ k.T)
                w = np.exp(z - z.max(1, keepdims=True))
                w /= w.sum(1, keepdims=True)
                out[t, h * G:(h + 1) * G] = w @ v
                o = vo[p_, h, s_][:, None]
                mag[0, t, h * G:(h + 1) * G] = w @ np.abs(v)
                mag[1, t, h * G:(h + 1) * G] = w @ (np.abs(v) + 2 * o)      # s q <= |v| + |o|
        return out, mag, owned
