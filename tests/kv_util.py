"""Ragged batches over a paged cache for the KV-cache tests: the host oracle's
cache and the same bytes on the device, and the error bound of the attention."""
import numpy as np
import torch

import oracle
from gpu_util import DEV, dev
from workloads import f32_to_bf16_bits

U_BF16 = 2.0 ** -8       # half a step of bf16, relative to the value


def bf16(a):
    """(values fp64 of a rounded to bf16, device tensor builder)"""
    bits = f32_to_bf16_bits(np.asarray(a, np.float32))
    return oracle.product.bf16_to_f64(bits), bits


def dev_bf16(bits):
    return dev(bits.view(np.int16)).view(torch.bfloat16)


def rows(rng, shape):
    x = rng.standard_normal(shape).astype(np.float32)
    x[..., :3] *= 4
    x[..., -1] += 2          # a channel with a mean
    return x


class Batch:
    """Sequences with lens[b] tokens (new[b] of them the rows of this call), shuffled pages, spare pages between."""

    def __init__(self, rng, lens, new, page_size, heads, head_dim, bits, starts=True, lead=0, spare=3, width=None,
                 prefix=0, fill=True):
        self.lens, self.new = np.array(lens, np.int32), np.array(new, np.int32)
        need = [-(-int(n) // page_size) for n in lens]
        pre = -(-prefix // page_size)
        self.n_pages = sum(need) + pre + spare
        order = rng.permutation(self.n_pages)
        self.pages = np.full((len(lens), width or max(1, max(need))), -1, np.int32)
        at = 0
        for b, n in enumerate(need):
            self.pages[b, :n] = order[at:at + n]
            at += n
        self.prefix, self.prefix_pages = prefix, order[at:at + pre].astype(np.int32)
        self.starts = np.concatenate([[lead], lead + np.cumsum(new)]).astype(np.int32) if starts else None
        self.T = int(lead + sum(new))
        self.geom = (self.n_pages, page_size, heads, head_dim, bits)
        self.ref = oracle.kvcache.Cache(*self.geom)
        if fill:                       # every slot of every page holds a row, the spare pages' too
            for i in range(2):
                x, _ = bf16(rows(rng, (self.n_pages, heads, page_size, head_dim)))
                q, s, o = oracle.kvcache.quantize_rows(x, bits)
                self.ref.codes[i][:] = oracle.kvcache.pack_codes(q, bits)
                self.ref.meta[i][:] = oracle.kvcache.pack_meta(s, o)

    def device(self, cg):
        bufs = []
        for i in range(2):
            bufs += [dev(self.ref.codes[i].reshape(-1)), dev(self.ref.meta[i].view(np.int32).reshape(-1))]
        self.cache = cg.make_qcache(*self.geom, *bufs)
        self.d_pages, self.d_lens = dev(self.pages), dev(self.lens)
        self.d_starts = None if self.starts is None else dev(self.starts)
        self.d_prefix = dev(self.prefix_pages) if self.prefix else None
        return self

    def host_buffers(self):
        torch.cuda.synchronize()
        k, km, v, vm = (t.cpu().numpy() for t in self.cache._tensors)
        shape = self.ref.meta[0].shape
        return ([x.reshape(self.ref.codes[0].shape) for x in (k, v)],
                [x.view(np.uint32).reshape(shape) for x in (km, vm)])


def logit_size(batch, Q, scale):
    """A = max scale * sum_i |q_i| |k_i| over a query row and any row of the cache (finite ones), per [T][Hq]."""
    kmax = np.nan_to_num(np.abs(batch.ref.values(0)), nan=0.0).max(axis=(0, 1, 2))
    return abs(scale) * (np.abs(Q) @ kmax)


def attend_bound(batch, Q, scale, mag):
    """What an fp32 output may be off by, element by element.

    Roundings: a key value to 11 bits (relative 2^-11 at most), a query is exact; so a logit is off by at most
    2^-11 A, A = scale sum |q||k|, and a few 2^-24 of sums of at most 128 products whose size the offset form
    s*q + o raises to at most 8 A: 128 * 2^-24 * 8 A = 2^-14 A.  A weight exp(z - m) / sum is then off by a
    factor of at most exp(2 d), d = (2^-11 + 2^-14) A.  A weight is rounded to 11 bits and a value to 11 bits:
    2^-11 each.  Sums over the keys in fp32: below 2^-14 for the lengths here (at most 2^10 terms of size mag
    per partial sum).  All of that relative to mag[0] = sum p |v|.

    A value may also be summed as its two parts, (p s) q and p o, which can cancel down to a v far smaller than
    either: a weight p s carried in two bf16 parts is off by 2^-8 * 2^-8 of itself at most, and the fp32 sums of
    the parts by 2^-14 of them, so (2^-16 + 2^-14) mag[1], mag[1] >= sum p (s q + |o|)."""
    d = (2.0 ** -11 + 2.0 ** -14) * logit_size(batch, Q, scale)
    assert d.max() < 0.25
    return (np.expm1(2 * d)[..., None] + 2.0 ** -10 + 2.0 ** -14) * (mag[0] * 1.01) + (2.0 ** -16 + 2.0 ** -14) * mag[1] + 1e-30


def check_attend(batch, Q, got32, ref, mag, owned, scale):
    err = np.abs(got32.astype(np.float64) - ref)[owned]
    bound = attend_bound(batch, Q, scale, mag)[owned]
    worst = float(np.max(err / np.maximum(bound, 1e-300))) if err.size else 0.0
    assert np.all(np.isfinite(got32[owned])), "not finite"
    assert worst <= 1.0, f"error {err.max():.3e}, {worst:.2f} of the bound"
    return worst


__all__ = ["Batch", "bf16", "dev_bf16", "rows", "check_attend", "attend_bound", "DEV", "U_BF16"]
