"""Plain fp64 forms of the steps between projections and cache, for the GPU
tests, with the bounds their tolerances come from.  A rounding to bf16 is off
by at most 2^-8 of the value (half a step of 8 significant bits), one to fp32
by 2^-24; a product of two bf16 values is exact in fp32."""
import math

import torch

DEV = torch.device("cuda:0") if torch.cuda.is_available() else None
BF16_U = 2.0 ** -8


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def randn(shape, seed, dtype=torch.bfloat16, scale=1.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(dtype)


def segments(starts, T, B):
    """(sequence, first row, behind its last row) of sequences that own rows; starts is a list or None."""
    if starts is None:
        return [(b, b, b + 1) for b in range(B)]
    return [(b, starts[b], min(starts[b + 1], T)) for b in range(B) if min(starts[b + 1], T) > starts[b]]


# ------------------------------------------------------------------ adapters
def adapt_ref(A, B, scales, ranks, x, y, ids, starts):
    """(out, bound on |error| of an fp32 result), fp64.

    A sum over K of exact products in fp32: the products of 32 inputs are added to an accumulator at a time, so no value
    passes more than K / 32 + 32 additions there, 3 over the waves and 32 over the splits, each off by 2^-23 of the sum
    of magnitudes at most.  h in hi + lo: each rounding to bf16 leaves 2^-8 of what it rounds, so 2^-16 of h.  Then 2 r
    products, not exact here (h's parts times B are: 16 bits), and two roundings."""
    n, r, K = A.shape
    out, tol = y.double().clone(), y.double().abs() * 2.0 ** -23
    for b, s, e in segments(starts, x.shape[0], len(ids)):
        a = ids[b]
        if not 0 <= a < n:
            continue
        k = r if ranks is None else max(0, min(r, ranks[a]))
        Aa, Ba, xs = A[a, :k].double(), B[a, :, :k].double(), x[s:e].double()
        sc = scales[a].double()
        out[s:e] += (xs @ Aa.T) @ Ba.T * sc
        big = (xs.abs() @ Aa.abs().T) @ Ba.abs().T * sc.abs()
        tol[s:e] += big * ((K / 32 + 67) * 2.0 ** -23 + 2.0 ** -16 + (2 * r + 8) * 2.0 ** -23)
    return out, tol


# ------------------------------------------------------------ norm, rotation
def norm_rope_ref(x, w, eps, freqs, pairs, pos):
    """(out, bound on |error| of an fp32 result), fp64.  x [T][heads][D], pos [T] (fp64).

    The norm: 16 squares and 3 sums a lane, so 20 roundings of 2^-24 at most, half of them after the root, a root's and
    three products' own: below 2^-19 of a value.  The angle has three roundings of 2^-53 here
    and one there, 2^-20 radians for positions of 32 bits; its part of a turn is rounded to fp32 (2^-25 of a turn, 2^-22
    radians), sine and cosine to 2^-22: below 2^-18.6 of either value of a pair with the norm's, and two roundings."""
    x = x.double()
    n = x if w is None else x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps) * w.double()
    out, size = n.clone(), n.abs()
    half = 0 if freqs is None else freqs.numel()
    if half:
        i = torch.arange(half, device=x.device)
        ia, ib = (2 * i, 2 * i + 1) if pairs else (i, i + half)
        ang = pos.double()[:, None] * freqs
        c, s = torch.cos(ang)[:, None], torch.sin(ang)[:, None]
        a, b = n[..., ia], n[..., ib]
        out[..., ia], out[..., ib] = a * c - b * s, b * c + a * s
        size[..., ia] = size[..., ib] = a.abs() + b.abs()
    return out, size * 2.0 ** -18


# ------------------------------------------------------------------- prompts
def prompt_ref(Q, K, V, starts, scale):
    """(out, bound on |error| of an fp32 result), fp64; rows nobody owns are NaN in both.

    A logit: D exact products, at most D / 16 + 16 additions off by 2^-23 of the magnitudes' sum, one more product, the
    exponential (2^-22): the relative error of a weight is that of the logit (times ln 2 in the log2 domain, so below).
    Rounded to bf16: 2^-8.  The sums over keys: n / 16 + 32 additions of 2^-23 each, in the numerator and below."""
    T, Hq, D = Q.shape
    H = K.shape[1]
    out = torch.full((T, Hq, D), math.nan, dtype=torch.float64, device=Q.device)
    tol = out.clone()
    seqs = [(0, 0, T)] if starts is None else segments(starts, T, len(starts) - 1)
    for _, s, e in seqs:
        n = e - s
        later = torch.ones((n, n), dtype=torch.bool, device=Q.device).triu(1)
        for h in range(Hq):
            q, k, v = Q[s:e, h].double(), K[s:e, h // (Hq // H)].double(), V[s:e, h // (Hq // H)].double()
            z = (q @ k.T * scale).masked_fill(later, -math.inf)
            w = torch.softmax(z, -1)
            off = (q.abs() @ k.abs().T * abs(scale)).masked_fill(later, 0).amax(-1, keepdim=True)
            err = off * (D / 16 + 18) * 2.0 ** -23 * 2 + 2.0 ** -8 + (n / 16 + 32) * 2.0 ** -22 + 2.0 ** -20
            out[s:e, h] = w @ v
            tol[s:e, h] = (w @ v.abs()) * err
    return out, tol


def check(got, want, tol, what=""):
    """|got - want| <= tol, and half a step of bf16 more where the output is bf16."""
    g = got.double()
    if got.dtype == torch.bfloat16:
        tol = tol * (1 + BF16_U) + want.abs() * BF16_U + 2.0 ** -134
    bad = ~((g - want).abs() <= tol + 1e-37)
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[0].tolist(), float(g[bad][0]), float(want[bad][0]), float(tol[bad][0]))
