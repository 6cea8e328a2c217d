"""Attention over the KV cache where logits are far from zero, and where one
weight is large and many are small (include/qcache.h)."""
import math

import pytest
import torch

from layer_util import DEV, check, i32, randn

pytestmark = pytest.mark.gpu


def far_cache(gpu, lens, H, D, bits, top, scale, page=32):
    """A cache whose keys differ in coordinate 3 only (a few steps of 2^-6 apart), its page table, and the keys and
    values it holds, per sequence.  Returns the power of two of queries that brings logits to 2^top, too."""
    n = sum(lens)
    g = torch.Generator(device=DEV)
    g.manual_seed(top + bits)
    K = torch.zeros((n, H, D), device=DEV)
    K[..., 3] = (1 + torch.randint(0, 64, (n, H), generator=g, device=DEV) / 64.0) * 2.0 ** 10
    K[..., 3] *= torch.randint(0, 2, (n, H), generator=g, device=DEV) * 2 - 1
    V = randn((n, H, D), top, torch.float32)
    width = -(-max(lens) // page)
    pages = i32([[b * width + p for p in range(width)] for b in range(len(lens))])
    cache = gpu.make_qcache(len(lens) * width, page, H, D, bits)
    starts = [0]
    for m in lens:
        starts.append(starts[-1] + m)
    gpu.qcache_write(cache, K, V, pages, i32(lens), i32(starts))
    kc, vc = gpu.qcache_read(cache, pages, i32(lens), i32(starts), rows=n, dtype=torch.float32)
    return cache, pages, starts, kc, vc, top - 10 - round(math.log2(abs(scale)))


def winners(q, k, v, scale, sees):
    """The mean of the values of the largest logits: those here are single products, 2^-7 apart or equal."""
    z = q[:, 3:4] * k[:, 3].double() * scale
    z = z.masked_fill(~sees, -math.inf)
    w = (z == z.amax(-1, keepdim=True)).double()
    return w / w.sum(-1, keepdim=True) @ v.double()


RANGE = [(1.0, t) for t in (17, 24, 29, 30, 31, 40, 70)] + [(-2.0 ** 40, t) for t in (29, 30, 40, 110)]


def queries(rows, heads, D, up):
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    q = torch.zeros((rows, heads, D), dtype=torch.float64, device=DEV)
    q[..., 3] = (torch.randint(0, 2, (rows, heads), generator=g, device=DEV).double() * 2 - 1) * 2.0 ** up
    return q


def far_logits(gpu, D, H, G, lens, new, bits, scale, top):
    """out = V of the largest logit, the mean of V where several are equal: values and weights of 11 bits (2^-11 each
    where many rows are attended to), sums far below."""
    cache, pages, starts, kc, vc, up = far_cache(gpu, lens, H, D, bits, top, scale)
    rows = [0]
    for m in new:
        rows.append(rows[-1] + m)
    q = queries(rows[-1], H * G, D, up)
    out = gpu.qcache_attend(cache, q.bfloat16(), pages, i32(lens), i32(rows), scale=scale, out_dtype=torch.float32)
    for b, (n, m) in enumerate(zip(lens, new)):
        at = torch.arange(n, device=DEV)
        sees = at[None] <= torch.arange(n - m, n, device=DEV)[:, None]
        for h in range(H * G):
            k, v = (t[starts[b]:starts[b + 1], h // G] for t in (kc, vc))
            want = winners(q[rows[b]:rows[b + 1], h], k, v, scale, sees)
            tol = torch.full_like(want, float(v.abs().max()) * (2.0 ** -10 + 2.0 ** -14))
            check(out[rows[b]:rows[b + 1], h], want, tol, (b, h))


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("scale,top", RANGE)
@pytest.mark.parametrize("D,H,G,lens,new", [(128, 1, 4, [200, 90], [50, 90]), (64, 2, 8, [700, 40], [300, 20]),
                                            (128, 2, 8, [1500], [1100]), (128, 1, 4, [5000], [60])])
def test_far_logits_of_many_rows(gpu, D, H, G, lens, new, bits, scale, top):
    far_logits(gpu, D, H, G, lens, new, bits, scale, top)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("scale,top", RANGE)
@pytest.mark.parametrize("D,H,G,lens,new", [(128, 1, 4, [300, 33], [1, 1]), (64, 2, 8, [40, 517], [1, 4]), (128, 2, 4, [6000], [1]),
                                            (64, 1, 3, [900] * 9, [2] * 9)])
def test_far_logits_of_few_rows(gpu, D, H, G, lens, new, bits, scale, top):
    far_logits(gpu, D, H, G, lens, new, bits, scale, top)


@pytest.mark.parametrize("scale,top", RANGE)
@pytest.mark.parametrize("new", [1, 40])
def test_far_logits_behind_a_prefix(gpu, scale, top, new):
    """The first sequence is the prefix of the others."""
    D, H, G, lens, bits = 128, 1, 8, [701, 60, 90, 200], 8
    cache, pages, starts, kc, vc, up = far_cache(gpu, lens, H, D, bits, top, scale)
    q = queries(3 * new, H * G, D, up)
    out = gpu.qcache_attend_shared(cache, q.bfloat16(), pages[0].contiguous(), 701, pages[1:].contiguous(), i32(lens[1:]),
                                   i32([0, new, 2 * new, 3 * new]), scale=scale, out_dtype=torch.float32)
    for b, n in enumerate(lens[1:]):
        own = slice(starts[b + 1], starts[b + 2])
        k, v = torch.cat((kc[:701], kc[own]))[:, 0], torch.cat((vc[:701], vc[own]))[:, 0]
        sees = torch.arange(701 + n, device=DEV)[None] <= torch.arange(701 + n - new, 701 + n, device=DEV)[:, None]
        for h in range(H * G):
            want = winners(q[b * new:(b + 1) * new, h], k, v, scale, sees)
            tol = torch.full_like(want, float(v.abs().max()) * (2.0 ** -10 + 2.0 ** -14))
            check(out[b * new:(b + 1) * new, h], want, tol, (b, h))
