"""The steps between projections and cache at the ends of their arguments'
ranges, and over values that are not finite (include/qlayer.h)."""
import math

import pytest
import torch

from layer_util import DEV, check, i32, prompt_ref, randn
from test_gpu_prompt import SHARED, qkv, starts_of, verify

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------- prompts
def peaks(starts, H, G, D, top, scale):
    """Q, K, V whose logits are single products of 8 bits around +-2^top, and the result: of logits that far apart the
    largest takes all the weight, and equal ones share it.  out = V of it (the mean of their V) with 2^-23 of each
    addition and the quotient: n < 2^12 equal ones, added 16 at a time, stay below 2^-14."""
    T = starts[-1]
    g = torch.Generator(device=DEV)
    g.manual_seed(top)
    sign = lambda *s: torch.randint(0, 2, s, generator=g, device=DEV).double() * 2 - 1
    up = round(top - math.log2(abs(scale))) // 2
    q = torch.zeros((T, H * G, D), dtype=torch.float64, device=DEV)
    k = torch.zeros((T, H, D), dtype=torch.float64, device=DEV)
    q[..., 3] = sign(T, H * G) * 2.0 ** up
    k[..., 3] = sign(T, H) * (1 + torch.randint(0, 128, (T, H), generator=g, device=DEV) / 128.0) * 2.0 ** (top - round(math.log2(abs(scale))) - up)
    V = randn((T, H, D), top + 1)
    want = torch.empty((T, H * G, D), dtype=torch.float64, device=DEV)
    for s, e in zip(starts, starts[1:]):
        later = torch.ones((e - s, e - s), dtype=torch.bool, device=DEV).triu(1)
        for h in range(H * G if e > s else 0):
            z = (q[s:e, h, 3:4] * k[s:e, h // G, 3] * scale).masked_fill(later, -math.inf)
            w = (z == z.amax(-1, keepdim=True)).double()
            want[s:e, h] = w / w.sum(-1, keepdim=True) @ V[s:e, h // G].double()
    return q.bfloat16(), k.bfloat16(), V, want


@pytest.mark.parametrize("D,H,G,lens", [(128, 1, 1, [1]), (64, 2, 3, [70, 1, 300])] + SHARED)
@pytest.mark.parametrize("top", [17, 24, 31, 40, 80, 118])
@pytest.mark.parametrize("scale", [1.0, -0.3, 2.0 ** 45])
def test_far_logits(gpu, D, H, G, lens, top, scale):
    starts = starts_of(lens)
    Q, K, V, want = peaks(starts, H, G, D, top, scale)
    got = gpu.qprompt_attend(Q, K, V, i32(starts), scale=scale, out_dtype=torch.float32)
    tol = torch.full_like(want, float(V.float().abs().max()) * 2.0 ** -14)
    check(got, want, tol, (top, scale))


@pytest.mark.parametrize("D,H,G,lens", SHARED)
def test_far_logits_beside_others(gpu, D, H, G, lens):
    """Rows of ordinary logits in the tiles of rows with far ones: the same bits as without them."""
    starts = starts_of(lens)
    T = starts[-1]
    Q, K, V = qkv(T, H * G, H, D, 40)
    K[..., 3] = (1 + torch.arange(T, device=DEV) % 60).bfloat16()[:, None]
    Q[..., 3] = 0
    alone = gpu.qprompt_attend(Q, K, V, i32(starts))
    verify(alone, Q, K, V, starts)
    far = (torch.arange(T * H * G, device=DEV) % 7 == 2).view(T, H * G)
    Q[far] = 0                               # their logits are that one product
    Q[..., 3] = torch.where(far, 2.0 ** 60, 0.0).bfloat16()
    got = gpu.qprompt_attend(Q, K, V, i32(starts))
    assert torch.equal(got[~far], alone[~far])
    for s, e in zip(starts, starts[1:]):
        for t in range(s, e, 23):
            for h in range(0, H * G, max(1, H * G // 8)):
                if far[t, h]:
                    seen = K[s:t + 1, h // G, 3].float()
                    want = V[s:t + 1, h // G][seen == seen.max()].double().mean(0)
                    check(got[t, h], want, torch.full_like(want, 2.0 ** -14 * float(V.float().abs().max())), (t, h))


@pytest.mark.parametrize("D,H,G,lens", [(64, 2, 1, [1, 70]), (128, 1, 8, [40, 200])] + SHARED)
def test_logits_of_minus_infinity(gpu, D, H, G, lens):
    """A key whose products are all -inf weighs nothing; a row that sees no other key is NaN."""
    starts = starts_of(lens)
    Q, K, V = qkv(starts[-1], H * G, H, D, 41)
    Q[..., 5] = Q[..., 5].abs() + 0.5
    cut = []                                 # of every sequence the first few keys
    for s, e in zip(starts, starts[1:]):
        n = min(e - s, 3 + (e - s) // 3)
        K[s:s + n, :, 5] = -math.inf
        cut.append(n)
    got = gpu.qprompt_attend(Q, K, V, i32(starts), out_dtype=torch.float32)
    for s, e, n in zip(starts, starts[1:], cut):
        assert bool(got[s:s + n].isnan().all())
        if e > s + n:                        # the others see only what comes behind
            want, tol = prompt_ref(Q[s + n:e], K[s + n:e], V[s + n:e], None, D ** -0.5)
            check(got[s + n:e], want, tol)


@pytest.mark.parametrize("D,H,G,lens", [(64, 2, 1, [1, 70]), (128, 1, 8, [40, 200])] + SHARED)
def test_logits_of_plus_infinity(gpu, D, H, G, lens):
    """A row that sees one is NaN; the others do not feel it."""
    starts = starts_of(lens)
    Q, K, V = qkv(starts[-1], H * G, H, D, 44)
    Q[..., 5] = Q[..., 5].abs() + 0.5
    clean = gpu.qprompt_attend(Q, K, V, i32(starts))
    sees = torch.zeros(starts[-1], dtype=torch.bool, device=DEV)
    for s, e in zip(starts, starts[1:]):
        if e > s:
            K[s + (e - s) // 2, :, 5] = math.inf
            sees[s + (e - s) // 2:e] = True
    got = gpu.qprompt_attend(Q, K, V, i32(starts))
    assert bool(got[sees].isnan().all()) and torch.equal(got[~sees], clean[~sees])


@pytest.mark.parametrize("scale", [0.0, 1e-42, -1e-40, 1e-38])
@pytest.mark.parametrize("D,H,G,lens", [(64, 2, 2, [1, 90, 300]), (128, 1, 8, [150]), (128, 1, 2, [1, 1700])])
def test_scales_near_zero(gpu, D, H, G, lens, scale):
    """Over products up to the largest there may be: a scale of 0 makes all weights equal."""
    starts = starts_of(lens)
    Q, K, V = qkv(starts[-1], H * G, H, D, 42)
    Q = (Q.float().clamp(-3.9, 3.9) * 2.0 ** 55).bfloat16()
    K = (K.float().clamp(-3.9, 3.9) * 2.0 ** 60).bfloat16()
    assert float((Q.double().abs().amax((0, 1)) * K.double().abs().amax((0, 1))).sum()) < 2.0 ** 126
    got = gpu.qprompt_attend(Q, K, V, i32(starts), scale=scale, out_dtype=torch.float32)
    verify(got, Q, K, V, starts, torch.tensor(scale, dtype=torch.float32).item())


@pytest.mark.parametrize("D", [64, 128])
def test_one_large_weight_and_many_small_ones(gpu, D):
    """Weights of 2^-24.17 beside one of 1: each is lost if it is added to a sum by itself.  All values are 1, and so is
    the result.  Sums between 1 and 1.01: the numerator takes at most n / 16 additions off by 2^-23 each, the sum of the
    weights n / 32 in each of two lanes, off by 2^-24, and the rounding of the small weights (2^-8) is 2^-8 * 0.007."""
    T = 1 << 17
    Q = torch.zeros((T, 1, D), dtype=torch.bfloat16, device=DEV)
    K, V = torch.zeros_like(Q), torch.ones_like(Q)
    Q[..., 0] = 1.0
    K[0, 0, 0] = 16.75
    out = gpu.qprompt_attend(Q, K, V, scale=1.0, out_dtype=torch.float32)
    off = float((out.double() - 1).abs().max())
    assert off <= T / 16 * 2.0 ** -23 + T / 32 * 2.0 ** -24 + 2.0 ** -8 * 0.007 + 2.0 ** -20, off


@pytest.mark.parametrize("D", [64, 128])
def test_a_workgroup_with_a_second_tile(gpu, D):
    """More tiles than the grid holds (2^22 over the heads): the workgroups of the first tiles, some of them long and
    with values that are not finite, go on with the last sequences."""
    H, lens = 1024, [300] * 8 + [1 + b % 2 for b in range(4300)] + [150] * 8
    starts = starts_of(lens)
    T, n = starts[-1], len(lens)
    assert T // 256 + n > (1 << 22) // H + 200
    Q, K, V = qkv(T, H, H, D, 43)
    for b in range(1, 250, 2):               # in the tiles before those of the last sequences
        V[starts[b], :, 5] = math.inf if b % 4 == 1 else math.nan
    got = gpu.qprompt_attend(Q, K, V, i32(starts))
    first = torch.tensor(starts[:-1], device=DEV)
    sick = torch.zeros(n, dtype=torch.bool, device=DEV)
    sick[1:250:2] = True
    # a sequence's first row sees itself only
    assert torch.equal(got[first[~sick]], V[first[~sick]])
    assert bool((~got[first[sick]][..., 5].isfinite()).all())
    second = first[8:8 + 4300][1::2] + 1
    second = second[~sick[8:8 + 4300][1::2]]
    for part in second.split(256):
        q, k0, k1 = Q[part].double(), K[part - 1].double(), K[part].double()
        z0, z1 = (q * k0).sum(-1, keepdim=True) * D ** -0.5, (q * k1).sum(-1, keepdim=True) * D ** -0.5
        w = torch.sigmoid(z1 - z0)
        v0, v1 = V[part - 1].double(), V[part].double()
        # weights off by 2^-8 of themselves (rounded to bf16), and by 2^-16 (logits and exponentials: prompt_ref's terms)
        check(got[part], v0 + (v1 - v0) * w, (v0.abs() * (1 - w) + v1.abs() * w) * (2.0 ** -8 + 2.0 ** -14))
    for b in (0, 2, n - 8, n - 1):
        s, e = starts[b], starts[b + 1]
        for h in (0, 517, H - 1):
            want, tol = prompt_ref(Q[s:e, h:h + 1], K[s:e, h:h + 1], V[s:e, h:h + 1], None, D ** -0.5)
            check(got[s:e, h:h + 1], want, tol, (b, h))


# ------------------------------------------------------------------ adapters
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rank,own", [(8, 8), (8, 3), (16, 5), (24, 24), (40, 33), (128, 100)])
@pytest.mark.parametrize("kind", ["few", "many", "requests", "tall"])
def test_infinities_through_an_adapter(gpu, kind, rank, own, dtype):
    """Infinities in x and A come out as the formula's: of the sign of B times them where all terms agree, else NaN."""
    K, N, n = 264, 70, 2
    T = {"few": 9, "many": 50, "requests": 40, "tall": 150}[kind]
    starts = {"few": None, "many": None, "requests": [0] + list(range(9, 41)), "tall": [0, 100, 150]}[kind]
    ids = [0] * T if starts is None else [0] * (len(starts) - 1)
    A, B = randn((n, rank, K), 1).abs() + 0.125, randn((n, N, rank), 2)
    B[:, ::2] = B[:, ::2].abs() + 0.125
    B[:, 1::4] = -B[:, 1::4].abs() - 0.125
    A[:, own:], B[:, :, own:] = math.nan, math.inf          # behind the adapter's rank: anything
    x, y = randn((T, K), 3), randn((T, N), 4, dtype)
    rows = list(range(1, T, 4))
    x[rows[0::2], 7] = math.inf
    x[rows[1::2], K - 1] = -math.inf
    scales = torch.tensor([-0.5, 1.0], device=DEV)
    a = gpu.make_qadapters(A, B, scales, i32([own, own]))
    got = gpu.qadapt(a, x, y, i32(ids), None if starts is None else i32(starts))
    h = (x.double()[:, None] * A[0, :own].double()).sum(-1)
    want = y.double() - 0.5 * (h[:, None] * B[0, :, :own].double()).sum(-1)
    assert bool((want[rows][:, ::2].isinf()).all()) and bool(want[rows][:, 1::4].isinf().all())
    assert torch.equal(got[rows].double().nan_to_num(7.0, 1e300, -1e300), want[rows].nan_to_num(7.0, 1e300, -1e300))
    rest = [t for t in range(T) if t not in rows]
    assert bool(got[rest].isfinite().all())


@pytest.mark.parametrize("rank", [8, 16, 24, 64, 128])
@pytest.mark.parametrize("kind", ["few", "many", "tall"])
def test_the_inner_product_keeps_its_bits(gpu, kind, rank):
    """A x of 24 bits (three products 2^8 apart, below 2 in all) handed through a B of ones: every step is exact, so the
    fp32 result is A x itself, times the scale's power of two."""
    T, n, K, N = {"few": 5, "many": 70, "tall": 150}[kind], 2, 72, rank + 5
    g = torch.Generator(device=DEV)
    g.manual_seed(rank)
    A = torch.zeros((n, rank, K), device=DEV)
    A[..., 3:6] = 1 + torch.randint(0, 124, (n, rank, 3), generator=g, device=DEV) / 128.0
    x = torch.zeros((T, K), device=DEV)
    up = (2.0 ** torch.randint(-20, 20, (T,), generator=g, device=DEV).double()).float()
    assert bool((up.frexp()[0] == 0.5).all())
    x[:, 3], x[:, 4], x[:, 5] = up, -up * 2.0 ** -8, up * 2.0 ** -16
    B = torch.zeros((n, N, rank), device=DEV)
    out_of = torch.arange(N, device=DEV) % rank
    B[:, torch.arange(N, device=DEV), out_of] = 1.0
    ids = [t % 3 - 1 for t in range(T)] if kind != "tall" else [1, 0]
    starts = None if kind != "tall" else [0, 90, T]
    a = gpu.make_qadapters(A.bfloat16(), B.bfloat16(), torch.tensor([0.25, 2.0], device=DEV))
    got = gpu.qadapt(a, x.bfloat16(), torch.zeros((T, N), device=DEV), i32(ids), None if starts is None else i32(starts))
    of = torch.tensor(ids if starts is None else [1] * 90 + [0] * (T - 90), device=DEV)
    h = (A[of.clamp(min=0)].double() * x[:, None].double()).sum(-1)[:, out_of]
    want = torch.where(of[:, None] >= 0, h * torch.tensor([0.25, 2.0], device=DEV).double()[of.clamp(min=0)][:, None], 0.0)
    assert torch.equal(got.double(), want)
