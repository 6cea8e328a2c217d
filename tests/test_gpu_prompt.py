"""Causal attention of packed prompts on the GPU against softmax(q k) v in fp64
(include/qlayer.h: qprompt_attend)."""
import math

import pytest
import torch

from layer_util import DEV, check, i32, prompt_ref, randn

pytestmark = pytest.mark.gpu


def qkv(T, Hq, H, D, seed=0):
    return randn((T, Hq, D), seed), randn((T, H, D), seed + 1), randn((T, H, D), seed + 2)


def starts_of(lens, lead=0):
    s = [lead]
    for n in lens:
        s.append(s[-1] + n)
    return s


def verify(got, Q, K, V, starts, scale=None, what=""):
    want, tol = prompt_ref(Q, K, V, starts, Q.shape[2] ** -0.5 if scale is None else scale)
    m = ~want.isnan()
    check(got[m], want[m], tol[m], what)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,G", [(1, 1), (2, 1), (1, 3), (2, 5), (1, 8), (1, 64)])
@pytest.mark.parametrize("T", [1, 2, 31, 32, 33, 64, 100, 129, 257])
def test_one_prompt(gpu, D, H, G, T):
    Q, K, V = qkv(T, H * G, H, D, T)
    verify(gpu.qprompt_attend(Q, K, V), Q, K, V, None)


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D,H,G", [(64, 2, 4), (128, 2, 8), (128, 3, 1)])
@pytest.mark.parametrize("lens", [[1], [0, 1, 0], [5, 300, 0, 1, 77, 128], [64] * 9, [1] * 40, [700, 3, 450], [1100, 1]])
@pytest.mark.parametrize("lead,tail", [(0, 0), (3, 5)])
def test_packed_prompts(gpu, D, H, G, lens, lead, tail, out_dtype):
    starts = starts_of(lens, lead)
    T = starts[-1] + tail
    if T == 0:
        return
    Q, K, V = qkv(T, H * G, H, D, 1)
    # nobody's rows may hold anything
    for t in (Q, K, V):
        t[:lead] = float("nan")
        t[starts[-1]:] = float("inf")
    out = torch.full((T, H * G, D), 7.0, dtype=out_dtype, device=DEV)
    gpu.qprompt_attend(Q, K, V, i32(starts), out=out)
    verify(out, Q, K, V, starts)
    assert bool((out[:lead] == 7.0).all()) and bool((out[starts[-1]:] == 7.0).all())


@pytest.mark.parametrize("D,H,G,T", [(128, 1, 8, 3001), (64, 2, 1, 2500), (128, 2, 2, 2049)])
def test_long_prompts(gpu, D, H, G, T):
    Q, K, V = qkv(T, H * G, H, D, 2)
    verify(gpu.qprompt_attend(Q, K, V, out_dtype=torch.float32), Q, K, V, None)


def test_more_tiles_than_workgroups(gpu):
    lens = [200 + 17 * b for b in range(30)]
    starts = starts_of(lens)
    Q, K, V = qkv(starts[-1], 16, 8, 64, 3)
    verify(gpu.qprompt_attend(Q, K, V, i32(starts)), Q, K, V, starts)


@pytest.mark.parametrize("B", [64, 65, 256, 257, 1000])
def test_many_sequences(gpu, B):
    lens = [(b * 7) % 23 + (130 if b % 50 == 3 else 0) for b in range(B)]
    starts = starts_of(lens, 1)
    Q, K, V = qkv(starts[-1] + 2, 4, 2, 64, 33)
    out = torch.full((starts[-1] + 2, 4, 64), 3.0, dtype=torch.bfloat16, device=DEV)
    gpu.qprompt_attend(Q, K, V, i32(starts), out=out)
    verify(out, Q, K, V, starts)
    assert bool((out[:1] == 3.0).all()) and bool((out[-2:] == 3.0).all())


@pytest.mark.parametrize("scale", [0.0, 1e-30, 0.01, -0.2, 1.0, 30.0])
def test_scales(gpu, scale):
    Q, K, V = qkv(150, 4, 2, 64, 4)
    verify(gpu.qprompt_attend(Q, K, V, scale=scale), Q, K, V, None, scale)


@pytest.mark.parametrize("order", ["up", "down", "spike"])
def test_moving_maximum(gpu, order):
    """Logits that rise, fall or jump along the keys by far more than fp32's exponential takes."""
    T, D = 400, 64
    Q, K, V = qkv(T, 2, 1, D, 5)
    Q[..., 0] = 16.0
    ramp = torch.arange(T, device=DEV).float()
    K[:, 0, 0] = {"up": ramp, "down": -ramp, "spike": 300.0 * ((ramp % 97) == 50).float()}[order].bfloat16()
    verify(gpu.qprompt_attend(Q, K, V, scale=1.0, out_dtype=torch.float32), Q, K, V, None, 1.0)


def test_strides(gpu):
    T, Hq, H, D = 200, 6, 2, 128
    rows = randn((T, Hq + 2 * H, D), 6)
    Q, K, V = rows[:, :Hq], rows[:, Hq:Hq + H], rows[:, Hq + H:]
    out = torch.full((T, Hq + 3, D), 5.0, dtype=torch.bfloat16, device=DEV)
    got = gpu.qprompt_attend(Q, K, V, out=out[:, 2:2 + Hq])
    verify(got, Q, K, V, None)
    assert torch.equal(got, gpu.qprompt_attend(Q.contiguous(), K.contiguous(), V.contiguous()))
    assert bool((out[:, :2] == 5.0).all()) and bool((out[:, 2 + Hq:] == 5.0).all())


@pytest.mark.parametrize("D,H,G", [(64, 1, 4), (128, 2, 1), (128, 1, 8)])
@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("at", [0, 37, 130, 299, 300, 349])
def test_rows_before_a_value_that_is_not_finite(gpu, D, H, G, value, which, at):
    """Sequences of 300 and 50: the rows of another sequence and those before it are what they were, bit for bit."""
    starts = [0, 300, 350]
    Q, K, V = qkv(350, H * G, H, D, 7)
    clean = gpu.qprompt_attend(Q, K, V, i32(starts))
    (K if which == "k" else V)[at, 0, 5] = value
    got = gpu.qprompt_attend(Q, K, V, i32(starts))
    end = 300 if at < 300 else 350
    sees = torch.zeros((350, H * G), dtype=torch.bool, device=DEV)
    sees[at:end, :G] = True
    assert torch.equal(got[~sees], clean[~sees])
    if which == "v":
        assert bool((~got[sees][:, 5].isfinite()).all())
    elif math.isnan(value):
        assert bool(got[sees].isnan().all())


# sizes whose tiles' rows one wave has to itself (many heads; of 64 also with two workgroups a CU), or shares with one
# other or three (few heads, long)
SHARED = [(64, 96, 8, [300, 0, 50]), (64, 40, 2, [260, 30, 1] * 8), (64, 32, 8, [300, 0, 50]), (128, 24, 6, [280, 1, 60]), (128, 2, 4, [400, 90]), (64, 1, 1, [1500, 200]), (128, 1, 2, [1, 1700])]


@pytest.mark.parametrize("D,H,G,lens", SHARED)
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
def test_rows_of_one_or_several_waves(gpu, D, H, G, lens, out_dtype):
    starts = starts_of(lens, 2)
    T = starts[-1] + 3
    Q, K, V = qkv(T, H * G, H, D, 30)
    out = torch.full((T, H * G, D), 3.0, dtype=out_dtype, device=DEV)
    gpu.qprompt_attend(Q, K, V, i32(starts), out=out)
    verify(out, Q, K, V, starts)
    assert bool((out[:2] == 3.0).all()) and bool((out[-3:] == 3.0).all())


@pytest.mark.parametrize("D,H,G,lens", SHARED)
@pytest.mark.parametrize("value", [math.inf, math.nan])
@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("at", [0, 31, 100, 128, 250])
def test_values_that_are_not_finite_by_waves(gpu, D, H, G, lens, value, which, at):
    starts = starts_of(lens)
    T = starts[-1]
    Q, K, V = qkv(T, H * G, H, D, 31)
    clean = gpu.qprompt_attend(Q, K, V, i32(starts))
    (K if which == "k" else V)[at, H - 1, 5] = value
    got = gpu.qprompt_attend(Q, K, V, i32(starts))
    sees = torch.zeros((T, H * G), dtype=torch.bool, device=DEV)
    sees[at:next(s for s in starts if s > at), (H - 1) * G:] = True
    assert torch.equal(got[~sees], clean[~sees])
    if which == "v":
        assert bool((~got[sees][:, 5].isfinite()).all())
    elif math.isnan(value):
        assert bool(got[sees].isnan().all())


@pytest.mark.parametrize("D,H,G,lens", SHARED)
def test_rising_logits_by_waves(gpu, D, H, G, lens):
    starts = starts_of(lens)
    Q, K, V = qkv(starts[-1], H * G, H, D, 32)
    Q[..., 0] = 8.0
    K[..., 0] = (torch.arange(starts[-1], device=DEV) % 300).bfloat16()[:, None]
    verify(gpu.qprompt_attend(Q, K, V, i32(starts), scale=0.5, out_dtype=torch.float32), Q, K, V, starts, 0.5)


@pytest.mark.parametrize("lens", [[300], [40, 500, 3]])
def test_the_same_every_time(gpu, lens):
    starts = starts_of(lens)
    Q, K, V = qkv(starts[-1], 8, 2, 128, 8)
    first = gpu.qprompt_attend(Q, K, V, i32(starts))
    for _ in range(5):
        assert torch.equal(gpu.qprompt_attend(Q, K, V, i32(starts)), first)


def test_graph_follows_starts(gpu):
    T = 500
    Q, K, V = qkv(T, 8, 2, 64, 9)
    starts, out = i32([0, 0, 0, T]), torch.zeros((T, 8, 64), dtype=torch.bfloat16, device=DEV)
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        gpu.qprompt_attend(Q, K, V, starts, out=out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        gpu.qprompt_attend(Q, K, V, starts, out=out)
    for now in ([0, 10, 200, 500], [0, 499, 499, 500], [100, 200, 300, 400], [0, 0, 500, 500]):
        starts.copy_(i32(now))
        V.copy_(randn((T, 2, 64), now[1]))
        out.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        verify(out, Q, K, V, now, what=now)
        assert bool((out[:now[0]] == 0).all()) and bool((out[now[-1]:] == 0).all())
        again = torch.zeros_like(out)
        assert torch.equal(gpu.qprompt_attend(Q, K, V, starts, out=again), out)


def test_calls_at_once(gpu):
    sets = [qkv(900, 8, 2, 128, s) for s in (10, 20)]
    want = [gpu.qprompt_attend(*s) for s in sets]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], [[], []]
    for _ in range(6):
        for k in (0, 1):
            got[k].append(gpu.qprompt_attend(*sets[k], stream=streams[k]))
    torch.cuda.synchronize()
    for k in (0, 1):
        assert all(torch.equal(o, want[k]) for o in got[k])


def test_no_rows(gpu):
    out = gpu.qprompt_attend(*qkv(0, 8, 2, 64), i32([0, 0]))
    assert out.shape == (0, 8, 64)
