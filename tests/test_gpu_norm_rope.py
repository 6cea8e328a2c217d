"""Head norms and rotation on the GPU against the formula in fp64
(include/qlayer.h: qnorm_rope)."""
import pytest
import torch

from layer_util import DEV, check, i32, norm_rope_ref, randn

pytestmark = pytest.mark.gpu


def freqs_of(rot, base=1e4):
    return base ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot) if rot else None


def positions(lens, starts, T, offset):
    """Positions of all rows; NaN where nobody owns one."""
    p = torch.full((T,), float("nan"), dtype=torch.float64, device=DEV)
    for b, n in enumerate(lens):
        s, e = (b, b + 1) if starts is None else (starts[b], starts[b + 1])
        p[s:e] = torch.arange(n - (e - s), n, dtype=torch.float64, device=DEV) + offset
    return p


def verify(outs, ins, weights, eps, freqs, pairs, pos):
    m = ~pos.isnan()
    for o, x, w in zip(outs, ins, weights):
        if x is not None:
            want, tol = norm_rope_ref(x[m], w, eps, freqs, pairs, pos[m])
            check(o[m], want, tol)


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("ind,outd", [(i, o) for i in (torch.bfloat16, torch.float32) for o in (torch.bfloat16, torch.float32)])
@pytest.mark.parametrize("D,rot", [(64, 64), (64, 16), (64, 48), (128, 128), (128, 32), (128, 112), (128, 0)])
@pytest.mark.parametrize("Hq,Hk", [(1, 1), (8, 1), (5, 3), (64, 8)])
def test_heads_and_types(gpu, D, rot, Hq, Hk, ind, outd, pairs):
    lens = [1, 5, 1000, 131072, 0, 77, 3]
    Q, K = randn((7, Hq, D), 1, ind, 3.0), randn((7, Hk, D), 2, ind)
    qw, kw = randn((D,), 3), randn((D,), 4)
    fr = freqs_of(rot)
    outs = gpu.qnorm_rope(Q, K, i32(lens), freqs=fr, q_weight=qw, k_weight=kw, eps=1e-5, pairs=pairs, out_dtype=outd)
    verify(outs, (Q, K), (qw, kw), 1e-5, fr, pairs, positions(lens, None, 7, 0))


@pytest.mark.parametrize("weights", ["both", "q", "k", "none"])
@pytest.mark.parametrize("wd", [torch.bfloat16, torch.float32])
def test_weights(gpu, weights, wd):
    Q, K = randn((9, 6, 64), 1), randn((9, 2, 64), 2)
    qw = randn((64,), 3, wd) if weights in ("both", "q") else None
    kw = randn((64,), 4, wd) if weights in ("both", "k") else None
    lens, fr = list(range(40, 49)), freqs_of(64)
    outs = gpu.qnorm_rope(Q, K, i32(lens), freqs=fr, q_weight=qw, k_weight=kw, out_dtype=torch.float32)
    verify(outs, (Q, K), (qw, kw), 1e-6, fr, False, positions(lens, None, 9, 0))


@pytest.mark.parametrize("new", [[1], [300], [1, 0, 64, 2, 0, 33], [0, 5, 0], [1] * 130])
@pytest.mark.parametrize("lead,tail", [(0, 0), (4, 3)])
def test_ragged_rows(gpu, new, lead, tail):
    starts = [lead]
    for n in new:
        starts.append(starts[-1] + n)
    T = starts[-1] + tail
    lens = [n + 13 * b for b, n in enumerate(new)]
    Q, K = randn((T, 4, 128), 1), randn((T, 2, 128), 2)
    fr, w = freqs_of(128), randn((128,), 3)
    qo, ko = torch.full_like(Q, 9.0), torch.full_like(K, 9.0)
    outs = gpu.qnorm_rope(Q, K, i32(lens), i32(starts), freqs=fr, q_weight=w, k_weight=w, Qo=qo, Ko=ko, offset=50)
    pos = positions(lens, starts, T, 50)
    verify(outs, (Q, K), (w, w), 1e-6, fr, False, pos)
    nobody = pos.isnan()
    assert bool((qo[nobody] == 9.0).all()) and bool((ko[nobody] == 9.0).all())


@pytest.mark.parametrize("B", [300, 5000])
def test_many_sequences(gpu, B):
    new = [b % 4 for b in range(B)]
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    lens = [n + (b * 37) % 1000 for b, n in enumerate(new)]
    Q, K, fr = randn((starts[-1], 9, 64), 1), randn((starts[-1], 1, 64), 2), freqs_of(32)
    outs = gpu.qnorm_rope(Q, K, i32(lens), i32(starts), freqs=fr, pairs=True)
    verify(outs, (Q, K), (None, None), 1e-6, fr, True, positions(lens, starts, starts[-1], 0))


@pytest.mark.parametrize("offset", [0, 2 ** 20 - 1, 2 ** 31 - 1, -(2 ** 31) + 1])
def test_far_positions(gpu, offset):
    """Angles of positions of 31 bits; lens shorter than the new rows give negative ones."""
    lens = [2 ** 30, 1, 0, -5]
    starts = [0, 3, 6, 9, 12]
    Q = randn((12, 2, 64), 1, torch.float32)
    fr = freqs_of(64)
    (out, none) = gpu.qnorm_rope(Q, None, i32(lens), i32(starts), freqs=fr, offset=offset, out_dtype=torch.float32)
    assert none is None
    verify((out,), (Q,), (None,), 1e-6, fr, False, positions(lens, starts, 12, offset))


def test_keys_alone(gpu):
    K = randn((5, 3, 64), 1)
    fr, w, lens = freqs_of(32), randn((64,), 2), [3, 4, 5, 6, 7]
    none, out = gpu.qnorm_rope(None, K, i32(lens), freqs=fr, k_weight=w)
    assert none is None
    verify((out,), (K,), (w,), 1e-6, fr, False, positions(lens, None, 5, 0))


@pytest.mark.parametrize("ind", [torch.bfloat16, torch.float32])
def test_in_place_on_a_fused_projection(gpu, ind):
    """q and k as slices of one output, turned in place; v beside them stays."""
    T, Hq, Hk, D = 37, 5, 2, 128
    qkv = randn((T, Hq + 2 * Hk, D), 1, ind)
    was = qkv.clone()
    Q, K = qkv[:, :Hq], qkv[:, Hq:Hq + Hk]
    w, fr, starts, lens = randn((D,), 2), freqs_of(D), [0, 20, 37], [20, 400]
    want = gpu.qnorm_rope(Q, K, i32(lens), i32(starts), freqs=fr, q_weight=w, k_weight=w, out_dtype=ind)
    got = gpu.qnorm_rope(Q, K, i32(lens), i32(starts), freqs=fr, q_weight=w, k_weight=w, Qo=Q, Ko=K)
    assert got[0].data_ptr() == Q.data_ptr()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.equal(qkv[:, Hq + Hk:], was[:, Hq + Hk:])


@pytest.mark.parametrize("big", [2.0 ** 62, 2.0 ** 70, 2.0 ** 126])
@pytest.mark.parametrize("D", [64, 128])
def test_squares_beyond_fp32(gpu, big, D):
    Q = randn((6, 9, D), 1, torch.float32)
    Q[1] *= big / 8
    Q[2, 4] *= big / 8
    Q[3, :, 5] = big
    w = torch.ones(D, device=DEV)
    out, _ = gpu.qnorm_rope(Q, None, i32([1] * 6), q_weight=w, out_dtype=torch.float32)
    verify((out,), (Q,), (w,), 1e-6, None, False, positions([1] * 6, None, 6, 0))


def test_small_values_and_zeros(gpu):
    Q = randn((4, 3, 64), 1, torch.float32)
    Q[0] *= 1e-9
    Q[1] = 0
    w = torch.ones(64, device=DEV)
    out, _ = gpu.qnorm_rope(Q, None, i32([1] * 4), q_weight=w, eps=1e-20, out_dtype=torch.float32)
    verify((out,), (Q,), (w,), 1e-20, None, False, positions([1] * 4, None, 4, 0))


def test_values_that_are_not_finite_stay_in_their_head(gpu):
    Q = randn((8, 9, 128), 1)
    w, fr = randn((128,), 2), freqs_of(128)
    clean, _ = gpu.qnorm_rope(Q, None, i32([5] * 8), freqs=fr, q_weight=w)
    Q[3, 4, 7] = float("inf")
    Q[3, 6] = float("nan")
    got, _ = gpu.qnorm_rope(Q, None, i32([5] * 8), freqs=fr, q_weight=w)
    m = torch.ones((8, 9), dtype=torch.bool, device=DEV)
    m[3, 4] = m[3, 6] = False
    assert torch.equal(got[m], clean[m])
    assert bool(got[3, 6].isnan().all()) and bool(got[3, 4, 7].isnan())


def test_the_rest_of_a_head_is_not_turned(gpu):
    """An infinity behind rot stays one and where it is."""
    Q = randn((2, 1, 64), 1)
    Q[0, 0, 40] = float("inf")
    out, _ = gpu.qnorm_rope(Q, None, i32([9, 9]), freqs=freqs_of(32))
    assert torch.equal(out[..., 32:], Q[..., 32:])


def test_graph_follows_lens(gpu):
    Q, K, lens = randn((5, 8, 128), 1), randn((5, 2, 128), 2), i32([1] * 5)
    w, fr = randn((128,), 3), freqs_of(128)
    qo, ko = torch.empty_like(Q), torch.empty_like(K)
    st = torch.cuda.Stream()

    def call():
        gpu.qnorm_rope(Q, K, lens, freqs=fr, q_weight=w, k_weight=w, Qo=qo, Ko=ko)
    with torch.cuda.stream(st):
        call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        call()
    for rep in range(4):
        now = [10 * rep + b for b in range(5)]
        lens.copy_(i32(now))
        Q.copy_(randn((5, 8, 128), 30 + rep))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        verify((qo, ko), (Q, K), (w, w), 1e-6, fr, False, positions(now, None, 5, 0))


def test_another_stream(gpu):
    Q = randn((700, 8, 128), 1)
    fr, lens, st = freqs_of(128), i32(list(range(700))), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = [gpu.qnorm_rope(Q, None, lens, freqs=fr, stream=st)[0] for _ in range(4)]
    torch.cuda.current_stream().wait_stream(st)
    want, _ = gpu.qnorm_rope(Q, None, lens, freqs=fr)
    assert all(torch.equal(o, want) for o in outs)


def test_no_rows(gpu):
    qo, ko = gpu.qnorm_rope(randn((0, 8, 128), 1), randn((0, 2, 128), 1), i32([]))
    assert qo.shape == (0, 8, 128) and ko.shape == (0, 2, 128)
