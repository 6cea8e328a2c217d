"""Low-rank adapters beside a shared projection on the GPU against the formula
in fp64 (include/qlayer.h: qadapt)."""
import pytest
import torch

from layer_util import DEV, adapt_ref, check, i32, randn

pytestmark = pytest.mark.gpu


class Case:
    def __init__(self, K, N, r, n, ids, starts=None, T=None, ranks=None, dtype=torch.float32, seed=0):
        T = len(ids) if T is None else T
        self.K, self.N, self.r, self.n, self.T = K, N, r, n, T
        self.A = randn((n, r, K), seed, scale=K ** -0.5)
        self.B = randn((n, N, r), seed + 1)
        self.scales = randn((n,), seed + 2, torch.float32)
        self.x = randn((T, K), seed + 3)
        self.y = randn((T, N), seed + 4, dtype)
        self.ids, self.starts, self.ranks = ids, starts, ranks

    def handle(self, cg):
        return cg.make_qadapters(self.A, self.B, self.scales, None if self.ranks is None else i32(self.ranks))

    def run(self, cg, out=None, **kw):
        return cg.qadapt(self.handle(cg), self.x, self.y, i32(self.ids), None if self.starts is None else i32(self.starts),
                         out=out, **kw)

    def owned(self):
        m = torch.ones(self.T, dtype=torch.bool, device=DEV)
        if self.starts is not None:
            m[:] = False
            m[self.starts[0]:self.starts[-1]] = True
        return m

    def verify(self, got, y=None, what=""):
        want, tol = adapt_ref(self.A, self.B, self.scales, self.ranks, self.x, self.y if y is None else y, self.ids, self.starts)
        m = self.owned()
        check(got[m], want[m], tol[m], what)


SIZES = [(8, 1, 8), (8, 17, 128), (64, 64, 16), (264, 100, 24), (512, 512, 40), (1000, 333, 64), (2048, 1023, 8),
         (8192, 1024, 16), (4104, 257, 104)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("K,N,r", SIZES)
@pytest.mark.parametrize("T", [1, 3, 16, 17, 64, 65, 150])
def test_one_row_each(gpu, K, N, r, T, dtype):
    ids = [(5 * b + b // 7) % 7 - 1 for b in range(T)]       # -1 .. 5 of 5: without an adapter at both ends
    c = Case(K, N, r, 5, ids, dtype=dtype, seed=T)
    c.verify(c.run(gpu))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("K,N,r", SIZES)
@pytest.mark.parametrize("lens", [[1], [64], [65], [5, 0, 0, 130], [1] * 70, [0, 17, 16, 1, 63, 64, 200, 0],
                                  [100] + [1] * 40])
def test_segments(gpu, K, N, r, lens, dtype):
    starts = [0]
    for n in lens:
        starts.append(starts[-1] + n)
    ids = [(3 * b + 1) % 6 - 1 for b in range(len(lens))]
    c = Case(K, N, r, 4, ids, starts, starts[-1], dtype=dtype, seed=len(lens))
    c.verify(c.run(gpu))


@pytest.mark.parametrize("ids", [[0] * 200, list(range(200)), [b % 2 for b in range(200)], [-1] * 200,
                                 [199 - b for b in range(200)]])
def test_one_adapter_or_many(gpu, ids):
    c = Case(256, 320, 16, 200, ids, seed=3)
    c.verify(c.run(gpu))


@pytest.mark.parametrize("T", [1025, 3001])
def test_many_single_rows(gpu, T):
    c = Case(128, 96, 8, 40, [(b * b) % 41 for b in range(T)], seed=4)
    c.verify(c.run(gpu))


@pytest.mark.parametrize("starts", [None, [0, 40, 40, 41, 100]])
def test_ranks_of_their_own(gpu, starts):
    """What lies behind an adapter's rank is not looked at, be it NaN."""
    r, ranks = 48, [0, 1, 7, 16, 17, 33, 48, 99, -5]
    ids = [3, 8, 0, 5] if starts else [b % 10 for b in range(100)]
    c = Case(200, 130, r, len(ranks), ids, starts, 100, ranks, seed=5)
    for a, k in enumerate(ranks):
        k = max(0, min(r, k))
        c.A[a, k:] = float("nan")
        c.B[a, :, k:] = float("inf")
    c.verify(c.run(gpu))


@pytest.mark.parametrize("B", [300, 5000])
@pytest.mark.parametrize("long", [0, 700])
def test_many_requests(gpu, B, long):
    """Requests of 0 to 4 rows, one of them long."""
    starts = [0]
    for b in range(B):
        starts.append(starts[-1] + b % 5 + (long * B // 10 if b == 77 else 0))
    c = Case(72, 50, 16, 9, [(b * 3) % 11 - 1 for b in range(B)], starts, starts[-1], seed=16)
    c.verify(c.run(gpu))


def test_ids_outside_the_set(gpu):
    c = Case(64, 40, 8, 3, [-1, 3, 2 ** 31 - 1, -2 ** 31, 2], seed=6)
    got = c.run(gpu)
    assert torch.equal(got[:4], c.y[:4])
    c.verify(got)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("starts", [None, [7, 30, 30, 90]])
def test_in_place_and_rows_of_nobody(gpu, starts, dtype):
    ids = [1, 0, -1] if starts else [b % 4 - 1 for b in range(95)]
    c = Case(136, 75, 16, 3, ids, starts, 95, dtype=dtype, seed=7)
    fresh = c.run(gpu)
    y0, m = c.y.clone(), c.owned()
    got = c.run(gpu, out=c.y)
    assert got.data_ptr() == c.y.data_ptr()
    assert torch.equal(got[m], fresh[m]) and torch.equal(got[~m], y0[~m])
    c.verify(got, y0)
    # a given output keeps what nobody owns
    c.y = y0
    out = torch.full_like(y0, 777.0)
    c.run(gpu, out=out)
    assert torch.equal(out[m], fresh[m]) and bool((out[~m] == 777.0).all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shift", [0, 1, 3])
def test_strides(gpu, dtype, shift):
    """Columns of one fused output, beginning anywhere; what lies beside them stays."""
    c = Case(72, 130, 24, 3, [b % 3 for b in range(33)], dtype=dtype, seed=8)
    want = c.run(gpu)
    X = randn((33, 72 + 16), 1)
    X[:, 8:80] = c.x
    Y = torch.full((33, 200 + shift), 5.0, dtype=dtype, device=DEV)
    Y[:, shift:shift + 130] = c.y
    got = gpu.qadapt(c.handle(gpu), X[:, 8:80], Y[:, shift:shift + 130], i32(c.ids), out=Y[:, shift:shift + 130])
    assert torch.equal(got, want)
    assert bool((Y[:, :shift] == 5.0).all()) and bool((Y[:, shift + 130:] == 5.0).all())


def test_values_that_are_not_finite_stay_in_their_row(gpu):
    c = Case(128, 96, 16, 2, [b % 2 for b in range(40)], seed=9)
    clean = c.run(gpu)
    c.x[5, 3] = float("inf")
    c.x[6] = float("nan")
    c.y[7, 2] = float("inf")
    got = c.run(gpu)
    keep = [b for b in range(40) if b not in (5, 6, 7)]
    assert torch.equal(got[keep], clean[keep])
    assert bool(got[6].isnan().all()) and bool((~got[5].isfinite()).all()) and bool(got[7, 2].isinf())
    assert torch.equal(got[7, 3:], clean[7, 3:])


def test_the_same_every_time(gpu):
    c = Case(8192, 1000, 64, 6, [b % 7 for b in range(50)], seed=10)
    first = c.run(gpu)
    for _ in range(5):
        assert torch.equal(c.run(gpu), first)


def test_far_into_a_large_set(gpu):
    """Adapters that begin beyond 4 GiB of A and of B."""
    n, r, K, N = 40, 128, 496 * 1024, 440 * 1024
    A = torch.zeros((n, r, K), dtype=torch.bfloat16, device=DEV)
    B = torch.zeros((n, N, r), dtype=torch.bfloat16, device=DEV)
    assert A[n - 1].data_ptr() - A.data_ptr() > 2 ** 32 and B[n - 1].data_ptr() - B.data_ptr() > 2 ** 32
    A[n - 1], B[n - 1] = randn((r, K), 1, scale=K ** -0.5), randn((N, r), 2)
    x, y = randn((2, K), 3), randn((2, N), 4, torch.float32)
    a = gpu.make_qadapters(A, B, torch.ones(n, device=DEV))
    got = gpu.qadapt(a, x, y, i32([n - 1, 0]))
    want, tol = adapt_ref(A[-1:], B[-1:], torch.ones(1, device=DEV), None, x, y, [0, -1], None)
    check(got, want, tol)


@pytest.mark.parametrize("single", [True, False])
def test_graph_follows_ids_and_rows(gpu, single):
    """A captured call reads ids, starts and values at every replay; the program's own work runs between."""
    T = 90
    c = Case(512, 200, 16, 4, [0] * T if single else [0, 0, 0], None if single else [0, 0, 0, T], T, seed=11)
    h, ids = c.handle(gpu), i32(c.ids)
    starts = None if single else i32(c.starts)
    ws = torch.empty(gpu.qadapt_ws(h, ids.numel(), T), dtype=torch.uint8, device=DEV)
    out = torch.empty_like(c.y)
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        gpu.qadapt(h, c.x, c.y, ids, starts, out=out, ws=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        gpu.qadapt(h, c.x, c.y, ids, starts, out=out, ws=ws)
    for rep in range(4):
        c.ids = [(b * (rep + 1)) % 5 - 1 for b in range(ids.numel())]
        ids.copy_(i32(c.ids))
        if not single:
            c.starts = [0, 10 * rep, 30 + 7 * rep, T]
            starts.copy_(i32(c.starts))
        c.x.copy_(randn((T, 512), 20 + rep))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        c.verify(out, what=rep)
        assert torch.equal(out, c.run(gpu))


def test_streams_and_workspaces_of_their_own(gpu):
    """Two calls at once, each with its stream: neither sees the other's workspace."""
    cs = [Case(4096, 2048, 32, 3, [b % 3 for b in range(64)], seed=s) for s in (12, 13)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(6):
        for k in (0, 1):
            got[k].append(cs[k].run(gpu, stream=streams[k]))
    torch.cuda.synchronize()
    for k in (0, 1):
        for o in got[k]:
            cs[k].verify(o)


def test_beside_a_compressed_projection(gpu):
    """The projection's own outputs, fp32 and bf16, take the adapters in place."""
    K, N = 512, 300
    W = randn((N, K), 1, torch.float32, 0.02)
    codes, meta = gpu.qpack_group(W, 4, 64)
    c = Case(K, N, 16, 3, [0, 2, -1, 1, 0], seed=14)
    for dt in (torch.float32, torch.bfloat16):
        y = gpu.qgemv_group(codes, meta, N, K, 4, 64, c.x, y_dtype=dt)
        y0 = y.clone()
        gpu.qadapt(c.handle(gpu), c.x, y, i32(c.ids), out=y)
        c.verify(y, y0)


def test_no_rows(gpu):
    c = Case(64, 40, 8, 3, [0], seed=15)
    out = gpu.qadapt(c.handle(gpu), c.x[:0], c.y[:0], i32([]))
    assert out.shape == (0, 40)
