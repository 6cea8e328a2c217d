"""A layer's attention path as it is used: projections with adapters, head norms
and rotation, prompt attention, the cache, then single tokens."""
import pytest
import torch

from layer_util import DEV, adapt_ref, check, i32, norm_rope_ref, prompt_ref, randn

pytestmark = pytest.mark.gpu


class Layer:
    """512 inputs, 4 query heads and 2 KV heads of 64, 4-bit weights, three adapters of rank 16."""
    K, Hq, H, D = 512, 4, 2, 64

    def __init__(self, cg):
        self.cg, self.N = cg, (self.Hq + 2 * self.H) * self.D
        self.codes, self.meta = cg.qpack_group(randn((self.N, self.K), 1, torch.float32, self.K ** -0.5), 4, 64)
        self.A, self.B = randn((3, 16, self.K), 2, scale=self.K ** -0.5), randn((3, self.N, 16), 3, scale=0.2)
        self.scales = torch.tensor([1.0, -0.5, 2.0], device=DEV)
        self.adapters = cg.make_qadapters(self.A, self.B, self.scales)
        self.qw, self.kw = randn((self.D,), 4).abs(), randn((self.D,), 5).abs()
        self.freqs = 1e4 ** (-torch.arange(0, self.D, 2, dtype=torch.float64, device=DEV) / self.D)
        self.w = cg.make_qweight_group(self.codes, self.meta, self.N, self.K, 4, 64)

    def rows(self, x, ids, starts, lens):
        """(q, k, v) of the new tokens x; and what qadapt was given."""
        cg = self.cg
        y = (cg.qgemm_prefill(self.w, x) if starts is not None else
             cg.qgemv_group(self.codes, self.meta, self.N, self.K, 4, 64, x))
        y0 = y.clone()
        cg.qadapt(self.adapters, x, y, ids, starts, out=y)
        qkv = y.view(-1, self.Hq + 2 * self.H, self.D)
        q, k = cg.qnorm_rope(qkv[:, :self.Hq], qkv[:, self.Hq:self.Hq + self.H], lens, starts, freqs=self.freqs,
                             q_weight=self.qw, k_weight=self.kw)
        return q, k, qkv[:, self.Hq + self.H:].bfloat16(), y0, y


def test_prompts_then_single_tokens(gpu):
    L = Layer(gpu)
    lens = [70, 1, 133]
    starts = [0, 70, 71, 204]
    ids = [2, -1, 0]
    x = randn((204, L.K), 6)
    q, k, v, y0, y = L.rows(x, i32(ids), i32(starts), i32(lens))
    want, tol = adapt_ref(L.A, L.B, L.scales, None, x, y0, ids, starts)
    check(y, want, tol, "adapters")
    pos = torch.cat([torch.arange(n, device=DEV) for n in lens]).double()
    qkv = y.view(204, -1, L.D)
    for got, rows, w in ((q, qkv[:, :L.Hq], L.qw), (k, qkv[:, L.Hq:L.Hq + L.H], L.kw)):
        want, tol = norm_rope_ref(rows, w, 1e-6, L.freqs, False, pos)
        check(got, want, tol, "norms")
    out = gpu.qprompt_attend(q, k, v, i32(starts))
    want, tol = prompt_ref(q, k, v, starts, L.D ** -0.5)
    check(out, want, tol, "prompts")

    # into the cache: 8-bit rows are off by half a step, a step is the row's range over 255 (and a bit for its fp16 constants)
    cache = gpu.make_qcache(16, 64, L.H, L.D, 8)
    pages = i32([[3, 5, 7, 0], [1, 2, 4, 6], [8, 9, 10, 11]])
    gpu.qcache_write(cache, k, v, pages, i32(lens), i32(starts))
    kc, vc = gpu.qcache_read(cache, pages, i32(lens), i32(starts), rows=204, dtype=torch.float32)
    assert float((kc - k.float()).abs().max()) <= float(k.float().abs().max()) * 2 / 255
    again = gpu.qcache_attend(cache, q, pages, i32(lens), i32(starts))
    want, tol = prompt_ref(q, kc, vc, starts, L.D ** -0.5)
    check(again, want, tol + cache_tol(q, kc, vc), "the cache's rows")

    # one new token each: the same rows at their places, seen through the cache
    lens = [n + 1 for n in lens]
    x1 = randn((3, L.K), 7)
    q1, k1, v1, y0, y1 = L.rows(x1, i32(ids), None, i32(lens))
    want, tol = adapt_ref(L.A, L.B, L.scales, None, x1, y0, ids, None)
    check(y1, want, tol, "adapters, single tokens")
    want, tol = norm_rope_ref(y1.view(3, -1, L.D)[:, :L.Hq], L.qw, 1e-6, L.freqs, False, i32(lens).double() - 1)
    check(q1, want, tol, "norms, single tokens")
    gpu.qcache_write(cache, k1, v1, pages, i32(lens))
    step = gpu.qcache_attend(cache, q1, pages, i32(lens), out_dtype=torch.float32)
    longer = [0, 71, 73, 207]
    kc, vc = gpu.qcache_read(cache, pages, i32(lens), i32(longer), rows=207, dtype=torch.float32)
    for b in range(3):
        rows = slice(longer[b], longer[b + 1])
        qs = torch.cat([q[starts[b]:starts[b + 1]], q1[b:b + 1]])
        want, tol = prompt_ref(qs, kc[rows], vc[rows], None, L.D ** -0.5)
        check(step[b], want[-1], tol[-1] + cache_tol(qs, kc, vc), "single tokens")


def cache_tol(q, k, v):
    """What attention over the cache may be off beyond a prompt's bound: keys, values and weights of 11 bits, so 2^-11 of
    a logit's terms from keys (at most |q| |k| scale in all, twice in a quotient) and 2^-11 of the values twice over."""
    terms = float(q.float().norm(dim=-1).max() * k.norm(dim=-1).max()) * q.shape[2] ** -0.5
    return float(v.abs().max()) * (terms * 2.0 ** -10 + 2.0 ** -10)


@pytest.mark.parametrize("tokens", [1, 5])
def test_a_captured_step(gpu, tokens):
    """The whole step of single tokens in one graph, replayed as the sequences grow."""
    L = Layer(gpu)
    ids, x, lens = i32([b % 4 - 1 for b in range(tokens)]), randn((tokens, L.K), 8), i32([1] * tokens)
    cache = gpu.make_qcache(4 * tokens, 16, L.H, L.D, 8)
    pages = i32([[4 * b + p for p in range(4)] for b in range(tokens)])
    twin = gpu.make_qcache(4 * tokens, 16, L.H, L.D, 8)
    out = torch.empty((tokens, L.Hq, L.D), dtype=torch.bfloat16, device=DEV)

    def step(c, o):
        q, k, v, _, _ = L.rows(x, ids, None, lens)
        gpu.qcache_write(c, k, v, pages, lens)
        return gpu.qcache_attend(c, q, pages, lens, out=o)
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        step(cache, out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        step(cache, out)
    for n in range(1, 40):
        lens.fill_(n)
        x.copy_(randn((tokens, L.K), 100 + n))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(step(twin, None), out), n
