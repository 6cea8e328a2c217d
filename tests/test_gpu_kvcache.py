"""The quantized, paged KV cache on the GPU against the fp64 oracle: codes and
constants bit for bit, rows read back exactly, attention within the bound of
its roundings."""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import dev, host, say
from kv_util import Batch, bf16, check_attend, dev_bf16, rows

pytestmark = pytest.mark.gpu


def _same_bytes(batch, what=""):
    codes, meta = batch.host_buffers()
    for i, n in enumerate("kv"):
        assert np.array_equal(meta[i], batch.ref.meta[i]), f"{what} {n} constants differ"
        assert np.array_equal(codes[i], batch.ref.codes[i]), f"{what} {n} codes differ"


# ------------------------------------------------------------------- write
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("head_dim", [64, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_write(gpu, bits, head_dim, dtype):
    rng = np.random.default_rng(bits * 1000 + head_dim)
    H = 3
    # whole prompts, one token, nothing, a chunk behind old tokens, more rows than tokens (two have no place)
    b = Batch(rng, [33, 1, 0, 70, 5], [33, 1, 0, 9, 7], 16, H, head_dim, bits, lead=2).device(gpu)
    say(f"write b{bits} d{head_dim} {dtype}")
    x = [rows(rng, (b.T + 3, H, head_dim)) for _ in range(2)]
    if dtype == torch.bfloat16:
        (k, kb), (v, vb) = bf16(x[0]), bf16(x[1])
        K, V = dev_bf16(kb), dev_bf16(vb)
    else:
        k, v = x
        K, V = dev(k), dev(v)
    b.ref.write(k, v, b.pages, b.lens, b.starts)
    gpu.qcache_write(b.cache, K, V, b.d_pages, b.d_lens, b.d_starts)
    _same_bytes(b)


@pytest.mark.parametrize("page_size", [16, 32, 64, 128, 256])
def test_write_single_tokens_strided(gpu, page_size):
    """One token per sequence out of a fused projection; idle sequences and holes in the page table are skipped."""
    rng = np.random.default_rng(page_size)
    H, D = 5, 128
    lens = [1, 16, 17, 0, page_size, page_size + 1, 2 * page_size, 3]
    b = Batch(rng, lens, [1] * len(lens), page_size, H, D, 8, starts=False)
    b.pages[7, 0] = -1
    b.pages[1, 0] = b.n_pages              # outside the cache
    b.device(gpu)
    qkv, bits = bf16(rows(rng, (len(lens), 20 + 2 * H, D)))
    t = dev_bf16(bits)
    b.ref.write(qkv[:, 20:20 + H], qkv[:, 20 + H:], b.pages, b.lens)
    gpu.qcache_write(b.cache, t[:, 20:20 + H], t[:, 20 + H:], b.d_pages, b.d_lens)
    _same_bytes(b)


@pytest.mark.parametrize("bits", [4, 8])
def test_write_special_rows(gpu, bits):
    """Constant, zero, huge, tiny, one-sided, tied and non-finite rows."""
    rng = np.random.default_rng(7)
    D = 64
    x = rng.standard_normal((24, D)).astype(np.float32)
    x[0] = 0
    x[1] = 1.7
    x[2] = -0.0
    x[3] *= 1e5                             # beyond what is stored
    x[4] *= 1e-5
    x[5] *= 1e-7                            # near fp16's smallest
    x[6] *= 1e-12
    x[7] = np.abs(x[7])
    x[8] = -np.abs(x[8])
    x[9, 5] = np.inf
    x[10, 63] = np.nan
    x[11, 0] = -np.inf
    L = (1 << bits) - 1
    x[12] = (np.arange(D) % (2 * L + 1)) * 0.5 - 3          # every half-way point of a grid of steps 1
    x[12, :2] = [-3, L - 3]
    x[13] = (np.arange(D) % (2 * L + 1)) * 0.125
    x[13, :2] = [0, L * 0.25]
    x[14] = 3.0e38
    x[15, 1:] = 0
    x[16] = 65280
    x[16, 3] = -65280
    x[17] = np.float32(1) + np.arange(D) * np.float32(2 ** -20)
    x[18] = -5.5
    x[18, 1] = 2.0 ** -30
    x[19] = 6.1e-5
    x[20] = rng.integers(-3, 4, D) * 2.0 ** -24
    x = x.reshape(24, 1, D)
    b = Batch(rng, [24], [24], 32, 1, D, bits, fill=False).device(gpu)
    b.ref.write(x, x[::-1], b.pages, b.lens, b.starts)
    gpu.qcache_write(b.cache, dev(x), dev(np.ascontiguousarray(x[::-1])), b.d_pages, b.d_lens, b.d_starts)
    codes, meta = b.host_buffers()
    for i in range(2):
        nan = np.isnan(oracle.kvcache.unpack_meta(b.ref.meta[i])[0])
        s, o = oracle.kvcache.unpack_meta(meta[i])
        assert np.array_equal(np.isnan(s), nan) and np.array_equal(np.isnan(o), nan)
        assert np.array_equal(meta[i][~nan], b.ref.meta[i][~nan])
        assert np.array_equal(codes[i], b.ref.codes[i])
    # and back: the non-finite rows read as NaN, the rest as their levels
    K, V = gpu.qcache_read(b.cache, b.d_pages, b.d_lens, b.d_starts, rows=24, dtype=torch.float32)
    k, v, _ = b.ref.read(24, b.pages, b.lens, b.starts)
    for got, want in ((host(K), k), (host(V), v)):
        assert np.array_equal(np.isnan(got), np.isnan(want))
        assert np.array_equal(got[~np.isnan(want)], want.astype(np.float32)[~np.isnan(want)])


def test_cache_is_what_the_group_packer_makes(gpu):
    """4-bit rows of 64 are format-1 groups of 64: qunpack_group reads the cache, qpack_group writes the same bytes."""
    rng = np.random.default_rng(3)
    b = Batch(rng, [64], [64], 64, 1, 64, 4, spare=0, fill=False).device(gpu)
    x = rows(rng, (64, 1, 64))
    gpu.qcache_write(b.cache, dev(x), dev(x), b.d_pages, b.d_lens, b.d_starts)
    codes, meta = gpu.qpack_group(dev(x.reshape(64, 64)), 4, 64)
    assert torch.equal(codes, b.cache._tensors[0]) and torch.equal(meta, b.cache._tensors[1])
    _, w = gpu.qunpack_group(*b.cache._tensors[:2], 64, 64, 4, 64, want_w=True)
    K, _ = gpu.qcache_read(b.cache, b.d_pages, b.d_lens, b.d_starts, rows=64, dtype=torch.float32)
    assert torch.equal(w.view(64, 1, 64), K)


# -------------------------------------------------------------------- read
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("head_dim", [64, 128])
def test_read(gpu, bits, head_dim):
    rng = np.random.default_rng(bits + head_dim)
    H, lens = 2, [40, 0, 1, 100, 3]
    new = [40, 0, 1, 17, 6]                 # the whole, nothing, the tail, more than there is
    b = Batch(rng, lens, new, 32, H, head_dim, bits, lead=3)
    b.pages[3, 2] = -7                      # a hole under the tail
    b.device(gpu)
    say(f"read b{bits} d{head_dim}")
    T = b.T + 4                             # rows behind the last sequence
    k, v, owned = b.ref.read(T, b.pages, b.lens, b.starts)
    for dtype in (torch.float32, torch.bfloat16):
        big = torch.full((T, 2 * H + 1, head_dim), 7.0, dtype=dtype, device="cuda")
        K, V = big[:, :H], big[:, H + 1:]
        gpu.qcache_read(b.cache, b.d_pages, b.d_lens, b.d_starts, K=K, V=V)
        assert torch.all(big[:, H] == 7.0)  # between the slices
        for got, want in ((K, k), (V, v)):
            assert torch.all(got[torch.from_numpy(~owned).cuda()] == 7.0)
            want32 = torch.from_numpy(want.astype(np.float32))
            assert torch.equal(got.cpu()[owned], want32.to(dtype)[owned])


# ------------------------------------------------------------------ attend
def _attend(gpu, b, rng, group, lead_rows=0, scale=None, shared=False, q_mul=1.0):
    H, D = b.geom[2], b.geom[3]
    T = b.T + lead_rows
    q, bits = bf16(q_mul * rng.standard_normal((T, H * group, D)))
    Q = dev_bf16(bits)
    kw = dict(scale=scale)
    if shared:
        call = lambda **k: gpu.qcache_attend_shared(b.cache, Q, b.d_prefix, b.prefix, b.d_pages, b.d_lens, b.d_starts, **kw, **k)  # noqa: E731
        ref, mag, owned = b.ref.attend(q, b.pages, b.lens, b.starts, scale, b.prefix_pages, b.prefix)
    else:
        call = lambda **k: gpu.qcache_attend(b.cache, Q, b.d_pages, b.d_lens, b.d_starts, **kw, **k)  # noqa: E731
        ref, mag, owned = b.ref.attend(q, b.pages, b.lens, b.starts, scale)
    out = torch.full((T, H * group, D), 7.0, device="cuda")
    assert call(out=out) is out
    got = host(out)
    assert np.all(got[~owned] == 7.0), "a row that no sequence owns was written"
    worst = check_attend(b, q, got, ref, mag, owned, D ** -0.5 if scale is None else scale)
    none = owned & (mag[0].max(axis=(1, 2)) == 0)
    assert np.all(got[none] == 0.0)         # rows that see nothing
    o16 = call()
    own = torch.from_numpy(owned).cuda()
    assert torch.equal(o16[own], out[own].bfloat16()), "bf16 output is not the fp32 one rounded"
    assert torch.equal(call(out_dtype=torch.float32)[own], out[own]), "two calls differ"
    return worst


GEOMS = [(16, 2, 128, 8, 8), (16, 2, 128, 4, 8), (64, 1, 64, 8, 4), (32, 3, 64, 4, 1), (256, 1, 128, 8, 5), (128, 2, 64, 4, 16)]


@pytest.mark.parametrize("page_size,heads,head_dim,bits,group", GEOMS)
def test_attend_one_token(gpu, page_size, heads, head_dim, bits, group):
    rng = np.random.default_rng(page_size + head_dim)
    lens = [1, 2, 0, 15, 16, 17, 31, 33, 64, 127, 130, 257, 300]
    say(f"attend one p{page_size} h{heads} d{head_dim} b{bits} g{group}")
    b = Batch(rng, lens, [1] * len(lens), page_size, heads, head_dim, bits, starts=False).device(gpu)
    _attend(gpu, b, rng, group)


@pytest.mark.parametrize("page_size,heads,head_dim,bits,group", GEOMS)
def test_attend_some_tokens(gpu, page_size, heads, head_dim, bits, group):
    """Drafted tokens, chunks, whole prompts, rows without tokens: ragged, causal."""
    rng = np.random.default_rng(page_size * 3 + head_dim)
    say(f"attend some p{page_size} h{heads} d{head_dim} b{bits} g{group}")
    b = Batch(rng, [70, 5, 0, 33, 150, 1], [3, 5, 0, 2, 7, 4], page_size, heads, head_dim, bits, lead=1).device(gpu)
    _attend(gpu, b, rng, group, lead_rows=2)


@pytest.mark.parametrize("page_size,heads,head_dim,bits,group", GEOMS)
def test_attend_chunk(gpu, page_size, heads, head_dim, bits, group):
    rng = np.random.default_rng(page_size * 5 + head_dim)
    say(f"attend chunk p{page_size} h{heads} d{head_dim} b{bits} g{group}")
    b = Batch(rng, [150, 1, 97, 0, 65], [70, 1, 97, 3, 33], page_size, heads, head_dim, bits, lead=5).device(gpu)
    _attend(gpu, b, rng, group, lead_rows=1)


@pytest.mark.parametrize("bits", [4, 8])
def test_attend_long_and_split(gpu, bits):
    """One sequence much longer than the others: the work over its keys is split and joined."""
    rng = np.random.default_rng(bits)
    say(f"attend long b{bits}")
    b = Batch(rng, [6000, 7, 1025], [1, 1, 1], 64, 2, 128, bits, starts=False).device(gpu)
    _attend(gpu, b, rng, 8)
    b = Batch(rng, [2500, 40], [40, 2], 16, 1, 64, bits).device(gpu)
    _attend(gpu, b, rng, 4)


@pytest.mark.parametrize("page_size,heads,head_dim,bits,group", GEOMS)
@pytest.mark.parametrize("prefix", [1, 77, 700])
def test_attend_shared(gpu, page_size, heads, head_dim, bits, group, prefix):
    rng = np.random.default_rng(page_size + prefix)
    say(f"shared p{page_size} h{heads} d{head_dim} b{bits} g{group} prefix {prefix}")
    lens = [1, 0, 40, 129, 16, 3, 64, 0, 17]
    b = Batch(rng, lens, [1] * len(lens), page_size, heads, head_dim, bits, starts=False, prefix=prefix).device(gpu)
    _attend(gpu, b, rng, group, shared=True)
    b = Batch(rng, [90, 5, 0, 33], [12, 5, 0, 2], page_size, heads, head_dim, bits, lead=2, prefix=prefix).device(gpu)
    _attend(gpu, b, rng, group, lead_rows=3, shared=True)


def test_attend_holes(gpu):
    """Pages outside the cache hide their tokens; a sequence of which nothing is left is zero."""
    rng = np.random.default_rng(11)
    for new, starts in (([1, 1, 1], False), ([3, 40, 2], True)):
        b = Batch(rng, [100, 60, 20], new, 16, 2, 128, 8, starts=starts, prefix=50)
        b.pages[0, 1:3] = -1
        b.pages[1, 0] = b.n_pages
        b.pages[1, 3] = 2 ** 31 - 1
        b.pages[2, :] = -2 ** 31
        b.prefix_pages[1] = -5
        b.device(gpu)
        _attend(gpu, b, rng, 4)
        _attend(gpu, b, rng, 4, shared=True)


def test_attend_table_narrower_than_lens(gpu):
    rng = np.random.default_rng(12)
    b = Batch(rng, [100, 20], [1, 1], 16, 1, 64, 8, starts=False)
    b.pages = np.ascontiguousarray(b.pages[:, :3])       # 48 positions; rows 48.. have no place
    b.device(gpu)
    _attend(gpu, b, rng, 2)
    b = Batch(rng, [100, 20], [70, 20], 16, 1, 64, 8)
    b.pages = np.ascontiguousarray(b.pages[:, :3])
    b.device(gpu)
    _attend(gpu, b, rng, 2)


@pytest.mark.parametrize("new", [[1, 1], [5, 3], [60, 40]])
def test_attend_nan_only_where_it_is_seen(gpu, new):
    """NaN rows behind a sequence's end, in its later tokens and in other pages reach nothing else."""
    rng = np.random.default_rng(13)
    H, D, G = 2, 128, 4
    b = Batch(rng, [70, 45], new, 16, H, D, 8)
    nan = np.uint32(0x7E007E00)
    used = np.zeros(b.ref.meta[0].shape, bool)
    for s, n in enumerate(b.lens):
        for p in range(n):
            used[b.pages[s, p // 16], :, p % 16] = True
    for m in b.ref.meta:
        m[~used] = nan                       # every slot that no token holds
    b.device(gpu)
    _attend(gpu, b, rng, G)
    # the last token of sequence 0 goes bad: only the rows that see it are NaN
    page, slot = b.pages[0, 69 // 16], 69 % 16
    for i in range(2):
        keep = b.ref.meta[i].copy()
        b.ref.meta[i][page, 1, slot] = nan
        b.device(gpu)
        q, bits = bf16(rng.standard_normal((b.T, H * G, D)))
        out = host(gpu.qcache_attend(b.cache, dev_bf16(bits), b.d_pages, b.d_lens, b.d_starts, out_dtype=torch.float32))
        bad = np.isnan(out).any(-1)
        want = np.zeros_like(bad)
        want[new[0] - 1, G:2 * G] = True
        assert np.array_equal(bad, want), (i, np.argwhere(bad != want)[:5])
        b.ref.meta[i][:] = keep


def test_attend_large_and_small_logits(gpu):
    """Logits of hundreds (one key takes all), all equal logits, and a scale of zero."""
    rng = np.random.default_rng(14)
    for lens, new in (([200, 33], [1, 1]), ([200, 90], [50, 90])):
        b = Batch(rng, lens, new, 32, 1, 128, 8).device(gpu)
        _attend(gpu, b, rng, 4, scale=0.0)
        _attend(gpu, b, rng, 4, scale=-0.05)
        _attend(gpu, b, rng, 4, q_mul=1e-3)
        # logits of hundreds: the bound's logit term is no bound any more, the largest logit decides
        q, bits = bf16(60 * rng.standard_normal((b.T, 4, 128)))
        out = host(gpu.qcache_attend(b.cache, dev_bf16(bits), b.d_pages, b.d_lens, b.d_starts, out_dtype=torch.float32))
        ref, _, _ = b.ref.attend(q, b.pages, b.lens, b.starts)
        assert np.isfinite(out).all()
        # a row whose two largest logits are 4 or more apart than the logits' error (2^-10 A) is its key's value
        # up to weights below e^-4 that the reference has as well: compare those that are clear by 20
        A = 60 * 6.0
        clear = 0
        kv = b.ref.values(0)
        for t, s, pos in b.ref.rows(b.lens, b.starts):
            k = np.stack([kv[b.pages[s, j // 32], 0, j % 32] for j in range(pos + 1)])
            z = np.sort((q[t] @ k.T) * 128 ** -0.5, axis=1)
            for g in range(4):
                if pos == 0 or z[g, -1] - z[g, -2] > 20 + A * 2.0 ** -9:
                    clear += 1
                    assert np.allclose(out[t, g], ref[t, g], rtol=2.0 ** -10, atol=2.0 ** -9)
        assert clear > 0


# ------------------------------------------------------- the set in its use
def test_prompts_then_tokens(gpu):
    """Prompts enter the cache, are attended to in chunks, then tokens are appended one by one: every step's bytes
    and outputs against the oracle."""
    rng = np.random.default_rng(21)
    H, D, G, P = 2, 128, 4, 16
    total, prompt, chunk = [61, 30, 47], [50, 20, 40], 23
    b = Batch(rng, total, [1, 1, 1], P, H, D, 8, fill=False).device(gpu)
    lens = np.zeros(3, np.int32)
    x = [[bf16(rows(rng, (n, h, D))) for n in total] for h in (H, H, H * G)]
    while not np.array_equal(lens, total):
        new = [min(chunk, p - n) if n < p else (1 if n < t else 0) for n, p, t in zip(lens, prompt, total)]
        part = [np.concatenate([x[i][s][0][lens[s]:lens[s] + new[s]] for s in range(3)]) for i in range(3)]
        dpart = [dev_bf16(np.concatenate([x[i][s][1][lens[s]:lens[s] + new[s]] for s in range(3)])) for i in range(3)]
        lens = (lens + new).astype(np.int32)
        starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        b.ref.write(part[0], part[1], b.pages, lens, starts)
        gpu.qcache_write(b.cache, dpart[0], dpart[1], b.d_pages, dev(lens), dev(starts))
        _same_bytes(b)
        out = host(gpu.qcache_attend(b.cache, dpart[2], b.d_pages, dev(lens), dev(starts), out_dtype=torch.float32))
        ref, mag, owned = b.ref.attend(part[2], b.pages, lens, starts)
        check_attend(b, part[2], out, ref, mag, owned, D ** -0.5)


def test_shared_is_the_concatenation(gpu):
    """Attention behind a shared prefix equals attention over page tables that begin with the prefix's pages."""
    rng = np.random.default_rng(22)
    H, D, G, P = 2, 64, 8, 32
    pre = 3 * P
    b = Batch(rng, [40, 1, 77], [1, 1, 1], P, H, D, 4, starts=False, prefix=pre).device(gpu)
    q, bits = bf16(rng.standard_normal((3, H * G, D)))
    one = host(gpu.qcache_attend_shared(b.cache, dev_bf16(bits), b.d_prefix, pre, b.d_pages, b.d_lens, out_dtype=torch.float32))
    joined = np.concatenate([np.tile(b.prefix_pages, (3, 1)), b.pages], 1).astype(np.int32)
    lens = (b.lens + pre).astype(np.int32)
    two = host(gpu.qcache_attend(b.cache, dev_bf16(bits), dev(joined), dev(lens), out_dtype=torch.float32))
    ref, mag, owned = b.ref.attend(q, joined, lens)
    check_attend(b, q, one, ref, mag, owned, D ** -0.5)
    check_attend(b, q, two, ref, mag, owned, D ** -0.5)


# ----------------------------------------------------- streams and capture
def _capture(fn):
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        with torch.cuda.graph(g, stream=s):
            fn()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    return g


def test_captured_step(gpu):
    """A decode step (write, attend, attend behind a prefix) captured once and replayed while the sequences grow."""
    rng = np.random.default_rng(31)
    H, D, G, P, B = 2, 128, 8, 16, 3
    b = Batch(rng, [700, 40, 95], [1] * B, P, H, D, 8, starts=False, prefix=100).device(gpu)
    lens = dev(np.array([600, 1, 60], np.int32))
    K, V, Q = (torch.empty((B, n, D), dtype=torch.bfloat16, device="cuda") for n in (H, H, H * G))
    out = [torch.empty((B, H * G, D), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    ws = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in (
        gpu.qcache_attend_ws(b.cache, B, B, b.pages.shape[1], H * G),
        gpu.qcache_attend_ws(b.cache, B, B, b.pages.shape[1], H * G, 100))]

    def step(o, w):
        gpu.qcache_write(b.cache, K, V, b.d_pages, lens)
        gpu.qcache_attend(b.cache, Q, b.d_pages, lens, out=o[0], ws=w[0])
        gpu.qcache_attend_shared(b.cache, Q, b.d_prefix, 100, b.d_pages, lens, out=o[1], ws=w[1])

    K.normal_(), V.normal_(), Q.normal_()
    step(out, ws)
    torch.cuda.synchronize()
    g = _capture(lambda: step(out, ws))
    for i in range(4):
        lens += 1
        K.normal_(), V.normal_(), Q.normal_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        got, cache = [o.clone() for o in out], [t.clone() for t in b.cache._tensors]
        eager = [torch.empty_like(o) for o in out]
        step(eager, [None, None])
        for a, e in zip(got + cache, eager + list(b.cache._tensors)):
            assert torch.equal(a, e), f"replay {i}"


def test_other_stream(gpu):
    """An explicit stream that is not the current one: temporaries stay alive until it is done with them."""
    rng = np.random.default_rng(32)
    b = Batch(rng, [500, 60], [1, 1], 16, 2, 128, 4, starts=False).device(gpu)
    q, bits = bf16(rng.standard_normal((2, 16, 128)))
    Q = dev_bf16(bits)
    want = gpu.qcache_attend(b.cache, Q, b.d_pages, b.d_lens)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    outs = []
    for _ in range(4):
        outs.append(gpu.qcache_attend(b.cache, Q, b.d_pages, b.d_lens, stream=s))
        torch.full((1 << 20,), 255, dtype=torch.uint8, device="cuda")     # would reuse a freed workspace
    K, V = gpu.qcache_read(b.cache, b.d_pages, b.d_lens, stream=s)
    s.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    k, v, _ = b.ref.read(2, b.pages, b.lens)
    assert torch.equal(K.cpu(), torch.from_numpy(k.astype(np.float32)).bfloat16())
    assert torch.equal(V.cpu(), torch.from_numpy(v.astype(np.float32)).bfloat16())


def test_two_streams_at_once(gpu):
    rng = np.random.default_rng(33)
    b = Batch(rng, [3000, 60], [1, 1], 64, 2, 128, 8, starts=False).device(gpu)
    Q = [dev_bf16(bf16(rng.standard_normal((2, 16, 128)))[1]) for _ in range(2)]
    want = [gpu.qcache_attend(b.cache, q, b.d_pages, b.d_lens) for q in Q]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            outs[i].append(gpu.qcache_attend(b.cache, Q[i], b.d_pages, b.d_lens, stream=s))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i]) for o in outs[i])


def test_bad_starts_stay_in_bounds(gpu):
    """starts that do not ascend or leave the rows own what they say, and nothing outside the buffers is touched."""
    rng = np.random.default_rng(34)
    b = Batch(rng, [30, 40, 20], [4, 4, 4], 16, 1, 64, 8).device(gpu)
    q, bits = bf16(rng.standard_normal((12, 4, 64)))
    for starts in ([5, 3, 9, 2], [-4, 2, 6, 100], [0, 0, 0, 0], [2 ** 31 - 1, -2 ** 31, 7, 12]):
        st = dev(np.array(starts, np.int32))
        guard = torch.full((14, 4, 64), 7.0, device="cuda")
        gpu.qcache_attend(b.cache, dev_bf16(bits), b.d_pages, b.d_lens, st, out=guard[1:13])
        gpu.qcache_read(b.cache, b.d_pages, b.d_lens, st, K=guard[1:13, :1], V=guard[1:13, 1:2])
        torch.cuda.synchronize()
        assert torch.all(guard[0] == 7.0) and torch.all(guard[13] == 7.0)
