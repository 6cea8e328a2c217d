"""Attention over the KV cache on every path a call can take: each tile height,
keys decoded beforehand, many sequences, far pages, strided rows, the same page
in several tables, captured ragged calls."""
import numpy as np
import pytest
import torch

from gpu_util import dev, host, say
from kv_util import Batch, bf16, check_attend, dev_bf16, rows

pytestmark = pytest.mark.gpu

NAN = np.uint32(0x7E007E00)


def _nan_where_no_token_is(b):
    """Slots that no token holds are NaN: nothing may come of them."""
    P = b.geom[1]
    used = np.zeros(b.ref.meta[0].shape, bool)
    for s, n in enumerate(b.lens):
        for p in range(0, int(n), P):
            if 0 <= b.pages[s, p // P] < b.n_pages:
                used[b.pages[s, p // P], :, :min(P, int(n) - p)] = True
    for i in range(b.prefix):
        used[b.prefix_pages[i // P], :, i % P] = True
    for m in b.ref.meta:
        m[~used] = NAN


def _attend(gpu, b, rng, group, extra=0, shared=False):
    H, D = b.geom[2], b.geom[3]
    q, bits = bf16(rng.standard_normal((b.T + extra, H * group, D)))
    Q = dev_bf16(bits)
    out = torch.full(Q.shape, 7.0, device="cuda")
    if shared:
        gpu.qcache_attend_shared(b.cache, Q, b.d_prefix, b.prefix, b.d_pages, b.d_lens, b.d_starts, out=out)
        ref, mag, owned = b.ref.attend(q, b.pages, b.lens, b.starts, None, b.prefix_pages, b.prefix)
    else:
        gpu.qcache_attend(b.cache, Q, b.d_pages, b.d_lens, b.d_starts, out=out)
        ref, mag, owned = b.ref.attend(q, b.pages, b.lens, b.starts)
    got = host(out)
    assert np.all(got[~owned] == 7.0)
    check_attend(b, q, got, ref, mag, owned, D ** -0.5)
    assert np.all(got[owned & (mag[0].max(axis=(1, 2)) == 0)] == 0.0)
    return got


# rows of a KV head and sequence on average: 12, 26, 86, 256, 884
@pytest.mark.parametrize("tokens", [6, 15, 50, 150, 520])
@pytest.mark.parametrize("head_dim", [64, 128])
@pytest.mark.parametrize("bits", [4, 8])
def test_every_height(gpu, tokens, head_dim, bits):
    rng = np.random.default_rng(tokens * 7 + head_dim + bits)
    say(f"height {tokens} tokens d{head_dim} b{bits}")
    new = [tokens + 3, 0, tokens - 3, tokens + tokens // 2, tokens // 2]
    lens = [tokens + 1703, 0, tokens - 3, tokens // 2 + 77, tokens // 2 + 401]    # the fourth has rows before its start
    new = [n + tokens // 4 + 1 for n in new[:1]] + new[1:]
    b = Batch(rng, lens, new, 32, 1, head_dim, bits, lead=2)
    b.pages[4, 1] = -3                     # a hole
    _nan_where_no_token_is(b)
    _attend(gpu, b.device(gpu), rng, 2, extra=3)


@pytest.mark.parametrize("page_size", [16, 64, 256])
@pytest.mark.parametrize("head_dim", [64, 128])
@pytest.mark.parametrize("bits", [4, 8])
def test_decoded_beforehand(gpu, page_size, head_dim, bits):
    """Whole prompts whose keys are decoded once for all tiles: page and step boundaries, holes, a sequence of one token."""
    rng = np.random.default_rng(page_size)
    b = Batch(rng, [257, 1, 128, 640], [257, 1, 128, 200], page_size, 2, head_dim, bits)
    b.pages[3, 0] = b.n_pages
    if page_size == 16:
        b.pages[0, 5] = -1
    _nan_where_no_token_is(b)
    _attend(gpu, b.device(gpu), rng, 16)


def test_rows_of_sequences_that_are_not_whole_tiles(gpu):
    """Groups that do not divide a tile, up to 64 query heads for a KV head."""
    for group, new in ((3, [1, 1, 1]), (7, [4, 1, 9]), (64, [1, 1, 1]), (64, [3, 7, 1]), (11, [61, 30, 7])):
        rng = np.random.default_rng(group + new[0])
        say(f"group {group} {new}")
        b = Batch(rng, [130, 31, 900], new, 16, 1, 128, 8, prefix=33)
        _nan_where_no_token_is(b)
        b.device(gpu)
        _attend(gpu, b, rng, group)
        _attend(gpu, b, rng, group, shared=True)


@pytest.mark.parametrize("page_size,width", [(16, 8), (64, 40)])
def test_many_sequences(gpu, page_size, width):
    """More sequences than a wave has lanes, idle ones among them; short page tables and long ones."""
    rng = np.random.default_rng(page_size)
    B = 150
    lens = [int(n) for n in rng.integers(0, 129, B)]
    lens[3] = lens[64] = lens[149] = 0
    if width == 40:
        lens[70] = 2300
    b = Batch(rng, lens, [1] * B, page_size, 1, 64, 8, starts=False, width=width, prefix=70)
    _nan_where_no_token_is(b)
    b.device(gpu)
    _attend(gpu, b, rng, 2)
    _attend(gpu, b, rng, 2, shared=True)
    new = [min(n, int(k)) for n, k in zip(lens, rng.integers(0, 5, B))]
    r = Batch(rng, lens, new, page_size, 1, 64, 4, width=width, prefix=70)
    _nan_where_no_token_is(r)
    r.device(gpu)
    _attend(gpu, r, rng, 4)
    _attend(gpu, r, rng, 4, shared=True)


def test_many_rows_of_many_sequences(gpu):
    """Ragged chunks of 70 sequences, keys decoded beforehand: steps are counted over more than 64 sequences."""
    rng = np.random.default_rng(70)
    new = [int(n) for n in rng.integers(20, 60, 70)]
    lens = [n + int(k) for n, k in zip(new, rng.integers(0, 150, 70))]
    b = Batch(rng, lens, new, 16, 1, 64, 8)
    _nan_where_no_token_is(b)
    _attend(gpu, b.device(gpu), rng, 64)


def test_far_pages(gpu):
    """Codes behind 2^32 bytes: the same tokens in a small cache and at the end of a large one, bit for bit."""
    H, D, P, B = 1, 128, 256, 3
    small = gpu.make_qcache(8, P, H, D, 8, device="cuda")
    n = 2 ** 32 // (P * D) + 40
    far = gpu.make_qcache(n, P, H, D, 8, device="cuda")
    assert far._tensors[0].numel() > 2 ** 32
    torch.manual_seed(1)
    pages = torch.tensor([[0, 3], [5, 6], [7, 1]], dtype=torch.int32, device="cuda")
    far_pages = n - 1 - pages * 3
    lens = torch.tensor([300, 512, 20], dtype=torch.int32, device="cuda")
    starts = torch.tensor([0, 300, 812, 832], dtype=torch.int32, device="cuda")
    K, V = (torch.randn(832, H, D, device="cuda").bfloat16() for _ in range(2))
    for c, p in ((small, pages), (far, far_pages)):
        gpu.qcache_write(c, K, V, p, lens, starts)
    both = [gpu.qcache_read(c, p, lens, starts, rows=832) for c, p in ((small, pages), (far, far_pages))]
    assert torch.equal(both[0][0], both[1][0]) and torch.equal(both[0][1], both[1][1])
    assert torch.count_nonzero(both[0][0]) > 0
    for T, st, group in ((B, None, 8), (832, starts, 2), (832, starts, 8)):      # few rows, tiles, decoded beforehand
        Q = torch.randn(T, H * group, D, device="cuda").bfloat16()
        a, b = (gpu.qcache_attend(c, Q, p, lens, st) for c, p in ((small, pages), (far, far_pages)))
        assert torch.equal(a, b)
        a, b = (gpu.qcache_attend_shared(c, Q, p[1], 260, p, lens, st) for c, p in ((small, pages), (far, far_pages)))
        assert torch.equal(a, b)


def test_strided_rows(gpu):
    """Queries out of a fused projection, outputs into a slice: the rest of it stays."""
    rng = np.random.default_rng(5)
    H, D, G = 2, 64, 4
    for lens, new in (([40, 300], [1, 1]), ([70, 300], [70, 60])):
        b = Batch(rng, lens, new, 16, H, D, 8).device(gpu)
        q, bits = bf16(rng.standard_normal((b.T, H * G + 3, D)))
        fused = dev_bf16(bits)
        ref, mag, owned = b.ref.attend(q[:, 1:1 + H * G], b.pages, b.lens, b.starts)
        big = torch.full((b.T, H * G + 2, D), 7.0, device="cuda")
        gpu.qcache_attend(b.cache, fused[:, 1:1 + H * G], b.d_pages, b.d_lens, b.d_starts, out=big[:, 1:1 + H * G])
        assert torch.all(big[:, 0] == 7.0) and torch.all(big[:, -1] == 7.0)
        check_attend(b, q[:, 1:1 + H * G], host(big[:, 1:1 + H * G].contiguous()), ref, mag, owned, D ** -0.5)


def test_the_same_pages_in_several_tables(gpu):
    """Two sequences that share all pages, one that lists a page twice, a prefix that is also somebody's own page."""
    rng = np.random.default_rng(6)
    for new, starts in (([1, 1, 1], False), ([30, 9, 20], True)):
        b = Batch(rng, [60, 60, 64], new, 16, 2, 128, 4, starts=starts, prefix=32)
        b.pages[1] = b.pages[0]
        b.pages[2, 2] = b.pages[2, 1]
        b.prefix_pages[0] = b.pages[0, 0]
        b.device(gpu)
        _attend(gpu, b, rng, 4)
        _attend(gpu, b, rng, 4, shared=True)


@pytest.mark.parametrize("tokens", [4, 40, 150])
def test_captured_ragged(gpu, tokens):
    """Chunks captured once and replayed with other lens and starts: the work is divided on the device."""
    rng = np.random.default_rng(tokens)
    H, D, G, B = 1, 64, 16, 4
    b = Batch(rng, [tokens * 5] * B, [tokens] * B, 16, H, D, 8, prefix=50).device(gpu)
    T = tokens * B
    Q = torch.empty(T, H * G, D, dtype=torch.bfloat16, device="cuda")
    out = [torch.full((T, H * G, D), 7.0, device="cuda") for _ in range(2)]
    lens, starts = torch.zeros_like(b.d_lens), torch.zeros(B + 1, dtype=torch.int32, device="cuda")

    def both(o):
        gpu.qcache_attend(b.cache, Q, b.d_pages, lens, starts, out=o[0])
        gpu.qcache_attend_shared(b.cache, Q, b.d_prefix, b.prefix, b.d_pages, lens, starts, out=o[1])

    Q.normal_()
    both(out)
    torch.cuda.synchronize()
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        with torch.cuda.graph(g, stream=s):
            both(out)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    for i in range(4):
        cut = np.sort(rng.integers(0, T + 1, B - 1))
        n = np.diff(np.concatenate([[0], cut, [T]]))
        starts.copy_(dev(np.concatenate([[0], np.cumsum(n)]).astype(np.int32)))
        lens.copy_(dev(np.minimum(n + rng.integers(0, 3 * tokens, B), 5 * tokens).astype(np.int32)))
        Q.normal_()
        for o in out:
            o.fill_(7.0)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        eager = [torch.full_like(o, 7.0) for o in out]
        both(eager)
        for a, e in zip(out, eager):
            assert torch.equal(a, e), f"replay {i}"
        ref, mag, owned = b.ref.attend(host(Q.float()).astype(np.float64), b.pages, host(lens), host(starts))
        check_attend(b, host(Q.float()).astype(np.float64), host(out[0]), ref, mag, owned, D ** -0.5)


def test_write_then_read_grows_page_by_page(gpu):
    """One token at a time over three pages: every earlier row stays as it was."""
    rng = np.random.default_rng(9)
    H, D, P, n = 3, 64, 16, 40
    b = Batch(rng, [n, n - 9], [1, 1], P, H, D, 4, starts=False, fill=False).device(gpu)
    x, bits = bf16(rows(rng, (n, 2, H, D)))
    before = None
    for i in range(9, n):
        lens = dev(np.array([i + 1, i - 8], np.int32))
        t = dev_bf16(bits[i])
        gpu.qcache_write(b.cache, t, t, b.d_pages, lens)
        b.ref.write(x[i], x[i], b.pages, np.array([i + 1, i - 8]))
        K, V = gpu.qcache_read(b.cache, b.d_pages, lens, dev(np.array([0, i - 8, 2 * (i - 8)], np.int32)),
                               rows=2 * (i - 8), dtype=torch.float32)
        assert torch.equal(K, V)
        if before is not None:
            assert torch.equal(K.view(2, i - 8, H, D)[:, :-1], before)
        before = K.view(2, i - 8, H, D)
    codes, meta = b.host_buffers()
    for i in range(2):
        assert np.array_equal(meta[i], b.ref.meta[i]) and np.array_equal(codes[i], b.ref.codes[i])


@pytest.mark.parametrize("power", [-40, 50])
def test_query_range(gpu, power):
    """Queries far from 1 with a scale that brings the logits back: few rows and many."""
    rng = np.random.default_rng(power + 100)
    for lens, new in (([300, 33], [1, 1]), ([200, 90], [50, 90])):
        b = Batch(rng, lens, new, 32, 1, 128, 8).device(gpu)
        q, bits = bf16(rng.standard_normal((b.T, 4, 128)) * 2.0 ** power)
        scale = 128 ** -0.5 * 2.0 ** -power
        out = host(gpu.qcache_attend(b.cache, dev_bf16(bits), b.d_pages, b.d_lens, b.d_starts, scale=scale,
                                     out_dtype=torch.float32))
        ref, mag, owned = b.ref.attend(q, b.pages, b.lens, b.starts, scale)
        check_attend(b, q, out, ref, mag, owned, scale)


@pytest.mark.parametrize("below", [10.4, 24.6, 31.0])
@pytest.mark.parametrize("new", [1, 60])
def test_many_small_weights(gpu, below, new):
    """One key far above all the others, whose weights of 2^-below each make the whole output: the first key's value
    is zero, all others are one."""
    rng = np.random.default_rng(1)
    n, H, D, G = 3000, 1, 128, 4
    b = Batch(rng, [n], [new], 64, H, D, 8, fill=False)
    k, v = np.zeros((n, H, D)), np.ones((n, H, D))
    k[0], v[0] = 1.0, 0.0
    b.ref.write(k, v, b.pages, b.lens, np.array([0, n]))
    b.device(gpu)
    q, bits = bf16(np.full((new, H * G, D), below * np.log(2) * 128 ** -0.5))
    out = host(gpu.qcache_attend(b.cache, dev_bf16(bits), b.d_pages, b.d_lens, b.d_starts, out_dtype=torch.float32))
    ref, mag, owned = b.ref.attend(q, b.pages, b.lens, b.starts)
    assert ref.max() < 1e-3 * 2.0 ** (10.4 - below) * 3000
    check_attend(b, q, out, ref, mag, owned, 128 ** -0.5)


def test_queries_that_are_not_finite(gpu):
    """A query row with a NaN or an infinity comes out not finite, the rows beside it as ever."""
    rng = np.random.default_rng(2)
    for lens, new in (([300, 33], [1, 1]), ([200, 90], [50, 90])):
        b = Batch(rng, lens, new, 32, 2, 64, 8).device(gpu)
        q, bits = bf16(rng.standard_normal((b.T, 8, 64)))
        bits = bits.copy()
        bad = np.zeros((b.T, 8), bool)
        for t, h, word in ((0, 1, 0x7FC0), (1, 6, 0x7F80), (b.T - 1, 3, 0xFF80)):
            bits[t, h, 5] = word
            bad[t, h] = True
        out = host(gpu.qcache_attend(b.cache, dev_bf16(bits), b.d_pages, b.d_lens, b.d_starts, out_dtype=torch.float32))
        ref, mag, owned = b.ref.attend(q, b.pages, b.lens, b.starts)
        assert not np.isfinite(out[bad]).all(-1).any()
        out[bad] = ref[bad]
        check_attend(b, q, out, ref, mag, owned, 64 ** -0.5)


@pytest.mark.parametrize("lens", [[30, 3], [1700, 3]])
def test_long_prefix_for_few(gpu, lens):
    """A prefix much longer than what follows it, cut into many parts; own tables short (one launch) and long."""
    for bits, group in ((8, 8), (4, 16), (8, 2)):
        rng = np.random.default_rng(bits * group)
        b = Batch(rng, lens, [1, 1], 64, 2, 128, bits, starts=False, prefix=5003)
        _nan_where_no_token_is(b)
        _attend(gpu, b.device(gpu), rng, group, shared=True)


def test_more_heads_than_workgroups(gpu):
    rng = np.random.default_rng(600)
    b = Batch(rng, [40, 7], [1, 1], 16, 600, 64, 8, starts=False, prefix=20).device(gpu)
    _attend(gpu, b, rng, 2)
    _attend(gpu, b, rng, 2, shared=True)
    b = Batch(rng, [170, 7], [30, 1], 16, 600, 64, 4, prefix=20).device(gpu)
    _attend(gpu, b, rng, 2)
    _attend(gpu, b, rng, 2, shared=True)
    x, bits = bf16(rows(rng, (31, 600, 64)))
    b.ref.write(x, x, b.pages, b.lens, b.starts)
    gpu.qcache_write(b.cache, dev_bf16(bits), dev_bf16(bits), b.d_pages, b.d_lens, b.d_starts)
    codes, meta = b.host_buffers()
    for i in range(2):
        assert np.array_equal(meta[i], b.ref.meta[i]) and np.array_equal(codes[i], b.ref.codes[i])


def test_lens_that_make_no_sense(gpu):
    """Negative and huge lengths: nothing, and as far as the table goes."""
    rng = np.random.default_rng(8)
    lo, hi = -2 ** 31, 2 ** 31 - 1
    for new, starts in (([1] * 5, False), ([9, 4, 30, 1, 2], True)):
        b = Batch(rng, [33, 48, 20, 48, 5], new, 16, 2, 64, 8, starts=starts, prefix=20).device(gpu)
        b.lens = np.array([lo, hi, -1, 1000, 5], np.int32)
        b.d_lens = dev(b.lens)
        _attend(gpu, b, rng, 4)
        _attend(gpu, b, rng, 4, shared=True)
        T = b.T
        K, V = gpu.qcache_read(b.cache, b.d_pages, b.d_lens, b.d_starts, rows=T, dtype=torch.float32)
        k, v, owned = b.ref.read(T, b.pages, b.lens, b.starts)
        assert owned.all() and np.array_equal(host(K), k.astype(np.float32)) and np.array_equal(host(V), v.astype(np.float32))


@pytest.mark.parametrize("B", [1, 2, 3, 7])
def test_few_long_sequences(gpu, B):
    """A few sequences with many workgroups each, of very different lengths, some without tokens: one row and more."""
    rng = np.random.default_rng(B)
    lens = [4001, 1, 2047, 0, 129, 3100, 640][:B]
    for bits, group, new in ((8, 8, 1), (4, 5, 3), (8, 4, 7), (4, 16, 1)):
        say(f"{B} sequences, b{bits} g{group}, {new} tokens")
        b = Batch(rng, lens, [min(n, new) if new > 1 else 1 for n in lens], 16, 2, 128 if bits == 8 else 64, bits,
                  starts=new > 1)
        _nan_where_no_token_is(b)
        _attend(gpu, b.device(gpu), rng, group)
