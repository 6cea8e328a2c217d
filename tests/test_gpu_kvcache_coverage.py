"""Attention over the KV cache counts every key a row sees once, on every path:
whole tiles, tiles cut anywhere, pieces of one tile, keys decoded beforehand,
a prefix in front of each."""
import numpy as np
import pytest
import torch

from gpu_util import host, say
from kv_cover import CASES, make
from kv_util import Batch, bf16, check_attend, dev_bf16

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name", CASES)
def test_every_key_once(gpu, name):
    say(name)
    b, group = make(name)
    b.device(gpu)
    H, D = b.geom[2], b.geom[3]
    rng = np.random.default_rng(1)
    Q = dev_bf16(bf16(rng.standard_normal((b.T, H * group, D)))[1])
    for shared in ([False, True] if b.prefix else [False]):
        out = torch.full(Q.shape, 7.0, device="cuda")
        if shared:
            gpu.qcache_attend_shared(b.cache, Q, b.d_prefix, b.prefix, b.d_pages, b.d_lens, b.d_starts, out=out)
        else:
            gpu.qcache_attend(b.cache, Q, b.d_pages, b.d_lens, b.d_starts, out=out)
        got = host(out).astype(np.float64)
        counts, owned = b.counts(shared)
        assert np.all(got[~owned] == 7.0)
        for h in range(H * group):
            bad = b.wrong(got[owned, h], counts[owned]) | ~np.isfinite(got[owned, h])
            assert not bad.any(), (shared, h, np.argwhere(bad)[:5])


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("head_dim", [64, 128])
def test_decoded_beforehand_behind_a_prefix(gpu, bits, head_dim):
    """Prompts whose keys are decoded once for all their tiles, behind a prefix, against the oracle; slots without a
    token are NaN."""
    rng = np.random.default_rng(bits + head_dim)
    b = Batch(rng, [300, 150, 1], [70, 40, 1], 16, 1, head_dim, bits, prefix=210, lead=1)
    used = np.zeros(b.ref.meta[0].shape, bool)
    for table, n in [(b.pages[s], n) for s, n in enumerate(b.lens)] + [(b.prefix_pages, 210)]:
        for j in range(int(n)):
            used[table[j // 16], :, j % 16] = True
    for m in b.ref.meta:
        m[~used] = np.uint32(0x7E007E00)
    b.device(gpu)
    q, qb = bf16(rng.standard_normal((b.T, 64, head_dim)))     # 37 rows a sequence on average, 64 heads: 2368 rows
    out = torch.full((b.T, 64, head_dim), 7.0, device="cuda")
    gpu.qcache_attend_shared(b.cache, dev_bf16(qb), b.d_prefix, 210, b.d_pages, b.d_lens, b.d_starts, out=out)
    ref, mag, owned = b.ref.attend(q, b.pages, b.lens, b.starts, None, b.prefix_pages, 210)
    got = host(out)
    assert np.all(got[~owned] == 7.0)
    check_attend(b, q, got, ref, mag, owned, head_dim ** -0.5)
