"""Attention over the KV cache at the ends of its arguments' ranges."""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import host, say
from kv_util import Batch, bf16, check_attend, dev_bf16

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("sign", [1, -1])
def test_largest_scale_and_rows(gpu, bits, sign):
    """A scale of 2^45 over keys of +-65280, whose s is the largest there is, and queries that bring the logits back;
    few rows and many."""
    rng = np.random.default_rng(bits)
    for lens, new in (([300, 33], [1, 1]), ([200, 90], [50, 90])):
        say(f"scale {sign} * 2^45, b{bits}, {new}")
        b = Batch(rng, lens, new, 32, 1, 128, bits, fill=False)
        n = sum(lens)
        k = rng.uniform(-65280, 65280, (n, 1, 128))
        k[:, :, 100:102] = 65280.0, -65280.0
        b.ref.write(k, rng.standard_normal((n, 1, 128)), b.pages, b.lens, np.concatenate([[0], np.cumsum(lens)]))
        b.device(gpu)
        x = np.zeros((b.T, 4, 128))
        for i in range(4):                   # scale sum |q||k| is at most 128 then
            x[:, i, [3 + i, 40, 77, 127 - i]] = 2.0 ** -56 * rng.choice([-1, 1], (b.T, 4))
        q, qb = bf16(x)
        scale = sign * 2.0 ** 45
        out = host(gpu.qcache_attend(b.cache, dev_bf16(qb), b.d_pages, b.d_lens, b.d_starts, scale=scale,
                                     out_dtype=torch.float32))
        ref, mag, owned = b.ref.attend(q, b.pages, b.lens, b.starts, scale)
        check_attend(b, q, out, ref, mag, owned, scale)


@pytest.mark.parametrize("bits", [4, 8])
def test_buffers_filled_by_hand(gpu, bits):
    """Constants at the ends of their range, of either sign, and codes as they come: few rows, many, and read back."""
    rng = np.random.default_rng(bits)
    top = (1 << bits) - 1
    for lens, new in (([300, 33], [1, 1]), ([200, 90], [50, 90])):
        b = Batch(rng, lens, new, 32, 1, 64, bits, fill=False)
        shape = b.ref.meta[0].shape
        for i in range(2):
            sign = rng.choice([-1.0, 1.0], shape)
            s = np.nextafter(np.float16(2 * 65504 / top), np.float16(0))          # s * top - 65504 stays below 65504
            s = np.where(rng.random(shape) < 0.5, s, np.float16(0.01)).astype(np.float16)
            o = np.where(s > 1, np.float16(-65504), rng.choice([-65504, 0, 3, 65000], shape)).astype(np.float16)
            s, o = (sign * s).astype(np.float16), (sign * o).astype(np.float16)
            assert np.abs(s.astype(np.float64) * top + o.astype(np.float64)).max() <= 65504
            b.ref.meta[i][:] = oracle.kvcache.pack_meta(s, o)
            b.ref.codes[i][:] = oracle.kvcache.pack_codes(rng.integers(0, top + 1, shape + (64,)).astype(np.uint8), bits)
        b.device(gpu)
        say(f"by hand b{bits} {new}")
        q, qb = bf16(rng.standard_normal((b.T, 4, 64)))
        out = host(gpu.qcache_attend(b.cache, dev_bf16(qb), b.d_pages, b.d_lens, b.d_starts, scale=1e-5,
                                     out_dtype=torch.float32))
        ref, mag, owned = b.ref.attend(q, b.pages, b.lens, b.starts, 1e-5)
        check_attend(b, q, out, ref, mag, owned, 1e-5)
        K, V = gpu.qcache_read(b.cache, b.d_pages, b.d_lens, b.d_starts, rows=b.T, dtype=torch.float32)
        k, v, _ = b.ref.read(b.T, b.pages, b.lens, b.starts)
        assert np.array_equal(host(K), k.astype(np.float32)) and np.array_equal(host(V), v.astype(np.float32))
