"""Attention over the KV cache at the ends of its arguments' ranges."""
import numpy as np
import pytest
import torch

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
