"""The marked batches on the CPU: what they expect is what the oracle computes,
and one key too few or too many is outside their tolerance."""
import numpy as np
import pytest

from kv_cover import CASES, Marked, make


@pytest.mark.parametrize("prefix", [0, 35])
def test_expected_is_the_oracle(prefix):
    rng = np.random.default_rng(3)
    b = Marked(rng, [70, 3, 0, 41], [5, 3, 2, 40], 16, 2, 64, 8, holes=[(0, 1)], prefix=prefix, lead=1)
    q = rng.standard_normal((b.T, 4, 64))
    args = (b.prefix_pages, prefix) if prefix else (None, 0)
    out, _, owned = b.ref.attend(q, b.pages, b.lens, b.starts, None, *args)
    counts, own = b.counts(bool(prefix))
    assert np.array_equal(owned, own)
    assert np.allclose(out[own], b.expected(counts)[own][:, None], rtol=1e-12, atol=0)


@pytest.mark.parametrize("name", CASES)
def test_one_key_shows(name):
    """Every mark a row sees, with one of its keys left out or counted twice: the row's output is noticed as wrong."""
    b, _ = make(name)
    counts, owned = b.counts(b.prefix > 0)
    counts = counts[owned & (counts.sum(1) > 1)]
    if len(counts) > 40:
        counts = counts[np.unique(np.linspace(0, len(counts) - 1, 40).astype(int))]
    assert not b.wrong(b.expected(counts), counts).any()
    for by in (-1, 1):
        for d in np.flatnonzero(counts.any(0)):
            off = counts.copy()
            off[:, d] += by * (counts[:, d] > 0)
            hit = counts[:, d] > 0
            assert b.wrong(b.expected(off), counts)[hit].any(1).all(), (d, by)


@pytest.mark.parametrize("name", CASES)
def test_a_run_of_keys_shows(name):
    """The last row of each sequence with 32, 64, 128, ... neighbouring keys of its sequence left out."""
    b, _ = make(name)
    counts, owned = b.counts(b.prefix > 0)
    last = {s: t for t, s, _ in b.ref.rows(b.lens, b.starts)}
    for s, t in last.items():
        seen = b.seen[s]
        for n in (32, 64, 128, 256, 384, 512, 1024):
            for k in range(0, len(seen) - 1 - n, 32):
                run = seen[k + n] - seen[k]
                if run.any() and counts[t].sum() > run.sum():
                    assert b.wrong(b.expected(counts[t:t + 1] - run), counts[t:t + 1]).any(), (s, n, k)
