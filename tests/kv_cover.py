"""Batches that show which keys an attention row counted.

All keys of a head are equal, so every key a row sees has the same weight, and
a value row is one in a single coordinate, its mark: a permutation for the
first head_dim positions of a sequence, random behind them.  Coordinate d of an
output is then a * (keys of that mark seen) / (keys seen), a the stored value of
one.  A key that is left out, counted twice or seen by a row that must not see
it changes its mark's coordinate by one key in those few that share the mark,
and a whole run of keys changes the marks' proportions."""
import numpy as np

import oracle
from kv_util import Batch

class Marked(Batch):
    def __init__(self, rng, lens, new, page_size, heads, head_dim, bits, holes=(), **kw):
        super().__init__(rng, lens, new, page_size, heads, head_dim, bits, fill=False, **kw)
        for b, i in holes:
            self.pages[b, i] = -1
        D, P = head_dim, page_size
        key, one = np.full((1, D), 0.75), np.zeros((D, D))
        np.fill_diagonal(one, 1.0)
        kq, ks, ko = oracle.kvcache.quantize_rows(key, bits)
        vq, vs, vo = oracle.kvcache.quantize_rows(one, bits)
        self.a = float(oracle.kvcache.row_values(vq, vs, vo)[0, 0])
        kc, km = oracle.kvcache.pack_codes(kq, bits)[0], oracle.kvcache.pack_meta(ks, ko)[0]
        vc, vm = oracle.kvcache.pack_codes(vq, bits), oracle.kvcache.pack_meta(vs, vo)
        for m in self.ref.meta:
            m[:] = 0x7E007E00                  # a slot without a token is NaN
        self.seen = []                         # per sequence: marks seen after 0, 1, ... keys
        tables = [(self.pages[b], int(n)) for b, n in enumerate(self.lens)]
        pre = [(self.prefix_pages, self.prefix)] if self.prefix else []
        for table, n in tables + pre:
            n = min(n, len(table) * P)
            mark = np.concatenate([rng.permutation(D), rng.integers(0, D, max(0, n - D))])
            one = np.zeros((n + 1, D))
            for j in range(n):
                page = table[j // P]
                if 0 <= page < self.n_pages:
                    d = mark[j]
                    self.ref.codes[0][page, :, j % P], self.ref.meta[0][page, :, j % P] = kc, km
                    self.ref.codes[1][page, :, j % P], self.ref.meta[1][page, :, j % P] = vc[d], vm[d]
                    one[j + 1, d] = 1
            self.seen.append(np.cumsum(one, 0))
        self.pre_seen = self.seen.pop()[-1] if pre else np.zeros(D)

    def counts(self, shared):
        """[T][D] keys of every mark that a row sees, and which rows are owned."""
        n, owned = np.zeros((self.T, self.geom[3])), np.zeros(self.T, bool)
        for t, b, pos in self.ref.rows(self.lens, self.starts):
            s = self.seen[b]
            n[t] = s[min(max(pos + 1, 0), len(s) - 1)] + (self.pre_seen if shared else 0)
            owned[t] = True
        return n, owned

    def expected(self, counts):
        total = counts.sum(1, keepdims=True)
        return self.a * counts / np.maximum(total, 1)

    def tolerance(self, counts):
        """Relative.  The logits of a row are equal to the bit, and with them its weights before they are rounded for
        the product: to 11 bits, half a step 2^-11 (or to 16 in two parts, less); a value to 11 bits, 2^-11.  Sums of
        equal terms in fp32, at most half the keys in one register: n / 2 * 2^-24 for the weights and as much for the
        products; joins, the division and powers of two: below 2^-20."""
        return 2 * 2.0 ** -11 + counts.sum(1, keepdims=True) * 2.0 ** -24 + 2.0 ** -20

    def wrong(self, got, counts):
        """Elements of got [T][D] that are not what these counts give; an output without a key of its mark is 0."""
        want = self.expected(counts)
        return np.abs(got - want) > self.tolerance(counts) * want


# name: page size, heads, head_dim, bits, query heads per KV head, lens, new rows, prefix, (sequence, page) holes
CASES = {
    "whole tables, a workgroup each": (16, 2, 128, 8, 8, [517, 1500, 33, 0, 1], 1, 0, [(1, 40)]),
    "whole tables, more than workgroups": (64, 8, 64, 4, 4, [(37 * i) % 620 for i in range(90)], 1, 0, []),
    "whole tables, 32 rows": (32, 2, 64, 8, 4, [700, 350, 9, 40], 6, 0, []),
    "pieces of one tile each, 8 rows": (16, 2, 128, 8, 8, [4001, 2047, 129], 1, 0, [(0, 77)]),
    "pieces of one tile each, 16 rows": (64, 1, 64, 4, 16, [3100, 1, 640, 2047], 1, 0, []),
    "pieces of one tile each, 32 rows": (32, 8, 128, 4, 5, [2500, 5], 5, 0, []),
    "cut anywhere, 8 rows": (32, 8, 128, 8, 8, [6000, 17, 0, 1025, 3500, 2, 4097, 900], 1, 0, [(0, 3), (4, 60)]),
    "cut anywhere, 16 rows": (256, 8, 128, 4, 4, [6000, 17, 3, 1025, 3500, 4, 4097, 900], 3, 0, []),
    "cut anywhere, 32 rows": (16, 8, 64, 8, 10, [4097, 2, 2, 1025, 3500, 7, 2900, 900], 2, 0, [(3, 1)]),
    "tiles of 128 rows": (16, 2, 64, 4, 8, [3500, 90, 0, 1300], 11, 0, [(0, 100)]),
    "tiles of 256 rows": (64, 2, 128, 8, 8, [2900, 120, 1700], 100, 0, [(2, 5)]),
    "tiles of 256 rows, 4 bits": (16, 1, 64, 4, 4, [2900, 333, 1], 200, 0, []),
    "decoded beforehand": (32, 2, 128, 8, 16, [1500, 257, 900], 200, 0, [(0, 20)]),
    "decoded beforehand, 4 bits": (256, 1, 64, 4, 16, [1500, 257, 900], 190, 0, []),
    "prefix and own keys in one launch, 32 rows": (16, 2, 128, 8, 8, [40, 0, 700, 5], 1, 5003, []),
    "prefix and own keys in one launch, 16 rows": (64, 4, 64, 4, 4, [40, 3, 7, 500], 1, 701, []),
    "prefix before long sequences": (64, 2, 128, 4, 8, [1700, 3, 0], 1, 1003, []),
    "prefix before many": (32, 8, 128, 8, 8, [(13 * i) % 500 for i in range(40)], 1, 4229, []),
    "prefix before chunks": (16, 2, 64, 8, 4, [700, 60, 210], 50, 777, [(0, 3)]),
    "prefix before prompts decoded beforehand": (16, 1, 128, 8, 16, [600, 257], 200, 1401, []),
    "prefix before prompts decoded beforehand, 4 bits": (64, 2, 64, 4, 32, [300, 190], 150, 333, []),
}


def make(name):
    page, heads, D, bits, group, lens, new, prefix, holes = CASES[name]
    rng = np.random.default_rng(len(name))
    rows = [1] * len(lens) if new == 1 else [min(n, new) for n in lens]
    lead = 0 if new == 1 else 2
    return Marked(rng, lens, rows, page, heads, D, bits, holes, starts=new > 1, prefix=prefix, lead=lead), group
