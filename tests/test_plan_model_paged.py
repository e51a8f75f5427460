"""A CPU model of the plan that gda_prefill_paged derives on the device.

The device code (Costs, cut_at, share_of and the planning warp, and the joining kernel's list of parts in
gda_prefill_paged.cu) decides, from cu_seqlens and kv_indptr alone, which share (a pair of CTAs with blocks of
256 rows and tiles of 128 keys, or a CTA with 128 and 64) computes which tiles of which block, and where the parts of a block that a share's end cuts go.  This model restates the same
rules in integers and checks their invariants: every tile of every block is computed exactly once, a block
without tiles too; each share leaves at most one part in each of its two places; the joining kernel's list of a
block's parts is exactly what the shares left, in the order of the shares; the tiles hold every position that a
row of the block sees.  (The GPU tests check the device code itself.)"""
import random

import pytest

ITEM_COST = 10
PAIR, LONE = (256, 128, 76), (128, 64, 152)   # rows of a block, keys of a tile, shares


class Batch:
    def __init__(self, new, lens, G, Hkv, window=0, keep=0, Tq=None, nnz=None, cu=None, indptr=None,
                 kernel=PAIR):
        self.rows, self.tile, self.n_shares = kernel
        self.G, self.Hkv, self.window, self.keep = G, Hkv, window, keep
        if cu is None:
            cu, indptr = [0], [0]
            for n, L in zip(new, lens):
                cu.append(cu[-1] + n)
                indptr.append(indptr[-1] + L)
        self.cu, self.indptr = cu, indptr
        self.Tq, self.nnz, self.B = cu[-1] if Tq is None else Tq, indptr[-1] if nnz is None else nnz, len(cu) - 1

    def seq(self, b):
        """(new tokens, positions), clamped to the tensors."""
        q0 = min(max(self.cu[b], 0), self.Tq)
        kb = min(max(self.indptr[b], 0), self.nnz)
        return max(min(self.cu[b + 1], self.Tq) - q0, 0), max(min(self.indptr[b + 1], self.nnz) - kb, 0)

    def blocks(self, s):
        return -(-s[0] * self.G // self.rows)

    def range(self, s, i):
        """(lo, hi, f, tl, n) of block i."""
        nq, L = s
        ta, tb = i * self.rows // self.G, min(nq - 1, (i * self.rows + self.rows - 1) // self.G)
        hi = max(L - nq + tb + 1, 0)
        lo = min(max(L - nq + ta - self.window + 1, 0), hi) if self.window > 0 else 0
        tl = lo // self.tile
        f = min(-(-min(self.keep, lo) // self.tile), tl)
        return lo, hi, f, tl, f + -(-hi // self.tile) - tl

    def costs(self, s):
        mt = self.blocks(s)
        knee = first = rise = 0
        if mt > 0:
            n0 = self.range(s, 0)[4]
            first = 2 * n0 + ITEM_COST
            if mt > 1:
                knee = mt - 1
                if self.window > 0:
                    knee = min(knee, max(0, self.window - s[1] + s[0]) * self.G // self.rows + 1)
                d = (2 * (self.range(s, knee)[4] - n0)) << 16
                rise = abs(d) // knee * (1 if d >= 0 else -1)    # (C's division)

        def before(i):
            k = min(i, knee)
            return first * i + ((rise * (k * (k - 1) // 2 + (i - k) * knee)) >> 16)
        return mt, before

    def cut_at(self, b, x):
        s = self.seq(b)
        mt, before = self.costs(s)
        per_head = before(mt)
        h, x = divmod(x, per_head)
        lo, hi = 0, mt - 1
        while lo < hi:
            mid = (lo + hi + 1) >> 1
            if before(mid) <= x:
                lo = mid
            else:
                hi = mid - 1
        at = before(lo)
        cost = before(lo + 1) - at
        return (b, h, lo, self.range(s, lo)[4] * (x - at) // cost if cost > 0 else 0)

    def shares(self, shares):
        """[used], each share's (start, end)."""
        costs = []
        for b in range(self.B):
            mt, before = self.costs(self.seq(b))
            assert mt == 0 or all(before(i + 1) > before(i) for i in range(mt)), "a block costs something"
            costs.append(self.Hkv * before(mt))
        total = sum(costs)
        assert total * shares < 1 << 63
        used = max(1, min(shares, total * self.tile // 256))

        def place(y):
            at = total * y // used if y < used else total
            upto = 0
            for b, c in enumerate(costs):
                if upto <= at < upto + c:
                    return self.cut_at(b, at - upto)
                upto += c
            return (self.B, 0, 0, 0)
        return used, [(place(y), place(y + 1)) for y in range(shares)]

    def items(self, x, start, end):
        """The planning warp's items of share x: (b, h, i, ta, tb, part)."""
        at = list(start)
        while True:
            last = tuple(at[:3]) == tuple(end[:3])
            if at[0] >= self.B or (last and end[3] <= at[3]):
                return
            s = self.seq(at[0])
            n = self.range(s, at[2])[4]
            ta, tb = at[3], end[3] if last else n
            yield at[0], at[1], at[2], ta, tb, (2 * x if ta > 0 else 2 * x + 1 if tb < n else -1)
            if last:
                return
            at[3] = 0
            at[2] += 1
            if at[2] < self.blocks(s):
                continue
            at[2] = 0
            at[1] += 1
            if at[1] < self.Hkv:
                continue
            at[1] = 0
            at[0] += 1
            while at[0] < self.B and self.seq(at[0])[0] == 0:
                at[0] += 1

    def check(self, shares=None):
        shares = shares or self.n_shares
        used, cuts = self.shares(shares)
        done, left = {}, {}
        for x, (start, end) in enumerate(cuts):
            for b, h, i, ta, tb, part in self.items(x, start, end):
                n = self.range(self.seq(b), i)[4]
                assert 0 <= ta <= tb <= n and (n == 0 or ta < tb)
                done.setdefault((b, h, i), []).append((ta, tb))
                if part >= 0:
                    assert part not in left, "one part to a place"
                    left[part] = (b, h, i)
                else:
                    assert (ta, tb) == (0, n)
        for b in range(self.B):
            s = self.seq(b)
            for i in range(self.blocks(s)):
                lo, hi, f, tl, n = self.range(s, i)
                for h in range(self.Hkv):
                    got = sorted(done.pop((b, h, i)))
                    assert got[0][0] == 0 and got[-1][1] == n and all(a[1] == c[0] for a, c in zip(got, got[1:]))
                # the tiles, [0, f) and [tl, th), hold every position that a row sees, each once
                th = tl + n - f
                assert 0 <= f <= tl and (n == 0 or (self.tile * tl <= lo and self.tile * th >= hi))
                assert lo == hi or n > 0
                assert f == tl or (min(self.keep, lo) if self.window else 0) <= self.tile * f
                for t in (i * self.rows // self.G, min(s[0] - 1, (i * self.rows + self.rows - 1) // self.G)):   # its first and last token
                    p = s[1] - s[0] + t
                    assert p < hi or p < 0
                    assert p < 0 or not self.window or max(p - self.window + 1, 0) >= lo
        assert not done, "no block that is not there"
        # the joining kernel: a block of it per share start after the first
        starts = [c[0] for c in cuts] + [(self.B, 0, 0, 0)]
        joined = set()
        for c in range(1, shares):
            me, before = starts[c], starts[c - 1]
            if c >= used or me[0] >= self.B or me[3] == 0 or (before[:3] == me[:3] and before[3] > 0):
                continue
            parts = [2 * (c - 1) + 1]
            for k in range(c, used):
                a = starts[k]
                z = starts[k + 1] if k + 1 < used else (self.B, 0, 0, 0)
                if a[:3] == me[:3] and (z[:3] != me[:3] or z[3] > a[3]):
                    parts.append(2 * k)
            assert me[:3] not in joined
            joined.add(me[:3])
            want = [p for p, item in sorted(left.items(), key=lambda e: (e[0] // 2, e[0] % 2)) if item == me[:3]]
            assert parts == want and len(parts) >= 2
        assert joined == set(left.values())


@pytest.mark.parametrize("kernel", (PAIR, LONE), ids=("pair", "lone"))
@pytest.mark.parametrize("G", (1, 3, 5, 8, 16, 48, 256, 300))
@pytest.mark.parametrize("window,keep", ((0, 0), (1, 0), (100, 4), (1024, 0), (4096, 300), (1 << 20, 5)))
def test_shapes(G, window, keep, kernel):
    for new, lens in (([1], [1]), ([1], [0]), ([5], [3]), ([1], [40000]), ([300], [300]), ([70], [33000]), ([0, 0, 7, 0], [5, 0, 9000, 3]),
                      ([1] * 64, [700 + 13 * b for b in range(64)]), ([2048, 1, 1, 500], [2048, 30000, 1, 5000])):
        Batch(new, lens, G, 2, window, keep, kernel=kernel).check()


@pytest.mark.parametrize("kernel", (PAIR, LONE), ids=("pair", "lone"))
@pytest.mark.parametrize("seed", range(40))
def test_random(seed, kernel):
    r = random.Random(seed)
    B = r.choice((1, 2, 5, 31, 32, 33, 90, 200))
    G, Hkv = r.choice((1, 2, 3, 4, 6, 8, 12, 16, 24)), r.choice((1, 2, 3, 8))
    top = r.choice((1, 5, 64, 700)) if B < 40 else r.choice((1, 5))
    new = [r.randrange(top + 1) if r.random() < .8 else 0 for _ in range(B)]
    lens = [max(n + r.randrange(-3, r.choice((1, 100, 9000)) + 1), 0) if r.random() < .9 else 0 for n in new]
    window = r.choice((0, 0, 1, 127, 128, 129, 1000, 5000))
    Batch(new, lens, G, Hkv, window, r.choice((0, 1, 4, 128, 600)), kernel=kernel).check(
        r.choice((1, 2, 7, 66, 76, 80, 152 if kernel is LONE else 78)))


@pytest.mark.parametrize("kernel", (PAIR, LONE), ids=("pair", "lone"))
@pytest.mark.parametrize("seed", range(12))
def test_offsets_out_of_range(seed, kernel):
    """Offsets that the tensors do not hold are clamped to them: the plan stays one of the same kind."""
    r = random.Random(seed)
    B, Tq, nnz = r.choice((1, 3, 40)), 500, 9000
    cu = sorted(r.randrange(-50, 600) for _ in range(B + 1))
    indptr = sorted(r.randrange(-500, 10000) for _ in range(B + 1))
    Batch(None, None, 8, 2, r.choice((0, 300)), 4, Tq, nnz, cu, indptr, kernel).check()


@pytest.mark.parametrize("kernel", (PAIR, LONE), ids=("pair", "lone"))
def test_long_cache(kernel):
    """A cache near 31 bits of positions, a prompt of a million tokens: the costs stay within 64 bits."""
    Batch([1, 5], [(1 << 31) - 1000, 100], 8, 2, kernel=kernel).check()
    Batch([1], [(1 << 31) - 1000], 1, 8, 1 << 30, 1000, kernel=kernel).check()
    b = Batch([1 << 20], [(1 << 31) - 1000], 16, 2, kernel=kernel)
    mt, before = b.costs(b.seq(0))
    assert before(mt) * b.Hkv * b.n_shares * b.tile < 1 << 63
