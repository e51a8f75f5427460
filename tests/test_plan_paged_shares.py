"""How even the shares of gda_prefill_paged's plan are, in the CPU model of it and as the device code leaves
them in the workspace.

A block's cost is taken as linear in its number up to the block from which on the tiles of a block stay as many
as they are: with a window that is where the window and the first visible tokens are both full, at position
window + keep."""
import pytest

from test_plan_model_paged import ITEM_COST, LONE, PAIR, Batch


class Plan(Batch):
    def costs(self, s):
        mt = self.blocks(s)
        knee = first = rise = 0
        if mt > 0:
            n0 = self.range(s, 0)[4]
            first = 2 * n0 + ITEM_COST
            if mt > 1:
                knee = mt - 1
                if self.window > 0:
                    knee = min(knee, max(0, self.window + self.keep - s[1] + s[0]) * self.G // self.rows + 1)
                d = (2 * (self.range(s, knee)[4] - n0)) << 16
                rise = abs(d) // knee * (1 if d >= 0 else -1)    # (C's division)

        def before(i):
            k = min(i, knee)
            return first * i + ((rise * (k * (k - 1) // 2 + (i - k) * knee)) >> 16)
        return mt, before

    def work(self, cuts):
        """Each share's work, in half tiles, from the shares' starts and ends."""
        return [sum(2 * (tb - ta) + ITEM_COST for _, _, _, ta, tb, _ in self.items(x, start, end))
                for x, (start, end) in enumerate(cuts)]

    def check_even(self, cuts):
        """A share may exceed the mean by: the constants of the two blocks that it shares with others (a cut block's
        constant is spent in each of its parts), a tile of its end's rounding, and less than a tile a block by which
        a block's tiles differ from the line that they are taken for."""
        work = self.work(cuts)
        blocks = max(sum(1 for _ in self.items(x, *c)) for x, c in enumerate(cuts))
        mean = sum(work) / len(cuts)
        assert max(work) <= mean + 2 * ITEM_COST + 2 * (blocks + 1), (max(work), mean, blocks)


# new tokens, positions, window, keep
UNEVEN = [([8192], [8192], 1024, 4096), ([4097, 4097], [4097, 4097], 256, 1024), ([3000, 500], [9000, 500], 100, 6500),
          ([4097, 4097], [4097, 4097], 1024, 16), ([6000], [6000], 5000, 1 << 30), ([2048], [30000], 512, 64)]


@pytest.mark.parametrize("kernel", (PAIR, LONE), ids=("pair", "lone"))
@pytest.mark.parametrize("case", UNEVEN, ids=str)
@pytest.mark.parametrize("G, Hkv", [(8, 2), (1, 8), (5, 1)])
def test_shares_are_even(kernel, case, G, Hkv):
    new, lens, window, keep = case
    b = Plan(new, lens, G, Hkv, window, keep, kernel=kernel)
    used, cuts = b.shares(b.n_shares)
    b.check()
    b.check_even(cuts[:used])


@pytest.mark.parametrize("kernel", (PAIR, LONE), ids=("pair", "lone"))
@pytest.mark.parametrize("G", (1, 3, 8, 48, 300))
@pytest.mark.parametrize("window,keep", ((1, 0), (1, 900), (100, 4), (1024, 300), (4096, 1 << 20), ((1 << 31) - 1, (1 << 31) - 1)))
def test_shapes(G, window, keep, kernel):
    for new, lens in (([1], [1]), ([1], [0]), ([5], [3]), ([300], [300]), ([70], [33000]), ([0, 0, 700, 0], [5, 0, 9000, 3]),
                      ([1] * 64, [700 + 13 * b for b in range(64)]), ([2048, 1, 1, 500], [2048, 30000, 1, 5000])):
        Plan(new, lens, G, 2, window, keep, kernel=kernel).check()


@pytest.mark.gpu
@pytest.mark.parametrize("case", UNEVEN + [([1, 40, 0, 3], [900, 4000, 7, 30000], 0, 0), ([1] * 40 + [300], [3000] * 41, 700, 70),
                                           ([9, 140, 3], [3, 20, 0], 5, 5), ([1] * 700, [50] * 700, 0, 0)], ids=str)
@pytest.mark.parametrize("empty", [0, 9000])
def test_the_devices_plan(gda, case, empty):
    """The table of shares that a call leaves in its workspace: the model's, and as even (with 9000 empty sequences a
    CTA takes an item)."""
    import torch
    new, lens, window, keep = case
    new, lens = list(new) + [0] * empty, list(lens) + [0] * empty
    Hq, Hkv, D = 8, 1, 256
    Tq, nnz = sum(new), sum(lens)
    lone = Tq * (Hq // Hkv) <= 128 * len(new)
    rows, tile, _ = LONE if lone else PAIR
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    n = min(sms, 160) if lone else min(sms // 2, 80)
    b = Plan(new, lens, Hq // Hkv, Hkv, window, keep, kernel=(rows, tile, n))
    if window >= nnz:
        b.window = 0
    dev = dict(device="cuda")
    pool = torch.zeros(16, Hkv, D, dtype=torch.bfloat16, **dev)
    ws = torch.empty(gda.prefill_paged_workspace_bytes(Tq, len(new), Hq, Hkv, D), dtype=torch.uint8, **dev)
    gda.prefill_paged(torch.zeros(Tq, Hq, D, dtype=torch.bfloat16, **dev), None, pool, pool,
                      torch.tensor(b.cu, dtype=torch.int32, **dev), torch.tensor(b.indptr, dtype=torch.int32, **dev),
                      torch.zeros(nnz, dtype=torch.int32, **dev), window=window, keep_first=keep, workspace=ws)
    assert gda.prefill_read_error() == 0
    table = ws[:(1 + 2 * n) * 16].view(torch.int32).view(-1, 4).tolist()
    used, cuts = b.shares(n)
    starts = [tuple(x) for x in table[1:1 + n]] + [(b.B, 0, 0, 0)]
    assert table[0][0] == used
    assert starts[:-1] == [c[0] for c in cuts]
    if case in UNEVEN:
        b.check_even([(starts[x], starts[x + 1]) for x in range(used)])
