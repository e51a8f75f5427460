"""The split plan of a 4-bit cache restated (test_plan_model.py has the BF16 and e4m3 ones): 16 S^2 > lmax, two CTAs
per SM, one wave of splits that keeps 95 % of the CTAs busy before anything else, and a segment start that costs 400
positions in the stream schedule."""
import random

import test_plan_model as base

PIECE_COST = 400


def uniform_splits(indptr, Hkv, grid, min_chunk):
    B = len(indptr) - 1
    units = B * Hkv
    if units > grid:
        return 0
    if units == 0:
        return 1
    lmax = max(indptr[b + 1] - indptr[b] for b in range(B))
    s_opt = 1
    while 16 * s_opt * s_opt <= lmax:
        s_opt *= 2
    wave = grid // units
    fills = 20 * wave * units >= 19 * grid
    if fills and 4 * lmax * B <= 5 * indptr[B] and min(s_opt, -(-lmax // min_chunk)) >= wave:
        return wave
    if not fills:
        return base.uniform_splits(indptr, Hkv, grid, min_chunk, kv8=True)
    # (the stream's bound per CTA does not apply to a wave that fills the CTAs)
    if 4 * lmax * B > 5 * indptr[B]:
        return 0
    return min(s_opt, max(1, -(-lmax // min_chunk)))


def test_the_wave_that_fills():
    ip = lambda n, B: [n * i for i in range(B + 1)]
    assert uniform_splits(ip(8192, 8), 2, 304, 64) == 19            # 304 of 304 CTAs
    assert uniform_splits(ip(131072, 8), 2, 304, 64) == 19          # at any length
    assert uniform_splits(ip(4096, 64), 2, 304, 64) == 2            # 256 of 304: the power of two
    assert uniform_splits(ip(300, 8), 2, 304, 64) == 5              # too short for a full wave: ceil(300 / 64)
    assert uniform_splits(ip(131072, 9), 2, 304, 64) == 0           # 288 of 304: the stream
    assert uniform_splits([0, 8192, 8192 + 100], 8, 304, 64) == 0   # far from equal: the stream


def test_pieces_cover_every_position_once():
    rng = random.Random(3)
    for _ in range(150):
        B, Hkv, grid = rng.randint(1, 40), rng.choice([1, 2, 3, 8]), 304
        top = rng.choice([1, 64, 700, 9000])
        equal = rng.random() < 0.5
        lens = [top if equal else rng.randint(0, top) for _ in range(B)]
        ip = [0]
        for n in lens:
            ip.append(ip[-1] + n)
        S = uniform_splits(ip, Hkv, grid, 64)
        assert S * B * Hkv <= grid or S == 1 or S == 0
        if S == 0:
            # the stream: force it in the model that knows it
            X = base.piece_cost(B, Hkv, grid, PIECE_COST)
            T = max(-(-base.stream_cost(Hkv * ip[-1], B, Hkv, X) // grid), 64)
            at = [base.position_at_cost(ip, Hkv, X, c * T) for c in range(grid + 1)]
            assert at[0] == 0 and at[-1] == Hkv * ip[-1] and all(a <= b for a, b in zip(at, at[1:]))
            continue
        pieces, _, _ = base.stage1_pieces(ip, Hkv, grid, 64, S)
        seen = {}
        for b, h, j0, j1, uid in pieces:
            assert 0 <= uid < base.AUTO_MAX_CTAS + B * Hkv
            seen.setdefault((b, h), []).append((j0, j1))
        for b, n in enumerate(lens):
            for h in range(Hkv):
                at = 0
                for j0, j1 in sorted(seen.get((b, h), [])):
                    assert j0 == at
                    at = j1
                assert at == n
