"""INT8 entry points without a GPU: their refusals (checked in the order the
header gives) and the tile lists that the grouped kernels form from the
device's offsets, restated here."""
import ctypes

import numpy as np
import pytest

from block_scaled_fp4_05_b200 import fp4

P = ctypes.c_void_p
A16 = P(1 << 20)       # 16-byte aligned dummy address (never dereferenced)
A1 = P((1 << 20) + 1)
A2 = P((1 << 20) + 2)


def no_gpu():
    import torch
    return not torch.cuda.is_available()


def test_new_symbols_are_declared_and_exported():
    names = fp4.declared_symbols()
    for n in ("fp4_quantize_int8", "fp4_gemm_int8", "fp4_gemm_int8_grouped"):
        assert n in names and hasattr(fp4.lib(), n)


# (in, dtype, rows_in, cols, ld, row_index, rows, codes, ld_codes, scales, stream)
@pytest.mark.parametrize("args,want", [
    ((A16, 2, 4, 64, 64, None, 4, A16, 64, A16, None), 1),          # type
    ((A16, 0, -1, 64, 64, None, -1, A16, 64, A16, None), 1),        # negative
    ((A16, 0, 4, 64, 56, None, 4, A16, 64, A16, None), 1),          # ld < cols
    ((A16, 0, 4, 64, 64, None, 4, A16, 48, A16, None), 1),          # ld_codes < cols
    ((A16, 0, 4, 64, 64, None, 5, A16, 64, A16, None), 1),          # rows differ without an index
    ((None, 0, 4, 64, 64, None, 4, A16, 64, A16, None), 1),         # no input
    ((A16, 0, 4, 64, 64, None, 4, None, 64, A16, None), 1),         # no codes
    ((A16, 0, 4, 64, 64, None, 4, A16, 64, None, None), 1),         # no scales
    ((A16, 0, 1 << 31, 64, 64, None, 1 << 31, A16, 64, A16, None), 2),
    ((A1, 0, 4, 64, 64, None, 4, A16, 64, A16, None), 3),
    ((A16, 0, 4, 64, 68, None, 4, A16, 64, A16, None), 3),          # ld % 8
    ((A16, 0, 4, 64, 64, None, 4, A16, 72, A16, None), 3),          # ld_codes % 16
    ((A16, 0, 4, 64, 64, None, 4, A1, 64, A16, None), 3),
    ((A16, 0, 4, 64, 64, None, 4, A16, 64, A2, None), 3),
    ((A16, 0, 4, 64, 64, A2, 8, A16, 64, A16, None), 3),
    ((None, 0, 0, 64, 64, None, 0, None, 64, None, None), 0),       # no rows
    ((A16, 0, 4, 61, 64, None, 4, A16, 64, A16, None), 6),          # valid, but no device here
    ((None, 1, 0, 64, 64, A16, 4, A16, 64, A16, None), 6),          # every index is outside
])
def test_quantize_int8_refusals(args, want):
    if want == 6 and not no_gpu():
        pytest.skip("a device is present")
    assert fp4.lib().fp4_quantize_int8(*args) == want


GOOD = dict(A=A16, lda=64, sA=A16, B=A16, ldb=64, sB=A16, M=4, N=16, K=64, bias=None, out=0, D=A16, ldd=16, kernel=0)

DENSE_REFUSALS = [
    (dict(kernel=3), 1), (dict(kernel=0x200), 1), (dict(out=2), 1), (dict(M=-1), 1), (dict(K=-1), 1),
    (dict(lda=48), 1), (dict(ldb=48), 1), (dict(ldd=8), 1), (dict(A=None), 1), (dict(B=None), 1),
    (dict(D=None), 1), (dict(sA=None), 1), (dict(sB=None), 1),
    (dict(K=131072, lda=131072, ldb=131072), 2), (dict(M=1 << 31), 2), (dict(lda=1 << 40), 2), (dict(ldd=1 << 39), 2),
    (dict(M=1 << 30, N=1 << 20, ldd=1 << 20), 2),
    (dict(lda=72), 3), (dict(ldb=72), 3), (dict(ldd=20), 3), (dict(A=A1), 3), (dict(B=A1), 3), (dict(D=A1), 3),
    (dict(sA=A2), 3), (dict(sB=A2), 3), (dict(bias=A2), 3),
    (dict(M=0), 0), (dict(N=0), 0),
    (dict(), 6), (dict(K=0), 6), (dict(K=61, N=13), 6), (dict(kernel=0x102), 6), (dict(K=131071, lda=131072, ldb=131072), 6),
]


@pytest.mark.parametrize("change,want", DENSE_REFUSALS)
def test_gemm_int8_refusals(change, want):
    if want == 6 and not no_gpu():
        pytest.skip("a device is present")
    a = {**GOOD, **change}
    assert fp4.lib().fp4_gemm_int8(a["A"], a["lda"], a["sA"], a["B"], a["ldb"], a["sB"], a["M"], a["N"], a["K"],
                                   a["bias"], a["out"], a["D"], a["ldd"], a["kernel"], None) == want


@pytest.mark.parametrize("change,want", DENSE_REFUSALS + [
    (dict(E=-1), 1), (dict(offsets=None), 1), (dict(stride=-16), 1),
    (dict(stride=15 * 64 + 48), 1),                       # experts would overlap
    (dict(E=513), 2), (dict(stride=1 << 40), 2), (dict(stride=16 * 64 + 8), 3), (dict(offsets=A2), 3),
    (dict(E=0), 0), (dict(E=0, offsets=None), 0), (dict(E=1, stride=0), 6), (dict(E=512), 6),
])
def test_gemm_int8_grouped_refusals(change, want):
    if want == 6 and not no_gpu():
        pytest.skip("a device is present")
    a = {**GOOD, "offsets": A16, "E": 4, "stride": 1 << 39, **change}
    assert fp4.lib().fp4_gemm_int8_grouped(a["A"], a["lda"], a["sA"], a["B"], a["ldb"], a["stride"], a["sB"],
                                           a["offsets"], a["E"], a["M"], a["N"], a["K"], a["bias"], a["out"],
                                           a["D"], a["ldd"], a["kernel"], None) == want


# ---- the grouped kernels' bounds and tile lists, restated ----
def expert_bounds(offsets, M):
    """As 32 lanes form them, 32 experts at a time: first and end row of each."""
    E, reached, out = len(offsets) - 1, 0, []
    for e0 in range(0, E, 32):
        lo, hi = np.zeros(32, np.int64), np.zeros(32, np.int64)
        for lane in range(32):
            if e0 + lane < E:
                lo[lane] = min(max(offsets[e0 + lane], 0), M)
                hi[lane] = min(max(offsets[e0 + lane + 1], 0), M)
        top = np.maximum.accumulate(np.maximum(lo, hi))
        before = np.concatenate([[0], top[:-1]])
        first = np.maximum(np.maximum(before, reached), lo)
        end = np.maximum(np.maximum(first, hi), reached)
        out += [(int(f), int(g)) for f, g in list(zip(first, end))[: E - e0]]
        reached = max(reached, int(top[31]))
    return out


def bounds_wanted(offsets, M):
    b = np.maximum.accumulate(np.clip(np.asarray(offsets, np.int64), 0, M))
    return list(zip(b[:-1].tolist(), b[1:].tolist()))


def test_expert_bounds_are_clamped_and_never_decrease():
    rng = np.random.default_rng(0)
    for _ in range(300):
        E, M = int(rng.integers(1, 130)), int(rng.integers(0, 500))
        kind = rng.integers(3)
        o = rng.integers(0, M + 1, E + 1)
        if kind == 0:
            o = np.sort(o)
        elif kind == 1:
            o = rng.integers(-(2 ** 31), 2 ** 31, E + 1)
        assert expert_bounds(o.tolist(), M) == bounds_wanted(o, M)


@pytest.mark.parametrize("nt", [16, 32, 64, 128, 256])
def test_every_row_is_in_one_tile_and_the_bound_on_tiles_holds(nt):
    rng = np.random.default_rng(1)
    for _ in range(60):
        E, M, tiles_n, rg = int(rng.integers(1, 80)), int(rng.integers(1, 3000)), int(rng.integers(1, 5)), int(rng.integers(1, 9))
        o = np.sort(rng.integers(0, M + 1, E + 1))
        bounds = expert_bounds(o.tolist(), M)
        seen = np.zeros((M, tiles_n), np.int64)
        listed = 0
        for first, end in bounds:
            mt = (end - first + nt - 1) // nt
            listed += mt
            for t in range(mt * tiles_n):
                span = rg * tiles_n
                grp, within = divmod(t, span)
                m0 = grp * rg
                gm = min(mt - m0, rg)
                row, col = first + (m0 + within % gm) * nt, within // gm
                seen[row:min(row + nt, end), col] += 1
        inside = np.zeros(M, bool)
        for first, end in bounds:
            inside[first:end] = True
        assert (seen[inside] == 1).all() and (seen[~inside] == 0).all()
        assert listed <= M // nt + min(E, M)   # what the launch provides for


def test_a_stride_too_small_by_more_than_64_bits_is_refused():
    # (N - 1) * ldb leaves 64 bits: wrapped around it would be negative
    N = 1 << 30
    assert fp4.lib().fp4_gemm_int8_grouped(A16, 64, A16, A16, 1 << 39, 1 << 39, A16, A16, 2, 4, N, 64, None, 0, A16, N,
                                           0, None) == 1


@pytest.mark.parametrize("change,want", [
    (dict(kernel=0), 1), (dict(kernel=3), 1), (dict(kernel=1, tile=48), 1), (dict(kernel=1, tile=0), 1),
    (dict(kernel=1, tile=288), 1), (dict(kernel=1, tile=64, split=2), 1), (dict(kernel=1, tile=64, K=0), 1),
    (dict(kernel=2, tile=48), 1), (dict(kernel=2, tile=256), 1), (dict(kernel=2, split=3), 1), (dict(kernel=2, split=0), 1),
    (dict(kernel=2, split=16, K=4096, lda=4096, ldb=4096), 1), (dict(kernel=2, split=2, K=128, lda=128, ldb=128), 1),
    (dict(E=2), 1), (dict(E=-1), 1), (dict(stride=-16), 1), (dict(E=513, offsets=A16), 2), (dict(A=A1), 3), (dict(M=0), 0),
    (dict(), 6), (dict(kernel=0x102), 6), (dict(kernel=1, tile=224), 6), (dict(kernel=2, split=2, K=129, lda=144, ldb=144), 6),
    (dict(kernel=2, K=0), 6), (dict(E=2, offsets=A16, stride=1 << 20), 6),
])
def test_selftest_gemm_int8_refusals(change, want):
    if want == 6 and not no_gpu():
        pytest.skip("a device is present")
    a = {**GOOD, "kernel": 2, "tile": 32, "split": 1, "offsets": None, "E": 1, "stride": 0, **change}
    assert fp4.lib().fp4_selftest_gemm_int8(a["kernel"], a["tile"], a["split"], a["A"], a["lda"], a["sA"], a["B"], a["ldb"],
                                            a["stride"], a["sB"], a["offsets"], a["E"], a["M"], a["N"], a["K"], a["bias"],
                                            a["out"], a["D"], a["ldd"], None) == want


# ---- the pair kernel's work items, restated: tiles, halves of the last wave,
# token boxes and the epilogue's chunks ----
def pair_items(bounds, tiles_n, bt, pairs, rg):
    """(expert, row, row end, channel tile, width) of every item, as `locate` finds them."""
    mts = [(end - first + bt - 1) // bt for first, end in bounds]
    tiles = sum(mts) * tiles_n
    rem = tiles % pairs
    split_from = tiles - rem if 2 * rem <= pairs else tiles
    for item in range(2 * tiles - split_from):
        t, half, halved = item, 0, item >= split_from
        if halved:
            half, t = (item - split_from) & 1, split_from + (item - split_from) // 2
        e = 0
        while t >= mts[e] * tiles_n:
            t -= mts[e] * tiles_n
            e += 1
        first, end = bounds[e]
        group = min(rg, max(mts))
        grp, within = divmod(t, group * tiles_n)
        gm = min(mts[e] - grp * group, group)
        row, col = first + (grp * group + within % gm) * bt, within // gm
        width = min(bt, (end - row + 31) & ~31)
        if halved:
            upper = (width // 2 + 31) & ~31
            row += half * upper
            width = width - upper if half else upper
        yield e, row, end, col, width


@pytest.mark.parametrize("bt", range(32, 257, 32))
def test_pair_items_cover_every_row_once_and_their_boxes_fit(bt):
    rng = np.random.default_rng(bt)
    for _ in range(40):
        E, tiles_n = int(rng.integers(1, 9)), int(rng.integers(1, 30))
        counts = rng.integers(0, 4 * bt, E) * (rng.random(E) < 0.8)
        o = np.concatenate([[0], np.cumsum(counts)])
        if o[-1] == 0:
            continue
        bounds = list(zip(o[:-1].tolist(), o[1:].tolist()))
        most = int(o[-1] // bt + min(E, o[-1])) * tiles_n
        seen = np.zeros((int(o[-1]), tiles_n), np.int64)
        for e, row, end, col, width in pair_items(bounds, tiles_n, bt, min(most, 74), int(rng.integers(1, 9))):
            if width == 0:
                continue
            assert width % 32 == 0 and 32 <= width <= bt        # what the pair MMA takes
            box = (width * 4 + bt - 1) // bt                    # quarters of a CTA's share of the widest tile
            assert 1 <= box <= 4 and width // 2 <= box * (bt // 8) <= bt // 2 and bt // 8 * box <= 256
            chunks = [(width // 32 - half + 1) >> 1 for half in (0, 1)]
            assert sorted(h + 2 * c for h in (0, 1) for c in range(chunks[h])) == list(range(width // 32)) and max(chunks) <= 4
            seen[row:min(row + width, end), col] += 1
        assert (seen == 1).all()
        assert (bt // 2 * 128) % 1024 == 0                      # a stage's tiles start where the swizzle does
